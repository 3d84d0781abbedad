"""tcl_i8_quant, tcl_i8_product and tcl_i8_linear against their definitions in
64 bits.

The integers of the quantiser and the sums of the product are exact, so the
quantiser must agree bit for bit, and a product only rounds: the integer sum
to fp32 and two fp32 multiplications (2^-24 each, relative), and for a bf16
output one more (2^-8).
"""
import numpy as np
import pytest
import torch

from tenant_composite_lora_amd import tclora

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def tol(dtype):
    """Half a step of the output type (finfo.eps / 2, relative) after three
    half steps of fp32."""
    t = 3 * torch.finfo(torch.float32).eps / 2
    return t if dtype == torch.float32 else t + torch.finfo(dtype).eps / 2 * (1 + t)


def quant64(x):
    """The definition: scale rounded to fp32, then the real quotient."""
    x = x.double().cpu()
    amax = x.abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    s = (amax / 127).float()
    n = torch.round(x / s.double()[:, None])
    n = torch.where((s > 0)[:, None], n, 0).clamp(-127, 127)
    bad = ~torch.isfinite(x).all(1)
    s[bad] = float("nan")
    n[bad] = 0
    return n.to(torch.int8), s


def product64(W, ws, q, s):
    return (q.double().cpu() @ W.double().cpu().T) * s.double().cpu()[:, None] * ws.double().cpu()


def close(got, want, dtype):
    got = got.double().cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    # the smallest normal's rounding is absolute below it
    tiny = torch.finfo(torch.float32).tiny * torch.finfo(dtype).eps
    err = ((got - want).abs() - tol(dtype) * want.abs())[~nan]
    assert err.numel() == 0 or float(err.max()) <= tiny, float(err.max())


def weight(seed, d_out, d_in, full=False):
    g = torch.Generator().manual_seed(seed)
    W = torch.randint(-128 if full else -127, 128, (d_out, d_in), generator=g, dtype=torch.int32)
    ws = torch.rand(d_out, generator=g) * 0.01 + 1e-4
    return W.to(torch.int8).to(DEV), ws.to(DEV)


def acts(seed, T, d, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, d, generator=g) * torch.exp2(torch.randint(-3, 4, (T, 1), generator=g))
            ).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 16), (3, 48), (5, 4096), (2, 16384), (2, 16400), (1, 40000),
                                 (1025, 16), (1031, 4112), (2051, 112), (4100, 80)])
def test_quant_is_the_definition(T, d, dtype):
    x = acts(T * 7 + d, T, d, DT[dtype])
    q, s = tclora.i8_quant(x)
    n, want = quant64(x)
    assert torch.equal(s.cpu().view(torch.int32), want.view(torch.int32))
    assert torch.equal(q.cpu(), n)


def test_quant_ties_and_their_neighbours():
    """A scale of 1 (largest magnitude 127): halves are ties, to even; fp32
    values one step beside a half go to their own side."""
    h = np.arange(-126.5, 127, 1.0, dtype=np.float32)
    up, dn = np.nextafter(h, np.float32(1e9)), np.nextafter(h, np.float32(-1e9))
    rows = []
    for v in (h, up, dn):
        rows.append(np.concatenate([[127.0], v, np.zeros(1)])[:256].astype(np.float32))
    x = torch.from_numpy(np.stack([np.pad(r, (0, 256 - len(r))) for r in rows])).to(DEV)
    # other scales whose quotients fall next to ties
    extra = []
    for a in (254.0, 1.0, 3.3, 1e-30, 1e30):
        s = np.float32(a / 127)
        t = (h.astype(np.float64) * float(s)).astype(np.float32)
        extra.append(np.pad(np.concatenate([[np.float32(a)], t]), (0, 256 - 1 - len(t))))
    x = torch.cat([x, torch.from_numpy(np.stack(extra).astype(np.float32)).to(DEV)])
    q, s = tclora.i8_quant(x)
    n, want = quant64(x)
    assert torch.equal(s.cpu(), want)
    assert torch.equal(q.cpu(), n)


def test_quant_special_rows():
    x = torch.zeros(6, 64)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3, 9] = -float("inf")
    x[4] = 1e-44          # the scale is zero after rounding, or subnormal
    x[4, 0] = 1.2e-43
    x[5] = torch.linspace(-3e38, 3e38, 64)
    x = x.to(DEV)
    q, s = tclora.i8_quant(x)
    assert s[0].item() == 0 and not q[0].any()
    assert torch.isnan(s[1:4]).all() and not q[1:4].any()
    n, want = quant64(x)
    # (the last row's range is beyond fp32: linspace makes infinities of it)
    assert torch.allclose(s.cpu()[4:], want[4:], rtol=0, atol=0, equal_nan=True)
    assert torch.equal(q.cpu()[4:], n[4:])
    W, ws = weight(3, 64, 64)
    y = tclora.i8_product(tclora.I8Weight(W, ws), q, s, y_dtype=torch.float32)
    assert not y[0].any() and torch.isnan(y[1:4]).all()
    close(y[4:], product64(W, ws, n[4:], want[4:]), torch.float32)


@pytest.mark.parametrize("T", [1, 3, 4, 5])
def test_linear_special_rows(T):
    """Zero rows, infinities and NaNs through the one-launch form and the two
    launches: each row on its own."""
    x = acts(4, T, 96, torch.float32)
    x[0] = 0
    if T > 1:
        x[1, 3], x[T - 1, 95] = float("nan"), -float("inf")
    W, ws = weight(4, 40, 96)
    y = tclora.i8_linear(tclora.I8Weight(W, ws), x, y_dtype=torch.float32)
    n, s = quant64(x)
    assert not y[0].any()
    close(y, product64(W, ws, n, s), torch.float32)


def test_quant_leaves_columns_behind_d():
    x = acts(1, 4, 48, torch.bfloat16)
    buf = torch.full((4, 80), 7, dtype=torch.int8, device=DEV)
    tclora.i8_quant(x, q=buf[:, :48])
    assert (buf[:, 48:] == 7).all()
    assert torch.equal(buf[:, :48].cpu(), quant64(x)[0])


SHAPES = [(1, 16, 8), (1, 4096, 1024), (2, 48, 40), (7, 144, 136), (16, 256, 1000),
          (17, 1040, 264), (32, 4112, 512), (33, 512, 4104), (64, 4096, 4096), (65, 336, 1032),
          (129, 2064, 72), (177, 1424, 520), (256, 128, 256), (257, 144, 136), (300, 4112, 392),
          (515, 400, 1032), (1025, 272, 264), (2048, 528, 264), (260, 64, 4104)]


@pytest.mark.parametrize("pack", [True, False])
@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_in,d_out", SHAPES)
def test_product(T, d_in, d_out, y, pack):
    W, ws = weight(T + d_out, d_out, d_in, full=True)
    g = torch.Generator().manual_seed(T * d_in)
    q = torch.randint(-128, 128, (T, d_in), generator=g, dtype=torch.int32).to(torch.int8).to(DEV)
    s = (torch.rand(T, generator=g) + 0.01).to(DEV)
    got = tclora.i8_product(tclora.I8Weight(W, ws, pack), q, s, y_dtype=DT[y])
    close(got, product64(W, ws, q, s), DT[y])


@pytest.mark.parametrize("T", [3, 70, 300])
def test_product_strides_and_bounds(T):
    """Rows wider than the operands: the padding of q is not read into the
    sums, the padding of y and the rows behind it stay as they were."""
    d_in, d_out = 208, 136
    W, ws = weight(9, d_out, d_in)
    qb = torch.full((T + 2, 256), 99, dtype=torch.int8, device=DEV)
    q = qb[:T, :d_in]
    q.copy_(torch.randint(-127, 128, (T, d_in), dtype=torch.int32))
    s = torch.rand(T, device=DEV) + 0.1
    yb = torch.full((T + 3, 160), -5.0, device=DEV)
    tclora.i8_product(tclora.I8Weight(W, ws), q, s, y=yb[:T, :d_out])
    close(yb[:T, :d_out], product64(W, ws, q, s), torch.float32)
    assert (yb[T:] == -5).all() and (yb[:, d_out:] == -5).all()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_product_longest_rows_do_not_overflow(T):
    d_in = 131056
    W = torch.full((8, d_in), -128, dtype=torch.int8, device=DEV)
    q = torch.full((T, d_in), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(8, device=DEV)
    y = tclora.i8_product(tclora.I8Weight(W, one), q, torch.ones(T, device=DEV),
                          y_dtype=torch.float32)
    assert (y == float(d_in) * 16384).all()


@pytest.mark.parametrize("x,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,d_in,d_out", [(1, 4096, 1024), (1, 16, 8), (2, 80, 24), (3, 14336, 264),
                                          (2, 16384, 40), (2, 16400, 40), (4, 16384, 40), (4, 8208, 1032),
                                          (5, 272, 136), (64, 1024, 4096),
                                          (300, 1040, 520), (4097, 400, 4104),
                                          (2100, 48, 8200)])
def test_linear(T, d_in, d_out, x, y):
    W, ws = weight(5, d_out, d_in)
    a = acts(T, T, d_in, DT[x])
    got = tclora.i8_linear(tclora.I8Weight(W, ws), a, y_dtype=DT[y])
    n, s = quant64(a)
    close(got, product64(W, ws, n, s), DT[y])


@pytest.mark.parametrize("d_out,d_in", [(8, 16), (16, 64), (40, 80), (264, 1040)])
def test_packed_copy(d_out, d_in):
    """The documented order, zeros behind rows and columns."""
    W, ws = weight(1, d_out, d_in, full=True)
    got = tclora.I8Weight(W, ws).W_p.view(torch.int8).cpu()
    R, C = -(-d_out // 16), -(-d_in // 64)
    want = torch.zeros(R * 16, C * 64, dtype=torch.int8)
    want[:d_out, :d_in] = W.cpu()
    want = want.view(R, 16, C, 4, 16).permute(0, 2, 3, 1, 4)  # [R, C, chunk, row, 16]
    assert torch.equal(got, want.reshape(-1))


def test_empty_batch_and_empty_weight():
    W, ws = weight(5, 16, 32)
    w = tclora.I8Weight(W, ws)
    assert tclora.i8_linear(w, torch.empty(0, 32, device=DEV)).shape == (0, 16)
    w0 = tclora.I8Weight(W[:0], ws[:0])
    assert tclora.i8_linear(w0, acts(1, 3, 32, torch.float32)).shape == (3, 0)


@pytest.mark.parametrize("T", [8, 300])
def test_linear_in_a_graph_and_on_another_stream(T):
    W, ws = weight(6, 1032, 528)
    w = tclora.I8Weight(W, ws)
    x = acts(2, T, 528, torch.bfloat16)
    y = torch.empty(T, 1032, device=DEV)
    call = tclora.I8Call(w, x, y)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for i in range(4):
        x.copy_(acts(20 + i, T, 528, torch.bfloat16))
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        replayed = y.clone()
        eager = tclora.i8_linear(w, x, y_dtype=torch.float32)
        assert torch.equal(replayed, eager)
        n, s = quant64(x)
        close(replayed, product64(W, ws, n, s), torch.float32)


def test_results_repeat_bit_for_bit():
    W, ws = weight(8, 520, 2064)
    w = tclora.I8Weight(W, ws)
    for T in (9, 200, 700):
        x = acts(T, T, 2064, torch.bfloat16)
        a = tclora.i8_linear(w, x)
        # a token's row does not depend on its batch
        b = tclora.i8_linear(w, x[3:9])
        assert torch.equal(tclora.i8_linear(w, x), a) and torch.equal(a[3:9], b)
        assert torch.equal(tclora.i8_linear(w, x[3:6]), a[3:6])


@pytest.mark.parametrize("T,d_out", [(1, 72), (2, 72), (40, 72), (2100, 1288)])
def test_scales_at_any_float(T, d_out):
    """Channel scales need no more than their own alignment."""
    W, ws = weight(9, d_out, 96)
    off = torch.empty(d_out + 1, device=DEV)[1:]
    off.copy_(ws)
    assert off.data_ptr() % 16 == 4
    x = acts(3, T, 96, torch.bfloat16)
    assert torch.equal(tclora.i8_linear(tclora.I8Weight(W, off), x, y_dtype=torch.float32),
                       tclora.i8_linear(tclora.I8Weight(W, ws), x, y_dtype=torch.float32))


@pytest.mark.parametrize("raw", [False, True])
def test_another_stream_leaves_freed_memory_to_its_readers(raw):
    """Memory that the current stream still reads may be handed to a call on
    another stream, which must not write it before that."""
    W, ws = weight(10, 2048, 256)
    w = tclora.I8Weight(W, ws)
    x = acts(4, 512, 256, torch.bfloat16)
    want = tclora.i8_linear(w, x)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.full((512, 2048), 3.0, dtype=torch.bfloat16, device=DEV)
    torch.cuda._sleep(20_000_000)
    copy = old.clone()
    del old  # (the allocator hands the block to the next of its size)
    got = tclora.i8_linear(w, x, stream=st.cuda_stream if raw else st)
    torch.cuda.synchronize()
    assert bool((copy == 3.0).all()) and torch.equal(got, want)


@pytest.mark.parametrize("T,d_out", [(300, 12000), (1030, 4104), (2300, 4096), (4100, 4096),
                                     (4400, 4072), (5200, 4096), (600, 32768),
                                     (72, 14336), (100, 14328), (333, 4096), (560, 4088)])
def test_tiles_of_every_size_and_split_batches(T, d_out):
    """Batches whose tokens go to one kernel or, past a whole round of large
    tiles, to two."""
    W, ws = weight(11, d_out, 80)
    x = acts(5, T, 80, torch.bfloat16)
    y = tclora.i8_linear(tclora.I8Weight(W, ws), x, y_dtype=torch.float32)
    n, s = quant64(x)
    close(y, product64(W, ws, n, s), torch.float32)


def test_workspace_outlives_its_call_on_another_current_stream():
    """A call made on one stream, run on another and dropped: its workspace is
    not handed out before the work has run."""
    W, ws = weight(12, 256, 4096)
    w = tclora.I8Weight(W, ws)
    x = acts(6, 512, 4096, torch.bfloat16)
    want = tclora.i8_linear(w, x)
    y = torch.zeros_like(want)
    call = tclora.I8Call(w, x, y)
    n, at = call.ws.numel(), call.ws.data_ptr()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        call()
    del call
    junk = [torch.full((n,), 85, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert all(j.data_ptr() != at for j in junk)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_two_calls_at_once():
    """Calls on two streams share the weight, each with a workspace of its own."""
    W, ws = weight(13, 1024, 2048)
    w = tclora.I8Weight(W, ws)
    xs = [acts(7 + i, 700, 2048, torch.bfloat16) for i in range(2)]
    want = [tclora.i8_linear(w, x) for x in xs]
    ys = [torch.zeros_like(o) for o in want]
    calls = [tclora.I8Call(w, x, y) for x, y in zip(xs, ys)]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, c in zip(st, calls):
            c(s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, o) for y, o in zip(ys, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(7, 1024), (7, 1040), (5, 2048), (1027, 2064), (3, 4112), (512, 4112),
                                 (513, 4112), (2, 33008), (515, 16400)])
def test_quant_by_rows_of_every_length(T, d, dtype):
    """Each number of waves a row, rows beyond what they keep, odd row counts."""
    test_quant_is_the_definition(T, d, dtype)


@pytest.mark.parametrize("T", [1, 2, 20, 40, 300, 2100])
@pytest.mark.parametrize("d_in", [16, 32, 48])
def test_rows_shorter_than_a_block(T, d_in):
    """Operands in plain rows, whose lanes past the row's end find no block of
    their own, in every kernel."""
    d_out = 8200 if T == 2100 else 264
    W, ws = weight(14, d_out, d_in, full=True)
    x = acts(8, T, d_in, torch.bfloat16)
    n, s = quant64(x)
    w = tclora.I8Weight(W, ws, pack=False)
    want = product64(W, ws, n, s)
    close(tclora.i8_linear(w, x, y_dtype=torch.float32), want, torch.float32)
    close(tclora.i8_product(w, n.to(DEV), s.to(DEV), y_dtype=torch.float32), want, torch.float32)


@pytest.mark.parametrize("d", [128, 4096])
def test_quant_next_to_ties_at_small_scales(d):
    """Scales around and below the smallest normal number: the quotients
    nearest to every tie, on it and a step of fp32 to either side."""
    r = np.random.default_rng(15)
    rows = []
    for lo, hi in ((-149, -140), (-140, -132), (-132, -126), (-126, -125), (-125, -99)):
        for _ in range(40):
            top = np.float32(127 * 2.0 ** r.uniform(lo, hi))
            s = np.float32(np.float64(top) / 127)
            v = (np.float64(s) * (r.integers(0, 127, d - 1) + 0.5)).astype(np.float32)
            v = np.where(r.random(d - 1) < 0.5, np.nextafter(v, np.float32(1)), v)
            v = np.where(r.random(d - 1) < 0.5, np.nextafter(v, np.float32(0)), v)
            v = np.minimum(v, top) * r.choice([-1, 1], d - 1).astype(np.float32)
            rows.append(np.concatenate([[top], v]).astype(np.float32))
    rows.append(np.zeros(d, np.float32))
    rows[-1][:2] = 2.5094301558894677e-38, 2.1636421034566686e-38
    x = torch.from_numpy(np.stack(rows)).to(DEV)
    q, s = tclora.i8_quant(x)
    # (the real quotient: an fp64 division rounds the neighbours of some ties)
    want = (x.double().cpu().abs().amax(1) / 127).float()
    assert torch.equal(s.cpu().view(torch.int32), want.view(torch.int32))
    xi = (x.cpu().numpy().astype(np.float64) * 2.0 ** 149).astype(np.int64)
    si = (want.numpy().astype(np.float64) * 2.0 ** 149).astype(np.int64)[:, None]
    a = np.abs(xi)
    n, rem = a // np.maximum(si, 1), a % np.maximum(si, 1)
    n = n + ((2 * rem > si) | ((2 * rem == si) & (n % 2 == 1)))
    n = np.where(si > 0, np.sign(xi) * np.minimum(n, 127), 0)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), n)


def test_quant_of_as_many_tokens_as_are_allowed():
    """2^24 - 1 tokens of rows longer than a pair of waves takes at a time."""
    T, d = (1 << 24) - 1, 2064
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 104 GB of memory")
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 1, 4095, 1 << 23, (1 << 23) + 1, T - 2, T - 1], device=DEV)
    x[at] = acts(16, len(at), d, torch.bfloat16)
    q, s = tclora.i8_quant(x)
    n, want = quant64(x[at])
    assert torch.equal(q[at].cpu(), n) and torch.equal(s[at].cpu(), want)
    rows = torch.ones(T, dtype=torch.bool, device=DEV)
    rows[at] = False
    assert not s[rows].any()
    del x, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,d_in,d_out", [(33, 4096, 24576), (64, 4112, 32768), (49, 4096, 32776),
                                          (64, 4080, 24584)])
def test_few_tokens_of_wide_weights(T, d_in, d_out):
    """Both sides of the sizes where blocks and tiles change places."""
    W, ws = weight(17, d_out, d_in)
    x = acts(9, T, d_in, torch.bfloat16)
    n, s = quant64(x)
    # (sums of products of 8-bit numbers: exact in 64 bits on the GPU as well)
    sums = (n.to(DEV).double() @ W.double().t()).cpu()
    want = sums * s.double()[:, None] * ws.double().cpu()
    close(tclora.i8_linear(tclora.I8Weight(W, ws), x, y_dtype=torch.float32), want, torch.float32)
