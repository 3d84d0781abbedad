"""tcl_i4_linear against the product with (n - z) s in 64 bits.

Tolerance.  A group's sums of x (16 + n) and of x are fp32: up to 2 L roundings
for L columns, each at most 2^-24 of a partial sum, which is at most P = 31 |x|_1
of the group (the second sum enters 16 + z times, and is at most |x|_1: (16 + z)
|x|_1).  The two are joined and added over the groups with a few more roundings
of numbers no larger than P s.  Roundings have independent signs, so that their
sum has a standard deviation below sqrt(2 L + 4) 2^-24 (31 + 16 + z) |x|_1 s a
group, groups add as squares, and eight deviations are allowed.  (Weights
rounded to bf16 would show: 2^-9 of each is some ten times as much.)  Then y is
rounded once: 2^-24 or 2^-8 of its value.
"""
import numpy as np
import pytest
import torch

from tenant_composite_lora_amd import tclora

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def weight(seed, d_out, d_in, group, zeros=False, full=False):
    """(W, scale, zero) on the GPU and the integers [d_out, d_in] on the CPU."""
    g = torch.Generator().manual_seed(seed)
    n = (torch.randint(0, 16, (d_out, d_in), generator=g) if full else
         (torch.randn(d_out, d_in, generator=g) * 2.7 + 7.5).round().clamp(0, 15)).to(torch.uint8)
    scale = (0.5 + torch.rand(d_out, d_in // group, generator=g)) * 0.01
    zero = torch.randint(0, 16, scale.shape, generator=g, dtype=torch.uint8) if zeros else None
    W = n[:, 0::2] | n[:, 1::2] << 4
    return (W.to(DEV), scale.to(DEV), None if zero is None else zero.to(DEV)), n


def acts(seed, T, d):
    g = torch.Generator().manual_seed(1000 + seed)
    x = torch.randn(T, d, generator=g) * (1 + 11 * (torch.rand(d, generator=g) < 0.02))
    return x.to(torch.bfloat16).to(DEV)


def product64(w, n, x):
    """(y, bound of what comes before its rounding) in 64 bits, on the GPU."""
    _, scale, zero = w
    G = scale.shape[1]
    L = n.shape[1] // G
    z = torch.full_like(scale, 8).double() if zero is None else zero.double()
    s = scale.double()
    xd = x.double()
    w64 = ((n.to(DEV).double().view(len(n), G, L) - z[..., None]) * s[..., None]).view(len(n), -1)
    norm = xd.abs().view(len(x), G, L).sum(-1)
    dev = (norm.square() @ ((47 + z) * s).square().T).sqrt()
    return xd @ w64.T, 8 * (2 * L + 4) ** 0.5 * 2.0 ** -24 * dev


def close(got, want, tol):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - want).abs() - (tol * (1 + half) + want.abs() * half)
    assert err.numel() == 0 or float(err.max()) <= 2.0 ** -130, float(err.max())


CASES = [(1, 4096, 1024, 128), (1, 32, 8, 32), (2, 96, 40, 32), (7, 128, 16, 128), (16, 4096, 4096, 64),
         (17, 1056, 264, 32), (23, 14336, 512, 32), (32, 576, 1000, 64), (33, 4096, 14336, 128),
         (64, 2048, 2056, 512), (65, 224, 136, 32), (100, 1280, 1280, 256), (130, 4096, 520, 128),
         (177, 448, 4096, 64), (257, 1024, 264, 1024), (300, 160, 3000, 32), (513, 2048, 1032, 128),
         (1000, 960, 776, 64)]


@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,d_in,d_out,group", CASES)
def test_linear(T, d_in, d_out, group, zeros, y):
    w, n = weight(T + d_in, d_out, d_in, group, zeros, full=T % 2 == 1)
    x = acts(T, T, d_in)
    close(tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=DT[y]), *product64(w, n, x))


@pytest.mark.parametrize("T", [1, 8, 15, 16, 24, 31, 47, 48, 63, 64, 95, 128, 129, 192, 255, 256, 384, 640, 2049])
@pytest.mark.parametrize("d_out", [8, 520, 4096])
def test_tokens_and_channels_around_the_tiles(T, d_out):
    w, n = weight(T, d_out, 384, 128, True)
    x = acts(T, T, 384)
    close(tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32), *product64(w, n, x))


# (calls that take tiles of 64 and of 128 tokens, whole and ragged, blocks of
# three widths, and columns split over workgroups)
@pytest.mark.parametrize("T,d_out", [(1024, 4096), (1000, 4000), (2048, 4096), (2030, 4104), (500, 14336),
                                     (700, 7000), (33, 6200), (64, 14336), (300, 2600)])
@pytest.mark.parametrize("d_in,group", [(96, 32), (192, 64), (640, 128), (768, 384), (64, 64), (32, 32)])
def test_many_tokens(T, d_out, d_in, group):
    w, n = weight(T + d_in, d_out, d_in, group, d_in % 3 == 0, full=True)
    x = acts(T, T, d_in)
    y = torch.full((T + 1, d_out), 7.0, device=DEV)
    tclora.i4_linear(tclora.I4Weight(*w), x, y=y[:T])
    close(y[:T], *product64(w, n, x))
    assert (y[T] == 7).all()


@pytest.mark.parametrize("T", [17, 40, 64])
@pytest.mark.parametrize("d_in,d_out,group", [(8192, 1024, 128), (14336, 72, 32), (9216, 2048, 64),
                                              (16128, 4096, 384), (8224, 520, 32)])
def test_long_rows(T, d_in, d_out, group):
    w, n = weight(T, d_out, d_in, group, T == 40)
    x = acts(T, T, d_in)
    close(tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32), *product64(w, n, x))


@pytest.mark.parametrize("T", [1, 20, 64, 200])
@pytest.mark.parametrize("d_in", [32, 64, 96, 160, 224, 416, 1120])
def test_rows_that_end_inside_a_block(T, d_in):
    """Columns behind d_in hold NaNs: they are not part of any product."""
    w, n = weight(d_in, 72, d_in, 32, True)
    wide = torch.full((T, d_in + 136), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :d_in] = acts(T, T, d_in)
    x = wide[:, :d_in]
    close(tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32), *product64(w, n, x))


@pytest.mark.parametrize("T,d_out", [(17, 25592), (64, 25592), (1000, 4088), (2040, 4088)])
@pytest.mark.parametrize("d_in,group", [(96, 32), (416, 32), (448, 64), (1152, 384)])
def test_laid_out_activations(T, d_out, d_in, group):
    """Wide outputs and many tokens: NaNs behind the rows, zero points up to
    255, scales of any size, rows that are not finite."""
    w, n = weight(T, d_out, d_in, group, True, full=True)
    W, s, z = w
    z.copy_(torch.randint(0, 256, z.shape, dtype=torch.uint8))
    s[0], s[1], s[2], s[3] = 0, -s[1], s[2] * 1e20, s[3] * 1e-30
    wide = torch.full((T, d_in + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    x = wide[:, :d_in].copy_(acts(T, T, d_in))
    x[T // 2, 5], x[1, d_in - 1] = float("inf"), float("nan")
    rest = [t for t in range(T) if t not in (1, T // 2)]
    y = tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32)
    close(y[rest], *product64(w, n, x[rest]))


@pytest.mark.parametrize("T", [3, 40, 70, 300])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_strides_and_bounds(T, y):
    d_in, d_out = 256, 136
    w, n = weight(9, d_out, d_in, 64, True)
    xb = torch.full((T + 2, d_in + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    yb = torch.full((T + 2, d_out + 8), 5.0, dtype=DT[y], device=DEV)
    xb[:T, :d_in] = acts(9, T, d_in)
    tclora.I4Call(tclora.I4Weight(*w), xb[:T, :d_in], yb[:T, :d_out])()
    close(yb[:T, :d_out], *product64(w, n, xb[:T, :d_in]))
    assert (yb[T:] == 5).all() and (yb[:, d_out:] == 5).all()


@pytest.mark.parametrize("T,d_in,d_out,group", [(3, 256, 72, 64), (20, 256, 72, 128), (20, 8192, 72, 128),
                                                (20, 256, 25600, 32), (20, 256, 25600, 128), (24, 256, 65536, 128)])
def test_offsets_beyond_32_bits(T, d_in, d_out, group):
    w, n = weight(19, d_out, d_in, group, True)
    far = (1 << 31) // 2 + 64 if T < 4 else 1 << 27
    x = torch.empty((T - 1) * far + d_in, dtype=torch.bfloat16, device=DEV).as_strided((T, d_in), (far, 1))
    y = torch.empty((T - 1) * far + d_out, dtype=torch.float32, device=DEV).as_strided((T, d_out), (far, 1))
    x.copy_(acts(19, T, d_in))
    tclora.I4Call(tclora.I4Weight(*w), x, y)()
    close(y.clone(), *product64(w, n, x.contiguous()))
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [5, 50, 200])
def test_rows_that_are_not_finite_stay_alone(T):
    w, n = weight(3, 264, 512, 128)
    x = acts(3, T, 512)
    x[1, 7] = float("inf")
    x[3, 300] = float("nan")
    x[4] = 0
    y = tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32)
    assert not torch.isfinite(y[[1, 3]]).any() and (y[4] == 0).all()
    rest = [i for i in range(T) if i not in (1, 3)]
    close(y[rest], *product64(w, n, x[rest]))


@pytest.mark.parametrize("T", [4, 64, 200])
def test_zero_points_and_scales_at_any_value(T):
    """Zero points up to 255, scales of both signs, of zero and far apart."""
    w, n = weight(4, 264, 640, 64, True, full=True)
    W, s, z = w
    z.copy_(torch.randint(0, 256, z.shape, dtype=torch.uint8))
    s[0] = 0
    s[1] *= -1
    s[2] *= 1e20
    s[3] *= 1e-30
    x = acts(4, T, 640)
    close(tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32), *product64(w, n, x))


@pytest.mark.parametrize("T", [3, 64, 200])
def test_activations_with_an_offset(T):
    """All of one sign, where the two sums of a group nearly cancel."""
    w, n = weight(5, 264, 1024, 128, full=True)
    x = (acts(5, T, 1024).abs() + 4).to(torch.bfloat16)
    close(tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32), *product64(w, n, x))


@pytest.mark.parametrize("T", [3, 64, 200, 2048])
@pytest.mark.parametrize("size", [1e-36, 1e-38, 3e-39, 1e30])
def test_activations_at_the_ends_of_their_range(T, size):
    """Next to and below the smallest normal number, with scales that bring the
    results back; and large ones."""
    w, n = weight(14, 4096 if T == 2048 else 264, 256, 64, True, full=True)
    w[1].mul_(1e30 if size < 1 else 1e-25)
    x = (acts(14, T, 256).double() * size).to(torch.bfloat16)
    y, tol = product64(w, n, x)
    # (what falls below 2^-149 in a sum is lost there: up to 2 L times, on both
    # sides of the correction)
    s = w[1].double().abs().sum(1)
    close(tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32), y,
          tol + 2.0 ** -149 * 2 * 64 * (1 + 16 + 255) * s)


def test_packed_copy_holds_the_weight():
    for d_out, d_in, group, zeros in ((40, 352, 32, True), (16, 128, 128, False), (8, 64, 64, True)):
        w, n = weight(6, d_out, d_in, group, zeros)
        p = tclora.I4Weight(*w).W_p.cpu().numpy()
        ct, kb, G = -(-d_out // 32), 2 * -(-d_in // 128), d_in // group
        want = np.zeros((ct, kb, 64, 4), np.uint32)
        full = np.zeros((ct * 32, kb * 64), np.uint32)
        full[:d_out, :d_in] = n.numpy()
        for lane in range(64):
            for i, eight in enumerate((0, 4, 2, 6)):
                k = 8 * (eight + lane // 32) + np.arange(kb) * 64
                rows = full[np.arange(ct) * 32 + lane % 32]
                u = np.zeros((ct, kb), np.uint64)
                for j in range(8):
                    u |= rows[:, k + j].astype(np.uint64) << np.uint64(3 + 4 * (j // 2) + 16 * (j % 2))
                want[:, :, lane, i] = (u | u >> np.uint64(32)).astype(np.uint32)
        nw = ct * kb * 1024
        assert np.array_equal(p[:nw].view(np.uint32).reshape(want.shape), want)
        s = np.zeros((ct * 32, G), np.float32)
        s[:d_out] = w[1].cpu().numpy()
        got = p[nw:nw + ct * G * 128].view(np.float32).reshape(ct, G, 32)
        assert np.array_equal(got, s.reshape(ct, 32, G).transpose(0, 2, 1))
        if zeros:
            z = np.full((ct * 32, G), 8, np.uint8)
            z[:d_out] = w[2].cpu().numpy()
            got = p[nw + ct * G * 128:nw + ct * G * 160].reshape(ct, G, 32)
            assert np.array_equal(got, z.reshape(ct, 32, G).transpose(0, 2, 1))


def test_empty_batch_and_empty_weight():
    w, _ = weight(7, 16, 64, 32)
    y = tclora.i4_linear(tclora.I4Weight(*w), acts(7, 0, 64))
    assert y.shape == (0, 16)
    w0 = tclora.I4Weight(w[0][:0], w[1][:0])
    assert tclora.i4_linear(w0, acts(7, 3, 64)).shape == (3, 0)


@pytest.mark.parametrize("T,d_in,d_out", [(1, 1024, 1032), (64, 1024, 1032), (300, 1024, 1032),
                                          (40, 8192, 1032), (600, 1024, 4096), (1024, 1024, 4096)])
def test_in_a_graph_and_bit_for_bit(T, d_in, d_out):
    w, n = weight(8, d_out, d_in, 128, True)
    p = tclora.I4Weight(*w)
    x = acts(8, T, d_in)
    y = torch.empty(T, d_out, device=DEV)
    call = tclora.I4Call(p, x, y)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for i in range(4):
        x.copy_(acts(20 + i, T, d_in))
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, tclora.i4_linear(p, x, y_dtype=torch.float32))
        close(got, *product64(w, n, x))


@pytest.mark.parametrize("d_in", [2048, 8192])
def test_two_calls_at_once(d_in):
    w, _ = weight(10, 2048, d_in, 128)
    p = tclora.I4Weight(*w)
    xs = [acts(30 + i, t, d_in) for i, t in enumerate((64, 300))]
    want = [tclora.i4_linear(p, x) for x in xs]
    calls = [tclora.I4Call(p, x, torch.empty_like(y)) for x, y in zip(xs, want)]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, c in zip(st, calls):
            c(s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.y, y) for c, y in zip(calls, want))


def test_a_token_does_not_depend_on_its_batch():
    """Rows of one batch size are the same wherever they stand in it."""
    w, _ = weight(11, 520, 1024, 64, True)
    p = tclora.I4Weight(*w)
    for T in (5, 40, 300):
        x = acts(11, T, 1024)
        y = tclora.i4_linear(p, x, y_dtype=torch.float32)
        perm = torch.randperm(T, device=DEV)
        assert torch.equal(tclora.i4_linear(p, x[perm], y_dtype=torch.float32), y[perm])


@pytest.mark.parametrize("d_in", [1024, 8192])
@pytest.mark.parametrize("raw", [False, True])
def test_on_another_stream(raw, d_in):
    """Weight, packed copy and result made on the way belong to the stream of
    the call, also when everything is dropped right behind it."""
    w, _ = weight(12, 512, d_in, 128, True)
    x = acts(12, 32, d_in)
    want = tclora.i4_linear(tclora.I4Weight(*w), x)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = st.cuda_stream if raw else st
    for _ in range(3):
        torch.cuda._sleep(2_000_000)
        junk = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (1 << 15, 1 << 18, 1 << 20)]
        kept = [j.clone() for j in junk]
        del junk
        p = tclora.I4Weight(*w, stream=s)
        got = tclora.i4_linear(p, x, stream=s)
        del p
        over = [torch.full((n,), 9, dtype=torch.uint8, device=DEV) for n in (1 << 15, 1 << 18, 1 << 20)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(bool((k == 7).all()) for k in kept)
        del got, over


def test_binding_refusals():
    (W, s, z), _ = weight(13, 16, 128, 32, True)
    p = tclora.I4Weight(W, s, z)
    x = acts(13, 4, 128)
    for bad in ((W.to(torch.int8), s, z), (W, s.double(), z), (W, s, z.int()), (W, s.to(torch.bfloat16), z)):
        with pytest.raises(TypeError):
            tclora.I4Weight(*bad)
    for bad in ((W[:, ::2], s, z), (W, s[:8], z), (W, s, z[:, :2]), (W, s[:, :3].contiguous(), None),
                (W, s.cpu(), z), (W, s.t(), None), (W[0], s, z)):
        with pytest.raises(ValueError):
            tclora.I4Weight(*bad)
    with pytest.raises(tclora.TclError) as e:  # a group of 16
        tclora.I4Weight(W, torch.ones(16, 8, device=DEV))
    assert e.value.code == tclora.EUNSUPPORTED
    with pytest.raises(TypeError):
        tclora.i4_linear(p, x.float())
    with pytest.raises(TypeError):
        tclora.i4_linear(p, x, y_dtype=torch.float16)
    with pytest.raises(ValueError):
        tclora.i4_linear(p, x[:, :64])
    with pytest.raises(ValueError):
        tclora.i4_linear(p, x, y=torch.empty(4, 8, device=DEV))
    with pytest.raises(ValueError):
        tclora.i4_linear(p, x, y=torch.empty(4, 16))
