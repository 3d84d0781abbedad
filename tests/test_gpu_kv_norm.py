"""tcl_kv_append_norm against the norm and the rotation in 64 bits.

A normed element x r w is computed in fp32.  The sum of squares has D / 8 + 4
additions in a row at most (16 products a lane, up to four joins, the order of
a lane's own 16): 20 roundings of 2^-24 of a sum of positive numbers, halved by
the root, with the division, the sum with eps, the reciprocal root (two units)
and two products: 10 + 1 + 1 + 2 + 2 = 16 roundings of 2^-24 relative to the
element's value.  The rotation then adds what it adds to the plain append
(2^-22 + 3 * 2^-24 relative to |a| + |b|), and the result is rounded to bf16.
"""
import pytest
import torch

from tenant_composite_lora_amd import tclora
from test_gpu_kv import DEV, DT, FP32, HALF, inv_freq, make, rotate64

pytestmark = pytest.mark.gpu
NORM = 16 * 2.0 ** -24


def norm64(x, w, eps, D):
    """x [T, heads * D] normed by head in 64 bits, on the CPU."""
    x = x.double().cpu().reshape(x.shape[0], -1, D)
    if w is None:
        return x
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()


def check_normed(got, x, w, eps, pos, inv, D, inter):
    n = norm64(x, w, eps, D)
    want, mag = rotate64(n.flatten(1), pos, inv, D, inter)
    got = got.double().cpu().reshape(want.shape)
    base = torch.maximum(mag, n.abs())
    tol = (mag * FP32 + (0 if w is None else base * NORM)) * (1 + HALF) + want.abs() * HALF
    finite = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan())
    err = ((got - want).abs() - tol)[finite]
    assert err.numel() == 0 or float(err.max()) <= 2.0 ** -130, float(err.max())


def run_and_check(cache, rows, slot, pos, inv, wq, wk, eps=1e-6, inter=False, live=None):
    q, k, v = rows
    D, T = cache.head_dim, k.shape[0]
    K0, V0 = cache.K.clone(), cache.V.clone()
    qo = tclora.kv_append(cache, k, v, pos, slot, tclora.Rope(inv, inter), q=q,
                          norm=tclora.HeadNorm(wq, wk, eps))
    if live is None:
        live = torch.ones(T, dtype=torch.bool, device=slot.device)
    check_normed(qo, q, wq, eps, pos, inv, D, inter)
    s = slot[live]
    page, off = s // cache.page_size, s % cache.page_size
    if s.numel():
        check_normed(cache.K[page, off].flatten(1), k[live], wk, eps, pos[live], inv, D, inter)
        assert torch.equal(cache.V[page, off].flatten(1), v[live].to(torch.bfloat16))
    K1, V1 = cache.K.clone(), cache.V.clone()
    K1[page, off], V1[page, off] = K0[page, off], V0[page, off]
    for x, y in ((K1, K0), (V1, V0)):  # (bits: a NaN equals itself)
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def weights(seed, Hq, Hkv, D, by_head=False):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(*((h, D) if by_head else (D,)), generator=g)).to(DEV)
            for h in (Hq, Hkv)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter,by_head", [(False, False), (True, True)])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,head_major", [
    (1, 32, 8, 128, 128, 16, True), (1, 1, 1, 16, 16, 1, False), (7, 14, 2, 64, 32, 32, False),
    (33, 6, 3, 96, 48, 64, True), (5, 4, 4, 256, 256, 128, True), (130, 3, 1, 80, 64, 8, False),
    (257, 8, 8, 48, 0, 1024, True), (64, 40, 8, 32, 32, 16, True), (3, 5, 5, 240, 16, 16, True),
    (2, 200, 100, 256, 128, 16, False)])
def test_append(T, Hq, Hkv, D, rot, page, head_major, inter, by_head, dtype):
    cache, rows, slot = make(T + D, T, Hq, Hkv, D, page, DT[dtype], head_major)
    pos = torch.randint(0, 100000, (T,), dtype=torch.int32, device=DEV)
    run_and_check(cache, rows, slot, pos, inv_freq(rot) if rot else None,
                  *weights(T, Hq, Hkv, D, by_head), inter=inter)


@pytest.mark.parametrize("which", ["q", "k", "none"])
def test_one_side_only(which):
    cache, rows, slot = make(3, 19, 6, 2, 128, 16, torch.float32)
    wq, wk = weights(3, 6, 2, 128)
    run_and_check(cache, rows, slot, torch.arange(19, dtype=torch.int32, device=DEV), inv_freq(128),
                  wq if which == "q" else None, wk if which == "k" else None)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e-10, 1e15, 1e19, 1e30])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_heads_whose_squares_leave_fp32(scale, eps):
    cache, rows, slot = make(4, 16, 4, 2, 96, 16, torch.float32)
    rows = [(r * scale) for r in rows[:2]] + [rows[2]]
    run_and_check(cache, rows, slot, torch.arange(16, dtype=torch.int32, device=DEV), inv_freq(64),
                  *weights(4, 4, 2, 96), eps=eps)


def test_zeros_and_what_is_not_finite_stay_in_their_head():
    cache, (q, k, v), slot = make(5, 8, 4, 2, 64, 16, torch.bfloat16)
    q[0, :64] = 0
    q[1, 64] = float("inf")
    q[2, 130] = float("nan")
    k[3, :] = 0
    k[4, 5] = float("-inf")
    pos = torch.zeros(8, dtype=torch.int32, device=DEV)
    run_and_check(cache, (q, k, v), slot, pos, None, *weights(5, 4, 2, 64))
    # without eps a head of zeros has no norm
    run_and_check(cache, (q, k, v), slot, pos, None, *weights(5, 4, 2, 64), eps=0.0)


def test_padding_strides_in_place():
    cache, (q, k, v), slot = make(7, 40, 6, 2, 64, 32, torch.bfloat16, pad=8, gap=8)
    slot[::3] = -1
    slot[1] = cache.n_pages * cache.page_size
    live = (slot >= 0) & (slot < cache.n_pages * cache.page_size)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    wq, wk = weights(7, 6, 2, 64)
    run_and_check(cache, (q, k, v), slot, pos, inv_freq(64), wq, wk, live=live)
    norm, rope = tclora.HeadNorm(wq, wk), tclora.Rope(inv_freq(64))
    want = tclora.kv_append(cache, k, v, pos, slot, rope, q=q, norm=norm)
    K = cache.K.clone()
    assert tclora.kv_append(cache, k, v, pos, slot, rope, norm=norm) is None
    assert torch.equal(cache.K, K)
    assert tclora.kv_append(cache, k, v, pos, slot, rope, q=q, q_out=q, norm=norm) is q
    assert torch.equal(q, want)


def test_weights_by_head_without_queries():
    cache, (q, k, v), slot = make(12, 9, 6, 2, 64, 16, torch.bfloat16)
    pos, rope = torch.arange(9, dtype=torch.int32, device=DEV), tclora.Rope(inv_freq(64))
    norm = tclora.HeadNorm(*weights(12, 6, 2, 64, True))
    tclora.kv_append(cache, k, v, pos, slot, rope, q=q, norm=norm)
    K = cache.K.clone()
    cache.K.zero_()
    assert tclora.kv_append(cache, k, v, pos, slot, rope, norm=norm) is None
    page, off = slot // 16, slot % 16
    assert torch.equal(cache.K[page, off], K[page, off])


def test_empty_batch():
    cache, (q, k, v), slot = make(9, 0, 4, 2, 64, 16, torch.bfloat16)
    out = tclora.kv_append(cache, k, v, slot.to(torch.int32), slot, q=q,
                           norm=tclora.HeadNorm(*weights(9, 4, 2, 64)))
    assert out.shape == (0, 256)


def test_graph_replays_follow_the_inputs():
    cache, (q, k, v), slot = make(10, 16, 8, 2, 128, 16, torch.bfloat16)
    pos = torch.arange(16, dtype=torch.int32, device=DEV)
    inv, norm = inv_freq(128), tclora.HeadNorm(*weights(10, 8, 2, 128))
    call = tclora.AppendCall(cache, k, v, pos, slot, tclora.Rope(inv), q=q, norm=norm)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call()
    for i in range(4):
        gen = torch.Generator().manual_seed(i)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen))
        norm.w_q.add_(0.1)
        pos.add_(1)
        slot.copy_(torch.randperm(cache.n_pages * 16, generator=gen)[:16])
        K0, V0 = cache.K.clone(), cache.V.clone()
        g.replay()
        torch.cuda.synchronize()
        K1, V1, q1 = cache.K.clone(), cache.V.clone(), call.q_out.clone()
        cache.K.copy_(K0), cache.V.copy_(V0)
        eager = tclora.kv_append(cache, k, v, pos, slot, tclora.Rope(inv), q=q, norm=norm)
        assert torch.equal(eager, q1) and torch.equal(cache.K, K1) and torch.equal(cache.V, V1)


def test_binding_refusals():
    cache, (q, k, v), slot = make(11, 4, 4, 2, 64, 16, torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    wq, wk = weights(11, 4, 2, 64, True)
    for bad in ((wq[:3], wk), (wq, wk[:, :32].contiguous()), (wk, wk), (wq, wk[0][:16].contiguous()),
                (wq.cpu(), wk)):
        with pytest.raises(ValueError):
            tclora.kv_append(cache, k, v, pos, slot, q=q, norm=tclora.HeadNorm(*bad))
    with pytest.raises(ValueError):
        tclora.HeadNorm(wq.t(), wk)
    with pytest.raises(TypeError):
        tclora.HeadNorm(wq.to(torch.bfloat16), wk)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(tclora.TclError):
            tclora.kv_append(cache, k, v, pos, slot, q=q, norm=tclora.HeadNorm(wq, wk, eps))
