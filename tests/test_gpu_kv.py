"""tcl_kv_append against the rotation in 64 bits.

Copied elements are rounded to bf16 once (bf16 sources stay bit for bit).  A
rotated element a cos - b sin is computed in fp32: the angle's sine and cosine
are off by 2^-22 at most (the angle's own rounding to fp32, 2^-24 * pi, and
two units of the functions), two products and their difference round at
2^-24 each, all relative to |a| + |b|; then one rounding to bf16, 2^-8 at most
relative to the value.
"""
import numpy as np
import pytest
import torch

from tenant_composite_lora_amd import tclora

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FP32 = 2.0 ** -22 + 3 * 2.0 ** -24
HALF = torch.finfo(torch.bfloat16).eps / 2


def rotate64(x, pos, inv, D, inter):
    """(rotated, |a| + |b| of every element) in 64 bits, on the CPU."""
    x = x.double().cpu().reshape(x.shape[0], -1, D)
    out, mag = x.clone(), x.abs()
    if inv is None:
        return out, mag * 0
    r = 2 * inv.numel()
    ang = pos.double().cpu()[:, None, None] * inv.double().cpu()
    ia = torch.arange(0, r, 2) if inter else torch.arange(r // 2)
    ib = ia + 1 if inter else ia + r // 2
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * ang.cos() - b * ang.sin()
    out[..., ib] = b * ang.cos() + a * ang.sin()
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    mag[..., r:] = 0
    return out, mag


def check_rotated(got, x, pos, inv, D, inter):
    want, mag = rotate64(x, pos, inv, D, inter)
    got = got.double().cpu().reshape(want.shape)
    err = (got - want).abs() - (mag * FP32 * (1 + HALF) + want.abs() * HALF)
    assert float(err.max()) <= 2.0 ** -130, float(err.max())


def make(seed, T, Hq, Hkv, D, page, dtype, head_major=True, pad=0, spare=2, gap=0):
    g = torch.Generator().manual_seed(seed)
    n_pages = -(-max(T, 1) // page) + spare
    shape = [n_pages, Hkv, page, D + gap] if head_major else [n_pages, page, Hkv, D + gap]
    K, V = (torch.randn(shape, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    if head_major:
        K, V = K.transpose(1, 2), V.transpose(1, 2)
    K, V = K[..., :D], V[..., :D]
    rows = [torch.randn(T, h * D + pad, generator=g).to(dtype).to(DEV)[:, :h * D]
            for h in (Hq, Hkv, Hkv)]
    slot = torch.randperm(n_pages * page, generator=g)[:T].to(DEV)
    return tclora.KVCache(K, V), rows, slot


def inv_freq(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().to(DEV)


def run_and_check(cache, rows, slot, pos, inv, inter=False, live=None):
    q, k, v = rows
    D, T = cache.head_dim, k.shape[0]
    K0, V0 = cache.K.clone(), cache.V.clone()
    qo = tclora.kv_append(cache, k, v, pos, slot, tclora.Rope(inv, inter), q=q)
    if live is None:
        live = torch.ones(T, dtype=torch.bool, device=slot.device)
    check_rotated(qo, q, pos, inv, D, inter)
    s = slot[live]
    page, off = s // cache.page_size, s % cache.page_size
    if s.numel():
        check_rotated(cache.K[page, off].flatten(1), k[live], pos[live], inv, D, inter)
        assert torch.equal(cache.V[page, off].flatten(1), v[live].to(torch.bfloat16))
    # every other slot as it was
    K1, V1 = cache.K.clone(), cache.V.clone()
    K1[page, off], V1[page, off] = K0[page, off], V0[page, off]
    assert torch.equal(K1, K0) and torch.equal(V1, V0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,head_major", [
    (1, 32, 8, 128, 128, 16, True), (1, 1, 1, 16, 16, 1, False), (7, 14, 2, 64, 32, 32, False),
    (33, 6, 3, 96, 48, 64, True), (5, 4, 4, 256, 256, 128, True), (130, 3, 1, 128, 64, 8, False),
    (257, 8, 8, 64, 0, 1024, True), (64, 40, 8, 128, 128, 16, True)])
def test_append(T, Hq, Hkv, D, rot, page, head_major, inter, dtype):
    cache, rows, slot = make(T + D, T, Hq, Hkv, D, page, DT[dtype], head_major)
    pos = torch.randint(0, 100000, (T,), dtype=torch.int32, device=DEV)
    run_and_check(cache, rows, slot, pos, inv_freq(rot) if rot else None, inter)


@pytest.mark.parametrize("at", [0, 1, 1 << 20, (1 << 31) - 40])
def test_far_positions(at):
    cache, rows, slot = make(3, 32, 4, 2, 128, 16, torch.float32)
    pos = torch.arange(at, at + 32, dtype=torch.int32, device=DEV)
    run_and_check(cache, rows, slot, pos, inv_freq(128))


def test_negative_positions():
    cache, rows, slot = make(4, 16, 2, 2, 64, 16, torch.float32)
    run_and_check(cache, rows, slot, torch.arange(-16, 0, dtype=torch.int32, device=DEV),
                  inv_freq(64))


def test_padding_tokens_write_nothing():
    """Slots below 0 and behind the last page are padding."""
    cache, rows, slot = make(5, 40, 4, 2, 128, 16, torch.bfloat16)
    slot[::3] = -1
    slot[1] = cache.n_pages * cache.page_size
    slot[2] = 1 << 40
    slot[4] = -(1 << 62)
    live = (slot >= 0) & (slot < cache.n_pages * cache.page_size)
    run_and_check(cache, rows, slot, torch.arange(40, dtype=torch.int32, device=DEV),
                  inv_freq(128), live=live)
    cache, rows, slot = make(6, 4, 4, 2, 64, 16, torch.bfloat16)
    slot.fill_(-1)
    run_and_check(cache, rows, slot, torch.arange(4, dtype=torch.int32, device=DEV), inv_freq(64),
                  live=slot >= 0)


@pytest.mark.parametrize("head_major", [True, False])
def test_strides(head_major):
    """Wider rows of q, k, v and gaps between the cache's heads."""
    cache, rows, slot = make(7, 19, 6, 2, 64, 32, torch.float32, head_major, pad=8, gap=8)
    run_and_check(cache, rows, slot, torch.arange(19, dtype=torch.int32, device=DEV),
                  inv_freq(64))


def test_queries_in_place_and_none():
    cache, (q, k, v), slot = make(8, 21, 6, 2, 64, 16, torch.bfloat16)
    pos, rope = torch.arange(21, dtype=torch.int32, device=DEV), tclora.Rope(inv_freq(64))
    want = tclora.kv_append(cache, k, v, pos, slot, rope, q=q)
    K, V = cache.K.clone(), cache.V.clone()
    cache.K.zero_(), cache.V.zero_()
    assert tclora.kv_append(cache, k, v, pos, slot, rope) is None
    page, off = slot // 16, slot % 16
    assert torch.equal(cache.K[page, off], K[page, off])
    assert torch.equal(cache.V[page, off], V[page, off])
    assert tclora.kv_append(cache, k, v, pos, slot, rope, q=q, q_out=q) is q
    assert torch.equal(q, want)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: its last page."""
    n_pages = (1 << 31) // (1024 * 128) + 3
    K = torch.zeros(n_pages, 1024, 1, 128, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    k = torch.randn(3, 128, device=DEV).to(torch.bfloat16)
    last = n_pages * 1024
    slot = torch.tensor([last - 1, last - 1025, last], device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    tclora.kv_append(tclora.KVCache(K, V), k, k, pos, slot)
    for cache in (K, V):
        flat = cache.view(-1, 128)
        assert torch.equal(flat[last - 1], k[0]) and torch.equal(flat[last - 1025], k[1])
        flat[last - 1].zero_(), flat[last - 1025].zero_()
        assert not cache.view(torch.int16).any()


def test_empty_batch():
    cache, rows, slot = make(9, 0, 4, 2, 64, 16, torch.bfloat16)
    q, k, v = rows
    out = tclora.kv_append(cache, k, v, slot.to(torch.int32), slot, q=q)
    assert out.shape == (0, 256)


def test_graph_replays_follow_the_inputs():
    cache, (q, k, v), slot = make(10, 16, 8, 2, 128, 16, torch.bfloat16)
    pos = torch.arange(16, dtype=torch.int32, device=DEV)
    inv = inv_freq(128)
    call = tclora.AppendCall(cache, k, v, pos, slot, tclora.Rope(inv), q=q)
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
        pos.add_(1)
        slot.copy_(torch.randperm(cache.n_pages * 16, generator=gen)[:16])
        K0, V0 = cache.K.clone(), cache.V.clone()
        g.replay()
        torch.cuda.synchronize()
        K1, V1, q1 = cache.K.clone(), cache.V.clone(), call.q_out.clone()
        cache.K.copy_(K0), cache.V.copy_(V0)
        eager = tclora.kv_append(cache, k, v, pos, slot, tclora.Rope(inv), q=q)
        assert torch.equal(eager, q1) and torch.equal(cache.K, K1) and torch.equal(cache.V, V1)


def test_binding_refusals():
    cache, (q, k, v), slot = make(11, 4, 4, 2, 64, 16, torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (dict(k=k[:3]), dict(v=v[:, :64]), dict(pos=pos[:2]), dict(slot=slot.to(torch.int32)),
                dict(pos=pos.long()), dict(q=q[:, :100]), dict(q=q[:2]), dict(pos=pos.cpu()),
                dict(q_out=q)):
        a = {**dict(k=k, v=v, pos=pos, slot=slot), **bad}
        with pytest.raises(ValueError):
            tclora.kv_append(cache, a["k"], a["v"], a["pos"], a["slot"], q=a.get("q"),
                             q_out=a.get("q_out"))
    with pytest.raises(TypeError):
        tclora.kv_append(cache, k, v.float(), pos, slot)
    with pytest.raises(TypeError):
        tclora.KVCache(cache.K.float(), cache.V.float())
    with pytest.raises(ValueError):
        tclora.KVCache(cache.K, cache.V.contiguous().clone())
    with pytest.raises(ValueError):
        one = cache.K[:, :, :1].expand(-1, -1, 2, -1)
        tclora.KVCache(one, one)
