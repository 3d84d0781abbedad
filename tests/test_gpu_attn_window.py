"""tcl_attn_window_apply against the softmax over each token's own set of
visible keys in 64 bits, key by key.  Tolerances are those of the attention
without windows (derived beside its tests): a row's error does not depend on
which keys it sees, only on their count through the sums bounded there."""
import numpy as np
import pytest
import torch

from tenant_composite_lora_amd import tclora
from test_gpu_attn import CHUNKS, DECODE, DEV, HALF, Batch

pytestmark = pytest.mark.gpu


class Windowed(Batch):
    def __init__(self, seed, groups, Hq, Hkv, D, page, window, sinks, **kw):
        self.window, self.sinks = window, sinks
        super().__init__(seed, groups, Hq, Hkv, D, page, **kw)

    def plan(self):
        return tclora.AttnPlan(self.cache, self.Hq, *self.table(), n_tokens=self.T,
                               window=self.window, sinks=self.sinks)

    def want(self, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        T, Hq, D, gq = self.T, self.Hq, self.D, self.Hq // self.Hkv
        o = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
        lse, tol = o[..., 0].clone(), o.clone()
        for s in range(len(self.seqs)):
            K, V = self.keys(self.Kh, s), self.keys(self.Vh, s)
            t0, t1 = int(self.seq_tok[s]), int(self.seq_tok[s + 1])
            n, L = t1 - t0, K.shape[0]
            for i in range(n):
                vis = max(0, L - n + i + 1)
                seen = [j for j in range(vis) if j >= vis - self.window or j < self.sinks]
                q = self.q[t0 + i].double().view(self.Hkv, gq, D)
                k, v = K[seen].transpose(0, 1), V[seen].transpose(0, 1)
                sc = (q @ k.transpose(1, 2)) * scale
                e = ((q.abs() @ k.abs().transpose(1, 2)) * abs(scale)).amax(-1) if vis else q[..., 0]
                E = (D + 2) * 2.0 ** -24 * e
                z = torch.logsumexp(sc, -1) if vis else torch.full((self.Hkv, gq), -float("inf"), dtype=torch.float64)
                w = torch.exp(sc - z[..., None]) if vis else sc
                ob, A = w @ v, w @ v.abs()
                o[t0 + i] = ob.reshape(Hq, D)
                lse[t0 + i] = z.reshape(Hq)
                tol[t0 + i] = ((2 * E[..., None] + 2.0 ** -19 + HALF) * A + HALF * ob.abs()).reshape(Hq, D)
        return o, lse, tol


def run(b, scale=None):
    plan = b.plan()
    assert plan.status() == tclora.OK
    o = torch.full((b.T, b.Hq * b.D), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((b.T, b.Hq), 77.0, device=DEV)
    tclora.attention(plan, b.qd, o=o, lse=lse, scale=scale)
    b.check(o, lse, scale)
    n = int(b.seq_tok[-1])
    assert (o[n:] == 77).all() and (lse[n:] == 77).all()
    return o


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 4), (65, 0), (130, 70), (400, 16)])
@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [
    (8, 2, 64, 16, True), (4, 4, 128, 16, False), (14, 2, 64, 32, False), (6, 2, 256, 16, True),
    (32, 1, 64, 16, True), (3, 1, 128, 1, False)])
@pytest.mark.parametrize("name", DECODE)
def test_decode(name, Hq, Hkv, D, page, head_major, window, sinks):
    run(Windowed(len(name) + D, DECODE[name], Hq, Hkv, D, page, window, sinks, head_major=head_major))


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (33, 1), (64, 64), (100, 130)])
@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [
    (8, 2, 64, 16, True), (4, 1, 128, 32, False), (14, 2, 64, 16, False), (3, 1, 256, 64, True),
    (4, 4, 128, 16, True)])
@pytest.mark.parametrize("name", CHUNKS)
def test_chunks(name, Hq, Hkv, D, page, head_major, window, sinks):
    run(Windowed(len(name) * D, CHUNKS[name], Hq, Hkv, D, page, window, sinks, head_major=head_major))


def test_long_chunks_and_prefixes():
    """Tiles whose sinks, windows and items lie many steps apart."""
    run(Windowed(50, [(1500, [(300, 900), (1, 700), (1, 3), (9, 2000)]), (4000, [(1, 5), (1, 9)] * 6)],
                 8, 2, 64, 16, 500, 70))
    run(Windowed(51, [(700, [(140, 140), (1, 1)]), (0, [(1, 5000)])], 4, 2, 128, 32, 1000, 900))


@pytest.mark.parametrize("gq", [1, 2, 5, 16, 17, 33, 128])
def test_heads_of_a_key_head(gq):
    run(Windowed(gq, [(90, [(1, 30), (1, 40), (4, 50)])], 2 * gq, 2, 64, 16, 50, 3))


@pytest.mark.parametrize("window", [5000, (1 << 31) - 1, 1 << 40])
def test_a_window_over_all_keys_is_no_window(window):
    """Bit for bit the attention without one."""
    for groups in (DECODE["several groups, one empty"], CHUNKS["short and long requests of a group"],
                   CHUNKS["more tokens than keys"]):
        b = Windowed(3, groups, 8, 2, 64, 16, window, 0)
        lse = [torch.zeros(b.T, 8, device=DEV) for _ in range(3)]
        want = tclora.attention(Batch.plan(b), b.qd, lse=lse[0])
        assert torch.equal(tclora.attention(b.plan(), b.qd, lse=lse[1]), want)
        b.window, b.sinks = 1, window
        assert torch.equal(tclora.attention(b.plan(), b.qd, lse=lse[2]), want)
        assert torch.equal(lse[0], lse[1]) and torch.equal(lse[0], lse[2])


def test_more_requests_and_groups_than_threads():
    r = np.random.default_rng(3)
    seqs = lambda n, q=1: [(q, q + int(x)) for x in r.integers(0, 8, n)]  # noqa: E731
    run(Windowed(31, [(int(p), seqs(30)) for p in r.integers(0, 40, 50)], 4, 2, 64, 16, 9, 2))
    run(Windowed(32, [(int(p), seqs(int(n))) for p, n in zip(r.integers(0, 9, 1100),
                                                              r.integers(0, 3, 1100))], 2, 1, 64, 8, 4, 1))
    run(Windowed(33, [(20, seqs(560, 3))], 64, 1, 64, 16, 6, 3))


def test_offsets_beyond_32_bits():
    b = Windowed(34, [(300, [(1, 90), (1, 70), (40, 100)])], 4, 2, 64, 32, 111, 5)
    want = tclora.attention(b.plan(), b.qd)
    b.check(want)
    pages, elems = b.cache.n_pages, 32 * 2 * 64
    big = (1 << 31) // elems + pages + 1
    K = torch.zeros(big, 2, 32, 64, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    K[big - pages:] = b.cache.K.transpose(1, 2)
    V[big - pages:] = b.cache.V.transpose(1, 2)
    t = b.table()
    for i in (3, 5):
        t[i] = torch.where(t[i] >= 0, t[i] + (big - pages), t[i])
    plan = tclora.AttnPlan(tclora.KVCache(K.transpose(1, 2), V.transpose(1, 2)), 4, *t, n_tokens=b.T,
                           window=111, sinks=5)
    assert plan.status() == tclora.OK
    assert torch.equal(tclora.attention(plan, b.qd), want)


def test_rows_behind_the_last_request_stay():
    run(Windowed(5, [(100, [(1, 4), (1, 9), (70, 80)])], 8, 2, 64, 16, 40, 4, pad_tokens=9))
    run(Windowed(5, [(0, [(0, 4)])], 8, 2, 64, 16, 2, 0, pad_tokens=3))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scale(scale):
    b = Windowed(6, [(150, [(1, 40), (1, 70), (20, 30)])], 4, 2, 64, 16, 33, 2)
    o = tclora.attention(b.plan(), b.qd, scale=scale)
    b.check(o, scale=scale)


@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [
    (8, 2, 64, 16, True), (4, 1, 128, 32, False), (3, 1, 256, 64, True), (32, 1, 128, 8, True)])
@pytest.mark.parametrize("where", ["V", "K"])
@pytest.mark.parametrize("window,sinks", [(20, 3), (90, 0)])
def test_infinities_and_nans_of_hidden_keys(where, Hq, Hkv, D, page, head_major, window, sinks):
    """Keys on both sides of the windows' and sinks' borders, and slots behind
    every length, hold infinities and NaNs: rows that do not see them are as
    ever, rows that do are what the sum gives in 64 bits."""
    b = Windowed(15, [(170, [(3, 60), (90, 100), (1, 9), (2, 70)]), (130, [(150, 20), (1, 0), (40, 70)])],
                 Hq, Hkv, D, page, window, sinks, head_major=head_major)
    X = b.Vh if where == "V" else b.Kh
    g = torch.Generator().manual_seed(1)
    kinds = torch.tensor([float("nan"), float("inf"), -float("inf")])
    used = torch.zeros(X.shape[:2], dtype=torch.bool)
    for pages, n, back in [(b.prefix_pages[i], p, (1, 25, 100, p - sinks, p - sinks + 1, p - 4))
                           for i, (p, _) in enumerate(b.groups)] + [
            (b.own_pages[i], s[1], (2, 21, 45, 61)) for i, s in enumerate(b.seqs)]:
        for j in range(n):
            used[int(pages[j // page]), j % page] = True
        for k in back:  # a few dimensions each
            if n > k > 0:
                d = torch.randint(0, D, (2,), generator=g)
                X[int(pages[(n - k) // page]), (n - k) % page, int(torch.randint(0, Hkv, (1,), generator=g)),
                  d] = kinds[torch.randint(0, 3, (2,), generator=g)].to(X.dtype)
    b.Kh[~used] = float("nan")
    b.Vh[~used] = float("nan")
    b.up(b.Kh, b.Vh)
    o = tclora.attention(b.plan(), b.qd).double().cpu().view(b.T, Hq, D)
    wo, _, tol = b.want()
    assert torch.equal(torch.isnan(o), torch.isnan(wo))
    inf = torch.isinf(wo)
    assert torch.equal(o[inf], wo[inf]) and bool(inf.any()) == (where == "V")
    ok = torch.isfinite(wo)
    # (a sink that is not finite reaches every row of its key head)
    assert bool(ok.any())
    assert float(((o - wo).abs() - tol)[ok].max()) <= 1e-30


def test_keys_before_the_windows_are_not_read():
    """Pages that no step touches hold NaNs everywhere: nothing changes."""
    b = Windowed(16, [(2000, [(1, 300), (1, 310), (70, 400)])], 8, 2, 64, 16, 130, 4)
    want = tclora.attention(b.plan(), b.qd)
    for pages, lo, hi in [(b.prefix_pages[0], 64, 2000)] + [(p, 0, 64) for p in b.own_pages]:
        for i in range(lo // 16, hi // 16):
            b.cache.K[int(pages[i])] = b.cache.V[int(pages[i])] = float("nan")
    b.check(want)
    assert torch.equal(tclora.attention(b.plan(), b.qd), want)


def test_a_plan_serves_its_window_only():
    b = Windowed(17, [(200, [(1, 40), (1, 90), (20, 30)])], 8, 2, 64, 16, 50, 4)
    plan, none = b.plan(), Batch.plan(b)
    o = torch.full((b.T, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    for p, limits in ((plan, (50, 5)), (plan, (51, 4)), (plan, ()), (none, (50, 4)), (none, (1 << 30, 0))):
        p.limits = limits
        tclora.attention(p, b.qd, o=o)
        assert (o == 3).all(), limits
    plan.limits = (50, 4)
    b.check(tclora.attention(plan, b.qd, o=o))


def test_bad_tables_change_nothing():
    for i, at, v in ((0, 1, 4), (1, 2, 2), (2, 0, -1), (4, 0, 65), (5, 0, -1), (3, 6, 200)):
        b = Windowed(9, [(100, [(1, 30), (2, 40)]), (50, [(1, 20)])], 4, 2, 64, 16, 10, 2)
        t = b.table()
        t[i].view(-1)[at] = v
        plan = tclora.AttnPlan(b.cache, 4, *t, n_tokens=b.T, window=10, sinks=2)
        o = torch.full((4, 256), 3.0, dtype=torch.bfloat16, device=DEV)
        assert plan.status() == tclora.EINVAL
        tclora.attention(plan, b.qd, o=o)
        assert (o == 3).all()


def test_remap_and_graph():
    """Batches of the same sizes mapped into one plan inside a graph while
    requests grow past their windows."""
    b = Windowed(10, [(200, [(1, 40), (1, 90), (1, 30)]), (64, [(1, 100), (1, 5)])], 8, 2, 128, 16, 96, 4,
                 extra=6)
    t = b.table()
    plan = tclora.AttnPlan(b.cache, 8, *t, n_tokens=b.T, window=96, sinks=4)
    call = tclora.AttnCall(plan, b.qd)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    plan.remap(*t, stream=st)
    call(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        plan.remap(*t)
        call()
    for step in range(4):
        for s, d in ((0, -1), (1, -3), (3, -17), (4, step % 2)):
            q, n = b.seqs[s]
            b.seqs[s] = (q, max(1, n + d))
        i = 0
        for gi, (p, ss) in enumerate(b.groups):
            b.groups[gi] = (p - 25 * gi - 40 * step, b.seqs[i:i + len(ss)])
            i += len(ss)
        b.groups = [(max(p, 0), ss) for p, ss in b.groups]
        for dst, src in zip(t, b.table()):
            dst.copy_(src)
        call.o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = call.o.clone()
        assert torch.equal(got, tclora.attention(b.plan(), b.qd))
        b.check(got)


def test_layers_with_and_without_windows_at_once():
    b = Windowed(11, [(700, [(1, 40)] * 20)], 8, 2, 128, 16, 128, 4)
    plans = [b.plan(), Batch.plan(b)]
    want = [tclora.attention(p, b.qd) for p in plans]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = [tclora.AttnCall(p, b.qd) for p in plans]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, c in zip(st, calls):
            c(s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.o, o) for c, o in zip(calls, want))


def test_refusals_and_empty_batches():
    b = Windowed(14, [(20, [(0, 3)])], 4, 2, 64, 16, 3, 1)
    run(b)
    t = b.table()
    for kw in (dict(window=0), dict(window=-1), dict(window=4, sinks=-1)):
        with pytest.raises(tclora.TclError) as e:
            tclora.AttnPlan(b.cache, 4, *t, n_tokens=b.T, **kw)
        assert e.value.code == tclora.EINVAL
    with pytest.raises(ValueError):
        tclora.AttnPlan(b.cache, 4, *t, n_tokens=b.T, sinks=2)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    plan = tclora.AttnPlan(b.cache, 4, z(1), z(1), z(0), z(0, 1), z(0), z(0, 1), n_tokens=5, window=2)
    assert plan.status() == tclora.OK
    o = torch.full((5, 256), 4.0, dtype=torch.bfloat16, device=DEV)
    tclora.attention(plan, torch.zeros_like(o), o=o)
    assert (o == 4).all()
