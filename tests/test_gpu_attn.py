"""tcl_attn_apply against softmax(scale q K') V in 64 bits, key by key.

Tolerance of a row.  Scores are fp32 sums of exact products of bf16 numbers:
off by at most (D + 2) * 2^-24 * sum |q k| * scale, which moves every weight
by that factor (E below); the base-2 exponential and the running maximum's
corrections add at most 2^-20.  Weights enter the second product rounded to
bf16 (2^-8 each; 2^-16 where a tile has at most 16 rows, not assumed here),
its sum and the sum of weights are fp32, and the result is rounded to bf16
once (2^-8 of itself).  With A = sum w |V| the error is at most
(2 E + 2^-19 + 2^-8) A + 2^-8 |o|.
"""
import numpy as np
import pytest
import torch

from tenant_composite_lora_amd import tclora

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = torch.finfo(torch.bfloat16).eps / 2


class Batch:
    """A random batch: q_len, own and prefix lengths per request / group."""

    def __init__(self, seed, groups, Hq, Hkv, D, page, head_major=True, pad_tokens=0, extra=1,
                 gap=0):
        """groups: [(prefix length, [(query tokens, own length), ...]), ...]"""
        g = torch.Generator().manual_seed(seed)
        self.groups, self.Hq, self.Hkv, self.D, self.page = groups, Hq, Hkv, D, page
        seqs = [s for _, ss in groups for s in ss]
        q = [s[0] for s in seqs]
        npg = lambda n: -(-n // page)  # noqa: E731
        n_pages = sum(npg(p) for p, _ in groups) + sum(npg(s[1]) for s in seqs) + 2
        shape = [n_pages, Hkv, page, D + gap] if head_major else [n_pages, page, Hkv, D + gap]
        K, V = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2))
        if head_major:
            K, V = K.transpose(1, 2), V.transpose(1, 2)
        ids = torch.randperm(n_pages, generator=g).tolist()

        def table(lens):
            w = max([npg(n) for n in lens] + [0]) + extra
            t = np.full((len(lens), w), -7, np.int32)  # behind the lengths: not page ids
            for r, n in enumerate(lens):
                for i in range(npg(n)):
                    t[r, i] = ids.pop()
            return t

        self.prefix_pages = table([p for p, _ in groups])
        self.own_pages = table([s[1] for s in seqs])
        self.seq_tok = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        self.group_seq = np.concatenate([[0], np.cumsum([len(ss) for _, ss in groups])]).astype(np.int32)
        self.T = int(self.seq_tok[-1]) + pad_tokens
        self.seqs = seqs
        self.q = torch.randn(self.T, Hq * D, generator=g).to(torch.bfloat16)
        self.Kh, self.Vh = K[..., :D], V[..., :D]
        self.up(K, V)

    def up(self, K, V):
        kd, vd = K.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if K.stride(2) > K.stride(1) else K.to(DEV), None
        vd = V.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if V.stride(2) > V.stride(1) else V.to(DEV)
        self.cache = tclora.KVCache(kd[..., :self.D], vd[..., :self.D])
        self.qd = self.q.to(DEV)

    def table(self):
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
        return [d(self.seq_tok), d(self.group_seq), d([p for p, _ in self.groups]),
                d(self.prefix_pages), d([s[1] for s in self.seqs]), d(self.own_pages)]

    def plan(self):
        return tclora.AttnPlan(self.cache, self.Hq, *self.table(), n_tokens=self.T)

    def keys(self, cache, s):
        g = int(np.searchsorted(self.group_seq, s, side="right")) - 1
        rows = []
        for pages, n in ((self.prefix_pages[g], self.groups[g][0]),
                         (self.own_pages[s], self.seqs[s][1])):
            for j in range(0, n, self.page):
                rows.append(cache[int(pages[j // self.page]), :min(self.page, n - j)])
        return (torch.cat(rows) if rows else cache[0, :0]).double()  # [L, Hkv, D]

    def want(self, scale=None):
        """(o, lse, bound) in 64 bits; NaN rows where no request owns the token."""
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
                q = self.q[t0 + i].double().view(self.Hkv, gq, D)
                k, v = K[:vis].transpose(0, 1), V[:vis].transpose(0, 1)
                sc = (q @ k.transpose(1, 2)) * scale            # [Hkv, gq, vis]
                e = ((q.abs() @ k.abs().transpose(1, 2)) * abs(scale)).amax(-1) if vis else q[..., 0]
                E = (D + 2) * 2.0 ** -24 * e
                z = torch.logsumexp(sc, -1) if vis else torch.full((self.Hkv, gq), -float("inf"), dtype=torch.float64)
                w = torch.exp(sc - z[..., None]) if vis else sc
                ob, A = w @ v, w @ v.abs()
                o[t0 + i] = ob.reshape(Hq, D)
                lse[t0 + i] = z.reshape(Hq)
                tol[t0 + i] = ((2 * E[..., None] + 2.0 ** -19 + HALF) * A
                               + HALF * ob.abs()).reshape(Hq, D)
        return o, lse, tol

    def check(self, o, lse=None, scale=None):
        wo, wl, tol = self.want(scale)
        own = ~torch.isnan(wl)
        got = o.double().cpu().view(self.T, self.Hq, self.D)
        err = ((got - wo).abs() - tol)[own]
        assert err.numel() == 0 or float(err.max()) <= 1e-30, float(err.max())
        if lse is not None:
            got = lse.double().cpu()
            none = torch.isinf(wl)
            assert torch.equal(got[none], wl[none])
            f = own & ~none
            # scores as above (E <= 2^-10 here), fp32 logarithm and exponentials
            lim = 2.0 ** -18 + 2.0 ** -20 * wl[f].abs() + (self.D + 2) * 2.0 ** -24 * 64
            assert bool(((got[f] - wl[f]).abs() <= lim).all())


def run(b, scale=None, want_lse=True):
    plan = b.plan()
    assert plan.status() == tclora.OK
    o = torch.full((b.T, b.Hq * b.D), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((b.T, b.Hq), 77.0, device=DEV) if want_lse else None
    tclora.attention(plan, b.qd, o=o, lse=lse, scale=scale)
    b.check(o, lse, scale)
    n = int(b.seq_tok[-1])
    assert (o[n:] == 77).all() and (lse is None or (lse[n:] == 77).all())
    return o


DECODE = {
    "one token, one key": [(0, [(1, 1)])],
    "no prefix": [(0, [(1, 5), (1, 64), (1, 65), (1, 300)])],
    "prefix of one request": [(130, [(1, 7)])],
    "shared prefix": [(200, [(1, 1), (1, 17), (1, 64), (1, 63)])],
    "prefix that ends inside a page and a step": [(77, [(1, 1), (1, 2)]), (1, [(1, 1), (1, 1)])],
    "many requests": [(500, [(1, 1 + 3 * i) for i in range(40)])],
    "several groups, one empty": [(64, [(1, 3)] * 3), (33, []), (0, [(1, 9)] * 2), (129, [(1, 70)] * 5)],
    "long": [(3000, [(1, 2500), (1, 10), (1, 700)])],
    "requests without tokens": [(90, [(1, 4), (0, 12), (1, 8)]), (20, [(0, 0)])],
}


@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [
    (8, 2, 64, 16, True), (4, 4, 128, 16, False), (8, 1, 128, 64, True), (14, 2, 64, 32, False),
    (6, 2, 256, 16, True), (32, 1, 64, 16, True), (3, 1, 128, 1, False)])
@pytest.mark.parametrize("name", DECODE)
def test_decode(name, Hq, Hkv, D, page, head_major):
    run(Batch(len(name) + D, DECODE[name], Hq, Hkv, D, page, head_major))


CHUNKS = {
    "two tokens": [(100, [(2, 2), (2, 30)])],
    "a prompt": [(0, [(150, 150)])],
    "a prompt behind a prefix": [(70, [(97, 97)])],
    "short and long requests of a group": [(300, [(1, 40), (200, 210), (3, 3), (30, 64), (1, 1)])],
    "odd": [(33, [(5, 9), (6, 6), (7, 70)]), (0, [(31, 33), (1, 2)])],
    "more tokens than keys": [(2, [(5, 1), (4, 0)]), (0, [(3, 0), (9, 4), (70, 3)]), (40, [(50, 5), (45, 2)])],
}


@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [
    (8, 2, 64, 16, True), (4, 1, 128, 32, False), (14, 2, 64, 16, False), (3, 1, 256, 64, True),
    (4, 4, 128, 16, True)])
@pytest.mark.parametrize("name", CHUNKS)
def test_chunks(name, Hq, Hkv, D, page, head_major):
    """Several query tokens a request, causal; rows that see no key are zero."""
    run(Batch(len(name) * D, CHUNKS[name], Hq, Hkv, D, page, head_major))


@pytest.mark.parametrize("gq", [1, 2, 5, 7, 16, 17, 33, 128])
def test_heads_of_a_key_head(gq):
    run(Batch(gq, [(90, [(1, 30), (1, 40), (4, 50)])], 2 * gq, 2, 64, 16))


def test_more_requests_and_groups_than_threads():
    """Mappings beyond one pass of the workgroup, and beyond its LDS tables."""
    r = np.random.default_rng(3)
    seqs = lambda n, q=1: [(q, q + int(x)) for x in r.integers(0, 8, n)]  # noqa: E731
    run(Batch(31, [(int(p), seqs(30)) for p in r.integers(0, 40, 50)], 4, 2, 64, 16))
    run(Batch(32, [(int(p), seqs(int(n))) for p, n in zip(r.integers(0, 9, 1100),
                                                           r.integers(0, 3, 1100))], 2, 1, 64, 8))
    # two tiles a request: more tiles than threads
    run(Batch(33, [(20, seqs(560, 3))], 64, 1, 64, 16))


def test_offsets_beyond_32_bits():
    """Pages at the end of a cache of more than 2^31 elements and 2^32 bytes:
    the same rows as from a cache that holds nothing else."""
    b = Batch(34, [(300, [(1, 90), (1, 70), (40, 100)])], 4, 2, 64, 32)
    want = tclora.attention(b.plan(), b.qd)
    b.check(want)
    pages, elems = b.cache.n_pages, 32 * 2 * 64
    big = (1 << 31) // elems + pages + 1
    K = torch.zeros(big, 2, 32, 64, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros_like(K)
    K[big - pages:] = b.cache.K.transpose(1, 2)
    V[big - pages:] = b.cache.V.transpose(1, 2)
    cache = tclora.KVCache(K.transpose(1, 2), V.transpose(1, 2))
    t = b.table()
    for i in (3, 5):
        t[i] = torch.where(t[i] >= 0, t[i] + (big - pages), t[i])
    plan = tclora.AttnPlan(cache, 4, *t, n_tokens=b.T)
    assert plan.status() == tclora.OK
    assert torch.equal(tclora.attention(plan, b.qd), want)


def test_rows_behind_the_last_request_stay():
    run(Batch(5, [(100, [(1, 4), (1, 9), (70, 80)])], 8, 2, 64, 16, pad_tokens=9))
    run(Batch(5, [(0, [(0, 4)])], 8, 2, 64, 16, pad_tokens=3))


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 3.0])
def test_scale(scale):
    run(Batch(6, [(150, [(1, 40), (1, 70), (20, 30)])], 4, 2, 64, 16), scale=scale, want_lse=False)


def test_strides():
    b = Batch(7, [(150, [(1, 40), (1, 70), (20, 30)])], 4, 2, 64, 16, gap=8)
    run(b)
    plan = b.plan()
    wide = torch.full((b.T, 3 * 256 + 8), 5.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 256:512] = b.qd
    o = tclora.attention(plan, wide[:, 256:512], o=wide[:, 512:768])
    b.check(o)
    assert (wide[:, :256] == 5).all() and (wide[:, 768:] == 5).all()
    o = tclora.attention(plan, wide[:, 256:512], o=wide[:, 256:512])  # in place
    b.check(o)


def test_extreme_scores():
    """Scores of some thousands: one key takes everything, no overflow."""
    b = Batch(8, [(150, [(1, 40), (1, 70), (20, 30), (90, 100)])], 4, 2, 64, 16)
    b.Kh.mul_(64)
    b.q.mul_(64)
    b.up(b.Kh, b.Vh)
    plan = b.plan()
    o = tclora.attention(plan, b.qd)
    wo, _, _ = b.want()
    assert torch.isfinite(o).all()
    # the exact winner of every row, up to near ties that 64 bits settle
    err = (o.double().cpu().view(wo.shape) - wo).abs().amax(-1)
    assert float((err > 0.05).double().mean()) < 0.01


@pytest.mark.parametrize("Hq,Hkv,D,page,head_major", [
    (8, 2, 64, 16, True), (4, 1, 128, 32, False), (3, 1, 256, 64, True), (32, 1, 128, 8, True)])
@pytest.mark.parametrize("where", ["V", "K"])
def test_infinities_and_nans_of_hidden_keys(where, Hq, Hkv, D, page, head_major):
    """Keys that only some rows see (the newest ones, the end of a prefix that
    a request without own keys does not reach) and slots behind every length
    hold infinities and NaNs: rows that do not see them are as ever, rows that
    do are what the sum gives in 64 bits."""
    b = Batch(15, [(70, [(3, 20), (90, 100), (1, 9), (2, 70)]), (130, [(150, 20), (1, 0), (40, 70)])],
              Hq, Hkv, D, page, head_major)
    X = b.Vh if where == "V" else b.Kh
    g = torch.Generator().manual_seed(1)
    kinds = torch.tensor([float("nan"), float("inf"), -float("inf")])
    used = torch.zeros(X.shape[:2], dtype=torch.bool)

    def slots(pages, n, at):
        return int(pages[at // page]), at % page

    for pages, n in [(b.prefix_pages[i], p) for i, (p, _) in enumerate(b.groups)] + [
            (b.own_pages[i], s[1]) for i, s in enumerate(b.seqs)]:
        for j in range(n):
            used[slots(pages, n, j)] = True
        for back in (1, 2, 5, 17):  # the last keys, a few dimensions each
            if n > back:
                pg, of = slots(pages, n, n - back)
                d = torch.randint(0, D, (3,), generator=g)
                X[pg, of, int(torch.randint(0, Hkv, (1,), generator=g)), d] = kinds[
                    torch.randint(0, 3, (3,), generator=g)].to(X.dtype)
    b.Kh[~used] = float("nan")
    b.Vh[~used] = float("nan")
    b.up(b.Kh, b.Vh)
    o = tclora.attention(b.plan(), b.qd).double().cpu().view(b.T, Hq, D)
    wo, _, tol = b.want()
    assert torch.equal(torch.isnan(o), torch.isnan(wo))
    inf = torch.isinf(wo)
    assert torch.equal(o[inf], wo[inf]) and bool(inf.any()) == (where == "V")
    ok = torch.isfinite(wo)
    assert float(ok.double().mean()) > 0.2
    # (a row's bound counts every visible |V|: where one is infinite only the
    # finite dimensions are held to theirs)
    assert float(((o - wo).abs() - tol)[ok].max()) <= 1e-30


def test_bad_tables_change_nothing():
    base = [(100, [(1, 30), (2, 40)]), (50, [(1, 20)])]
    o = torch.full((4, 256), 3.0, dtype=torch.bfloat16, device=DEV)

    def bad(**kw):
        b = Batch(9, base, 4, 2, 64, 16)
        t = dict(zip(("seq_tok", "group_seq", "prefix_len", "prefix_pages", "own_len", "own_pages"),
                     b.table()))
        for k, (i, v) in kw.items():
            t[k].view(-1)[i] = v
        plan = tclora.AttnPlan(b.cache, 4, *t.values(), n_tokens=b.T)
        assert plan.status() == tclora.EINVAL, kw
        tclora.attention(plan, b.qd, o=o)
        assert (o == 3).all(), kw

    n = 200
    for kw in (dict(seq_tok=(0, 1)), dict(seq_tok=(1, 4)), dict(seq_tok=(3, 5)),
               dict(group_seq=(0, 1)), dict(group_seq=(2, 2)), dict(group_seq=(1, 4)),
               dict(prefix_len=(0, -1)), dict(prefix_len=(1, 1000)), dict(own_len=(2, -5)),
               dict(own_len=(0, 65)), dict(own_pages=(0, -1)), dict(own_pages=(1, n)),
               dict(prefix_pages=(6, n)), dict(prefix_pages=(0, -2147483648))):
        bad(**kw)


def test_remap_and_graph():
    """One plan, batches of the same sizes mapped into it inside a graph."""
    b = Batch(10, [(200, [(1, 40), (1, 90), (1, 30)]), (64, [(1, 100), (1, 5)])], 8, 2, 128, 16,
              extra=6)
    t = b.table()
    plan = tclora.AttnPlan(b.cache, 8, *t, n_tokens=b.T)
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
        # lengths shrink and grow inside the pages
        for s, d in ((0, -1), (1, -3), (3, -17), (4, step % 2)):
            q, n = b.seqs[s]
            b.seqs[s] = (q, max(1, n + d))
        i = 0
        for gi, (p, ss) in enumerate(b.groups):
            b.groups[gi] = (p - 5 * gi - step, b.seqs[i:i + len(ss)])
            i += len(ss)
        for dst, src in zip(t, b.table()):
            dst.copy_(src)
        call.o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = call.o.clone()
        eager = tclora.attention(b.plan(), b.qd)
        assert torch.equal(got, eager)
        b.check(got)


def test_two_calls_at_once():
    """Two streams, a workspace each, one plan."""
    b = Batch(11, [(700, [(1, 40)] * 20)], 8, 2, 128, 16)
    plan = b.plan()
    want = tclora.attention(plan, b.qd)
    q2 = (b.qd * 0.5).contiguous()
    want2 = tclora.attention(plan, q2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    c1, c2 = tclora.AttnCall(plan, b.qd), tclora.AttnCall(plan, q2)
    torch.cuda.synchronize()
    for _ in range(5):
        c1(s1), c2(s2)
    torch.cuda.synchronize()
    assert torch.equal(c1.o, want) and torch.equal(c2.o, want2)


# (a test below has the same name: this one runs under another)
test_two_queries_at_once = test_two_calls_at_once


def test_layers_share_a_plan():
    b = Batch(12, [(120, [(1, 40), (1, 50)])], 8, 2, 64, 16)
    other = tclora.KVCache(b.cache.K.clone(), torch.zeros_like(b.cache.V))
    o = tclora.attention(b.plan(), b.qd, cache=other)
    assert not o.any()


def test_binding_refusals():
    b = Batch(13, [(120, [(1, 40), (1, 50)])], 8, 2, 64, 16)
    plan, t = b.plan(), b.table()
    with pytest.raises(ValueError):
        tclora.attention(plan, b.qd[:1])
    with pytest.raises(TypeError):
        tclora.attention(plan, b.qd.float())
    with pytest.raises(ValueError):
        tclora.attention(plan, b.qd, lse=torch.empty(2, 4, device=DEV))
    with pytest.raises(ValueError):
        tclora.AttnCall(plan, b.qd, cache=tclora.KVCache(b.cache.K[:3], b.cache.V[:3]))
    with pytest.raises(ValueError):
        plan.remap(t[0][:-1], t[1], *t[2:4], t[4][:-1], t[5][:-1])
    with pytest.raises(ValueError):
        tclora.AttnPlan(b.cache, 8, t[0].long(), *t[1:], n_tokens=b.T)
    with pytest.raises(ValueError):
        tclora.AttnPlan(b.cache, 8, t[0].cpu(), *t[1:], n_tokens=b.T)
    with pytest.raises(tclora.TclError) as e:
        tclora.AttnPlan(b.cache, 7, *t, n_tokens=b.T)
    assert e.value.code == tclora.EINVAL
    k96 = torch.zeros(4, 16, 2, 96, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(tclora.TclError) as e:
        tclora.AttnPlan(tclora.KVCache(k96, k96.clone()), 8, *t, n_tokens=b.T)
    assert e.value.code == tclora.EUNSUPPORTED


def test_empty_batches():
    b = Batch(14, [(20, [(0, 3)])], 4, 2, 64, 16)
    run(b)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    plan = tclora.AttnPlan(b.cache, 4, z(1), z(1), z(0), z(0, 1), z(0), z(0, 1), n_tokens=5)
    assert plan.status() == tclora.OK
    q = torch.zeros(5, 256, dtype=torch.bfloat16, device=DEV)
    o = torch.full_like(q, 4.0)
    tclora.attention(plan, q, o=o)
    assert (o == 4).all()


@pytest.mark.parametrize("raw", [False, True])
def test_plan_and_attention_on_another_stream(raw):
    """Plan, workspace and rows made on the way belong to the stream of the
    call, also when everything is dropped right behind it."""
    b = Batch(35, [(300, [(1, 90), (1, 70), (40, 100)])], 4, 2, 64, 32)
    want = tclora.attention(b.plan(), b.qd)
    t = b.table()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = st.cuda_stream if raw else st
    for _ in range(3):
        torch.cuda._sleep(2_000_000)
        junk = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (1 << 14, 1 << 20, b.qd.numel() * 2)]
        kept = [j.clone() for j in junk]
        del junk
        plan = tclora.AttnPlan(b.cache, 4, *t, n_tokens=b.T, stream=s)
        got = tclora.attention(plan, b.qd, stream=s)
        del plan
        over = [torch.full((n,), 9, dtype=torch.uint8, device=DEV) for n in (1 << 14, 1 << 20)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(bool((k == 7).all()) for k in kept)
        del got, over


def test_two_calls_at_once():
    """Two layers' attention on two streams through one plan, a workspace each."""
    b = Batch(37, [(300, [(1, 90), (1, 70), (40, 100)]), (64, [(1, 30), (1, 200)])], 8, 2, 128, 16)
    plan = b.plan()
    other = tclora.KVCache(b.cache.V, b.cache.K)
    want = [tclora.attention(plan, b.qd), tclora.attention(plan, b.qd, cache=other)]
    calls = [tclora.AttnCall(plan, b.qd), tclora.AttnCall(plan, b.qd, cache=other)]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, c in zip(st, calls):
            c(s)
    torch.cuda.synchronize()
    assert all(torch.equal(c.o, o) for c, o in zip(calls, want))


def test_no_prefix_pages_at_all():
    """Groups without prefixes may have a page table of no columns, requests
    without own keys likewise."""
    b = Batch(38, [(0, [(1, 20), (30, 40)]), (0, [(1, 5)])], 4, 2, 64, 16)
    want = tclora.attention(b.plan(), b.qd)
    t = list(b.table())
    t[3] = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    plan = tclora.AttnPlan(b.cache, 4, *t, n_tokens=b.T)
    assert plan.status() == tclora.OK
    assert torch.equal(tclora.attention(plan, b.qd), want)
    b = Batch(39, [(50, [(1, 0), (2, 0)]), (7, [(1, 0)])], 4, 2, 64, 16)
    want = tclora.attention(b.plan(), b.qd)
    t = list(b.table())
    t[5] = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    plan = tclora.AttnPlan(b.cache, 4, *t, n_tokens=b.T)
    assert plan.status() == tclora.OK
    assert torch.equal(tclora.attention(plan, b.qd), want)
