"""The attention half of a layer whose bookkeeping, norms, window and 4-bit base
weights all run on the GPU: pages and slots of the new tokens, 4-bit base
projection of queries, keys and values, the tenants' adapters on the same rows,
normed and rotated append, attention with a window and sinks, 4-bit output
projection, adapters again.

Every stage is compared with its definition in 64 bits on what the stage before
it left; the whole step, captured once, goes on by itself from replay to replay
(lengths, pages and positions are the GPU's) and stays bit for bit what eager
steps give, also when the pages have run out.
"""
import numpy as np
import pytest
import torch

from gpu_util import composites_to_dev, make_module, rel_err
from tenant_composite_lora_amd import tclora
from tenant_composite_lora_amd import workloads as W
from test_gpu_attn_window import Windowed
from test_gpu_i4 import close, product64, weight
from test_gpu_kv import inv_freq
from test_gpu_kv_norm import check_normed, weights
from test_gpu_layer_step import adapted
from test_gpu_parity import TOL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HKV, D, PAGE, DM, WINDOW, SINKS = 8, 2, 64, 16, 256, 48, 3
QKV = (HQ + 2 * HKV) * D
NEW = [1, 1, 1, 1, 9, 1, 2]
PREFIX, GROUPS = [70, 33, 0], [0, 3, 5, 7]


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


class Step:
    def __init__(self, steps):
        rng = np.random.default_rng(5)
        S, T = len(NEW), sum(NEW) + 2
        self.T, self.new, self.rows = sum(NEW), np.array(NEW), T
        self.own0 = np.array([8, 39, 16, 4, 10, 11, 5])
        have = -(-self.own0 // PAGE)
        last = -(-(self.own0 + steps * self.new) // PAGE)
        npre = [-(-p // PAGE) for p in PREFIX]
        n_pages = int(last.sum()) + sum(npre)
        ids, at = rng.permutation(n_pages), 0
        self.prefix_pages = np.zeros((3, max(npre)), np.int32)
        for g, n in enumerate(npre):
            self.prefix_pages[g, :n] = ids[at:at + n]
            at += n
        own_pages = np.zeros((S, int(last.max()) + 2), np.int32)
        for s, n in enumerate(have):
            own_pages[s, :n] = ids[at:at + n]
            at += n
        g = torch.Generator().manual_seed(3)
        K, V = (torch.randn(n_pages, HKV, PAGE, D, generator=g).to(torch.bfloat16).to(DEV).transpose(1, 2)
                for _ in range(2))
        self.cache = tclora.KVCache(K, V)
        self.own, self.used, self.own_pages = up(self.own0), up([at]), up(own_pages)
        self.map = tclora.MapCall(self.cache, up(NEW), up(GROUPS), up(PREFIX), self.own, self.own_pages,
                                  up(ids), self.used, T, own_len_out=self.own, used_out=self.used)
        # a tenant's composite: one to three adapters
        ads = [sorted(rng.choice(12, n, replace=False).tolist()) for n in (2, 1, 3)]
        als = [rng.normal(1, 0.3, len(a)).tolist() for a in ads]
        tenant = np.repeat(np.searchsorted(GROUPS, np.arange(S), side="right") - 1, NEW).tolist() + [0, 0]
        self.c = W.csr_from_token_lists([ads[t] for t in tenant], [als[t] for t in tenant], 12)
        self.plan = tclora.Plan(*composites_to_dev(self.c), 12, n_tokens=T, max_tuples=self.c.n_tuples())
        self.adapters = [W.random_case(30 + i, T=4, N=12, d_in=DM if i < 3 else HQ * D, d_out=n,
                                       r_max=8, max_pairs=2).modules[0]
                         for i, n in enumerate((HQ * D, HKV * D, HKV * D, DM))]
        self.mods = [make_module(m) for m in self.adapters]
        self.w = [weight(40, QKV, DM, 64, True), weight(41, DM, HQ * D, 128)]
        base = [tclora.I4Weight(*w) for w, _ in self.w]
        self.x = torch.zeros(T, DM, dtype=torch.bfloat16, device=DEV)
        self.qkv = torch.empty(T, QKV, device=DEV)
        self.y = torch.zeros(T, DM, device=DEV)
        self.inv = inv_freq(D)
        self.norm = tclora.HeadNorm(*weights(6, HQ, HKV, D))
        self.split = list(self.qkv.split([HQ * D, HKV * D, HKV * D], 1))
        self.first = tclora.I4Call(base[0], self.x, self.qkv)
        self.adapt = tclora.FusedCall(self.plan, self.mods[:3], [self.x] * 3, self.split)
        q, k, v = self.split
        self.append = tclora.AppendCall(self.cache, k, v, self.map.pos, self.map.slot,
                                        tclora.Rope(self.inv), q=q, norm=self.norm)
        self.map.seq_tok_ptr.zero_()
        self.table = [self.map.seq_tok_ptr, up(GROUPS), up(PREFIX), up(self.prefix_pages), self.own,
                      self.own_pages]
        self.aplan = tclora.AttnPlan(self.cache, HQ, *self.table, n_tokens=T, window=WINDOW, sinks=SINKS)
        self.o = torch.zeros(T, HQ * D, dtype=torch.bfloat16, device=DEV)
        self.attn = tclora.AttnCall(self.aplan, self.append.q_out, o=self.o)
        self.last = tclora.I4Call(base[1], self.o, self.y)
        self.adapt2 = tclora.FusedCall(self.plan, self.mods[3:], [self.o], [self.y])

    def inputs(self, step):
        g = torch.Generator().manual_seed(100 + step)
        self.x.copy_(torch.randn(self.x.shape, generator=g))

    def __call__(self):
        self.map()
        self.first()
        self.adapt()
        self.append()
        self.aplan.remap(*self.table)
        self.attn()
        self.last()
        self.adapt2()
        return self.y


def test_stages():
    s = Step(4)
    for step in range(3):
        s.inputs(step)
        s.map()
        assert s.map.status()[:2] == (tclora.OK, s.T)
        own = s.own0 + (step + 1) * s.new
        assert np.array_equal(s.own.cpu().numpy(), own)
        seq = np.repeat(np.arange(len(NEW)), NEW)
        ptr = np.concatenate([[0], np.cumsum(NEW)])
        assert np.array_equal(s.map.seq_tok_ptr.cpu().numpy(), ptr)
        key = own[seq] - s.new[seq] + np.arange(s.T) - ptr[seq]
        grp = np.searchsorted(GROUPS, seq, side="right") - 1
        assert np.array_equal(s.map.pos.cpu().numpy()[:s.T], np.array(PREFIX)[grp] + key)
        tab = s.own_pages.cpu().numpy()
        assert np.array_equal(s.map.slot.cpu().numpy()[:s.T], tab[seq, key // PAGE] * PAGE + key % PAGE)
        assert s.map.slot.tolist()[s.T:] == [-1, -1]
        # base projection, then adapters on the same rows
        s.first()
        close(s.qkv, *product64(*s.w[0], s.x))
        base = [t.clone() for t in s.split]
        s.adapt()
        for i in range(3):
            y0, delta = adapted(s, base[i], s.x, i, 0)
            assert rel_err(s.split[i].double().cpu().numpy() - y0, delta) <= TOL["bf16"]
        # norms, rotation, append
        rows = [t.clone() for t in s.split]
        s.append()
        pos, slot = s.map.pos[:s.T], s.map.slot[:s.T]
        check_normed(s.append.q_out, rows[0], s.norm.w_q, 1e-6, s.map.pos, s.inv, D, False)
        page, off = slot // PAGE, slot % PAGE
        check_normed(s.cache.K[page, off].flatten(1), rows[1][:s.T], s.norm.w_k, 1e-6, pos, s.inv, D, False)
        assert torch.equal(s.cache.V[page, off].flatten(1), rows[2][:s.T].to(torch.bfloat16))
        # attention over what the cache now holds
        s.aplan.remap(*s.table)
        assert s.aplan.status() == tclora.OK
        o = s.attn()
        b = Windowed.__new__(Windowed)
        b.window, b.sinks, b.Hq, b.Hkv, b.D, b.page, b.T = WINDOW, SINKS, HQ, HKV, D, PAGE, s.rows
        b.seqs = list(zip(NEW, own.tolist()))
        b.groups = [(p, b.seqs[GROUPS[i]:GROUPS[i + 1]]) for i, p in enumerate(PREFIX)]
        b.seq_tok, b.group_seq, b.prefix_pages, b.own_pages = ptr, np.array(GROUPS), s.prefix_pages, tab
        b.Kh, b.Vh, b.q = s.cache.K.cpu(), s.cache.V.cpu(), s.append.q_out.cpu()
        b.check(o)
        assert not o[s.T:].any()
        # output projection and its adapters
        s.last()
        close(s.y, *product64(*s.w[1], o))
        base = s.y.clone()
        s.adapt2()
        y0, delta = adapted(s, base, o, 3, 0)
        assert rel_err(s.y.double().cpu().numpy() - y0, delta) <= TOL["bf16"]


def test_captured_steps_go_on_by_themselves():
    steps = 5
    s, e = Step(steps), Step(steps)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for t in (s, e):
        t.inputs(0)
    with torch.cuda.stream(st):
        s()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s()
    e()  # (the first step, which the other took on its own stream)
    for step in range(1, steps + 2):
        s.inputs(step)
        e.inputs(step)
        s.y.fill_(float("nan"))
        K = s.cache.K.clone()
        g.replay()
        want = e()
        torch.cuda.synchronize()
        code = s.map.status()[0]
        assert code == (tclora.OK if step < steps else tclora.ENOSPC)
        assert torch.equal(s.y, want)
        assert torch.equal(s.cache.K, e.cache.K) and torch.equal(s.cache.V, e.cache.V)
        assert torch.equal(s.own, e.own) and torch.equal(s.own_pages, e.own_pages)
        if code != tclora.OK:  # nothing was appended, nobody grew
            assert torch.equal(s.cache.K, K)
            assert np.array_equal(s.own.cpu().numpy(), s.own0 + steps * s.new)
