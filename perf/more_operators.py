"""More operators of a layer step that are timed here: pages, positions and
slots of a batch's new tokens, the append with norms of queries and keys, the
attention with a sliding window and sinks, and products with 4-bit weights.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through the library.  ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _map(name, seqs, groups, long, new, own_len, page, pad=0, lens=0):
    """The step's bookkeeping: `long` of the requests bring up to `new` tokens
    each, the others one; a request holds up to own_len keys before; pad rows
    lie behind the last request's tokens."""
    return {"name": name, "kind": "map", "seqs": seqs, "groups": groups, "long": long,
            "new": new, "own": own_len, "page": page, "pad": pad, "lens": lens}


def _append(name, T, Hq, Hkv, D, rot, page, x="bf16", interleaved=False, head_major=True, start=0,
            by_head=False):
    """T new tokens' queries and keys normed by head and rotated, keys and
    values into the cache; by_head: norm weights of every head, not of one."""
    return {"name": name, "kind": "append", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "page": page, "x": x, "interleaved": interleaved, "head_major": head_major,
            "start": start, "by_head": by_head}


def _window(name, seqs, groups, q_len, prefix, own_len, window, sinks, Hq, Hkv, D, page,
            plan=False, head_major=True, lens=0):
    """seqs requests of `groups` tenants with up to q_len new tokens each that
    see their last `window` keys and the first `sinks`.  plan: the pass maps
    the batch too (the first layer of a step)."""
    return {"name": name, "kind": "window", "seqs": seqs, "groups": groups, "q_len": q_len,
            "prefix": prefix, "own": own_len, "window": window, "sinks": sinks, "Hq": Hq,
            "Hkv": Hkv, "D": D, "page": page, "plan": plan, "head_major": head_major,
            "lens": lens}


def _i4(name, T, d_in, d_out, group, zeros=False, y="bf16"):
    """y = base projection of T tokens by 4-bit weights, a scale (and a zero
    point) for every `group` weights of a channel."""
    return {"name": name, "kind": "i4", "T": T, "d_in": d_in, "d_out": d_out, "group": group,
            "zeros": zeros, "y": y}


def listed():
    return [
        # a decode step of several tenants: one token a request
        _map("map_decode", 64, 8, 0, 1, 2048, 16, lens=1),
        # a large mixed step: prompts beside decoding requests, padded rows
        _map("map_mixed", 1152, 24, 128, 512, 512, 16, pad=96, lens=2),
        # a decode batch's new keys and values
        _append("norm_decode", 64, 32, 8, 128, 128, 16, start=4096),
        # a prefill batch's, from fp32 projections, token-major pages
        _append("norm_prefill", 4224, 32, 8, 128, 128, 64, x="f32", head_major=False),
        # narrow heads of an odd number of units, partly rotated in
        # neighbouring pairs, weights by head, at far positions
        _append("norm_far", 999, 14, 2, 80, 32, 32, interleaved=True, start=1000003, by_head=True),
        # a few requests of one tenant, a short window, with its mapping
        _window("window_small", 3, 1, 1, 200, 340, 128, 4, 8, 2, 64, 16, plan=True, lens=1),
        # a decode batch of several tenants that outgrew the window or not yet
        _window("window_tenants", 64, 8, 1, 16384, 2048, 4096, 4, 32, 8, 128, 64, lens=3),
        # chunks of several requests' prompts behind their tenant's prefix
        _window("window_chunk", 8, 2, 512, 4096, 1024, 1024, 16, 32, 8, 128, 32,
                head_major=False, lens=4),
        # one request's token through a key or value projection: latency
        _i4("i4_token_kv", 1, 4096, 1024, 128),
        # a decode batch through an up projection; the apply adds to fp32 rows
        _i4("i4_decode_up", 64, 4096, 14336, 128, zeros=True, y="f32"),
        # a ragged small decode batch through a down projection, short groups
        _i4("i4_ragged_down", 23, 14336, 4096, 32),
        # a prefill batch through an up projection
        _i4("i4_prefill_up", 2048, 4096, 14336, 128),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))


def draw(rng):
    c = _draw(rng)
    del c["name"]
    return c


def _draw(rng):
    kind = rng.choice(["map", "append", "window", "window", "i4", "i4"])
    if kind == "i4":
        group = rng.choice([32, 64, 128])
        return _i4("", _log(rng, 1, 2048), _log(rng, 256, 14336, group),
                   _log(rng, 256, 4096, 8), group, rng.random() < 0.5, rng.choice(["bf16", "f32"]))
    page = rng.choice([16, 32, 64, 128])
    if kind == "map":
        seqs = _log(rng, 1, 1152)
        return _map("", seqs, rng.randint(1, min(24, seqs)), rng.randint(0, min(seqs, 96)),
                    _log(rng, 1, 512), _log(rng, 1, 512), page,
                    rng.choice([0, 1, rng.randint(2, 96)]), rng.randrange(1 << 30))
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([n for n in (1, 2, 3, 4, 7, 8) if Hkv * n * D <= 8192])
    if kind == "append":
        D = rng.choice([D, D, 16, 48, 80, 96, 192])
        row = D * (Hq + 2 * Hkv)
        return _append("", _log(rng, 1, min(4224, (4224 * 6144) // row)), Hq, Hkv, D,
                       rng.choice([D, max(16, D // 32 * 16), 16]), page,
                       rng.choice(["bf16", "f32"]), rng.random() < 0.5, rng.random() < 0.5,
                       _log(rng, 1, 1 << 20), rng.random() < 0.3)
    groups = rng.randint(1, 6)
    q_len = 1 if rng.random() < 0.6 else _log(rng, 2, 256)
    seqs = max(groups, _log(rng, 1, 48 if q_len == 1 else 6))
    return _window("", seqs, groups, q_len, _log(rng, 16, 8192), q_len + _log(rng, 1, 1024),
                   _log(rng, 16, 4096), rng.choice([0, 1, 4, 16, rng.randint(17, 200)]), Hq, Hkv,
                   D, page, rng.random() < 0.3, rng.random() < 0.5, rng.randrange(1 << 30))


def _cuts(r, B, G):
    """group of each of B requests, every group with one at least"""
    cut = np.sort(r.choice(np.arange(1, B), G - 1, replace=False)) if G > 1 else np.zeros(0, int)
    return np.searchsorted(cut, np.arange(B), side="right")


def _step(c):
    """Ragged lengths of a step: new tokens, keys before and tenant of each
    request, prefix of each tenant."""
    r = np.random.default_rng(c["lens"])
    B, G = c["seqs"], c["groups"]
    q = np.ones(B, int)
    q[r.permutation(B)[:c["long"]]] = r.integers(max(1, c["new"] // 4), c["new"] + 1, c["long"])
    return q, r.integers(0, c["own"] + 1, B), r.integers(0, 4096, G), _cuts(r, B, G)


def _lengths(c):
    """Ragged lengths of an attention case: new tokens, own keys (the new
    tokens among them) and tenant of each request, prefix of each tenant."""
    r = np.random.default_rng(c["lens"])
    B, G = c["seqs"], c["groups"]
    q = r.integers(max(1, c["q_len"] // 2), c["q_len"] + 1, B)
    o = np.maximum(q, r.integers(max(1, c["own"] // 4), c["own"] + 1, B))
    p = r.integers(max(1, c["prefix"] // 2), c["prefix"] + 1, G)
    return q, o, p, _cuts(r, B, G)


def work(c):
    e = {"bf16": 2, "f32": 4}
    if c["kind"] == "i4":
        T, i, o = c["T"], c["d_in"], c["d_out"]
        return {"bytes": 2 * T * i + i * o // 2 + (5 if c["zeros"] else 4) * o * (i // c["group"])
                + T * o * e[c["y"]], "flops": 2 * T * i * o}
    if c["kind"] == "append":
        D, H = c["D"], c["Hq"] + c["Hkv"]
        n = c["T"] * D * (H + c["Hkv"])
        w = 4 * D * (H if c["by_head"] else 2)
        return {"bytes": n * (e[c["x"]] + 2) + 12 * c["T"] + w,
                "flops": c["T"] * H * (4 * D + 3 * c["rot"])}
    if c["kind"] == "map":
        q, n, _, _ = _step(c)
        taken = int((-(-(n + q) // c["page"]) - -(-n // c["page"])).sum())
        T = int(q.sum()) + c["pad"]
        return {"bytes": 20 * c["seqs"] + 8 * c["groups"] + 8 * taken + 12 * T, "flops": 4 * T}
    q, o, p, g = _lengths(c)
    W, N = c["window"], c["sinks"]
    ts = np.repeat(np.arange(c["seqs"]), q)
    vis = (p[g] + o - q)[ts] + np.arange(len(ts)) - np.repeat(np.cumsum(q) - q, q) + 1
    seen = np.minimum(vis, W) + np.clip(np.minimum(N, vis) - np.maximum(vis - W, 0), 0, N) * (vis > W)
    # keys that some token sees, a tenant's prefix once
    first = np.maximum(0, p[g] + o - q + 1 - W)
    low = np.full(c["groups"], 1 << 40)
    np.minimum.at(low, g, first)
    union = lambda n, at, sink: np.where(sink >= at, n, n - at + sink)  # noqa: E731
    keys = (union(p, np.minimum(low, p), np.minimum(N, p)).sum()
            + union(o, np.clip(first - p[g], 0, o), np.clip(N - p[g], 0, o)).sum())
    return {"bytes": int(4 * c["Hq"] * c["D"] * q.sum() + 4 * c["Hkv"] * c["D"] * keys),
            "flops": int(4 * c["Hq"] * c["D"] * seen.sum())}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _cache(c, n_pages, gen, heads, D):
    """Keys and values [page, slot in the page, head, dim], in memory by head
    or by token inside a page."""
    shape = (n_pages, heads, c["page"], D) if c["head_major"] else (n_pages, c["page"], heads, D)
    kv = [torch.randn(shape, generator=gen, device="cuda", dtype=F32).to(BF16) for _ in range(2)]
    return [t.transpose(1, 2) if c["head_major"] else t for t in kv]


def _up(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _table(n, ids, at, wide=0):
    """Page tables of n[r] pages in row r, ids taken from ids[at:]."""
    t = np.zeros((len(n), max(1, wide, int(n.max()))), np.int32)
    for r, m in enumerate(n):
        t[r, :m] = ids[at:at + m]
        at += m
    return t, at


def _prepare_map(c, gen):
    q, n, p, g = _step(c)
    have, want = -(-n // c["page"]), -(-(n + q) // c["page"])
    T = int(q.sum()) + c["pad"]
    n_pages = int(want.sum()) + 7
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    pages, at = _table(have, ids.cpu().numpy(), 0, int(want.max()) + 1)
    # the list of free pages, the first of them taken by earlier steps
    st = {"n_new": _up(q), "group_seq_ptr": _up(np.searchsorted(g, np.arange(c["groups"] + 1))),
          "prefix_len": _up(p), "own_len": _up(n), "own_pages": _up(pages),
          "free_pages": ids, "used": _up([at]), "seq_group": _up(g), "T": T, "n_pages": n_pages}
    if own:
        from tenant_composite_lora_amd import tclora
        K, V = (torch.zeros(n_pages, c["page"], 1, 16, dtype=BF16, device="cuda") for _ in range(2))
        st["call"] = tclora.MapCall(tclora.KVCache(K, V), st["n_new"], st["group_seq_ptr"],
                                    st["prefix_len"], st["own_len"], st["own_pages"],
                                    st["free_pages"], st["used"], T)
    return st


def _prepare_append(c, gen):
    T, D = c["T"], c["D"]
    n_pages = -(-T // c["page"]) + 3
    # heads of different strength, as projections leave them
    q, k, v = ((torch.randn(T, h, D, generator=gen, device="cuda")
                * torch.exp(torch.randn(h, 1, generator=gen, device="cuda"))).reshape(T, h * D)
               .to(DTYPES[c["x"]]) for h in (c["Hq"], c["Hkv"], c["Hkv"]))
    wq, wk = (1 + 0.3 * torch.randn(*((h, D) if c["by_head"] else (D,)), generator=gen, device="cuda")
              for h in (c["Hq"], c["Hkv"]))
    K, V = _cache(c, n_pages, gen, c["Hkv"], D)
    pages = torch.randperm(n_pages, generator=gen, device="cuda")
    t = torch.arange(T, device="cuda") + 5
    pos = (torch.arange(T, device="cuda") + c["start"]).to(torch.int32)
    if T <= 128:  # a decode batch: every token of another request
        pos = torch.randint(c["start"], 2 * c["start"] + 2, (T,), generator=gen, device="cuda",
                            dtype=torch.int32)
    slot = pages[t // c["page"]] * c["page"] + t % c["page"]
    inv = (500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / max(1, c["rot"])))
    st = {"q": q, "k": k, "v": v, "wq": wq, "wk": wk, "eps": 1e-6, "K": K, "V": V, "pos": pos,
          "slot": slot, "inv": inv.to(F32).cuda()}
    if own:
        from tenant_composite_lora_amd import tclora
        rope = tclora.Rope(st["inv"], interleaved=c["interleaved"])
        norm = tclora.HeadNorm(wq, wk, eps=st["eps"])
        st["call"] = tclora.AppendCall(tclora.KVCache(K, V), k, v, pos, slot, rope, q=q, norm=norm)
    return st


def _prepare_window(c, gen):
    q, o, p, g = _lengths(c)
    page, D = c["page"], c["D"]
    npo, npp = -(-o // page), -(-p // page)
    n_pages = int(npo.sum() + npp.sum()) + 1
    K, V = _cache(c, n_pages, gen, c["Hkv"], D)
    K.mul_(1.5)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu().numpy()
    own_pages, at = _table(npo, ids, 0)
    prefix_pages, _ = _table(npp, ids, at)
    st = {"q": torch.randn(int(q.sum()), c["Hq"] * D, generator=gen, device="cuda").to(BF16),
          "K": K, "V": V, "seq_tok_ptr": _up(np.concatenate([[0], np.cumsum(q)])),
          "group_seq_ptr": _up(np.searchsorted(g, np.arange(c["groups"] + 1))),
          "prefix_len": _up(p), "prefix_pages": _up(prefix_pages), "own_len": _up(o),
          "own_pages": _up(own_pages), "tok_seq": _up(np.repeat(np.arange(c["seqs"]), q)),
          "seq_group": _up(g), "L": int((p[g] + o).max()), "Q": int(q.max())}
    if own:
        from tenant_composite_lora_amd import tclora
        table = [st[k] for k in ("seq_tok_ptr", "group_seq_ptr", "prefix_len", "prefix_pages",
                                 "own_len", "own_pages")]
        plan = tclora.AttnPlan(tclora.KVCache(K, V), c["Hq"], *table, n_tokens=int(q.sum()),
                               window=c["window"], sinks=c["sinks"])
        st["call"] = tclora.AttnCall(plan, st["q"])
        st["table"] = table
    return st


def _prepare_i4(c, gen):
    T, i, o, G = c["T"], c["d_in"], c["d_out"], c["d_in"] // c["group"]
    # activations with a few strong channels, weights as an export holds them:
    # column 2 j in the low half of byte j
    x = torch.randn(T, i, generator=gen, device="cuda")
    x *= 1 + 11 * (torch.rand(i, generator=gen, device="cuda") < 0.01)
    n = (torch.randn(o, i, generator=gen, device="cuda") * 2.7 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
    st = {"x": x.to(BF16), "W": n[:, 0::2] | n[:, 1::2] << 4, "zero": None,
          "scale": (0.5 + torch.rand(o, G, generator=gen, device="cuda")) * (0.02 / 2.7)}
    if c["zeros"]:
        st["zero"] = torch.randint(5, 11, (o, G), generator=gen, device="cuda", dtype=torch.uint8)
    if own:
        from tenant_composite_lora_amd import tclora
        y = torch.empty(T, o, dtype=DTYPES[c["y"]], device="cuda")
        st["call"] = tclora.I4Call(tclora.I4Weight(st["W"], st["scale"], st["zero"]), st["x"], y)
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"map": _prepare_map, "append": _prepare_append, "window": _prepare_window,
          "i4": _prepare_i4}[case["kind"]](case, gen)
    return st | {"case": case}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _plain_map(c, st):
    page, dev = c["page"], st["n_new"].device
    q, n, used = st["n_new"].long(), st["own_len"].long(), st["used"].long()
    ptr = torch.cat((q.new_zeros(1), q.cumsum(0)))
    # pages that each request takes, in order, from the list
    have, want = (n + page - 1) // page, (n + q + page - 1) // page
    first = (want - have).cumsum(0) - (want - have) + used
    j = torch.arange(st["own_pages"].shape[1], device=dev)
    new = (j >= have[:, None]) & (j < want[:, None])
    at = (first[:, None] + j - have[:, None]).clamp(0, st["free_pages"].shape[0] - 1)
    st["own_pages"].copy_(torch.where(new, st["free_pages"][at], st["own_pages"]))
    # tokens
    t = torch.arange(st["T"], device=dev)
    s = torch.searchsorted(ptr, t, right=True) - 1
    pad = t >= ptr[-1]
    s = s.clamp(max=q.shape[0] - 1)
    key = n[s] + t - ptr[s]
    pg = st["own_pages"][s, (key // page).clamp(max=st["own_pages"].shape[1] - 1)].long()
    pos = st["prefix_len"].long()[st["seq_group"].long()[s]] + key
    return {"seq_tok_ptr": ptr.to(torch.int32), "pos": pos.masked_fill(pad, 0).to(torch.int32),
            "slot": (pg * page + key % page).masked_fill(pad, -1),
            "own_len": (n + q).to(torch.int32),
            "used": (used + (want - have).sum()).to(torch.int32), "own_pages": st["own_pages"]}


def _plain_append(c, st):
    T, D, r = c["T"], c["D"], c["rot"]
    ang = st["pos"].double()[:, None] * st["inv"].double()
    cs, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def turned(t, w):
        t = t.float().reshape(T, -1, D)
        t = t * ((t * t).mean(-1, keepdim=True) + st["eps"]).rsqrt() * w
        a, b = (t[..., 0:r:2], t[..., 1:r:2]) if c["interleaved"] else (t[..., :r // 2], t[..., r // 2:r])
        a, b = a * cs - b * sn, b * cs + a * sn
        ab = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((ab, t[..., r:]), -1).to(BF16)

    page, off = st["slot"] // c["page"], st["slot"] % c["page"]
    st["K"][page, off] = turned(st["k"], st["wk"])
    st["V"][page, off] = st["v"].reshape(T, -1, D).to(BF16)
    return {"q": turned(st["q"], st["wq"]), "K": st["K"], "V": st["V"]}


def _plain_window(c, st):
    B, D, Hkv, page, L, Q = c["seqs"], c["D"], c["Hkv"], c["page"], st["L"], st["Q"]
    W, N = c["window"], c["sinks"]
    q, dev = st["q"].float(), st["q"].device
    ptr, P = st["seq_tok_ptr"].long(), st["prefix_len"].long()[st["seq_group"].long()][:, None]
    n_own, n_q = st["own_len"].long()[:, None], (ptr[1:] - ptr[:-1])[:, None]
    # the keys that some token of a request sees: the sinks, then those from
    # its first token's window on (positions j, the sinks among them left out)
    first = (P + n_own - n_q + 1 - W).clamp(min=0)
    n = min(N, L)
    j = torch.arange(min(L, W + Q - 1), device=dev) + first
    again = j < n
    j = torch.cat((torch.arange(n, device=dev).expand(B, n), j), 1)
    again = torch.cat((again.new_zeros(B, n), again), 1)
    jp = j.clamp(max=st["prefix_pages"].shape[1] * page - 1)
    jo = (j - P).clamp(0, st["own_pages"].shape[1] * page - 1)
    grp = st["seq_group"].long()[:, None]
    pg = torch.where(j < P, st["prefix_pages"].long()[grp, jp // page],
                     torch.gather(st["own_pages"].long(), 1, jo // page))
    off = torch.where(j < P, jp % page, jo % page)
    K, V = (t[pg, off].float().transpose(1, 2) for t in (st["K"], st["V"]))  # [B, Hkv, keys, D]
    # the queries of every request, padded to Q
    i = torch.arange(Q, device=dev)
    tok = (ptr[:-1, None] + i).clamp(max=q.shape[0] - 1)
    qs = q[tok].reshape(B, Q, Hkv, -1, D).transpose(1, 2).reshape(B, Hkv, -1, D)
    s = (qs @ K.transpose(-1, -2)).reshape(B, Hkv, Q, -1, j.shape[1]) / math.sqrt(D)
    vis = (P + n_own - n_q + i + 1)[..., None]  # [B, Q, 1]
    jj = j[:, None]
    hidden = again[:, None] | (jj >= vis) | ((jj >= N) & (jj < vis - W))
    s = s.masked_fill_(hidden[:, None, :, None], float("-inf"))
    w = (s - s.amax(-1, keepdim=True)).exp_()
    o = ((w.flatten(2, 3) @ V).reshape(B, Hkv, Q, -1, D) / w.sum(-1, keepdim=True))
    ts = st["tok_seq"].long()
    at = torch.arange(q.shape[0], device=dev) - ptr[ts]
    return o.transpose(1, 2)[ts, at].reshape(q.shape).to(BF16)


def _plain_i4(c, st):
    o, g = c["d_out"], c["group"]
    n = torch.stack((st["W"] & 15, st["W"] >> 4), -1).reshape(o, -1, g).float()
    z = 8.0 if st["zero"] is None else st["zero"].float()[..., None]
    w = ((n - z) * st["scale"][..., None]).reshape(o, -1)
    return (st["x"].float() @ w.t()).to(DTYPES[c["y"]])


def run(st):
    c = st["case"]
    if not own:
        return {"map": _plain_map, "append": _plain_append, "window": _plain_window,
                "i4": _plain_i4}[c["kind"]](c, st)
    if c["kind"] == "window" and c["plan"]:
        st["call"].plan.remap(*st["table"])
    out = st["call"]()
    if c["kind"] == "append":
        return {"q": out.reshape(c["T"], -1, c["D"]), "K": st["K"], "V": st["V"]}
    if c["kind"] == "map":
        return {k: getattr(out, k) for k in ("seq_tok_ptr", "pos", "slot", "own_len", "used")} | {
            "own_pages": st["own_pages"]}
    return out


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_map(c, st):
    page = c["page"]
    q, n, p, g = (st[k].tolist() for k in ("n_new", "own_len", "prefix_len", "seq_group"))
    free, used = st["free_pages"].tolist(), int(st["used"][0])
    pages = st["own_pages"].tolist()
    ptr, pos, slot = [0], [], []
    for s in range(c["seqs"]):
        for key in range(n[s], n[s] + q[s]):
            if key % page == 0:  # the first key of a page takes it from the list
                pages[s][key // page] = free[used]
                used += 1
            pos.append(p[g[s]] + key)
            slot.append(pages[s][key // page] * page + key % page)
        ptr.append(len(pos))
    pos += [0] * (st["T"] - len(pos))
    slot += [-1] * (st["T"] - len(slot))
    out = {"seq_tok_ptr": ptr, "pos": pos, "slot": slot,
           "own_len": [a + b for a, b in zip(n, q)], "used": [used], "own_pages": pages}
    return {k: torch.tensor(v, device="cuda") for k, v in out.items()}


def _exact_append(c, st):
    T, D, r = c["T"], c["D"], c["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(st["pos"].double(), st["inv"].double())).unsqueeze(1)

    def turned(t, w):
        t = t.double().view(T, -1, D)
        t = w.double() * t / torch.sqrt(torch.linalg.vector_norm(t, dim=2, keepdim=True) ** 2 / D
                                        + st["eps"])
        if c["interleaved"]:
            z = torch.view_as_complex(t[..., :r].reshape(T, -1, r // 2, 2).contiguous()) * turn
            t[..., :r] = torch.view_as_real(z).reshape(T, -1, r)
        else:
            z = torch.complex(t[..., :r // 2].contiguous(), t[..., r // 2:r].contiguous()) * turn
            t[..., :r // 2], t[..., r // 2:r] = z.real, z.imag
        return t

    out = {"q": turned(st["q"], st["wq"])}
    for name, src in (("K", turned(st["k"], st["wk"])), ("V", st["v"].double().view(T, -1, D))):
        cache = st[name].double()
        # slot s of the cache is row s of its pages laid end to end
        flat = cache.reshape(-1, c["Hkv"], D).clone()
        flat[st["slot"]] = src
        out[name] = flat.view(cache.shape)
    return out


def _exact_window(c, st):
    D, H, page = c["D"], c["Hq"] // c["Hkv"], c["page"]
    q, out = st["q"].double(), []
    ptr, grp = st["seq_tok_ptr"].tolist(), st["seq_group"].tolist()
    P, n_own = st["prefix_len"].tolist(), st["own_len"].tolist()

    def keys(cache, pages, n):
        return cache[pages[:-(-n // page)].long()].flatten(0, 1)[:n].double()

    for b in range(c["seqs"]):
        n = ptr[b + 1] - ptr[b]
        K, V = (torch.cat((keys(t, st["prefix_pages"][grp[b]], P[grp[b]]),
                           keys(t, st["own_pages"][b], n_own[b]))) for t in (st["K"], st["V"]))
        L = K.shape[0]
        ones = torch.ones(n, L, dtype=torch.bool, device="cuda")
        mask = ones.tril(L - n) & ones.triu(L - n - c["window"] + 1)
        mask[:, :c["sinks"]] |= ones.tril(L - n)[:, :c["sinks"]]
        qb = q[ptr[b]:ptr[b + 1]].view(n, -1, D)
        o = torch.empty_like(qb)
        for h in range(c["Hq"]):
            s = torch.mm(qb[:, h], K[:, h // H].T) * D ** -0.5
            s[~mask] = -torch.inf
            o[:, h] = torch.mm(torch.softmax(s, 1), V[:, h // H])
        out.append(o.reshape(n, -1))
    return torch.cat(out)


def _exact_i4(c, st):
    G = c["d_in"] // c["group"]
    w = torch.empty(c["d_out"], c["d_in"], dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = st["W"].remainder(16), st["W"].div(16, rounding_mode="floor")
    zero = torch.full((c["d_out"], G), 8) if st["zero"] is None else st["zero"]
    for k in range(G):
        at = slice(k * c["group"], (k + 1) * c["group"])
        w[:, at] = (w[:, at] - zero[:, k:k + 1].cuda()) * st["scale"][:, k:k + 1].double()
    return torch.mm(st["x"].double(), w.T)


def exact(case, seed):
    st = prepare(case, seed)
    return {"map": _exact_map, "append": _exact_append, "window": _exact_window,
            "i4": _exact_i4}[case["kind"]](case, st)
