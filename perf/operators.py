"""The operators around the batched LoRA apply that are timed here: int8 base
products, the rotated append to a paged key/value cache and the attention of a
batch whose requests share their tenant's prefix.

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
def _i8(name, T, d_in, d_out, x="bf16", y="bf16"):
    """y = base projection of T tokens: token scales and int8 rows from the
    activations, then the int8 product with channel scales."""
    return {"name": name, "kind": "i8", "T": T, "d_in": d_in, "d_out": d_out, "x": x, "y": y}


def _append(name, T, Hq, Hkv, D, rot, page, x="bf16", interleaved=False, head_major=True, start=0):
    """T new tokens' keys rotated into the cache, values copied, queries
    rotated; start is the first position."""
    return {"name": name, "kind": "append", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "page": page, "x": x, "interleaved": interleaved, "head_major": head_major,
            "start": start}


def _attn(name, seqs, groups, q_len, prefix, own_len, Hq, Hkv, D, page, plan=False,
          head_major=True, lens=0):
    """seqs requests of `groups` tenants with up to q_len new tokens each; a
    tenant's prefix has up to `prefix` keys, a request's own part up to
    own_len.  lens seeds the ragged lengths.  plan: the pass maps the batch
    too (the first layer of a step); otherwise it is one of the further
    layers."""
    return {"name": name, "kind": "attn", "seqs": seqs, "groups": groups, "q_len": q_len,
            "prefix": prefix, "own": own_len, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "plan": plan, "head_major": head_major, "lens": lens}


def listed():
    return [
        # one request's token through a key or value projection: latency
        _i8("i8_token_kv", 1, 4096, 1024),
        # a decode batch through an up projection; the apply adds to fp32 rows
        _i8("i8_decode_up", 64, 4096, 14336, y="f32"),
        # a ragged small prefill batch through a down projection
        _i8("i8_ragged_down", 177, 14336, 4096, x="f32"),
        # the mixed batch through the query projection and an up projection
        _i8("i8_prefill_q", 4224, 4096, 4096, y="f32"),
        _i8("i8_prefill_up", 4224, 4096, 14336),
        # a decode batch's new keys and values
        _append("append_decode", 64, 32, 8, 128, 128, 16, start=4096),
        # a prefill batch's, from fp32 projections, token-major pages
        _append("append_prefill", 4224, 32, 8, 128, 128, 64, x="f32", head_major=False),
        # partly rotated narrow heads in neighbouring pairs, at far positions
        _append("append_far", 999, 14, 2, 64, 32, 32, interleaved=True, start=1000003),
        # a few requests of one tenant with a short instruction
        _attn("attn_small", 3, 1, 1, 200, 40, 8, 2, 64, 16, lens=1),
        # a decode batch of one tenant with a long prefix, with its mapping
        _attn("attn_one_prefix", 64, 1, 1, 8192, 512, 32, 8, 128, 16, plan=True, lens=2),
        # a decode batch of several tenants, ragged prefixes and own parts
        _attn("attn_tenants", 64, 8, 1, 16384, 2048, 32, 8, 128, 64, lens=3),
        # chunks of several requests' prompts behind their tenant's prefix
        _attn("attn_chunk", 8, 2, 512, 4096, 1024, 32, 8, 128, 32, head_major=False, lens=4),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))


def draw(rng):
    c = _draw(rng)
    del c["name"]
    return c


def _draw(rng):
    kind = rng.choice(["i8", "i8", "append", "attn", "attn"])
    if kind == "i8":
        return _i8("", _log(rng, 1, 4224), _log(rng, 256, 14336, 16), _log(rng, 256, 4096, 8),
                   rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]))
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([n for n in (1, 2, 3, 4, 7, 8) if Hkv * n * D <= 8192])
    page = rng.choice([16, 32, 64, 128])
    if kind == "append":
        return _append("", _log(rng, 1, 4224), Hq, Hkv, D, rng.choice([D, D // 2, D // 4]), page,
                       rng.choice(["bf16", "f32"]), rng.random() < 0.5, rng.random() < 0.5,
                       _log(rng, 1, 1 << 20))
    groups = rng.randint(1, 6)
    q_len = 1 if rng.random() < 0.6 else _log(rng, 2, 256)
    seqs = max(groups, _log(rng, 1, 48 if q_len == 1 else 6))
    return _attn("", seqs, groups, q_len, _log(rng, 16, 8192), q_len + _log(rng, 1, 1024), Hq, Hkv,
                 D, page, rng.random() < 0.3, rng.random() < 0.5,
                 rng.randrange(1 << 30))


def _lengths(c):
    """Ragged lengths of an attention case: new tokens, own keys (the new
    tokens among them) and tenant of each request, prefix of each tenant."""
    r = np.random.default_rng(c["lens"])
    B, G = c["seqs"], c["groups"]
    q = r.integers(max(1, c["q_len"] // 2), c["q_len"] + 1, B)
    o = np.maximum(q, r.integers(max(1, c["own"] // 4), c["own"] + 1, B))
    p = r.integers(max(1, c["prefix"] // 2), c["prefix"] + 1, G)
    if G == 1:
        p[0] = c["prefix"]
    cut = np.sort(r.choice(np.arange(1, B), G - 1, replace=False)) if G > 1 else np.zeros(0, int)
    g = np.searchsorted(cut, np.arange(B), side="right")
    return q, o, p, g


def work(c):
    e = {"bf16": 2, "f32": 4}
    if c["kind"] == "i8":
        T, i, o = c["T"], c["d_in"], c["d_out"]
        return {"bytes": T * i * e[c["x"]] + i * o + 4 * o + T * o * e[c["y"]],
                "flops": 2 * T * i * o}
    if c["kind"] == "append":
        n = c["T"] * c["D"] * (c["Hq"] + 2 * c["Hkv"])
        return {"bytes": n * (e[c["x"]] + 2) + 12 * c["T"],
                "flops": 3 * c["T"] * c["rot"] * (c["Hq"] + c["Hkv"])}
    q, o, p, g = _lengths(c)
    kv, io = 4 * c["Hkv"] * c["D"], 4 * c["Hq"] * c["D"]
    seen = (q * (p[g] + o) - q * (q - 1) // 2).sum()
    return {"bytes": int(io * q.sum() + kv * (p.sum() + o.sum())),
            "flops": int(4 * c["Hq"] * c["D"] * seen)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _cache(c, n_pages, gen):
    """Keys and values [page, slot in the page, head, dim], in memory by head
    or by token inside a page."""
    shape = ((n_pages, c["Hkv"], c["page"], c["D"]) if c["head_major"]
             else (n_pages, c["page"], c["Hkv"], c["D"]))
    kv = [torch.randn(shape, generator=gen, device="cuda", dtype=F32).to(BF16) for _ in range(2)]
    return [t.transpose(1, 2) if c["head_major"] else t for t in kv]


def _prepare_i8(c, gen):
    T, i, o = c["T"], c["d_in"], c["d_out"]
    # activations with a few strong channels, weights as an export holds them
    x = torch.randn(T, i, generator=gen, device="cuda")
    x *= 1 + 11 * (torch.rand(i, generator=gen, device="cuda") < 0.01)
    W = (torch.randn(o, i, generator=gen, device="cuda") * 36).round_().clamp_(-127, 127)
    ws = (0.5 + torch.rand(o, generator=gen, device="cuda")) * (0.02 / 36)
    st = {"x": x.to(DTYPES[c["x"]]), "W": W.to(torch.int8), "ws": ws}
    if own:
        from tenant_composite_lora_amd import tclora
        y = torch.empty(T, o, dtype=DTYPES[c["y"]], device="cuda")
        st["call"] = tclora.I8Call(tclora.I8Weight(st["W"], ws), st["x"], y)
    return st


def _prepare_append(c, gen):
    T, D = c["T"], c["D"]
    n_pages = -(-T // c["page"]) + 3
    q, k, v = (torch.randn(T, h * D, generator=gen, device="cuda").to(DTYPES[c["x"]])
               for h in (c["Hq"], c["Hkv"], c["Hkv"]))
    K, V = _cache(c, n_pages, gen)
    pages = torch.randperm(n_pages, generator=gen, device="cuda")
    t = torch.arange(T, device="cuda") + 5
    pos = (torch.arange(T, device="cuda") + c["start"]).to(torch.int32)
    if T <= 128:  # a decode batch: every token of another request
        pos = torch.randint(c["start"], 2 * c["start"] + 2, (T,), generator=gen, device="cuda",
                            dtype=torch.int32)
    slot = pages[t // c["page"]] * c["page"] + t % c["page"]
    inv = (500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"]))
    st = {"q": q, "k": k, "v": v, "K": K, "V": V, "pos": pos, "slot": slot,
          "inv": inv.to(F32).cuda()}
    if own:
        from tenant_composite_lora_amd import tclora
        rope = tclora.Rope(st["inv"], interleaved=c["interleaved"])
        st["call"] = tclora.AppendCall(tclora.KVCache(K, V), k, v, pos, slot, rope, q=q)
    return st


def _prepare_attn(c, gen):
    q, o, p, g = _lengths(c)
    page, D = c["page"], c["D"]
    npo, npp = -(-o // page), -(-p // page)
    n_pages = int(npo.sum() + npp.sum()) + 1
    K, V = _cache(c, n_pages, gen)
    K.mul_(1.5)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu().numpy()

    def table(n, at):
        t = np.zeros((len(n), int(n.max())), np.int32)
        for r, m in enumerate(n):
            t[r, :m] = ids[at:at + m]
            at += m
        return t, at

    own_pages, at = table(npo, 0)
    prefix_pages, _ = table(npp, at)
    up = lambda a: torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    seq_tok = np.concatenate([[0], np.cumsum(q)])
    group_seq = np.searchsorted(g, np.arange(c["groups"] + 1), side="left")
    st = {"q": torch.randn(int(q.sum()), c["Hq"] * D, generator=gen, device="cuda").to(BF16),
          "K": K, "V": V, "seq_tok_ptr": up(seq_tok), "group_seq_ptr": up(group_seq),
          "prefix_len": up(p), "prefix_pages": up(prefix_pages), "own_len": up(o),
          "own_pages": up(own_pages), "tok_seq": up(np.repeat(np.arange(c["seqs"]), q)),
          "seq_group": up(g), "L": int((p[g] + o).max()), "Q": int(q.max())}
    if own:
        from tenant_composite_lora_amd import tclora
        table = [st[k] for k in ("seq_tok_ptr", "group_seq_ptr", "prefix_len", "prefix_pages",
                                 "own_len", "own_pages")]
        plan = tclora.AttnPlan(tclora.KVCache(K, V), c["Hq"], *table, n_tokens=int(q.sum()))
        st["call"] = tclora.AttnCall(plan, st["q"])
        st["table"] = table
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"i8": _prepare_i8, "append": _prepare_append, "attn": _prepare_attn}[case["kind"]](case, gen)
    return st | {"case": case}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _plain_i8(c, st):
    # in 64 bits up to the rounding: values lie next to a border
    x = st["x"].double()
    s = (x.abs().amax(1, keepdim=True) / 127).float()
    n = torch.where(s > 0, torch.round(x / s.double()).clamp(-127, 127), 0).float()
    y = (n @ st["W"].float().t()) * s * st["ws"]
    return y.to(DTYPES[c["y"]])


def _plain_append(c, st):
    T, D, r = c["T"], c["D"], c["rot"]
    ang = st["pos"].double()[:, None] * st["inv"].double()
    cs, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]

    def rotate(t):
        t = t.float().reshape(T, -1, D)
        a, b = (t[..., 0:r:2], t[..., 1:r:2]) if c["interleaved"] else (t[..., :r // 2], t[..., r // 2:r])
        a, b = a * cs - b * sn, b * cs + a * sn
        ab = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((ab, t[..., r:]), -1).to(BF16)

    page, off = st["slot"] // c["page"], st["slot"] % c["page"]
    st["K"][page, off] = rotate(st["k"])
    st["V"][page, off] = st["v"].reshape(T, -1, D).to(BF16)
    return {"q": rotate(st["q"]), "K": st["K"], "V": st["V"]}


def _plain_attn(c, st):
    B, D, Hkv, page, L, Q = c["seqs"], c["D"], c["Hkv"], c["page"], st["L"], st["Q"]
    q, dev = st["q"].float(), st["q"].device
    ptr, P = st["seq_tok_ptr"].long(), st["prefix_len"].long()[st["seq_group"].long()]
    n_own = st["own_len"].long()
    # the keys of every request, its tenant's prefix first, padded to L
    j = torch.arange(L, device=dev)
    jp = j.clamp(max=st["prefix_pages"].shape[1] * page - 1)
    jo = (j - P[:, None]).clamp(0, st["own_pages"].shape[1] * page - 1)
    pg = torch.where(j < P[:, None], st["prefix_pages"].long()[st["seq_group"].long()][:, jp // page],
                     torch.gather(st["own_pages"].long(), 1, jo // page))
    off = torch.where(j < P[:, None], jp % page, jo % page)
    K, V = (t[pg, off].float().transpose(1, 2) for t in (st["K"], st["V"]))  # [B, Hkv, L, D]
    # the queries of every request, padded to Q
    n_q = ptr[1:] - ptr[:-1]
    i = torch.arange(Q, device=dev)
    tok = (ptr[:-1, None] + i).clamp(max=q.shape[0] - 1)
    qs = q[tok].reshape(B, Q, Hkv, -1, D).transpose(1, 2).reshape(B, Hkv, -1, D)
    s = (qs @ K.transpose(-1, -2)).reshape(B, Hkv, Q, -1, L) / math.sqrt(D)
    seen = P[:, None] + n_own[:, None] - n_q[:, None] + i + 1
    hidden = j >= seen[:, None, :, None, None]
    s = s.masked_fill_(hidden, float("-inf"))
    w = (s - s.amax(-1, keepdim=True)).exp_()
    o = ((w.flatten(2, 3) @ V).reshape(B, Hkv, Q, -1, D) / w.sum(-1, keepdim=True))
    ts = st["tok_seq"].long()
    at = torch.arange(q.shape[0], device=dev) - ptr[ts]
    return o.transpose(1, 2)[ts, at].reshape(q.shape).to(BF16)


def run(st):
    c = st["case"]
    if own:
        if c["kind"] == "attn" and c["plan"]:
            st["call"].plan.remap(*st["table"])
        out = st["call"]()
        return {"q": out.reshape(c["T"], -1, c["D"]), "K": st["K"], "V": st["V"]} if c["kind"] == "append" else out
    return {"i8": _plain_i8, "append": _plain_append, "attn": _plain_attn}[c["kind"]](c, st)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_i8(c, st):
    x = st["x"].double()
    # a token's scale is held in 32 bits: its rounding is part of the definition
    s = (x.abs().max(dim=1, keepdim=True).values / 127).to(F32).double()
    n = torch.nan_to_num(torch.round(x / s)).clamp(-127, 127)
    return torch.mm(n, st["W"].double().T) * (s * st["ws"].double()[None, :])


def _exact_append(c, st):
    T, D, r = c["T"], c["D"], c["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(st["pos"].double(), st["inv"].double())).unsqueeze(1)

    def rotate(t):
        t = t.double().view(T, -1, D).clone()
        if c["interleaved"]:
            z = torch.view_as_complex(t[..., :r].reshape(T, -1, r // 2, 2).contiguous()) * turn
            t[..., :r] = torch.view_as_real(z).reshape(T, -1, r)
        else:
            z = torch.complex(t[..., :r // 2], t[..., r // 2:r]) * turn
            t[..., :r // 2], t[..., r // 2:r] = z.real, z.imag
        return t

    out = {"q": rotate(st["q"])}
    for name, src in (("K", rotate(st["k"])), ("V", st["v"].double().view(T, -1, D))):
        cache = st[name].double()
        # slot s of the cache is row s of its pages laid end to end
        flat = cache.reshape(-1, c["Hkv"], D).clone()
        flat[st["slot"]] = src
        out[name] = flat.view(cache.shape)
    return out


def _exact_attn(c, st):
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
        mask = torch.ones(n, L, dtype=torch.bool, device="cuda").tril(L - n)
        qb = q[ptr[b]:ptr[b + 1]].view(n, -1, D)
        o = torch.empty_like(qb)
        for h in range(c["Hq"]):
            s = torch.mm(qb[:, h], K[:, h // H].T) * D ** -0.5
            s[~mask] = -torch.inf
            o[:, h] = torch.mm(torch.softmax(s, 1), V[:, h // H])
        out.append(o.reshape(n, -1))
    return torch.cat(out)


def exact(case, seed):
    st = prepare(case, seed)
    return {"i8": _exact_i8, "append": _exact_append, "attn": _exact_attn}[case["kind"]](case, st)
