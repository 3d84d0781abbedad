"""The C ABI without a GPU: the library loads, exports every function the
header declares, and rejects bad arguments on the host before any HIP call."""
import ctypes
import os
import re

import numpy as np
import pytest

from tenant_composite_lora_amd import tclora

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tcl.h")


def declared_functions():
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tcl_[a-z_0-9]+)\s*\(", text)))


@pytest.fixture(scope="module")
def L():
    return tclora.lib()


def test_exports_every_declared_function(L):
    names = declared_functions()
    assert len(names) >= 12
    for n in names:
        assert hasattr(L, n), n
    assert sorted(tclora.EXPORTS) == names


def test_version(L):
    assert b"gfx950" in L.tcl_version()


def test_header_constants_match_binding():
    text = open(HEADER).read()
    consts = dict(re.findall(r"(TCL_E[A-Z]+|TCL_OK)\s*=\s*(-?\d+)", text))
    assert int(consts["TCL_OK"]) == tclora.OK
    assert int(consts["TCL_EINVAL"]) == tclora.EINVAL
    assert int(consts["TCL_EALIGN"]) == tclora.EALIGN
    assert int(consts["TCL_ENOSPC"]) == tclora.ENOSPC
    assert int(consts["TCL_EUNSUPPORTED"]) == tclora.EUNSUPPORTED
    assert int(consts["TCL_EHIP"]) == tclora.EHIP
    assert f"TCL_MAX_RANK {tclora.MAX_RANK}" in text
    assert f"TCL_MAX_PAIRS_PER_GROUP {tclora.MAX_PAIRS_PER_GROUP}" in text
    m = re.search(r"#define TCL_SCRATCH_BYTES \((\d+)u << (\d+)\)", text)
    assert m and int(m.group(1)) << int(m.group(2)) == tclora.SCRATCH_BYTES


def test_status_codes_match_oracle():
    import oracle as O
    assert (O.OK, O.EINVAL, O.ENOSPC, O.EUNSUPPORTED) == (
        tclora.OK, tclora.EINVAL, tclora.ENOSPC, tclora.EUNSUPPORTED)


def test_plan_bytes(L):
    out = ctypes.c_size_t(0)
    assert L.tcl_plan_bytes(32, 32, 96, 64, 96, ctypes.byref(out)) == 0
    small = out.value
    assert small > 0 and small % 256 == 0
    assert L.tcl_plan_bytes(4224, 4224, 10600, 256, 10600, ctypes.byref(out)) == 0
    assert out.value > small
    assert L.tcl_plan_bytes(0, 0, 0, 1, 0, ctypes.byref(out)) == 0
    for args in [(-1, 1, 1, 1, 1), (1, -1, 1, 1, 1), (1, 1, -1, 1, 1), (1, 1, 1, 0, 1),
                 (1, 1, 1, 1, -1), (1 << 25, 1, 1, 1, 1)]:
        assert L.tcl_plan_bytes(*args, ctypes.byref(out)) == tclora.EINVAL, args
        assert len(L.tcl_last_error()) > 0
    assert L.tcl_plan_bytes(1, 1, 1, 1, 1, None) == tclora.EINVAL


def _comp(T=3, G=2, NP=3, N=4, cap=4, ptr=0x1000):
    return tclora.Composites(T, G, NP, N, cap, ptr, ptr, ptr, ptr)


def test_plan_map_host_errors(L):
    h = ctypes.c_void_p(0)
    need = tclora.plan_bytes(3, 2, 3, 4, 4)
    # null composites / out
    assert L.tcl_plan_map(None, 0x10000, need, None, ctypes.byref(h)) == tclora.EINVAL
    c = _comp()
    assert L.tcl_plan_map(ctypes.byref(c), 0x10000, need, None, None) == tclora.EINVAL
    # null arrays
    c0 = tclora.Composites(3, 2, 3, 4, 4, None, 0x1000, 0x1000, 0x1000)
    assert L.tcl_plan_map(ctypes.byref(c0), 0x10000, need, None, ctypes.byref(h)) == tclora.EINVAL
    c1 = tclora.Composites(3, 2, 3, 4, 4, 0x1000, 0x1000, None, 0x1000)
    assert L.tcl_plan_map(ctypes.byref(c1), 0x10000, need, None, ctypes.byref(h)) == tclora.EINVAL
    # sizes
    cbad = _comp(N=0)
    assert L.tcl_plan_map(ctypes.byref(cbad), 0x10000, need, None, ctypes.byref(h)) == tclora.EINVAL
    # buffer
    assert L.tcl_plan_map(ctypes.byref(c), None, need, None, ctypes.byref(h)) == tclora.EINVAL
    assert L.tcl_plan_map(ctypes.byref(c), 0x10010, need, None, ctypes.byref(h)) == tclora.EALIGN
    assert L.tcl_plan_map(ctypes.byref(c), 0x10000, need - 1, None, ctypes.byref(h)) == tclora.ENOSPC
    assert b"needs" in L.tcl_last_error()
    assert h.value is None


def test_null_plan_rejected(L):
    m = tclora.ModuleDesc(4, 16, 16, 4, tclora.BF16, 0x1000, 0x2000, None)
    out = ctypes.c_size_t(0)
    assert L.tcl_workspace_bytes(None, ctypes.byref(m), 1, ctypes.byref(out)) == tclora.EINVAL
    assert L.tcl_shrink(None, ctypes.byref(m), 0x1000, 16, 0, 0x1000, None) == tclora.EINVAL
    assert L.tcl_expand(None, ctypes.byref(m), 0x1000, 0x1000, 16, 1, None) == tclora.EINVAL
    assert L.tcl_plan_status(None, None, None, None) == tclora.EINVAL
    c = tclora.Composites(4, 4, 4, 4, 4, 0x1000, 0x2000, 0x3000, 0x4000)
    ptrs = (ctypes.c_void_p * 1)(0x1000)
    lds = (ctypes.c_int64 * 1)(16)
    assert L.tcl_remap_apply(None, ctypes.byref(c), ctypes.byref(m), 1, ptrs, lds, 0, ptrs,
                             lds, 1, 0x1000, 1 << 20, None) == tclora.EINVAL
    assert L.tcl_remap_shrink(None, ctypes.byref(c), ctypes.byref(m), 1, ptrs, lds, 0, 0x1000,
                              1 << 20, None) == tclora.EINVAL
    assert L.tcl_plan_copy_out(None, *([None] * 9)) == tclora.EINVAL
    L.tcl_plan_free(None)


def test_load_ranks_host_errors(L):
    m = tclora.ModuleDesc(4, 16, 16, 8, tclora.BF16, 0x1000, 0x2000, None)
    k = np.array([0, 8, 9, 1], np.int32)          # 9 > r_max
    rc = L.tcl_module_load_ranks(ctypes.byref(m), k.ctypes.data_as(ctypes.c_void_p), 0x3000,
                                 None)
    assert rc == tclora.EINVAL and b"k[2]" in L.tcl_last_error()
    k = np.array([0, -1, 2, 1], np.int32)
    rc = L.tcl_module_load_ranks(ctypes.byref(m), k.ctypes.data_as(ctypes.c_void_p), 0x3000,
                                 None)
    assert rc == tclora.EINVAL
    assert L.tcl_module_load_ranks(ctypes.byref(m), None, 0x3000, None) == tclora.EINVAL


def test_gate_host_errors(L):
    """tcl_gate_topk rejects bad sizes and pointers on the host (no GPU)."""
    P = 0x1000

    def call(T=4, C=8, k=2, ldl=8, ldc=8, lg=P, cd=P, out=P):
        return L.tcl_gate_topk(lg, ldl, cd, ldc, T, C, k, out, out, out, out, None)

    assert call(T=-1) == tclora.EINVAL
    assert call(C=0) == tclora.EINVAL
    assert call(C=65, ldl=65, ldc=65) == tclora.EINVAL
    assert call(k=0) == tclora.EINVAL
    assert call(k=9) == tclora.EINVAL              # k > n_candidates
    assert call(ldl=7) == tclora.EINVAL
    assert call(ldc=7) == tclora.EINVAL
    assert call(lg=None) == tclora.EINVAL
    assert call(cd=None) == tclora.EINVAL
    assert call(out=None) == tclora.EINVAL
    assert call(T=1 << 30, k=4, C=8) == tclora.EINVAL  # T * k beyond 32-bit indexing
    assert call(lg=P + 2) == tclora.EALIGN
    assert b"gate" in L.tcl_last_error()


# ---------------------------------------------------------------------------
# host-resident composite tables: validated on the host, before any HIP call
# ---------------------------------------------------------------------------

def _mutations(seed, n):
    """Random tables with random defects (or none): every error class of the
    validation, alone and together, over a few hundred groups."""
    from tenant_composite_lora_amd import workloads as W
    rng = np.random.default_rng(seed)
    for i in range(n):
        T = int(rng.integers(0, 60))
        base = W.random_case(int(rng.integers(1 << 30)), T=max(T, 1), N=12, d_in=8, d_out=8,
                             r_max=2, max_pairs=6, empty_frac=0.2,
                             tokens_per_group=int(rng.integers(1, 4))).composites
        gt = base.group_tok_ptr.astype(np.int64).copy()
        gp = base.group_pair_ptr.astype(np.int64).copy()
        ad = base.pair_adapter.astype(np.int64).copy()
        al = base.pair_alpha.astype(np.float32).copy()
        N, Tn = base.n_adapters, base.n_tokens
        cap = None
        kinds = rng.choice(9, size=int(rng.integers(0, 3)), replace=False)
        for k in kinds:
            G, NP = len(gt) - 1, len(ad)
            if k == 0 and NP:
                ad[rng.integers(NP)] = rng.choice([-1, N, N + 7])
            elif k == 1 and NP:
                al[rng.integers(NP)] = rng.choice([np.nan, np.inf, -np.inf])
            elif k == 2 and G > 1:
                g = int(rng.integers(1, G))
                gt[g] = gt[g - 1] - 1 if gt[g - 1] > 0 else gt[g + 1] + 1
            elif k == 3 and G > 1:
                g = int(rng.integers(1, G))
                gp[g] = gp[g + 1] + 1
            elif k == 4:
                Tn += 1
            elif k == 5:
                for g in range(G):
                    if gp[g + 1] - gp[g] >= 2:
                        ad[gp[g] + 1] = ad[gp[g]]
                        break
            elif k == 6:
                # a group of 70 pairs appended (beyond the limit)
                ad = np.concatenate([ad, np.arange(70) % N + 0]).astype(np.int64)
                ad[-70:] = np.arange(70)
                N = max(N, 70)
                al = np.concatenate([al, np.ones(70, np.float32)])
                gp = np.concatenate([gp, [gp[-1] + 70]])
                gt = np.concatenate([gt, [gt[-1] + 1]])
                Tn += 1
            elif k == 7:
                P = int(np.sum(np.diff(gt).clip(0) * np.diff(gp).clip(0)))
                cap = max(P - 1, 0)
            elif k == 8:
                gp[-1] += 1
        yield i, gt, gp, ad, al, Tn, N, cap


def _validate_both(gt, gp, ad, al, T, N, cap):
    import oracle as O
    want = O.validate(gt, gp, ad.astype(np.int32), al, T, N, max_tuples=cap)
    rc, P, U = tclora.validate_composites(gt, gp, ad, al, N, n_tokens=T, max_tuples=cap)
    return want, rc, P, U


def test_host_validation_matches_oracle_on_hand_tables():
    """Every hand-made defect (and the defect-free tables) gets the oracle's
    code, including the precedence of EINVAL over EUNSUPPORTED over
    ENOSPC."""
    from test_gpu_parity import _bad_large_tables, _bad_tables, _pad_groups
    for name, (tp, pp, ad, al, T, cap) in _bad_tables().items():
        N = 80 if name.startswith("too_many_pairs") else 4
        for padded in (False, True):
            tq, pq = _pad_groups(tp, pp, 1100) if padded else (tp, pp)
            want, rc, _, _ = _validate_both(np.array(tq), np.array(pq), np.array(ad),
                                            np.array(al, np.float32), T, N, cap)
            assert rc == want, (name, padded, rc, want)
    for name, (tp, pp, ad, al, T, N, cap) in _bad_large_tables().items():
        want, rc, _, _ = _validate_both(tp, pp, ad, al, T, N, cap)
        assert rc == want, (name, rc, want)


def test_host_validation_matches_oracle_on_random_defects():
    import oracle as O
    seen = set()
    for i, gt, gp, ad, al, T, N, cap in _mutations(5, 400):
        want, rc, P, U = _validate_both(gt, gp, ad, al, T, N, cap)
        assert rc == want, (i, rc, want)
        seen.add(want)
        if rc == 0:
            pl = O.plan(gt, gp, ad.astype(np.int32), al)
            assert P == len(pl["tup_token"]) and U == len(pl["seg_adapter"])
    assert seen == {O.OK, O.EINVAL, O.EUNSUPPORTED, O.ENOSPC}


def test_host_plan_map_rejects_before_any_hip_call(L):
    """A bad host table is refused with its code before the library touches
    the GPU (this container has none: a HIP call would fail with EHIP)."""
    from test_gpu_parity import _bad_tables
    h = ctypes.c_void_p(0)
    for name, (tp, pp, ad, al, T, cap) in _bad_tables().items():
        if name == "fits_capacity":
            continue
        N = 80 if name.startswith("too_many_pairs") else 4
        arrs = tclora._host_table(tp, pp, ad, al)
        c = tclora._host_composites(arrs, T, N, cap if cap is not None else 16)
        import oracle as O
        want = O.validate(np.array(tp), np.array(pp), np.array(ad, np.int32),
                          np.array(al, np.float32), T, N, max_tuples=cap)
        assert want != 0
        rc = L.tcl_plan_map_host(ctypes.byref(c), 0x10000, 1 << 30, None, ctypes.byref(h))
        assert rc == want, (name, rc, want)
        assert h.value is None
        assert len(L.tcl_last_error()) > 0


def test_plan_info_and_status_async_host_errors(L):
    P, U = ctypes.c_int32(0), ctypes.c_int32(0)
    assert L.tcl_plan_info(None, ctypes.byref(P), ctypes.byref(U)) == tclora.EINVAL
    assert L.tcl_plan_status_async(None, 0x1000, None) == tclora.EINVAL
    assert L.tcl_plan_remap_host(None, None, None) == tclora.EINVAL


def test_module_init_host_errors(L):
    ok = dict(n=4, d_in=16, d_out=16, r=8, dt=tclora.BF16, A=0x1000, B=0x2000)

    def m(**kw):
        a = {**ok, **kw}
        return tclora.ModuleDesc(a["n"], a["d_in"], a["d_out"], a["r"], a["dt"], a["A"], a["B"],
                                 None)

    k = np.array([0, 8, 3, 1], np.int32)
    kp = k.ctypes.data_as(ctypes.c_void_p)
    assert L.tcl_module_init(None, kp, 0x3000, None) == tclora.EINVAL
    assert L.tcl_module_init(ctypes.byref(m(A=0)), kp, 0x3000, None) == tclora.EINVAL
    assert L.tcl_module_init(ctypes.byref(m(n=0)), kp, 0x3000, None) == tclora.EINVAL
    assert L.tcl_module_init(ctypes.byref(m(r=65)), kp, 0x3000, None) == tclora.EUNSUPPORTED
    assert L.tcl_module_init(ctypes.byref(m(r=0)), kp, 0x3000, None) == tclora.EUNSUPPORTED
    assert L.tcl_module_init(ctypes.byref(m(d_in=12)), kp, 0x3000, None) == tclora.EALIGN
    assert L.tcl_module_init(ctypes.byref(m(A=0x1008)), kp, 0x3000, None) == tclora.EALIGN
    assert L.tcl_module_init(ctypes.byref(m(dt=7)), kp, 0x3000, None) == tclora.EINVAL
    bad = np.array([0, 9, 3, 1], np.int32)
    assert L.tcl_module_init(ctypes.byref(m()), bad.ctypes.data_as(ctypes.c_void_p), 0x3000,
                             None) == tclora.EINVAL
    assert L.tcl_module_init(ctypes.byref(m()), kp, None, None) == tclora.EINVAL
    # no ranks: every adapter at r_max, no GPU call
    d = m()
    d.k_dev = 0x5000
    assert L.tcl_module_init(ctypes.byref(d), None, None, None) == tclora.OK
    assert d.k_dev is None


def test_bam_load_host_errors(L):
    """tcl_bam_load and tcl_bam_pool_init check everything on the host before
    any HIP call (the pointers here are never dereferenced)."""
    pool = tclora.ModuleDesc(4, 16, 16, 8, tclora.BF16, 0x1000, 0x2000, 0x3000, None)
    plain = tclora.ModuleDesc(4, 16, 16, 8, tclora.BF16, 0x1000, 0x2000, None, None)
    k = np.array([8, 3, 9, 0, 2], np.int32)       # adapter 2 has rank 9 > r_max
    kp = k.ctypes.data_as(ctypes.c_void_p)

    def load(desc, slots, ads, n_logical=5, kk=kp):
        s = np.ascontiguousarray(slots, np.int32)
        a = np.ascontiguousarray(ads, np.int32)
        return L.tcl_bam_load(ctypes.byref(desc), 0x4000, 0x5000, kk, n_logical, len(s),
                              s.ctypes.data, a.ctypes.data, None)

    assert load(plain, [0], [0]) == tclora.EINVAL               # not a slot pool
    assert b"slot pool" in L.tcl_last_error()
    assert load(pool, [4], [0]) == tclora.EINVAL                # slot out of range
    assert load(pool, [-1], [0]) == tclora.EINVAL
    assert load(pool, [0], [5]) == tclora.EINVAL                # adapter out of range
    assert load(pool, [1, 1], [0, 1]) == tclora.EINVAL          # slot twice
    assert load(pool, [0], [2]) == tclora.EINVAL                # rank beyond r_max
    assert b"rank 9" in L.tcl_last_error()
    assert load(pool, [0], [0], n_logical=0) == tclora.EINVAL
    assert load(pool, [], []) == tclora.OK                      # nothing to do
    assert L.tcl_bam_load(None, 0x4000, 0x5000, kp, 5, 0, None, None, None) == tclora.EINVAL
    assert L.tcl_bam_pool_init(ctypes.byref(plain), None, None, 0, None) == tclora.EINVAL
    assert L.tcl_bam_pool_init(ctypes.byref(plain), 0x3002, None, 0, None) == tclora.EALIGN
    assert L.tcl_bam_pool_init(ctypes.byref(plain), 0x3000, 0x6010, 1 << 20, None) == tclora.EALIGN
    assert L.tcl_bam_pool_init(ctypes.byref(plain), 0x3000, 0x6000, 16, None) == tclora.ENOSPC
    f32 = tclora.ModuleDesc(4, 16, 16, 8, tclora.F32, 0x1000, 0x2000, None, None)
    assert L.tcl_bam_pool_init(ctypes.byref(f32), 0x3000, 0x6000, 1 << 20, None) == \
        tclora.EUNSUPPORTED


def test_host_validation_ignores_the_unused_tail():
    """Pair entries at or beyond group_pair_ptr[G] are unused capacity: a
    tail of invalid ids, repeats and NaN weights changes neither the verdict
    nor the counts, on the host as in the oracle; a table whose pairs end
    beyond the arrays is EINVAL."""
    import oracle as O
    from tenant_composite_lora_amd import workloads as W
    rng = np.random.default_rng(31)
    for trial in range(40):
        T, N = int(rng.integers(1, 30)), int(rng.integers(2, 12))
        wl = W.random_case(300 + trial, T=T, N=N, d_in=8, d_out=8, r_max=4,
                           max_pairs=min(4, N), empty_frac=0.2)
        c = wl.composites
        gt, gp = c.group_tok_ptr.astype(np.int32), c.group_pair_ptr.astype(np.int32)
        ad, al = c.pair_adapter.astype(np.int32), c.pair_alpha.astype(np.float32)
        extra = int(rng.integers(1, 9))
        ad_t = np.concatenate([ad, rng.choice([-5, N, 10 ** 6, 0], extra).astype(np.int32)])
        al_t = np.concatenate([al, np.full(extra, np.nan, np.float32)])
        want_cut = O.validate(gt, gp, ad, al, T, N)
        want_tail = O.validate(gt, gp, ad_t, al_t, T, N)
        assert want_cut == want_tail == tclora.OK
        rc, P, U = tclora.validate_composites(gt, gp, ad_t, al_t, N, n_tokens=T)
        rc0, P0, U0 = tclora.validate_composites(gt, gp, ad, al, N, n_tokens=T)
        assert (rc, P, U) == (rc0, P0, U0) == (tclora.OK, P0, U0)
        # pairs that end beyond the arrays
        gp_bad = gp.copy()
        gp_bad[-1] = len(ad_t) + 1
        assert O.validate(gt, gp_bad, ad_t, al_t, T, N) == O.EINVAL
        assert tclora.validate_composites(gt, gp_bad, ad_t, al_t, N, n_tokens=T)[0] == \
            tclora.EINVAL


def test_i8_host_errors(L):
    """The int8 calls refuse bad arguments on the host (no GPU)."""
    P = 0x1000
    ok = dict(d_in=64, d_out=32, W=P, scale=P)

    def w(**kw):
        a = {**ok, **kw}
        return ctypes.byref(tclora.I8WeightDesc(a["d_in"], a["d_out"], a["W"], a["scale"],
                                                a.get("W_p")))

    def quant(x=P, ldx=64, xd=0, T=4, d=64, q=P, ldq=64, s=P):
        return L.tcl_i8_quant(x, ldx, xd, T, d, q, ldq, s, None)

    def prod(wt=None, q=P, ldq=64, s=P, T=4, y=P, ldy=32, yd=1):
        return L.tcl_i8_product(wt or w(), q, ldq, s, T, y, ldy, yd, None)

    def lin(wt=None, x=P, ldx=64, xd=0, T=4, y=P, ldy=32, yd=1, ws=0x10000, n=1 << 20):
        return L.tcl_i8_linear(wt or w(), x, ldx, xd, T, y, ldy, yd, ws, n, None)

    E, A, U = tclora.EINVAL, tclora.EALIGN, tclora.EUNSUPPORTED
    assert [quant(x=None), quant(q=None), quant(s=None), quant(T=-1), quant(d=8), quant(ldx=56),
            quant(ldq=48)] == [E] * 7
    assert [quant(d=40), quant(x=P + 8), quant(q=P + 8), quant(s=P + 2), quant(ldx=68),
            quant(ldq=72)] == [A] * 6
    assert quant(xd=2) == U and quant(T=0) == 0
    for f in (prod, lin):
        assert [f(y=None), f(T=-1), f(ldy=24), f(w(W=None)), f(w(scale=None)), f(w(d_in=0)),
                f(w(d_out=-8))] == [E] * 7
        assert [f(w(d_in=72)), f(w(d_out=36)), f(w(W=P + 4)), f(w(scale=P + 1)), f(y=P + 8),
                f(ldy=36)] == [A] * 6
        assert f(yd=2) == U and f(w(d_in=131072)) == U and f(T=0) == 0
    assert L.tcl_i8_product(None, P, 64, P, 4, P, 32, 1, None) == E
    assert L.tcl_i8_linear(None, P, 64, 0, 4, P, 32, 1, P, 99, None) == E
    assert [prod(q=None), prod(s=None), prod(ldq=48)] == [E] * 3
    assert [prod(q=P + 8), prod(s=P + 2), prod(ldq=72)] == [A] * 3
    assert [lin(x=None), lin(ldx=56), lin(ws=None)] == [E] * 3 and lin(xd=3) == U
    assert lin(ws=0x10010) == A and lin(n=64) == tclora.ENOSPC
    out = ctypes.c_size_t(0)
    assert L.tcl_i8_workspace_bytes(w(), 4, ctypes.byref(out)) == 0 and out.value == 1024 + 256
    assert L.tcl_i8_pack_bytes(w(), ctypes.byref(out)) == 0 and out.value == 2048
    assert L.tcl_i8_pack_bytes(w(d_in=80, d_out=8), ctypes.byref(out)) == 0 and out.value == 2048
    assert L.tcl_i8_pack_bytes(None, ctypes.byref(out)) == E and L.tcl_i8_pack_bytes(w(), None) == E
    assert L.tcl_i8_pack(w(), None, 4096, None) == E
    assert L.tcl_i8_pack(w(W=None, W_p=P), P, 4096, None) == E
    assert L.tcl_i8_pack(w(), P + 16, 4096, None) == A
    assert L.tcl_i8_pack(w(), P, 2047, None) == tclora.ENOSPC
    assert prod(w(W_p=P + 16)) == A and prod(w(W=None, W_p=P), T=0) == 0
    assert L.tcl_i8_workspace_bytes(w(), -1, ctypes.byref(out)) == E
    assert L.tcl_i8_workspace_bytes(None, 4, ctypes.byref(out)) == E
    assert L.tcl_i8_workspace_bytes(w(), 4, None) == E


def test_kv_append_host_errors(L):
    """tcl_kv_append refuses bad caches, rotations, rows and pointers on the
    host (no GPU)."""
    P = 0x1000
    E, A, U = tclora.EINVAL, tclora.EALIGN, tclora.EUNSUPPORTED

    def call(c=None, r=None, k=P, ldk=128, v=P, ldv=128, q=P, ldq=256, Hq=4, xd=0, qo=2 * P,
             ldqo=256, T=4, pos=P, slot=P, **kw):
        cd = dict(n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, stride_page=2048,
                  stride_slot=64, stride_head=1024, K=P, V=P)
        rd = dict(inv_freq=P, rot_dim=64, interleaved=0)
        cd.update({n: x for n, x in kw.items() if n in cd})
        rd.update({n: x for n, x in kw.items() if n in rd})
        cp = ctypes.byref(tclora.KVDesc(**cd)) if c is None else None
        rp = ctypes.byref(tclora.RopeDesc(**rd)) if r is None else None
        return L.tcl_kv_append(cp, rp, k, ldk, v, ldv, q, ldq, Hq, xd, qo, ldqo, T, pos, slot,
                               None)

    assert call(T=0) == 0 and call(T=0, rot_dim=0, inv_freq=None) == 0
    assert [call(c=0), call(r=0), call(T=-1), call(k=None), call(v=None), call(pos=None),
            call(slot=None), call(K=None), call(V=None), call(n_pages=0), call(n_kv_heads=0),
            call(stride_head=-8), call(ldk=120), call(ldv=64), call(Hq=0), call(qo=None),
            call(ldq=192), call(ldqo=192), call(inv_freq=None), call(qo=P, ldqo=264),
            call(qo=P, xd=1)] == [E] * 21
    assert [call(k=P + 8), call(v=P + 2), call(q=P + 8), call(qo=P + 8), call(K=P + 8),
            call(slot=P + 4), call(pos=P + 2), call(ldk=132), call(ldq=260), call(ldqo=260),
            call(stride_slot=68), call(inv_freq=P + 2)] == [A] * 12
    assert [call(page_size=24), call(page_size=0), call(page_size=2048), call(head_dim=72),
            call(head_dim=272), call(rot_dim=24), call(rot_dim=80), call(rot_dim=-16),
            call(xd=2)] == [U] * 9


def test_attn_host_errors(L):
    """The attention calls refuse bad sizes and pointers on the host (no GPU)."""
    P = 0x1000
    E, A, U = tclora.EINVAL, tclora.EALIGN, tclora.EUNSUPPORTED
    out = ctypes.c_size_t(0)

    def args(kw):
        cd = dict(n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, stride_page=2048,
                  stride_slot=64, stride_head=1024, K=P, V=P)
        bd = dict(n_seqs=3, n_groups=2, n_tokens=5, ld_prefix=4, ld_own=4, seq_tok_ptr=P,
                  group_seq_ptr=P, prefix_len=P, prefix_pages=P, own_len=P, own_pages=P)
        for d in (cd, bd):
            d.update({n: kw.pop(n) for n in list(kw) if n in d})
        return ctypes.byref(tclora.AttnBatch(**bd)), ctypes.byref(tclora.KVDesc(**cd))

    def nbytes(f=L.tcl_attn_plan_bytes, Hq=4, res=ctypes.byref(out), **kw):
        return f(*args(kw), Hq, res)

    assert nbytes() == 0
    need = out.value
    assert need % 256 == 0 and nbytes(L.tcl_attn_workspace_bytes) == 0
    ws = out.value
    assert ws >= 2 * 5 * 2 * 2 * 64 * 4

    def plan(Hq=4, p=0x10000, n=need, **kw):
        return L.tcl_attn_plan(*args(kw), Hq, p, n, None)

    def apply(Hq=4, p=0x10000, n=need, q=P, ldq=256, o=P, ldo=256, lse=None, scale=0.1,
              w=0x20000, wn=ws, **kw):
        return L.tcl_attn_apply(*args(kw), Hq, p, n, q, ldq, o, ldo, lse, scale, w, wn, None)

    for f in (nbytes, lambda **k: nbytes(L.tcl_attn_workspace_bytes, **k), plan, apply):
        assert [f(Hq=0), f(Hq=5), f(n_seqs=-1), f(n_tokens=-1), f(ld_own=-1), f(n_groups=0),
                f(seq_tok_ptr=None), f(group_seq_ptr=None), f(own_len=None), f(own_pages=None),
                f(prefix_len=None), f(prefix_pages=None), f(K=None)] == [E] * 13
        assert [f(seq_tok_ptr=P + 2), f(own_pages=P + 1), f(stride_head=4)] == [A] * 3
        assert [f(head_dim=96), f(page_size=3), f(Hq=2 * 129), f(ld_own=1 << 26),
                f(n_tokens=1 << 28), f(n_kv_heads=128, Hq=128, n_seqs=1 << 23)] == [U] * 6
    assert nbytes(res=None) == E and nbytes(L.tcl_attn_workspace_bytes, res=None) == E
    for f in (plan, apply):
        assert [f(p=None), f(p=0x10010), f(n=need - 1)] == [E, A, tclora.ENOSPC]
    assert [apply(q=None), apply(o=None), apply(w=None), apply(ldq=192), apply(ldo=248),
            apply(scale=float("nan")), apply(scale=float("inf"))] == [E] * 7
    assert [apply(q=P + 8), apply(o=P + 2), apply(lse=P + 2), apply(w=0x20010), apply(ldq=260),
            apply(ldo=260)] == [A] * 6
    assert apply(wn=ws - 1) == tclora.ENOSPC
    assert apply(n_tokens=0) == 0 and apply(n_seqs=0) == 0
    assert L.tcl_attn_status_async(None, P, None) == E
    assert L.tcl_attn_status_async(0x10000, None, None) == E
    assert L.tcl_attn_status_async(0x10010, P, None) == A


def test_launch_sizes_are_refused_on_the_host(L):
    """Batches whose launches would pass the grid's limits are refused before
    anything is launched (no GPU)."""
    P, U, N = 0x1000, tclora.EUNSUPPORTED, 1 << 24
    w = ctypes.byref(tclora.I8WeightDesc(64, 32, P, P, None))
    assert L.tcl_i8_quant(P, 64, 0, N, 64, P, 64, P, None) == U
    assert L.tcl_i8_product(w, P, 64, P, N, P, 32, 1, None) == U
    assert L.tcl_i8_linear(w, P, 64, 0, N, P, 32, 1, P, 1 << 40, None) == U
    c = tclora.KVDesc(4, 16, 2, 64, 2048, 64, 1024, P, P)
    r = tclora.RopeDesc(P, 64, 0)
    assert L.tcl_kv_append(ctypes.byref(c), ctypes.byref(r), P, 128, P, 128, None, 0, 0, 0, None, 0,
                           N, P, P, None) == U
    out = ctypes.c_size_t(0)

    def sizes(S, G, T, heads, Hq):
        c = tclora.KVDesc(4, 16, heads, 64, 2048, 64, 1024, P, P)
        b = tclora.AttnBatch(S, G, T, 4, 4, P, P, P, P, P, P)
        return L.tcl_attn_plan_bytes(ctypes.byref(b), ctypes.byref(c), Hq, ctypes.byref(out))

    assert [sizes(3, 2, N, 2, 4), sizes(N, 2, 5, 1, 1), sizes(N // 128, 2, 5, 128, 128),
            sizes(3, N // 128, 5, 128, 128), sizes(1, 1, N // 8, 8, 8 * 128)] == [U] * 5
    assert sizes(N // 256, 2, 5, 128, 128) == 0 and sizes(1, 1, N // 64, 8, 32) == 0
    w, c = ctypes.byref(tclora.AttnBatch(3, 2, 5, 4, 4, P, P, P, P, P, P)), ctypes.byref(c)
    assert L.tcl_attn_apply(w, c, 4, 0x10000, 1 << 40, P, 256, P, 256, None, 3e38, 0x20000, 1 << 40,
                            None) == tclora.EINVAL


def test_workspaces_of_the_base_operators_are_whole():
    """A given workspace counts by its bytes and has to be contiguous: what is
    expanded or strided does not hold what it counts (no GPU)."""
    import torch
    ws = torch.empty(1024, dtype=torch.uint8)
    assert tclora._fits("x", ws, 1024) and not tclora._fits("x", ws, 1025)
    assert tclora._fits("x", ws.view(torch.float32), 1024) and not tclora._fits("x", None, 0)
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), ws[::2], ws.view(32, 32).t()):
        with pytest.raises(ValueError):
            tclora._fits("x", bad, 16)


def test_i8_sizes_beyond_the_grid_are_refused(L):
    """Weights and results whose launches would pass the grid's limits (no
    GPU): the calls say so before anything is launched."""
    P, U = 0x1000, tclora.EUNSUPPORTED
    out = ctypes.c_size_t(0)

    def w(d_in, d_out):
        return ctypes.byref(tclora.I8WeightDesc(d_in, d_out, P, P, None))

    for n in (1 << 27, (1 << 31) - 8):
        assert L.tcl_i8_pack_bytes(w(16, n), ctypes.byref(out)) == U
        assert L.tcl_i8_workspace_bytes(w(16, n), 1, ctypes.byref(out)) == U
        assert L.tcl_i8_product(w(16, n), P, 16, P, 1, P, n, 1, None) == U
        assert L.tcl_i8_linear(w(16, n), P, 16, 0, 1, P, n, 1, 0x10000, 1 << 20, None) == U
    assert L.tcl_i8_pack_bytes(w(16, (1 << 27) - 8), ctypes.byref(out)) == 0
    big = 1 << 20
    assert L.tcl_i8_product(w(16, big), P, 16, P, 1 << 16, P, big, 1, None) == U
    assert L.tcl_i8_linear(w(16, big), P, 16, 0, 1 << 16, P, big, 1, 0x10000, 1 << 40, None) == U
    assert L.tcl_i8_pack_bytes(w(65536, big), ctypes.byref(out)) == 0 and out.value == 1 << 36
    assert L.tcl_i8_pack(w(65536, big), P, out.value, None) == U


def test_kv_append_norm_host_errors(L):
    """The append with norms refuses what the plain one refuses, and bad norms
    (no GPU)."""
    P = 0x1000
    E, A, U = tclora.EINVAL, tclora.EALIGN, tclora.EUNSUPPORTED

    def call(n=None, T=4, k=P, ldk=128, rot=64, head_dim=64, xd=0, **kw):
        nd = dict(w_q=P, w_k=P, stride_q=0, stride_k=64, eps=1e-6)
        nd.update(kw)
        c = tclora.KVDesc(4, 16, 2, head_dim, 2048, 64, 1024, P, P)
        r = tclora.RopeDesc(P, rot, 0)
        norm = ctypes.byref(tclora.HeadNormDesc(**nd)) if n is None else None
        return L.tcl_kv_append_norm(ctypes.byref(c), ctypes.byref(r), norm, k, ldk, P, 128, P, 256, 4, xd,
                                    2 * P, 256, T, P, P, None)

    assert call(T=0) == 0 and call(T=0, w_q=None, w_k=None, eps=0.0) == 0
    assert [call(n=0), call(eps=-1e-9), call(eps=float("nan")), call(eps=float("inf")),
            call(stride_q=-64), call(stride_k=-4), call(T=-1), call(k=None), call(ldk=120)] == [E] * 9
    assert [call(w_q=P + 8), call(w_k=P + 4), call(stride_q=2), call(stride_k=65), call(k=P + 8)] == [A] * 5
    assert [call(rot=24), call(head_dim=72), call(xd=2), call(T=1 << 24)] == [U] * 4


def test_kv_map_host_errors(L):
    """tcl_kv_map refuses bad sizes and pointers on the host (no GPU)."""
    P = 0x1000
    E, A, U = tclora.EINVAL, tclora.EALIGN, tclora.EUNSUPPORTED
    ints = ("n_new", "group_seq_ptr", "prefix_len", "own_len", "free_pages", "used", "own_pages",
            "seq_tok_ptr", "pos", "own_len_out", "used_out", "status")

    def call(c=None, b=None, n_pages=4, page_size=16, **kw):
        bd = dict(n_seqs=3, n_groups=2, n_tokens=5, n_free=4, ld_own=4, slot=P, **{n: P for n in ints})
        bd.update(kw)
        cp = ctypes.byref(tclora.KVDesc(n_pages, page_size, 1, 16, 256, 16, 16, P, P)) if c is None else None
        bp = ctypes.byref(tclora.MapBatch(**bd)) if b is None else None
        return L.tcl_kv_map(cp, bp, None)

    assert [call(c=0), call(b=0), call(n_pages=0)] == [E] * 3 and call(page_size=24) == U
    assert [call(**{n: -1}) for n in ("n_seqs", "n_groups", "n_tokens", "n_free", "ld_own")] == [E] * 5
    assert [call(**{n: None}) for n in (*ints, "slot")] == [E] * 13
    assert call(n_groups=0) == E
    assert [call(**{n: P + 2}) for n in ints] == [A] * 12 and call(slot=P + 4) == A
    N = 1 << 24
    assert [call(n_seqs=N), call(n_groups=N), call(n_tokens=N), call(ld_own=1 << 25)] == [U] * 4


def test_attn_window_host_errors(L):
    """The windowed attention refuses bad windows, and what the one without
    refuses (no GPU)."""
    P = 0x1000
    E, A, U = tclora.EINVAL, tclora.EALIGN, tclora.EUNSUPPORTED
    c = ctypes.byref(tclora.KVDesc(4, 16, 2, 64, 2048, 64, 1024, P, P))
    out = ctypes.c_size_t(0)

    def batch(**kw):
        bd = dict(n_seqs=3, n_groups=2, n_tokens=5, ld_prefix=4, ld_own=4, seq_tok_ptr=P,
                  group_seq_ptr=P, prefix_len=P, prefix_pages=P, own_len=P, own_pages=P)
        bd.update(kw)
        return ctypes.byref(tclora.AttnBatch(**bd))

    assert L.tcl_attn_plan_bytes(batch(), c, 4, ctypes.byref(out)) == 0
    need = out.value
    assert L.tcl_attn_workspace_bytes(batch(), c, 4, ctypes.byref(out)) == 0
    ws = out.value

    def plan(Hq=4, W=8, N=2, p=0x10000, n=need, **kw):
        return L.tcl_attn_window_plan(batch(**kw), c, Hq, W, N, p, n, None)

    def apply(Hq=4, W=8, N=2, p=0x10000, n=need, q=P, o=P, w=0x20000, wn=ws, ldq=256, **kw):
        return L.tcl_attn_window_apply(batch(**kw), c, Hq, W, N, p, n, q, ldq, o, 256, None, 0.1, w, wn, None)

    for f in (plan, apply):
        assert [f(W=0), f(W=-5), f(N=-1), f(Hq=5), f(n_seqs=-1), f(own_len=None), f(p=None)] == [E] * 7
        assert [f(p=0x10010), f(n=need - 1), f(own_pages=P + 1), f(n_tokens=1 << 28)] == [
            A, tclora.ENOSPC, A, U]
    assert [apply(q=None), apply(o=None), apply(w=None), apply(ldq=192)] == [E] * 4
    assert apply(wn=ws - 1) == tclora.ENOSPC and apply(q=P + 8) == A
    assert apply(n_tokens=0) == 0 and apply(n_seqs=0, W=(1 << 31) - 1, N=(1 << 31) - 1) == 0


def test_windows_beyond_32_bits(L):
    """Windows and sinks that 32 bits do not hold: more than all keys where they
    are positive, refused as any other where they are negative (no GPU)."""
    P = 0x10000
    c = ctypes.byref(tclora.KVDesc(4, 16, 2, 64, 2048, 64, 1024, P, P))
    b = ctypes.byref(tclora.AttnBatch(0, 0, 0, 4, 4))

    def rc(window, sinks=0):
        return L.tcl_attn_window_apply(b, c, 4, *tclora.window_limits(window, sinks), P, 1 << 30, P, 256, P,
                                       256, None, 0.1, P, 1 << 40, None)

    for big in (5, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, 1 << 40):
        assert rc(big) == 0 and rc(1, big) == 0
        assert tclora.window_limits(big, 0) == (min(big, (1 << 31) - 1), 0)
    for bad in (0, -1, -(1 << 31), 5 - (1 << 32), -(1 << 40)):
        assert rc(bad) == tclora.EINVAL
        assert bad == 0 or rc(1, bad) == tclora.EINVAL


def test_i4_host_errors(L):
    """The 4-bit calls refuse bad weights, sizes and pointers on the host (no
    GPU)."""
    P = 0x1000
    E, A, U = tclora.EINVAL, tclora.EALIGN, tclora.EUNSUPPORTED
    out = ctypes.c_size_t(0)

    def w(**kw):
        d = dict(d_in=128, d_out=32, group=32, zeros=1, W=P, scale=P, zero=P, W_p=P)
        d.update(kw)
        return ctypes.byref(tclora.I4WeightDesc(**d))

    def nbytes(**kw):
        return L.tcl_i4_pack_bytes(w(**kw), ctypes.byref(out))

    def pack(p=P, n=1 << 40, **kw):
        return L.tcl_i4_pack(w(**kw), p, n, None)

    def lin(x=P, ldx=128, T=4, y=P, ldy=32, yd=1, ws=P, n=1 << 40, **kw):
        return L.tcl_i4_linear(w(**kw), x, ldx, T, y, ldy, yd, ws, n, None)

    assert nbytes() == 0 and out.value == 2048 + 4 * 128 + 256  # (zero points: 128)
    assert nbytes(zeros=0, d_in=256, group=256) == 0 and out.value == 2 * 2048 + 256  # (scales: 128)
    assert L.tcl_i4_pack_bytes(w(), None) == E
    for f in (nbytes, pack, lin):
        assert [f(d_in=0), f(d_out=-8), f(d_in=96, group=64), f(zeros=2), f(zeros=-1)] == [E] * 5
        assert [f(group=0), f(group=16), f(group=48), f(group=96), f(group=192), f(group=-32),
                f(d_in=(1 << 20) + 32), f(d_out=1 << 26)] == [U] * 8
        assert [f(d_out=36), f(W=P + 8), f(scale=P + 2), f(W_p=P + 16)] == [A] * 4
    assert L.tcl_i4_pack_bytes(None, ctypes.byref(out)) == E
    assert L.tcl_i4_pack(None, P, 9, None) == E and L.tcl_i4_linear(None, P, 128, 4, P, 32, 1, P, 9, None) == E
    assert nbytes(d_in=1 << 20, d_out=1 << 18) == U
    assert [pack(p=None), pack(W=None), pack(scale=None), pack(zero=None)] == [E] * 4
    assert pack(p=P + 16) == A and pack(n=2047) == tclora.ENOSPC
    assert [lin(x=None), lin(y=None), lin(W_p=None), lin(T=-1), lin(ldx=120), lin(ldy=24)] == [E] * 6
    assert [lin(x=P + 8), lin(y=P + 4), lin(ldx=132), lin(ldy=36)] == [A] * 4
    assert [lin(yd=2), lin(T=1 << 24), lin(d_out=1 << 20, ldy=1 << 20, T=1 << 16)] == [U] * 3
    assert lin(T=0) == 0 and lin(d_out=0, x=None) == 0
    assert lin(T=0, W=None, scale=None, zero=None) == 0
    assert [L.tcl_i4_workspace_bytes(w(), T, ctypes.byref(out)) for T in (16, 17)] == [0, 0]
    for kw, n in ((dict(d_out=25600), 8192 + 512),  # 32 tokens: one block and one step of four groups
                  (dict(d_in=8192), 8 * 17 * 32 * 4)):  # parts of eight workgroups
        assert L.tcl_i4_workspace_bytes(w(**kw), 17, ctypes.byref(out)) == 0 and out.value == n
        kw = dict(T=17, ldx=8192, ldy=25600, **kw)
        assert [lin(ws=None, **kw), lin(ws=P + 16, **kw), lin(n=n - 1, **kw)] == [E, A, tclora.ENOSPC]
    assert L.tcl_i4_workspace_bytes(w(), 4, ctypes.byref(out)) == 0 and out.value == 0
    assert L.tcl_i4_workspace_bytes(w(), -1, ctypes.byref(out)) == E
    assert L.tcl_i4_workspace_bytes(None, 4, ctypes.byref(out)) == E
    assert L.tcl_i4_workspace_bytes(w(), 4, None) == E
