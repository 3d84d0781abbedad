"""Python binding of libtclora (ctypes).

Argument marshalling only: every step of the apply runs in the library's HIP
kernels.  PyTorch supplies device memory and the stream (the current torch
stream of the tensors' device).  The library must be built
(``python -m tenant_composite_lora_amd.build``); nothing here computes a
result on the host, and a missing library raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtclora.so")

OK, EINVAL, EALIGN, ENOSPC, EUNSUPPORTED, EHIP = 0, -1, -2, -3, -4, -5
BF16, F32 = 0, 1
MAX_RANK = 64
MAX_PAIRS_PER_GROUP = 64

_NAMES = {OK: "OK", EINVAL: "EINVAL", EALIGN: "EALIGN", ENOSPC: "ENOSPC",
          EUNSUPPORTED: "EUNSUPPORTED", EHIP: "EHIP"}

EXPORTS = ["tcl_last_error", "tcl_version", "tcl_plan_bytes", "tcl_plan_map", "tcl_plan_remap",
           "tcl_plan_status", "tcl_plan_copy_out", "tcl_plan_free", "tcl_module_load_ranks",
           "tcl_workspace_bytes", "tcl_shrink", "tcl_expand", "tcl_fused_apply",
           "tcl_fused_shrink", "tcl_fused_expand", "tcl_remap_apply", "tcl_remap_shrink",
           "tcl_gate_topk", "tcl_factor_workspace_bytes",
           "tcl_factor_balanced", "tcl_rank_uniform", "tcl_rank_spectral",
           "tcl_bam_create", "tcl_bam_free", "tcl_bam_acquire", "tcl_bam_slots", "tcl_lag_select",
           "tcl_module_init", "tcl_composites_validate", "tcl_plan_map_host",
           "tcl_plan_remap_host", "tcl_plan_info", "tcl_plan_status_async",
           "tcl_module_pack_bytes", "tcl_module_pack", "tcl_fused_apply_noalloc",
           "tcl_bam_pool_init", "tcl_bam_load",
           "tcl_i8_quant", "tcl_i8_product", "tcl_i8_workspace_bytes", "tcl_i8_linear",
           "tcl_i8_pack_bytes", "tcl_i8_pack",
           "tcl_kv_append", "tcl_attn_plan_bytes", "tcl_attn_workspace_bytes", "tcl_attn_plan",
           "tcl_attn_status_async", "tcl_attn_apply", "tcl_kv_append_norm", "tcl_kv_map",
           "tcl_attn_window_plan", "tcl_attn_window_apply",
           "tcl_i4_pack_bytes", "tcl_i4_pack", "tcl_i4_workspace_bytes", "tcl_i4_linear"]

# bytes of the static device workspace of tcl_fused_apply_noalloc
SCRATCH_BYTES = 32 << 20


class TclError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_NAMES.get(code, code)}: {msg}")
        self.code = code


class Composites(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("n_pairs", ctypes.c_int32), ("n_adapters", ctypes.c_int32),
                ("max_tuples", ctypes.c_int32),
                ("group_tok_ptr", ctypes.c_void_p), ("group_pair_ptr", ctypes.c_void_p),
                ("pair_adapter", ctypes.c_void_p), ("pair_alpha", ctypes.c_void_p)]


class ModuleDesc(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("d_in", ctypes.c_int32),
                ("d_out", ctypes.c_int32), ("r_max", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("A_t", ctypes.c_void_p),
                ("B_t", ctypes.c_void_p), ("k_dev", ctypes.c_void_p),
                ("B_k", ctypes.c_void_p)]


class I8WeightDesc(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("W", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("W_p", ctypes.c_void_p)]


class I4WeightDesc(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("group", ctypes.c_int32),
                ("zeros", ctypes.c_int32), ("W", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("zero", ctypes.c_void_p), ("W_p", ctypes.c_void_p)]


class KVDesc(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("stride_page", ctypes.c_int64), ("stride_slot", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("K", ctypes.c_void_p), ("V", ctypes.c_void_p)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class HeadNormDesc(ctypes.Structure):
    _fields_ = [("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p),
                ("stride_q", ctypes.c_int64), ("stride_k", ctypes.c_int64),
                ("eps", ctypes.c_float)]


class MapBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_seqs", "n_groups", "n_tokens", "n_free", "ld_own")] + [
        (n, ctypes.c_void_p) for n in ("n_new", "group_seq_ptr", "prefix_len", "own_len", "free_pages",
                                       "used", "own_pages", "seq_tok_ptr", "pos", "slot",
                                       "own_len_out", "used_out", "status")]


class AttnBatch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("n_tokens", ctypes.c_int32), ("ld_prefix", ctypes.c_int32),
                ("ld_own", ctypes.c_int32), ("seq_tok_ptr", ctypes.c_void_p),
                ("group_seq_ptr", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
                ("prefix_pages", ctypes.c_void_p), ("own_len", ctypes.c_void_p),
                ("own_pages", ctypes.c_void_p)]


_lib = None


def lib(path: Optional[str] = None):
    """Load libtclora.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} not found: build it with `python -m tenant_composite_lora_amd.build`")
    L = ctypes.CDLL(p)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.tcl_last_error.restype = ctypes.c_char_p
    L.tcl_version.restype = ctypes.c_char_p
    L.tcl_plan_bytes.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    L.tcl_plan_map.argtypes = [ctypes.POINTER(Composites), vp, sz, vp, ctypes.POINTER(vp)]
    L.tcl_plan_remap.argtypes = [vp, ctypes.POINTER(Composites), vp]
    L.tcl_plan_status.argtypes = [vp, vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    L.tcl_plan_copy_out.argtypes = [vp] * 9 + [vp]
    L.tcl_plan_free.argtypes = [vp]
    L.tcl_plan_free.restype = None
    L.tcl_module_load_ranks.argtypes = [ctypes.POINTER(ModuleDesc), vp, vp, vp]
    L.tcl_module_init.argtypes = [ctypes.POINTER(ModuleDesc), vp, vp, vp]
    L.tcl_composites_validate.argtypes = [ctypes.POINTER(Composites), ctypes.POINTER(i32),
                                          ctypes.POINTER(i32)]
    L.tcl_plan_map_host.argtypes = [ctypes.POINTER(Composites), vp, sz, vp, ctypes.POINTER(vp)]
    L.tcl_plan_remap_host.argtypes = [vp, ctypes.POINTER(Composites), vp]
    L.tcl_plan_info.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    L.tcl_plan_status_async.argtypes = [vp, vp, vp]
    L.tcl_module_pack_bytes.argtypes = [ctypes.POINTER(ModuleDesc), ctypes.POINTER(sz)]
    L.tcl_module_pack.argtypes = [ctypes.POINTER(ModuleDesc), vp, sz, vp]
    L.tcl_workspace_bytes.argtypes = [vp, ctypes.POINTER(ModuleDesc), i32, ctypes.POINTER(sz)]
    L.tcl_shrink.argtypes = [vp, ctypes.POINTER(ModuleDesc), vp, i64, i32, vp, vp]
    L.tcl_expand.argtypes = [vp, ctypes.POINTER(ModuleDesc), vp, vp, i64, i32, vp]
    L.tcl_fused_apply.argtypes = [vp, ctypes.POINTER(ModuleDesc), i32, ctypes.POINTER(vp),
                                  ctypes.POINTER(i64), i32, ctypes.POINTER(vp),
                                  ctypes.POINTER(i64), i32, vp, sz, vp]
    L.tcl_fused_apply_noalloc.argtypes = [vp, ctypes.POINTER(ModuleDesc), i32,
                                          ctypes.POINTER(vp), ctypes.POINTER(i64), i32,
                                          ctypes.POINTER(vp), ctypes.POINTER(i64), i32, vp]
    L.tcl_fused_shrink.argtypes = [vp, ctypes.POINTER(ModuleDesc), i32, ctypes.POINTER(vp),
                                   ctypes.POINTER(i64), i32, vp, sz, vp]
    L.tcl_fused_expand.argtypes = [vp, ctypes.POINTER(ModuleDesc), i32, vp, sz,
                                   ctypes.POINTER(vp), ctypes.POINTER(i64), i32, vp]
    L.tcl_remap_apply.argtypes = [vp, ctypes.POINTER(Composites), ctypes.POINTER(ModuleDesc),
                                  i32, ctypes.POINTER(vp), ctypes.POINTER(i64), i32,
                                  ctypes.POINTER(vp), ctypes.POINTER(i64), i32, vp, sz, vp]
    L.tcl_remap_shrink.argtypes = [vp, ctypes.POINTER(Composites), ctypes.POINTER(ModuleDesc),
                                   i32, ctypes.POINTER(vp), ctypes.POINTER(i64), i32, vp, sz, vp]
    L.tcl_gate_topk.argtypes = [vp, i64, vp, i64, i32, i32, i32, vp, vp, vp, vp, vp]
    L.tcl_factor_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    L.tcl_factor_balanced.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.tcl_rank_uniform.argtypes = [vp, vp, i32, i32, vp, ctypes.POINTER(i64)]
    L.tcl_rank_spectral.argtypes = [vp, i64, vp, vp, vp, i32, i64, vp]
    L.tcl_bam_create.argtypes = [i32, ctypes.POINTER(vp)]
    L.tcl_bam_free.argtypes = [vp]
    L.tcl_bam_free.restype = None
    L.tcl_bam_acquire.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp]
    L.tcl_bam_slots.argtypes = [vp, vp]
    L.tcl_bam_pool_init.argtypes = [ctypes.POINTER(ModuleDesc), vp, vp, sz, vp]
    L.tcl_bam_load.argtypes = [ctypes.POINTER(ModuleDesc), vp, vp, vp, i32, i32, vp, vp, vp]
    L.tcl_i8_quant.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, vp]
    L.tcl_i8_product.argtypes = [ctypes.POINTER(I8WeightDesc), vp, i64, vp, i32, vp, i64, i32, vp]
    L.tcl_i8_workspace_bytes.argtypes = [ctypes.POINTER(I8WeightDesc), i32, ctypes.POINTER(sz)]
    L.tcl_i8_pack_bytes.argtypes = [ctypes.POINTER(I8WeightDesc), ctypes.POINTER(sz)]
    L.tcl_i8_pack.argtypes = [ctypes.POINTER(I8WeightDesc), vp, sz, vp]
    L.tcl_i8_linear.argtypes = [ctypes.POINTER(I8WeightDesc), vp, i64, i32, i32, vp, i64, i32, vp,
                                sz, vp]
    L.tcl_i4_pack_bytes.argtypes = [ctypes.POINTER(I4WeightDesc), ctypes.POINTER(sz)]
    L.tcl_i4_pack.argtypes = [ctypes.POINTER(I4WeightDesc), vp, sz, vp]
    L.tcl_i4_workspace_bytes.argtypes = [ctypes.POINTER(I4WeightDesc), i32, ctypes.POINTER(sz)]
    L.tcl_i4_linear.argtypes = [ctypes.POINTER(I4WeightDesc), vp, i64, i32, vp, i64, i32, vp, sz, vp]
    L.tcl_kv_append.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(RopeDesc), vp, i64, vp, i64,
                                vp, i64, i32, i32, vp, i64, i32, vp, vp, vp]
    L.tcl_kv_append_norm.argtypes = [*L.tcl_kv_append.argtypes[:2], ctypes.POINTER(HeadNormDesc),
                                     *L.tcl_kv_append.argtypes[2:]]
    L.tcl_kv_map.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(MapBatch), vp]
    bp, cp = ctypes.POINTER(AttnBatch), ctypes.POINTER(KVDesc)
    L.tcl_attn_plan_bytes.argtypes = [bp, cp, i32, ctypes.POINTER(sz)]
    L.tcl_attn_workspace_bytes.argtypes = [bp, cp, i32, ctypes.POINTER(sz)]
    L.tcl_attn_plan.argtypes = [bp, cp, i32, vp, sz, vp]
    L.tcl_attn_status_async.argtypes = [vp, vp, vp]
    L.tcl_attn_apply.argtypes = [bp, cp, i32, vp, sz, vp, i64, vp, i64, vp, ctypes.c_float, vp, sz,
                                 vp]
    L.tcl_attn_window_plan.argtypes = [bp, cp, i32, i32, i32, vp, sz, vp]
    L.tcl_attn_window_apply.argtypes = [bp, cp, i32, i32, *L.tcl_attn_apply.argtypes[2:]]
    L.tcl_lag_select.argtypes = [vp, vp, vp, i32, vp, i32, ctypes.c_double, ctypes.c_double,
                                 i32, i32, vp, vp]
    if path is None:
        _lib = L
    return L


def check(rc: int) -> None:
    if rc != OK:
        raise TclError(rc, lib().tcl_last_error().decode(errors="replace"))


def _stream(dev: torch.device, stream=None) -> int:
    if stream is not None:
        return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    return int(torch.cuda.current_stream(dev).cuda_stream)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return BF16
    if t == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def plan_bytes(n_tokens: int, n_groups: int, n_pairs: int, n_adapters: int,
               max_tuples: int) -> int:
    out = ctypes.c_size_t(0)
    check(lib().tcl_plan_bytes(n_tokens, n_groups, n_pairs, n_adapters, max_tuples,
                               ctypes.byref(out)))
    return out.value


def _host_table(group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha):
    import numpy as np
    return (np.ascontiguousarray(group_tok_ptr, dtype=np.int32),
            np.ascontiguousarray(group_pair_ptr, dtype=np.int32),
            np.ascontiguousarray(pair_adapter, dtype=np.int32),
            np.ascontiguousarray(pair_alpha, dtype=np.float32))


def _host_composites(arrs, n_tokens: int, n_adapters: int, max_tuples: int) -> Composites:
    gtp, gpp, pa, pw = arrs
    ptr = lambda a: a.ctypes.data if a.size else None  # noqa: E731
    return Composites(int(n_tokens), gtp.shape[0] - 1, pa.shape[0], int(n_adapters),
                      int(max_tuples), ptr(gtp), ptr(gpp), ptr(pa), ptr(pw))


def validate_composites(group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha,
                        n_adapters: int, n_tokens: Optional[int] = None,
                        max_tuples: Optional[int] = None):
    """Host-side check of a HOST-resident table (tcl_composites_validate, no
    GPU): returns (status code, tuples, segments)."""
    arrs = _host_table(group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha)
    T = int(arrs[0][-1]) if n_tokens is None and arrs[0].size else int(n_tokens or 0)
    cap = (1 << 31) - 1 if max_tuples is None else int(max_tuples)
    c = _host_composites(arrs, T, n_adapters, cap)
    P, U = ctypes.c_int32(0), ctypes.c_int32(0)
    rc = lib().tcl_composites_validate(ctypes.byref(c), ctypes.byref(P), ctypes.byref(U))
    return rc, P.value, U.value


class Plan:
    """A mapped batch: tuples reordered by adapter id plus the token index.

    ``group_tok_ptr``, ``group_pair_ptr``, ``pair_adapter`` (int32) and
    ``pair_alpha`` (float32) are device tensors.  ``max_tuples`` bounds the
    tuple count; if omitted it is taken as n_tokens * max pairs per group
    computed from ``group_pair_ptr`` on the device (a small reduction)."""

    def __init__(self, group_tok_ptr: torch.Tensor, group_pair_ptr: torch.Tensor,
                 pair_adapter: torch.Tensor, pair_alpha: torch.Tensor, n_adapters: int,
                 n_tokens: Optional[int] = None, max_tuples: Optional[int] = None,
                 buf: Optional[torch.Tensor] = None, stream=None):
        dev = group_tok_ptr.device
        self.device = dev
        G = int(group_tok_ptr.shape[0]) - 1
        NP = int(pair_adapter.shape[0])
        if n_tokens is None:
            # the token count is the last CSR entry (a 4-byte read-back)
            n_tokens = int(group_tok_ptr[-1].item()) if group_tok_ptr.numel() else 0
        if max_tuples is None:
            if G > 0:
                tl = (group_tok_ptr[1:] - group_tok_ptr[:-1]).to(torch.int64)
                pl = (group_pair_ptr[1:] - group_pair_ptr[:-1]).to(torch.int64)
                max_tuples = int((tl * pl).sum().item())
            else:
                max_tuples = 0
        T = int(n_tokens)
        self.n_tokens, self.n_groups, self.n_pairs = T, G, NP
        self.n_adapters, self.max_tuples = int(n_adapters), int(max_tuples)
        nbytes = plan_bytes(T, G, NP, n_adapters, self.max_tuples)
        if buf is None:
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        self.buf = buf
        # keep the inputs alive until the mapping kernel has run
        self._inputs = (group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha)
        self._c = Composites(T, G, NP, int(n_adapters), self.max_tuples,
                             _ptr(group_tok_ptr), _ptr(group_pair_ptr), _ptr(pair_adapter),
                             _ptr(pair_alpha))
        h = ctypes.c_void_p(0)
        check(lib().tcl_plan_map(ctypes.byref(self._c), buf.data_ptr(), buf.numel(),
                                 _stream(dev, stream), ctypes.byref(h)))
        self.handle = h

    def remap(self, group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha, n_tokens: int,
              stream=None) -> None:
        G = int(group_tok_ptr.shape[0]) - 1
        NP = int(pair_adapter.shape[0])
        self._inputs = (group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha)
        self._c = Composites(int(n_tokens), G, NP, self.n_adapters, self.max_tuples,
                             _ptr(group_tok_ptr), _ptr(group_pair_ptr), _ptr(pair_adapter),
                             _ptr(pair_alpha))
        check(lib().tcl_plan_remap(self.handle, ctypes.byref(self._c), _stream(self.device, stream)))
        self.n_tokens, self.n_groups, self.n_pairs = int(n_tokens), G, NP

    @classmethod
    def from_host(cls, group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha,
                  n_adapters: int, device, n_tokens: Optional[int] = None,
                  max_tuples: Optional[int] = None, buf: Optional[torch.Tensor] = None,
                  stream=None) -> "Plan":
        """A plan from a HOST-resident table (numpy arrays): validated on the
        host (tcl_plan_map_host), then copied and mapped on the device."""
        import numpy as np
        arrs = _host_table(group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha)
        gtp, gpp, pa, pw = arrs
        G, NP = gtp.shape[0] - 1, pa.shape[0]
        T = int(gtp[-1]) if n_tokens is None else int(n_tokens)
        if max_tuples is None:
            max_tuples = int((np.diff(gtp.astype(np.int64)) * np.diff(gpp.astype(np.int64))).sum())
        self = cls.__new__(cls)
        self.device = torch.device(device)
        self.n_tokens, self.n_groups, self.n_pairs = T, G, NP
        self.n_adapters, self.max_tuples = int(n_adapters), int(max_tuples)
        nbytes = plan_bytes(T, G, NP, self.n_adapters, self.max_tuples)
        if buf is None:
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        self.buf = buf
        self._inputs = None
        self._c = _host_composites(arrs, T, self.n_adapters, self.max_tuples)
        h = ctypes.c_void_p(0)
        check(lib().tcl_plan_map_host(ctypes.byref(self._c), buf.data_ptr(), buf.numel(),
                                      _stream(self.device, stream), ctypes.byref(h)))
        self.handle = h
        return self

    def remap_host(self, group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha,
                   n_tokens: Optional[int] = None, stream=None) -> None:
        """Re-map with a HOST-resident table (tcl_plan_remap_host)."""
        arrs = _host_table(group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha)
        T = int(arrs[0][-1]) if n_tokens is None else int(n_tokens)
        c = _host_composites(arrs, T, self.n_adapters, self.max_tuples)
        check(lib().tcl_plan_remap_host(self.handle, ctypes.byref(c),
                                        _stream(self.device, stream)))
        self._inputs = None
        self.n_tokens, self.n_groups, self.n_pairs = T, arrs[0].shape[0] - 1, arrs[2].shape[0]

    def info(self):
        """(rc, tuples, segments) known on the host (tcl_plan_info)."""
        P, U = ctypes.c_int32(0), ctypes.c_int32(0)
        rc = lib().tcl_plan_info(self.handle, ctypes.byref(P), ctypes.byref(U))
        return rc, P.value, U.value

    def status_async(self, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Queues a copy of {code, tuples, segments, items} into a device int32
        tensor of 4 entries (tcl_plan_status_async); no synchronisation."""
        if out is None:
            out = torch.empty(4, dtype=torch.int32, device=self.device)
        check(lib().tcl_plan_status_async(self.handle, out.data_ptr(),
                                          _stream(self.device, stream)))
        return out

    def status(self, stream=None):
        P, U = ctypes.c_int32(0), ctypes.c_int32(0)
        rc = lib().tcl_plan_status(self.handle, _stream(self.device, stream), ctypes.byref(P),
                                   ctypes.byref(U))
        return rc, P.value, U.value

    def copy_out(self, stream=None) -> dict:
        """Host copy of the plan arrays (synchronises)."""
        import numpy as np
        rc, P, U = self.status(stream)
        check(rc)
        cap, N, T = self.max_tuples, self.n_adapters, self.n_tokens
        arrs = {
            "tup_token": np.zeros(cap, np.int32), "tup_adapter": np.zeros(cap, np.int32),
            "tup_alpha": np.zeros(cap, np.float32), "tup_slot": np.zeros(cap, np.int32),
            "seg_adapter": np.zeros(N, np.int32), "seg_begin": np.zeros(N + 1, np.int32),
            "tok_ptr": np.zeros(T + 1, np.int32), "tok_tuple": np.zeros(cap, np.int32),
        }
        order = ["tup_token", "tup_adapter", "tup_alpha", "tup_slot", "seg_adapter",
                 "seg_begin", "tok_ptr", "tok_tuple"]
        ptrs = [arrs[k].ctypes.data_as(ctypes.c_void_p) if arrs[k].size else None for k in order]
        check(lib().tcl_plan_copy_out(self.handle, *ptrs, _stream(self.device, stream)))
        return {
            "tup_token": arrs["tup_token"][:P], "tup_adapter": arrs["tup_adapter"][:P],
            "tup_alpha": arrs["tup_alpha"][:P], "tup_slot": arrs["tup_slot"][:P],
            "seg_adapter": arrs["seg_adapter"][:U], "seg_begin": arrs["seg_begin"][:U + 1],
            "tok_ptr": arrs["tok_ptr"], "tok_tuple": arrs["tok_tuple"][:P],
        }

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            try:
                lib().tcl_plan_free(h)
            except Exception:  # noqa: BLE001 - interpreter shutdown
                pass
            self.handle = None


class Module:
    """One projection's adapter pool: A_t [N, r_max, d_in], B_t [N, r_max,
    d_out] (rank-major, bf16 or fp32, on the GPU) and optional effective
    ranks k (host ints, loaded to the device once).  bf16 pools also get the
    rank-contiguous copy of B the prefill expand reads (tcl_module_pack)
    unless ``pack`` is False."""

    def __init__(self, A_t: torch.Tensor, B_t: torch.Tensor, k=None, stream=None,
                 pack: bool = True):
        if A_t.dim() != 3 or B_t.dim() != 3 or A_t.shape[:2] != B_t.shape[:2]:
            raise ValueError("A_t and B_t must be [N, r_max, d] with equal N and r_max")
        if A_t.dtype != B_t.dtype:
            raise ValueError("A_t and B_t must share a dtype")
        self.A_t = A_t.contiguous()
        self.B_t = B_t.contiguous()
        N, r, d_in = self.A_t.shape
        d_out = self.B_t.shape[2]
        self.desc = ModuleDesc(N, d_in, d_out, r, _dtype_code(A_t.dtype), self.A_t.data_ptr(),
                               self.B_t.data_ptr(), None)
        self.k_dev = None
        if k is not None:
            import numpy as np
            kh = np.ascontiguousarray(np.asarray(k, dtype=np.int32))
            if kh.shape != (N,):
                raise ValueError("k must have one entry per adapter")
            self.k_dev = torch.empty(N, dtype=torch.int32, device=A_t.device)
            check(lib().tcl_module_init(ctypes.byref(self.desc),
                                        kh.ctypes.data_as(ctypes.c_void_p),
                                        self.k_dev.data_ptr(), _stream(A_t.device, stream)))
        else:
            check(lib().tcl_module_init(ctypes.byref(self.desc), None, None,
                                        _stream(A_t.device, stream)))
        self.B_k = None
        if pack and self.desc.wdtype == BF16:
            nb = ctypes.c_size_t(0)
            check(lib().tcl_module_pack_bytes(ctypes.byref(self.desc), ctypes.byref(nb)))
            self.B_k = torch.empty(max(nb.value // 2, 8), dtype=torch.bfloat16,
                                   device=A_t.device)
            check(lib().tcl_module_pack(ctypes.byref(self.desc), self.B_k.data_ptr(), nb.value,
                                        _stream(A_t.device, stream)))

    @property
    def n_adapters(self):
        return self.desc.n_adapters

    @property
    def d_in(self):
        return self.desc.d_in

    @property
    def d_out(self):
        return self.desc.d_out

    @property
    def r_max(self):
        return self.desc.r_max


def shrink(plan: Plan, m: Module, x: torch.Tensor, z: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """z [max_tuples, r_max] fp32 in the plan's sorted-tuple order."""
    if z is None:
        z = torch.empty((max(plan.max_tuples, 1), m.r_max), dtype=torch.float32, device=x.device)
    check(lib().tcl_shrink(plan.handle, ctypes.byref(m.desc), x.data_ptr(), x.stride(0),
                           _dtype_code(x.dtype), z.data_ptr(), _stream(x.device, stream)))
    return z


def expand(plan: Plan, m: Module, z: torch.Tensor, y: torch.Tensor, stream=None) -> torch.Tensor:
    """y += aggregated alpha * B z, in place."""
    check(lib().tcl_expand(plan.handle, ctypes.byref(m.desc), z.data_ptr(), y.data_ptr(),
                           y.stride(0), _dtype_code(y.dtype), _stream(y.device, stream)))
    return y


def workspace_bytes(plan: Plan, mods: Sequence[Module]) -> int:
    arr = (ModuleDesc * len(mods))(*[m.desc for m in mods])
    out = ctypes.c_size_t(0)
    check(lib().tcl_workspace_bytes(plan.handle, arr, len(mods), ctypes.byref(out)))
    return out.value


class FusedCall:
    """Pre-marshalled arguments of tcl_fused_apply for repeated calls."""

    def __init__(self, plan: Plan, mods: Sequence[Module], xs: Sequence[torch.Tensor],
                 ys: Sequence[torch.Tensor], ws: Optional[torch.Tensor] = None):
        n = len(mods)
        assert len(xs) == n and len(ys) == n
        self.plan, self.mods, self.xs, self.ys = plan, list(mods), list(xs), list(ys)
        self.descs = (ModuleDesc * n)(*[m.desc for m in mods])
        self.xp = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
        self.yp = (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys])
        self.ldx = (ctypes.c_int64 * n)(*[x.stride(0) for x in xs])
        self.ldy = (ctypes.c_int64 * n)(*[y.stride(0) for y in ys])
        self.xd = _dtype_code(xs[0].dtype)
        self.yd = _dtype_code(ys[0].dtype)
        need = workspace_bytes(plan, mods)
        if ws is None or ws.numel() < need:
            ws = torch.empty(need, dtype=torch.uint8, device=xs[0].device)
        self.ws = ws
        self.n = n

    def __call__(self, stream=None):
        check(lib().tcl_fused_apply(self.plan.handle, self.descs, self.n, self.xp, self.ldx,
                                    self.xd, self.yp, self.ldy, self.yd, self.ws.data_ptr(),
                                    self.ws.numel(), _stream(self.xs[0].device, stream)))

    def noalloc(self, stream=None):
        """The same apply through tcl_fused_apply_noalloc: the library's static
        device workspace instead of self.ws."""
        check(lib().tcl_fused_apply_noalloc(self.plan.handle, self.descs, self.n, self.xp,
                                            self.ldx, self.xd, self.yp, self.ldy, self.yd,
                                            _stream(self.xs[0].device, stream)))

    def shrink(self, stream=None):
        """First half only: z of every module into the workspace."""
        check(lib().tcl_fused_shrink(self.plan.handle, self.descs, self.n, self.xp, self.ldx,
                                     self.xd, self.ws.data_ptr(), self.ws.numel(),
                                     _stream(self.xs[0].device, stream)))

    def expand(self, stream=None):
        """Second half only: y += aggregated alpha * B z from the workspace."""
        check(lib().tcl_fused_expand(self.plan.handle, self.descs, self.n, self.ws.data_ptr(),
                                     self.ws.numel(), self.yp, self.ldy, self.yd,
                                     _stream(self.xs[0].device, stream)))

    def _remap_table(self, group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha, n_tokens):
        plan = self.plan
        G = int(group_tok_ptr.shape[0]) - 1
        NP = int(pair_adapter.shape[0])
        plan._inputs = (group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha)
        plan._c = Composites(int(n_tokens), G, NP, plan.n_adapters, plan.max_tuples,
                             _ptr(group_tok_ptr), _ptr(group_pair_ptr), _ptr(pair_adapter),
                             _ptr(pair_alpha))
        return G, NP

    def remap_apply(self, group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha,
                    n_tokens: int, stream=None):
        """One step (tcl_remap_apply): re-map the plan with this composite
        table, then shrink and expand every module."""
        plan = self.plan
        G, NP = self._remap_table(group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha,
                                  n_tokens)
        check(lib().tcl_remap_apply(plan.handle, ctypes.byref(plan._c), self.descs, self.n,
                                    self.xp, self.ldx, self.xd, self.yp, self.ldy, self.yd,
                                    self.ws.data_ptr(), self.ws.numel(),
                                    _stream(self.xs[0].device, stream)))
        plan.n_tokens, plan.n_groups, plan.n_pairs = int(n_tokens), G, NP

    def remap_shrink(self, group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha,
                     n_tokens: int, stream=None):
        """First half of a step (tcl_remap_shrink); expand() completes it."""
        plan = self.plan
        G, NP = self._remap_table(group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha,
                                  n_tokens)
        check(lib().tcl_remap_shrink(plan.handle, ctypes.byref(plan._c), self.descs, self.n,
                                     self.xp, self.ldx, self.xd, self.ws.data_ptr(),
                                     self.ws.numel(), _stream(self.xs[0].device, stream)))
        plan.n_tokens, plan.n_groups, plan.n_pairs = int(n_tokens), G, NP


def fused_apply(plan: Plan, mods: Sequence[Module], xs: Sequence[torch.Tensor],
                ys: Sequence[torch.Tensor], ws: Optional[torch.Tensor] = None,
                stream=None) -> List[torch.Tensor]:
    FusedCall(plan, mods, xs, ys, ws)(stream)
    return list(ys)


def gate_topk(logits: torch.Tensor, candidates: torch.Tensor, k: int, stream=None):
    """tcl_gate_topk: the composite table of a token-level gate on the GPU.
    logits: fp32 [T, C]; candidates: int32 [T, C] adapter ids (< 0 = padding).
    Returns (group_tok_ptr, group_pair_ptr, pair_adapter, pair_alpha), device
    tensors ready for Plan / Plan.remap / FusedCall.remap_apply."""
    if logits.dim() != 2 or candidates.shape != logits.shape:
        raise ValueError("logits and candidates must both be [T, C]")
    if logits.dtype != torch.float32 or candidates.dtype != torch.int32:
        raise ValueError("logits must be float32 and candidates int32")
    T, C = logits.shape
    if T > 0 and (logits.stride(1) != 1 or candidates.stride(1) != 1):
        raise ValueError("logits and candidates must have contiguous rows")
    ldl, ldc = (logits.stride(0), candidates.stride(0)) if T > 0 else (C, C)
    dev = logits.device
    gtp = torch.empty(T + 1, dtype=torch.int32, device=dev)
    gpp = torch.empty(T + 1, dtype=torch.int32, device=dev)
    pa = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    pw = torch.empty(max(T * k, 1), dtype=torch.float32, device=dev)
    check(lib().tcl_gate_topk(logits.data_ptr(), ldl, candidates.data_ptr(),
                              ldc, T, C, k, gtp.data_ptr(), gpp.data_ptr(),
                              pa.data_ptr(), pw.data_ptr(), _stream(dev, stream)))
    return gtp, gpp, pa[:T * k], pw[:T * k]


def factor_balanced(B_t: torch.Tensor, A_t: torch.Tensor, stream=None):
    """tcl_factor_balanced: balanced factors of a batch of modules of one
    shape (LoRAForge, approach (3)).  B_t: bf16 [M, r, d_out] and A_t: bf16
    [M, r, d_in], contiguous, on one device.  Returns (F_t, T, sigma): the
    new B_t and A_t rows (bf16, same shapes), directions largest first, and
    the singular values (fp32 [M, r])."""
    if B_t.dtype != torch.bfloat16 or A_t.dtype != torch.bfloat16:
        raise TypeError("factor_balanced: B_t and A_t must be bfloat16")
    if B_t.dim() != 3 or A_t.dim() != 3 or B_t.shape[:2] != A_t.shape[:2]:
        raise ValueError("factor_balanced: B_t [M, r, d_out] and A_t [M, r, d_in] expected")
    if not (B_t.is_contiguous() and A_t.is_contiguous()):
        raise ValueError("factor_balanced: contiguous tensors expected")
    M, r, d_out = B_t.shape
    d_in = A_t.shape[2]
    L = lib()
    nb = ctypes.c_size_t()
    check(L.tcl_factor_workspace_bytes(M, d_out, d_in, r, ctypes.byref(nb)))
    dev = B_t.device
    F_t = torch.empty_like(B_t)
    T = torch.empty_like(A_t)
    sigma = torch.empty(M, r, dtype=torch.float32, device=dev)
    ws = torch.empty(max(nb.value, 1), dtype=torch.uint8, device=dev)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    check(L.tcl_factor_balanced(B_t.data_ptr(), A_t.data_ptr(), M, d_out, d_in, r,
                                F_t.data_ptr(), T.data_ptr(), sigma.data_ptr(), ws.data_ptr(),
                                nb.value, int(st.cuda_stream)))
    return F_t, T, sigma


def rank_uniform(ranks, costs, denominator: int):
    """tcl_rank_uniform (host): LoRAForge-U's kept ranks and budget P_U."""
    import numpy as np
    rk = np.ascontiguousarray(ranks, dtype=np.int32)
    cs = np.ascontiguousarray(costs, dtype=np.int64)
    u = np.empty(len(rk), dtype=np.int32)
    b = ctypes.c_int64()
    check(lib().tcl_rank_uniform(rk.ctypes.data, cs.ctypes.data, len(rk), int(denominator),
                                 u.ctypes.data, ctypes.byref(b)))
    return u, int(b.value)


def rank_spectral(sigma, ranks, costs, floors, budget: int):
    """tcl_rank_spectral (host): LoRAForge-S's kept ranks.  sigma: float64
    [M, ld] (row m's first ranks[m] entries are module m's spectrum)."""
    import numpy as np
    sg = np.ascontiguousarray(sigma, dtype=np.float64)
    rk = np.ascontiguousarray(ranks, dtype=np.int32)
    cs = np.ascontiguousarray(costs, dtype=np.int64)
    fl = np.ascontiguousarray(floors, dtype=np.int32)
    k = np.empty(len(rk), dtype=np.int32)
    ld = sg.shape[1] if sg.ndim == 2 else 0
    check(lib().tcl_rank_spectral(sg.ctypes.data, ld, rk.ctypes.data, cs.ctypes.data,
                                  fl.ctypes.data, len(rk), int(budget), k.ctypes.data))
    return k


class Bam:
    """tcl_bam_*: the adapter slot pool (host bookkeeping; the caller copies
    each loaded adapter into its slot)."""

    def __init__(self, n_slots: int):
        self.n_slots = int(n_slots)
        h = ctypes.c_void_p()
        check(lib().tcl_bam_create(self.n_slots, ctypes.byref(h)))
        self._h = h

    def acquire(self, adapters):
        """Returns (slot of each entry, [(slot, loaded adapter, evicted or -1)])."""
        import numpy as np
        a = np.ascontiguousarray(adapters, dtype=np.int32)
        n = len(a)
        so, ls, la, le = (np.empty(max(n, 1), np.int32) for _ in range(4))
        nl = ctypes.c_int32()
        check(lib().tcl_bam_acquire(self._h, a.ctypes.data, n, so.ctypes.data, ls.ctypes.data,
                                    la.ctypes.data, le.ctypes.data, ctypes.byref(nl)))
        k = nl.value
        return so[:n].copy(), list(zip(ls[:k].tolist(), la[:k].tolist(), le[:k].tolist()))

    def slots(self):
        import numpy as np
        out = np.empty(self.n_slots, np.int32)
        check(lib().tcl_bam_slots(self._h, out.ctypes.data))
        return out

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.tcl_bam_free(h)
            self._h = None


class SlotPool:
    """BAM on the GPU: n_slots device slots per module, filled from host pools.

    ``host_pools``: one (A_t, B_t, k) per module, A_t [N, r_max, d_in] and
    B_t [N, r_max, d_out] CPU tensors (bf16 or fp32; copied once into pinned
    memory here) over the N logical adapters, k their retained ranks (ints,
    or None for r_max).  ``modules`` are the device slot pools (tcl_module
    descriptors whose adapter ids are slots); load() makes a batch's adapters
    resident (tcl_bam_acquire, then tcl_bam_load for every module) and
    returns the slot of each adapter."""

    def __init__(self, n_slots: int, host_pools, device, stream=None):
        import numpy as np
        self.bam = Bam(n_slots)
        self.device = torch.device(device)
        self.n_logical = int(host_pools[0][0].shape[0])
        self.modules, self._host, self.h2d_bytes = [], [], 0
        for A_h, B_h, k in host_pools:
            if A_h.shape[0] != self.n_logical or B_h.shape[0] != self.n_logical:
                raise ValueError("every host pool holds the same logical adapters")
            A_p, B_p = A_h.contiguous().pin_memory(), B_h.contiguous().pin_memory()
            kh = None if k is None else np.ascontiguousarray(np.asarray(k, dtype=np.int32))
            _, r, d_in = A_p.shape
            d_out = B_p.shape[2]
            A_t = torch.zeros(n_slots, r, d_in, dtype=A_p.dtype, device=self.device)
            B_t = torch.zeros(n_slots, r, d_out, dtype=B_p.dtype, device=self.device)
            mod = Module(A_t, B_t, pack=False)
            mod.k_dev = torch.empty(n_slots, dtype=torch.int32, device=self.device)
            if mod.desc.wdtype == BF16:
                nb = ctypes.c_size_t(0)
                check(lib().tcl_module_pack_bytes(ctypes.byref(mod.desc), ctypes.byref(nb)))
                mod.B_k = torch.empty(max(nb.value // 2, 8), dtype=torch.bfloat16,
                                      device=self.device)
                bk, nbytes = mod.B_k.data_ptr(), nb.value
            else:
                bk, nbytes = None, 0
            check(lib().tcl_bam_pool_init(ctypes.byref(mod.desc), mod.k_dev.data_ptr(), bk,
                                          nbytes, _stream(self.device, stream)))
            self.modules.append(mod)
            self._host.append((A_p, B_p, kh))

    def load(self, adapters, stream=None):
        """Slots for the adapters of one batch (in the order given); the loads
        are queued on the stream.  Returns (slot of each entry, loads)."""
        import numpy as np
        slot_of, loads = self.bam.acquire(adapters)
        if loads:
            ls = np.ascontiguousarray([l[0] for l in loads], dtype=np.int32)
            la = np.ascontiguousarray([l[1] for l in loads], dtype=np.int32)
            for mod, (A_p, B_p, kh) in zip(self.modules, self._host):
                check(lib().tcl_bam_load(ctypes.byref(mod.desc), A_p.data_ptr(), B_p.data_ptr(),
                                         None if kh is None else kh.ctypes.data,
                                         self.n_logical, len(loads), ls.ctypes.data,
                                         la.ctypes.data, _stream(self.device, stream)))
                es = A_p.element_size()
                ks = [mod.r_max if kh is None else int(kh[a]) for a in la.tolist()]
                self.h2d_bytes += sum(ks) * (mod.d_in + mod.d_out) * es
        return slot_of, loads


def lag_select(now: float, theta: float, arrival, adapters, resident, max_batch: int,
               n_slots: int):
    """tcl_lag_select (host): the chosen request indices, in order."""
    import numpy as np
    arr = np.ascontiguousarray(arrival, dtype=np.float64)
    n = len(arr)
    ptr = np.zeros(n + 1, np.int32)
    ptr[1:] = np.cumsum([len(a) for a in adapters]) if n else []
    flat = np.ascontiguousarray(np.concatenate([np.asarray(a, np.int32) for a in adapters])
                                if n and ptr[-1] else np.zeros(1, np.int32), dtype=np.int32)
    res = np.ascontiguousarray(resident, dtype=np.int32) if len(resident) else np.zeros(1, np.int32)
    out = np.empty(max(1, min(int(max_batch), n)), np.int32)
    nc = ctypes.c_int32()
    check(lib().tcl_lag_select(arr.ctypes.data if n else None, ptr.ctypes.data, flat.ctypes.data,
                               n, res.ctypes.data, len(resident), float(now), float(theta),
                               int(max_batch), int(n_slots), out.ctypes.data, ctypes.byref(nc)))
    return out[:nc.value].tolist()


# ---------------------------------------------------------------------------
# the base model's operators around the apply
# ---------------------------------------------------------------------------
def _same_device(what: str, dev: torch.device, *tensors) -> None:
    if dev.type != "cuda":
        raise ValueError(f"{what}: tensors on the GPU expected")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"{what}: all tensors must be on {dev}")


def _rows(what: str, t: torch.Tensor, n: Optional[int] = None, d: Optional[int] = None) -> int:
    """Checks a [n, d] tensor of contiguous rows; returns its leading dimension."""
    if t.dim() != 2 or (n is not None and t.shape[0] != n) or (d is not None and t.shape[1] != d):
        want = "[rows, columns]" if d is None else f"[{'n' if n is None else n}, {d}]"
        raise ValueError(f"{what} must be {want}, got {list(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(what: str, t: torch.Tensor, n: int, dtype: torch.dtype) -> None:
    if t.shape != (n,) or t.dtype != dtype or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of {n} entries")


def _fits(what: str, ws: Optional[torch.Tensor], need: int) -> bool:
    """Whether a workspace was given and holds ``need`` bytes.  The calls write
    it from its first byte on, so its elements have to lie one behind another
    (an expanded tensor has more of them than memory)."""
    if ws is None:
        return False
    if not ws.is_contiguous():
        raise ValueError(f"{what}: ws must be contiguous")
    return ws.numel() * ws.element_size() >= need


def _stream_object(dev: torch.device, stream):
    if stream is None:
        return torch.cuda.current_stream(dev)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = _stream(dev, stream)
    return torch.cuda.ExternalStream(raw, dev) if raw else torch.cuda.default_stream(dev)


def _made_for(dev: torch.device, stream) -> None:
    """Before a call writes tensors that it makes itself: their memory may have
    been freed with work of the current stream still to run on it, so another
    stream waits for that work."""
    if stream is not None:
        s, current = _stream_object(dev, stream), torch.cuda.current_stream(dev)
        if s.cuda_stream != current.cuda_stream:
            s.wait_stream(current)


class _Made:
    """When an object made its tensors: their memory may have been freed with
    work of the stream of that time still to run on it, so the object's first
    call on another stream waits for what that stream held then.

    An event from before a capture cannot be waited for in it, nor one from a
    capture behind it: a captured call waits only where its object was made in
    the same capture (torch.cuda.graph waits for all earlier work itself).
    Objects that are called once, on the stream that they are made on, need
    none (_once)."""

    def __init__(self, dev: torch.device):
        with torch.cuda.device(dev):
            self.stream = torch.cuda.current_stream(dev)
            captured = torch.cuda.is_current_stream_capturing()
            self.event = None if captured else self.stream.record_event()
        self.waited = {int(self.stream.cuda_stream)}

    def before(self, s: torch.cuda.Stream) -> None:
        with torch.cuda.stream(s):
            captured = torch.cuda.is_current_stream_capturing()
        if self.event is not None:
            if not captured:
                s.wait_event(self.event)
                self.waited.add(int(s.cuda_stream))
        elif captured:
            with torch.cuda.stream(self.stream):
                captured = torch.cuda.is_current_stream_capturing()
            if captured:
                s.wait_stream(self.stream)


def _call(dev: torch.device, fn, args, stream, *own, made: Optional[_Made] = None) -> None:
    """fn(*args, stream) with ``dev`` the current device.  ``own``: tensors
    that the library's own objects made, each with the stream it was allocated
    on; one that the call uses on another stream, given or current, is kept
    until the work there has run.  ``made``: when the call's object made its
    own, which may have been just before."""
    i = dev.index
    st = torch._C._cuda_getCurrentRawStream(i) if stream is None else _stream(dev, stream)
    if made is not None and st not in made.waited:
        made.before(_stream_object(dev, stream))
    for t, home in own:
        if st != home:
            t.record_stream(_stream_object(dev, stream))
    if torch._C._cuda_getDevice() == i:
        rc = fn(*args, st)
    else:
        with torch.cuda.device(i):
            rc = fn(*args, st)
    if rc:
        check(rc)


def _packed(fn, args):
    """The arguments of a call that is made often, converted once."""
    return tuple(t(v) if isinstance(v, (int, float)) else v for v, t in zip(args, fn.argtypes))


class I8Weight:
    """An int8 base weight: W int8 [d_out, d_in] and its channel scales fp32
    [d_out], on the GPU (tcl_i8_weight).  The products read a copy in the
    matrix cores' order (tcl_i8_pack), made here unless ``pack`` is False;
    with it W itself is not kept.  The copy is made on ``stream`` or the
    current one: calls on others have to be ordered behind it."""

    def __init__(self, W: torch.Tensor, scale: torch.Tensor, pack: bool = True, stream=None):
        if W.dtype != torch.int8:
            raise TypeError("I8Weight: W must be int8")
        if W.dim() != 2 or not W.is_contiguous():
            raise ValueError("I8Weight: W must be [d_out, d_in], contiguous")
        _vector("I8Weight: scale", scale, W.shape[0], torch.float32)
        _same_device("I8Weight", W.device, scale)
        self.W, self.scale, self.device = W, scale, W.device
        self.d_out, self.d_in = W.shape
        self.desc = I8WeightDesc(self.d_in, self.d_out, W.data_ptr(), scale.data_ptr(), None)
        self.W_p = None
        self.home = _stream(W.device) if W.is_cuda else 0
        if pack and W.numel():
            n = ctypes.c_size_t(0)
            check(lib().tcl_i8_pack_bytes(ctypes.byref(self.desc), ctypes.byref(n)))
            self.W_p = torch.empty(n.value, dtype=torch.uint8, device=W.device)
            _made_for(W.device, stream)
            _call(W.device, lib().tcl_i8_pack,
                  (ctypes.byref(self.desc), self.W_p.data_ptr(), n.value), stream,
                  *((t, self.home) for t in (self.W_p, W)))
            self.W, self.desc.W = None, None

    def _own(self):
        return () if self.W_p is None else ((self.W_p, self.home),)


def i8_quant(x: torch.Tensor, q: Optional[torch.Tensor] = None,
             scale: Optional[torch.Tensor] = None, stream=None):
    """tcl_i8_quant: (q int8 [T, d], scale fp32 [T]) of x [T, d], bf16 or fp32."""
    ldx = _rows("i8_quant: x", x)
    T, d = x.shape
    own = []
    if q is None:
        q = torch.empty(T, d, dtype=torch.int8, device=x.device)
        own.append(q)
    if scale is None:
        scale = torch.empty(T, dtype=torch.float32, device=x.device)
        own.append(scale)
    if q.dtype != torch.int8:
        raise TypeError("i8_quant: q must be int8")
    ldq = _rows("i8_quant: q", q, T, d)
    _vector("i8_quant: scale", scale, T, torch.float32)
    _same_device("i8_quant", x.device, q, scale)
    if own:
        _made_for(x.device, stream)
    _call(x.device, lib().tcl_i8_quant,
          (x.data_ptr(), ldx, _dtype_code(x.dtype), T, d, q.data_ptr(), ldq, scale.data_ptr()),
          stream, *((t, _stream(x.device)) for t in own))
    return q, scale


def i8_product(w: I8Weight, q: torch.Tensor, scale: torch.Tensor,
               y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.bfloat16,
               stream=None) -> torch.Tensor:
    """tcl_i8_product: y [T, d_out] (written, not added to) of tokens q, scale."""
    if q.dtype != torch.int8:
        raise TypeError("i8_product: q must be int8")
    T = q.shape[0]
    ldq = _rows("i8_product: q", q, T, w.d_in)
    _vector("i8_product: scale", scale, T, torch.float32)
    own = []
    if y is None:
        y = torch.empty(T, w.d_out, dtype=y_dtype, device=q.device)
        own.append(y)
    ldy = _rows("i8_product: y", y, T, w.d_out)
    _same_device("i8_product", q.device, scale, y, w.scale)
    if own:
        _made_for(q.device, stream)
    _call(q.device, lib().tcl_i8_product,
          (ctypes.byref(w.desc), q.data_ptr(), ldq, scale.data_ptr(), T, y.data_ptr(), ldy,
           _dtype_code(y.dtype)), stream, *((t, _stream(q.device)) for t in own), *w._own())
    return y


class I8Call:
    """Pre-marshalled arguments of tcl_i8_linear for repeated calls: each call
    writes the base projection of x into y.  The workspace is the call's own
    (or ``ws``); calls that may run at the same time need one each."""

    def __init__(self, w: I8Weight, x: torch.Tensor, y: torch.Tensor,
                 ws: Optional[torch.Tensor] = None, *, _once: bool = False):
        T = x.shape[0]
        self.ldx = _rows("I8Call: x", x, T, w.d_in)
        self.ldy = _rows("I8Call: y", y, T, w.d_out)
        _same_device("I8Call", x.device, y, w.scale, ws)
        self.w, self.x, self.y, self.T = w, x, y, T
        self.xd, self.yd = _dtype_code(x.dtype), _dtype_code(y.dtype)
        need = ctypes.c_size_t(0)
        check(lib().tcl_i8_workspace_bytes(ctypes.byref(w.desc), T, ctypes.byref(need)))
        self._made = None
        if not _fits("I8Call", ws, need.value):
            ws = torch.empty(max(need.value, 256), dtype=torch.uint8, device=x.device)
            self._made = None if _once else _Made(x.device)
        self.ws, self.device = ws, x.device
        self._own = ((ws, _stream(x.device)), *w._own())
        self._fn = lib().tcl_i8_linear
        self._args = _packed(self._fn, (
            ctypes.byref(w.desc), x.data_ptr(), self.ldx, self.xd, T, y.data_ptr(), self.ldy,
            self.yd, ws.data_ptr(), ws.numel() * ws.element_size()))

    def __call__(self, stream=None) -> torch.Tensor:
        _call(self.device, self._fn, self._args, stream, *self._own, made=self._made)
        return self.y


def i8_linear(w: I8Weight, x: torch.Tensor, y: Optional[torch.Tensor] = None,
              y_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """tcl_i8_linear: the base projection of x [T, d_in]."""
    if y is None:
        y = torch.empty(x.shape[0], w.d_out, dtype=y_dtype, device=x.device)
        if stream is not None and x.is_cuda:
            y.record_stream(_stream_object(x.device, stream))
    return I8Call(w, x, y, _once=stream is None)(stream)


class I4Weight:
    """A 4-bit base weight with group scales (tcl_i4_weight): W uint8 [d_out,
    d_in / 2], the even column of a pair in the low half of its byte, scale
    fp32 [d_out, groups] and zero uint8 [d_out, groups] (None: 8), on the GPU.
    The products read a copy in the matrix cores' order (tcl_i4_pack), made
    here; W, scale and zero themselves are not kept.  The copy is made on
    ``stream`` or the current one: calls on others have to be ordered behind
    it."""

    def __init__(self, W: torch.Tensor, scale: torch.Tensor, zero: Optional[torch.Tensor] = None,
                 stream=None):
        if W.dtype != torch.uint8 or (zero is not None and zero.dtype != torch.uint8):
            raise TypeError("I4Weight: W and zero must be uint8")
        if scale.dtype != torch.float32:
            raise TypeError("I4Weight: scale must be float32")
        if W.dim() != 2 or not W.is_contiguous():
            raise ValueError("I4Weight: W must be [d_out, d_in / 2], contiguous")
        for name, t in (("scale", scale), ("zero", zero)):
            if t is not None and (t.dim() != 2 or t.shape != scale.shape or t.shape[0] != W.shape[0]
                                  or not t.is_contiguous()):
                raise ValueError(f"I4Weight: {name} must be [d_out, groups], contiguous")
        self.d_out, self.d_in, self.device = W.shape[0], 2 * W.shape[1], W.device
        if not scale.shape[1] or self.d_in % scale.shape[1]:
            raise ValueError("I4Weight: d_in must be whole groups")
        _same_device("I4Weight", W.device, scale, zero)
        self.group = self.d_in // scale.shape[1]
        self.desc = I4WeightDesc(self.d_in, self.d_out, self.group, int(zero is not None),
                                 W.data_ptr(), scale.data_ptr(), _ptr(zero), None)
        self.home = _stream(W.device)
        n = ctypes.c_size_t(0)
        check(lib().tcl_i4_pack_bytes(ctypes.byref(self.desc), ctypes.byref(n)))
        self.W_p = torch.empty(max(n.value, 256), dtype=torch.uint8, device=W.device)
        _made_for(W.device, stream)
        _call(W.device, lib().tcl_i4_pack, (ctypes.byref(self.desc), self.W_p.data_ptr(), n.value), stream,
              *((t, self.home) for t in (self.W_p, W, scale, zero) if t is not None))
        self.desc.W = self.desc.scale = self.desc.zero = None


class I4Call:
    """Pre-marshalled arguments of tcl_i4_linear for repeated calls: each call
    writes the base projection of x (bf16 [T, d_in]) into y (bf16 or fp32 [T,
    d_out]).  The workspace is the call's own (or ``ws``); calls that may run
    at the same time need one each."""

    def __init__(self, w: I4Weight, x: torch.Tensor, y: torch.Tensor,
                 ws: Optional[torch.Tensor] = None, *, _once: bool = False):
        if x.dtype != torch.bfloat16:
            raise TypeError("I4Call: x must be bfloat16")
        T = x.shape[0]
        self.ldx, self.ldy = _rows("I4Call: x", x, T, w.d_in), _rows("I4Call: y", y, T, w.d_out)
        _same_device("I4Call", x.device, y, w.W_p, ws)
        self.w, self.x, self.y, self.T, self.device = w, x, y, T, x.device
        need = ctypes.c_size_t(0)
        check(lib().tcl_i4_workspace_bytes(ctypes.byref(w.desc), T, ctypes.byref(need)))
        self._made = None
        if not need.value:
            ws = None
        elif not _fits("I4Call", ws, need.value):
            ws = torch.empty(need.value, dtype=torch.uint8, device=x.device)
            self._made = None if _once else _Made(x.device)
        self.ws = ws
        self._own = ((w.W_p, w.home),) + (() if ws is None else ((ws, _stream(x.device)),))
        self._fn = lib().tcl_i4_linear
        self._args = _packed(self._fn, (
            ctypes.byref(w.desc), x.data_ptr(), self.ldx, T, y.data_ptr(), self.ldy,
            _dtype_code(y.dtype), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size()))

    def __call__(self, stream=None) -> torch.Tensor:
        _call(self.device, self._fn, self._args, stream, *self._own, made=self._made)
        return self.y


def i4_linear(w: I4Weight, x: torch.Tensor, y: Optional[torch.Tensor] = None,
              y_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """tcl_i4_linear: the base projection of x [T, d_in] by a 4-bit weight."""
    if y is None:
        y = torch.empty(x.shape[0], w.d_out, dtype=y_dtype, device=x.device)
        if x.is_cuda:
            _made_for(x.device, stream)
            if stream is not None:
                y.record_stream(_stream_object(x.device, stream))
    return I4Call(w, x, y, _once=stream is None)(stream)


class KVCache:
    """One layer's paged key/value cache: K and V bf16 [n_pages, page_size,
    n_kv_heads, head_dim] views of one stride pattern, the last dimension
    contiguous (a tensor kept by head inside a page is passed transposed)."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor):
        if K.dtype != torch.bfloat16 or V.dtype != torch.bfloat16:
            raise TypeError("KVCache: K and V must be bfloat16")
        if K.dim() != 4 or K.shape != V.shape:
            raise ValueError("KVCache: K and V must both be [n_pages, page_size, heads, head_dim]")
        strides = [K.stride(i) if K.shape[i] > 1 else 0 for i in range(4)]
        if strides != [V.stride(i) if V.shape[i] > 1 else 0 for i in range(4)]:
            raise ValueError("KVCache: K and V must have the same strides")
        if strides[3] != 1 or any(K.shape[i] > 1 and strides[i] == 0 for i in range(3)):
            raise ValueError("KVCache: contiguous heads that do not overlap expected")
        _same_device("KVCache", K.device, V)
        self.K, self.V = K, V
        self.device = K.device
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = K.shape
        self.desc = KVDesc(*K.shape, *strides[:3], K.data_ptr(), V.data_ptr())


class Rope:
    """Position rotation: inv_freq fp32 [rot_dim / 2] on the GPU (None: no
    rotation); pairs (j, j + rot_dim / 2), or (2j, 2j + 1) if interleaved."""

    def __init__(self, inv_freq: Optional[torch.Tensor], interleaved: bool = False):
        n = 0 if inv_freq is None else inv_freq.numel()
        if n:
            _vector("Rope: inv_freq", inv_freq, n, torch.float32)
        self.inv_freq = inv_freq
        self.desc = RopeDesc(_ptr(inv_freq) if n else None, 2 * n, int(interleaved))


class HeadNorm:
    """Norms of queries and keys by head (tcl_head_norm): weights fp32
    [head_dim] for every head or [heads, head_dim], on the GPU; None leaves q
    (or k) as it is."""

    def __init__(self, w_q: Optional[torch.Tensor], w_k: Optional[torch.Tensor], eps: float = 1e-6):
        stride = []
        for name, w in (("w_q", w_q), ("w_k", w_k)):
            if w is not None and w.dtype != torch.float32:
                raise TypeError(f"HeadNorm: {name} must be float32")
            if w is not None and (w.dim() not in (1, 2) or not w.is_contiguous()):
                raise ValueError(f"HeadNorm: {name} must be [head_dim] or [heads, head_dim], contiguous")
            stride.append(0 if w is None or w.dim() == 1 else w.shape[1])
        self.w_q, self.w_k, self.eps = w_q, w_k, float(eps)
        self.desc = HeadNormDesc(_ptr(w_q), _ptr(w_k), *stride, self.eps)

    def fit(self, n_q_heads: int, n_kv_heads: int, head_dim: int) -> None:
        """Checks the weights against a call's heads (n_q_heads 0: it has no
        queries)."""
        for name, w, n in (("w_q", self.w_q, n_q_heads), ("w_k", self.w_k, n_kv_heads)):
            if w is not None and n and tuple(w.shape) not in ((head_dim,), (n, head_dim)):
                raise ValueError(f"HeadNorm: {name} must be [{head_dim}] or [{n}, {head_dim}], got "
                                 f"{list(w.shape)}")


class AppendCall:
    """Pre-marshalled arguments of tcl_kv_append for repeated calls: k, v [T,
    heads * head_dim] rows go to ``slot`` (int64 [T]) of the cache, k rotated
    to ``pos`` (int32 [T]); with q [T, q heads * head_dim] its rotated rows go
    to q_out (bf16, made here unless given).  With ``norm`` the heads of q and
    k are normed before they are rotated (tcl_kv_append_norm).  Each call
    returns q_out."""

    def __init__(self, cache: KVCache, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                 slot: torch.Tensor, rope: Optional[Rope] = None,
                 q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None, *,
                 norm: Optional[HeadNorm] = None, _once: bool = False):
        T, row = k.shape[0], cache.n_kv_heads * cache.head_dim
        self.ldk = _rows("AppendCall: k", k, T, row)
        self.ldv = _rows("AppendCall: v", v, T, row)
        if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
            raise TypeError("AppendCall: q, k and v must share a dtype")
        _vector("AppendCall: pos", pos, T, torch.int32)
        _vector("AppendCall: slot", slot, T, torch.int64)
        rope = rope or Rope(None)
        self.Hq, self.ldq, self.ldqo = 0, 0, 0
        self._made = None
        if q is not None:
            self.ldq = _rows("AppendCall: q", q, T)
            if q.shape[1] % cache.head_dim:
                raise ValueError("AppendCall: q must hold whole heads")
            self.Hq = q.shape[1] // cache.head_dim
            if q_out is None:
                q_out = torch.empty(T, q.shape[1], dtype=torch.bfloat16, device=k.device)
                self._made = _Made(k.device) if k.is_cuda and not _once else None
            if q_out.dtype != torch.bfloat16:
                raise TypeError("AppendCall: q_out must be bfloat16")
            self.ldqo = _rows("AppendCall: q_out", q_out, T, q.shape[1])
        elif q_out is not None:
            raise ValueError("AppendCall: q_out without q")
        _same_device("AppendCall", cache.device, k, v, pos, slot, q, q_out, rope.inv_freq)
        self.cache, self.rope, self.k, self.v, self.q = cache, rope, k, v, q
        self.pos, self.slot, self.q_out, self.T = pos, slot, q_out, T
        self.xd, self.device = _dtype_code(k.dtype), cache.device
        self._own = () if q_out is None else ((q_out, _stream(self.device)),)
        self.norm, by = norm, ()
        if norm is not None:
            norm.fit(self.Hq, cache.n_kv_heads, cache.head_dim)
            _same_device("AppendCall", cache.device, norm.w_q, norm.w_k)
            by = (ctypes.byref(norm.desc),)
        self._fn = lib().tcl_kv_append if norm is None else lib().tcl_kv_append_norm
        self._args = _packed(self._fn, (
            ctypes.byref(cache.desc), ctypes.byref(rope.desc), *by, k.data_ptr(), self.ldk,
            v.data_ptr(), self.ldv, _ptr(q), self.ldq, self.Hq, self.xd, _ptr(q_out), self.ldqo, T,
            pos.data_ptr(), slot.data_ptr()))

    def __call__(self, stream=None) -> Optional[torch.Tensor]:
        _call(self.device, self._fn, self._args, stream, *self._own, made=self._made)
        return self.q_out


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
              slot: torch.Tensor, rope: Optional[Rope] = None, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, stream=None,
              norm: Optional[HeadNorm] = None) -> Optional[torch.Tensor]:
    """tcl_kv_append, or tcl_kv_append_norm with ``norm``; returns the rotated
    queries (None without q)."""
    return AppendCall(cache, k, v, pos, slot, rope, q, q_out, norm=norm, _once=stream is None)(stream)


class MapCall:
    """Pre-marshalled arguments of tcl_kv_map for repeated calls: pages,
    positions and slots of a batch's new tokens.  int32 device tensors: n_new
    [n_seqs], group_seq_ptr [n_groups + 1], prefix_len [n_groups], own_len
    [n_seqs] (keys before the call), own_pages [n_seqs, m] (new pages are
    written into it), free_pages [n] and used [1], how many of them are taken.
    Each call returns this object, whose seq_tok_ptr [n_seqs + 1], pos int32
    and slot int64 [n_tokens] are what AppendCall and AttnPlan take, with
    own_len and used after the call.  ``own_len_out`` and ``used_out`` are made
    here unless given; given own_len and used themselves a captured call goes
    on by itself at each replay."""

    def __init__(self, cache: KVCache, n_new: torch.Tensor, group_seq_ptr: torch.Tensor,
                 prefix_len: torch.Tensor, own_len: torch.Tensor, own_pages: torch.Tensor,
                 free_pages: torch.Tensor, used: torch.Tensor, n_tokens: int,
                 own_len_out: Optional[torch.Tensor] = None,
                 used_out: Optional[torch.Tensor] = None, *, _once: bool = False):
        S, G, T = n_new.shape[0], group_seq_ptr.shape[0] - 1, int(n_tokens)
        for name, t, n in (("n_new", n_new, S), ("group_seq_ptr", group_seq_ptr, G + 1),
                           ("prefix_len", prefix_len, G), ("own_len", own_len, S), ("used", used, 1),
                           ("free_pages", free_pages, free_pages.numel()),
                           ("own_len_out", own_len_out, S), ("used_out", used_out, 1)):
            if t is not None:
                _vector(f"MapCall: {name}", t, n, torch.int32)
        if not 0 <= T < 1 << 31 or free_pages.numel() >= 1 << 31:
            raise ValueError("MapCall: n_tokens and the list of free pages must be counts below 2^31")
        if own_pages.dtype != torch.int32:
            raise ValueError("MapCall: own_pages must be int32")
        ld = _rows("MapCall: own_pages", own_pages, S) if own_pages.numel() else 0
        self.device = cache.device
        _same_device("MapCall", self.device, n_new, group_seq_ptr, prefix_len, own_len, own_pages,
                     free_pages, used, own_len_out, used_out)
        made = []

        def make(n, dtype=torch.int32):
            made.append(torch.empty(n, dtype=dtype, device=self.device))
            return made[-1]

        self.seq_tok_ptr, self.pos, self.slot = make(S + 1), make(T), make(T, torch.int64)
        self.own_len = make(S) if own_len_out is None else own_len_out
        self.used = make(1) if used_out is None else used_out
        self._status = make(4)
        self._made = None if _once else _Made(self.device)
        home = _stream(self.device)
        self._own = tuple((t, home) for t in made)
        self._in = (n_new, group_seq_ptr, prefix_len, own_len, own_pages, free_pages, used)
        self.cache, self.own_pages, self.n_tokens = cache, own_pages, T
        self.batch = MapBatch(S, G, T, free_pages.numel(), ld, *[_ptr(t) for t in (
            n_new, group_seq_ptr, prefix_len, own_len, free_pages, used, own_pages, self.seq_tok_ptr,
            self.pos, self.slot, self.own_len, self.used, self._status)])
        if own_pages.numel() and own_pages.shape[1] != ld:
            raise ValueError("MapCall: own_pages must be contiguous")
        self._fn = lib().tcl_kv_map
        self._args = (ctypes.byref(cache.desc), ctypes.byref(self.batch))

    def __call__(self, stream=None) -> "MapCall":
        _call(self.device, self._fn, self._args, stream, *self._own, made=self._made)
        return self

    def status(self):
        """(code, tokens, pages taken, pages left) of the last call;
        synchronises."""
        torch.cuda.synchronize(self.device)
        return tuple(self._status.tolist())


def kv_map(cache: KVCache, n_new: torch.Tensor, group_seq_ptr: torch.Tensor, prefix_len: torch.Tensor,
           own_len: torch.Tensor, own_pages: torch.Tensor, free_pages: torch.Tensor,
           used: torch.Tensor, n_tokens: int, own_len_out: Optional[torch.Tensor] = None,
           used_out: Optional[torch.Tensor] = None, stream=None) -> MapCall:
    """tcl_kv_map: the call, run, with its outputs."""
    return MapCall(cache, n_new, group_seq_ptr, prefix_len, own_len, own_pages, free_pages, used,
                   n_tokens, own_len_out, used_out, _once=stream is None)(stream)


def window_limits(window: int, sinks: int):
    """A window and its sinks as the library takes them, in 32 bits: what is
    above them is more than the keys there can be, what is below 0 stays so
    (and is refused)."""
    most = (1 << 31) - 1
    return max(-1, min(int(window), most)), max(-1, min(int(sinks), most))


class AttnPlan:
    """The mapping of an attention batch (tcl_attn_plan): requests in groups
    that share a prefix.  int32 device tensors: seq_tok_ptr [n_seqs + 1],
    group_seq_ptr [n_groups + 1], prefix_len [n_groups], prefix_pages
    [n_groups, m], own_len [n_seqs], own_pages [n_seqs, n].  One plan serves
    every layer whose cache has the sizes of ``cache``.  With ``window`` a
    token sees its last ``window`` keys and the request's first ``sinks``
    (tcl_attn_window_plan).  The mapping runs on ``stream`` or the current one:
    calls on others have to be ordered behind it, and the tables are read by
    them too."""

    def __init__(self, cache: KVCache, n_q_heads: int, seq_tok_ptr: torch.Tensor,
                 group_seq_ptr: torch.Tensor, prefix_len: torch.Tensor,
                 prefix_pages: torch.Tensor, own_len: torch.Tensor, own_pages: torch.Tensor,
                 n_tokens: int, stream=None, window: Optional[int] = None, sinks: int = 0):
        if window is None and sinks:
            raise ValueError("AttnPlan: sinks without a window")
        self.cache, self.n_q_heads, self.n_tokens = cache, int(n_q_heads), int(n_tokens)
        self.window, self.sinks = window, sinks
        self.limits = () if window is None else window_limits(window, sinks)
        self.device = cache.device
        self.home = _stream(self.device)
        self._set(seq_tok_ptr, group_seq_ptr, prefix_len, prefix_pages, own_len, own_pages)
        self._sizes = [getattr(self.batch, f) for f, _ in AttnBatch._fields_[:5]]
        n = ctypes.c_size_t(0)
        check(lib().tcl_attn_plan_bytes(ctypes.byref(self.batch), ctypes.byref(cache.desc),
                                        self.n_q_heads, ctypes.byref(n)))
        self.buf = torch.empty(n.value, dtype=torch.uint8, device=self.device)
        check(lib().tcl_attn_workspace_bytes(ctypes.byref(self.batch), ctypes.byref(cache.desc),
                                             self.n_q_heads, ctypes.byref(n)))
        self.workspace_bytes = n.value
        _made_for(self.device, stream)
        self._map(stream)

    def _set(self, *table):
        seq_tok_ptr, group_seq_ptr, prefix_len, prefix_pages, own_len, own_pages = table
        S, G = seq_tok_ptr.shape[0] - 1, group_seq_ptr.shape[0] - 1
        for name, t, n in (("seq_tok_ptr", seq_tok_ptr, S + 1),
                           ("group_seq_ptr", group_seq_ptr, G + 1),
                           ("prefix_len", prefix_len, G), ("own_len", own_len, S)):
            _vector(f"AttnPlan: {name}", t, n, torch.int32)
        ldp = _rows("AttnPlan: prefix_pages", prefix_pages, G) if prefix_pages.numel() else 0
        ldo = _rows("AttnPlan: own_pages", own_pages, S) if own_pages.numel() else 0
        if prefix_pages.dtype != torch.int32 or own_pages.dtype != torch.int32:
            raise ValueError("AttnPlan: page tables must be int32")
        if ((prefix_pages.numel() and prefix_pages.shape[1] != ldp)
                or (own_pages.numel() and own_pages.shape[1] != ldo)):
            raise ValueError("AttnPlan: page tables must be contiguous")
        _same_device("AttnPlan", self.device, *table)
        self.table = table
        self.batch = AttnBatch(S, G, self.n_tokens, ldp, ldo, *[t.data_ptr() for t in table])
        self.batch_ref = ctypes.byref(self.batch)

    def _map(self, stream):
        _call(self.device, lib().tcl_attn_window_plan if self.limits else lib().tcl_attn_plan,
              (ctypes.byref(self.batch), ctypes.byref(self.cache.desc), self.n_q_heads, *self.limits,
               self.buf.data_ptr(), self.buf.numel()), stream, (self.buf, self.home))

    def remap(self, seq_tok_ptr, group_seq_ptr, prefix_len, prefix_pages, own_len, own_pages,
              stream=None) -> None:
        """Maps a batch of the same sizes into this plan (no allocation; in a
        graph it follows what the tensors hold at each replay)."""
        old = self.table, self.batch, self.batch_ref
        self._set(seq_tok_ptr, group_seq_ptr, prefix_len, prefix_pages, own_len, own_pages)
        if [getattr(self.batch, f) for f, _ in AttnBatch._fields_[:5]] != self._sizes:
            self.table, self.batch, self.batch_ref = old
            raise ValueError("AttnPlan.remap: a batch of other sizes needs a plan of its own")
        self._map(stream)

    def status_async(self, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Queues a copy of {code, items, tiles, tokens that may share} into a
        device int32 tensor of 4 entries (tcl_attn_status_async)."""
        own = out is None
        if own:
            out = torch.empty(4, dtype=torch.int32, device=self.device)
        _vector("AttnPlan: status", out, 4, torch.int32)
        _same_device("AttnPlan", self.device, out)
        if own:
            _made_for(self.device, stream)
        _call(self.device, lib().tcl_attn_status_async, (self.buf.data_ptr(), out.data_ptr()),
              stream, (self.buf, self.home), *([(out, _stream(self.device))] if own else []))
        return out

    def status(self, stream=None) -> int:
        """The mapping's verdict (TCL_OK or TCL_EINVAL); synchronises."""
        out = self.status_async(stream=stream)
        torch.cuda.synchronize(self.device)
        return int(out[0].item())


class AttnCall:
    """Pre-marshalled arguments of tcl_attn_apply (tcl_attn_window_apply for
    a plan with a window) for repeated calls: each call writes o (bf16
    [n_tokens, q heads * head_dim], made here unless given) and, if given, lse
    (fp32 [n_tokens, q heads]).  ``cache`` is the
    layer's (the plan's by default); the workspace is the call's own, or
    ``ws``; calls that may run at the same time need one each."""

    def __init__(self, plan: AttnPlan, q: torch.Tensor, o: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                 cache: Optional[KVCache] = None, ws: Optional[torch.Tensor] = None, *,
                 _once: bool = False):
        cache = cache or plan.cache
        if any(getattr(cache, f) != getattr(plan.cache, f)
               for f in ("n_pages", "page_size", "n_kv_heads", "head_dim")):
            raise ValueError("AttnCall: the cache's sizes are not the plan's")
        T, row = plan.n_tokens, plan.n_q_heads * cache.head_dim
        made = o is None
        if o is None:
            o = torch.empty(T, row, dtype=torch.bfloat16, device=q.device)
        if q.dtype != torch.bfloat16 or o.dtype != torch.bfloat16:
            raise TypeError("AttnCall: q and o must be bfloat16")
        self.ldq, self.ldo = _rows("AttnCall: q", q, T, row), _rows("AttnCall: o", o, T, row)
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, plan.n_q_heads)
                                or not lse.is_contiguous()):
            raise ValueError("AttnCall: lse must be float32 [n_tokens, q heads], contiguous")
        _same_device("AttnCall", plan.device, q, o, lse, cache.K, ws)
        self.plan, self.cache, self.q, self.o, self.lse = plan, cache, q, o, lse
        self.scale = cache.head_dim ** -0.5 if scale is None else float(scale)
        if not _fits("AttnCall", ws, plan.workspace_bytes):
            ws = torch.empty(max(plan.workspace_bytes, 256), dtype=torch.uint8, device=plan.device)
            made = True
        self.ws = ws
        self._made = _Made(plan.device) if made and not _once else None
        home = _stream(plan.device)
        self._own = ((ws, home), (o, home), (plan.buf, plan.home))
        self._fn = lib().tcl_attn_window_apply if plan.limits else lib().tcl_attn_apply
        self._args = _packed(self._fn, (
            None, ctypes.byref(cache.desc), plan.n_q_heads, *plan.limits, plan.buf.data_ptr(), plan.buf.numel(),
            q.data_ptr(), self.ldq, o.data_ptr(), self.ldo, _ptr(lse), self.scale, ws.data_ptr(),
            ws.numel() * ws.element_size()))[1:]

    def __call__(self, stream=None) -> torch.Tensor:
        p = self.plan  # (the batch's tables are the plan's last ones)
        _call(p.device, self._fn, (p.batch_ref, *self._args), stream, *self._own, made=self._made)
        return self.o


def attention(plan: AttnPlan, q: torch.Tensor, o: Optional[torch.Tensor] = None,
              lse: Optional[torch.Tensor] = None, scale: Optional[float] = None,
              cache: Optional[KVCache] = None, stream=None) -> torch.Tensor:
    """tcl_attn_apply: attention of the plan's batch over the cache."""
    return AttnCall(plan, q, o, lse, scale, cache, _once=stream is None)(stream)
