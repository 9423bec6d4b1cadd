"""etree -- target-model verification of a draft token tree on NVIDIA B200 (sm_100a).

Thin ctypes binding of ``libetree.so``; argument marshalling only.  Every step of the
computation runs in the library's CUDA kernels.  PyTorch supplies device memory and streams.
The binding never falls back to anything else: without the built library (or without a CUDA
device) every entry point raises.

Entry points (same names as the C ABI in ``include/etree.h``)::

    etree_workspace_size(batch, hq, hkv, head_dim, hidden_dim, vocab) -> int
    etree_workspace_init(workspace, stream=None)
    etree_verify_attn(batch, q, k_tree, v_tree, k_cache, v_cache, scale, out, lse, workspace)
    etree_lmhead_accept(batch, hidden, w_lm, temperature, q_draft, seed, step, accept_len, path,
                        out_tokens, node_argmax, node_gap, workspace)
    etree_lmhead_accept_tree(batch, hidden, w_lm, temperature, q_draft, seed, step, accept_len,
                             path, out_tokens, zbuf, workspace)
    etree_kv_compact(batch, accept_len, path, k_tree, v_tree, k_cache, v_cache, n_layers,
                     tree_layer_stride, cache_layer_stride, kv_len_out, workspace)
    etree_page_plan(cu_new, kv_len, page_size, num_pages, pages_held, free_ring, ring_state,
                    block_table, pages_held_out, ring_state_out, slot_cap, slot_map, workspace)
    etree_kv_store(slot_map, k, v, k_pool, v_pool, workspace)
    etree_verify_attn_diff(batch, q, k_tree, v_tree, k_cache, v_cache, scale, lam, norm_w,
                           norm_eps, out_scale, out, lse, workspace)
    etree_verify_attn_diff_paged(batch, block_table, page_size, q, ...)
    etree_w4_linear(x, wq, scales, zeros, group, bias, out, workspace)
    etree_device_status(workspace, stream=None) -> (status, detail)
"""
from __future__ import annotations

import ctypes as C
import os

import torch

__all__ = [
    "EtreeError", "Batch", "make_batch", "lib", "library_path", "etree_workspace_size",
    "etree_workspace_init", "etree_verify_attn", "etree_verify_attn_noalloc",
    "etree_lmhead_accept", "etree_lmhead_accept_tree", "etree_lmhead_accept_timed",
    "etree_kv_compact",
    "etree_verify_attn_paged", "etree_kv_compact_paged", "etree_verify_cost", "etree_plan_tree",
    "cost_table", "load_cost_table", "etree_lowrank_workspace_size",
    "etree_lowrank_candidates", "etree_page_plan", "etree_kv_store",
    "etree_attn_diff_workspace_size", "etree_verify_attn_diff", "etree_verify_attn_diff_paged",
    "etree_w4_workspace_size", "etree_w4_linear", "etree_device_status", "etree_selftest_timeout", "etree_strerror",
    "etree_version", "etree_attn_plan", "STATUS",
]

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(HERE, "libetree.so")

STATUS = {0: "ETREE_OK", -1: "ETREE_EINVAL", -2: "ETREE_EUNSUPPORTED", -3: "ETREE_ECUDA",
          -4: "ETREE_EDEVICE", -5: "ETREE_ETIMEOUT", -6: "ETREE_ENOSPACE"}
DETAIL = {0: "none", 1: "bad parent", 2: "bad node count", 3: "bad kv_len", 4: "capacity",
          5: "not a chain", 6: "bad path", 7: "attention wait", 8: "gemm wait", 9: "bad token",
          10: "logit rows", 11: "bad page", 12: "self-test wait", 13: "walk wait", 14: "free ring",
          15: "bad slot", 16: "product wait"}

EXPORTS = ["etree_workspace_size", "etree_workspace_init", "etree_verify_attn",
           "etree_verify_attn_paged", "etree_kv_compact_paged", "etree_verify_cost",
           "etree_plan_tree", "etree_lowrank_workspace_size", "etree_lowrank_candidates",
           "etree_lmhead_accept", "etree_lmhead_accept_tree", "etree_lmhead_accept_timed",
           "etree_kv_compact", "etree_device_status", "etree_strerror",
           "etree_version", "etree_last_error", "etree_attn_plan", "etree_verify_attn_noalloc",
           "etree_selftest_timeout", "etree_page_plan", "etree_kv_store",
           "etree_attn_diff_workspace_size", "etree_verify_attn_diff",
           "etree_verify_attn_diff_paged", "etree_w4_workspace_size", "etree_w4_linear"]


class EtreeError(RuntimeError):
    def __init__(self, status: int, msg: str = ""):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {msg}")


class Batch(C.Structure):
    _fields_ = [("B", C.c_int32), ("n_total", C.c_int32), ("n_max", C.c_int32),
                ("kv_len_max", C.c_int32), ("cu_nodes", C.c_void_p), ("parent", C.c_void_p),
                ("tokens", C.c_void_p), ("kv_len", C.c_void_p), ("slot_base", C.c_void_p),
                ("slot_cap", C.c_void_p)]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libetree.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise EtreeError(-3, f"{_LIB_PATH} is missing: run `python -m "
                             "draft_tree_verification_masked_b200._build` first")
    L = C.CDLL(_LIB_PATH)
    vp, i32, i64, u64, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_uint64, C.c_float
    bp = C.POINTER(Batch)
    L.etree_workspace_size.argtypes = [bp, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int]
    L.etree_workspace_size.restype = C.c_size_t
    L.etree_workspace_init.argtypes = [vp, C.c_size_t, vp]
    L.etree_workspace_init.restype = C.c_int
    L.etree_verify_attn.argtypes = [bp, vp, vp, vp, vp, vp, i64, C.c_int, C.c_int, C.c_int, f32,
                                    vp, vp, vp, C.c_size_t, vp]
    L.etree_verify_attn.restype = C.c_int
    L.etree_lmhead_accept.argtypes = [bp, vp, vp, C.c_int, C.c_int, f32, vp, u64, u64, vp, vp,
                                      vp, vp, vp, vp, C.c_size_t, vp]
    L.etree_lmhead_accept.restype = C.c_int
    L.etree_lmhead_accept_tree.argtypes = [bp, vp, vp, C.c_int, C.c_int, f32, vp, u64, u64, vp,
                                           vp, vp, vp, C.c_int32, vp, C.c_size_t, vp]
    L.etree_lmhead_accept_tree.restype = C.c_int
    L.etree_lmhead_accept_timed.argtypes = [bp, vp, vp, C.c_int, C.c_int, f32, vp, u64, u64, vp,
                                            vp, vp, vp, vp, vp, C.c_int32, C.c_int32,
                                            C.POINTER(C.c_void_p), vp, C.c_size_t, vp]
    L.etree_lmhead_accept_timed.restype = C.c_int
    L.etree_kv_compact.argtypes = [bp, vp, vp, vp, vp, vp, vp, C.c_int, i64, i64, C.c_int,
                                   C.c_int, vp, vp, C.c_size_t, vp]
    L.etree_kv_compact.restype = C.c_int
    L.etree_verify_attn_paged.argtypes = [bp, vp, C.c_int32, C.c_int32, vp, vp, vp, vp, vp, i64,
                                          C.c_int, C.c_int, C.c_int, f32, vp, vp, vp, C.c_size_t,
                                          vp]
    L.etree_verify_attn_paged.restype = C.c_int
    L.etree_lowrank_workspace_size.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int]
    L.etree_lowrank_workspace_size.restype = C.c_size_t
    L.etree_lowrank_candidates.argtypes = [vp, C.c_int, C.c_int, vp, vp, C.c_int, vp, C.c_int,
                                           C.c_int, vp, vp, vp, C.c_size_t, vp]
    L.etree_lowrank_candidates.restype = C.c_int
    L.etree_verify_cost.argtypes = [C.POINTER(CostTable), C.c_double, C.c_double, C.c_double,
                                    C.POINTER(C.c_double)]
    L.etree_verify_cost.restype = C.c_int
    L.etree_plan_tree.argtypes = [C.POINTER(CostTable), C.c_int32, C.c_int32,
                                  C.POINTER(C.c_float), C.c_int32, C.c_float, C.c_float,
                                  C.c_int32, C.c_int32, C.c_int32, C.POINTER(TreePlan)]
    L.etree_plan_tree.restype = C.c_int
    L.etree_kv_compact_paged.argtypes = [bp, vp, C.c_int32, C.c_int32, vp, vp, vp, vp, vp, vp,
                                         i64, C.c_int, i64, i64, C.c_int, C.c_int, vp, vp,
                                         C.c_size_t, vp]
    L.etree_kv_compact_paged.restype = C.c_int
    L.etree_page_plan.argtypes = [i32, i32, vp, vp, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                  vp, C.c_size_t, vp]
    L.etree_page_plan.restype = C.c_int
    L.etree_kv_store.argtypes = [vp, i32, vp, i64, vp, i64, vp, vp, i64, C.c_int, C.c_int, vp,
                                 C.c_size_t, vp]
    L.etree_kv_store.restype = C.c_int
    L.etree_attn_diff_workspace_size.argtypes = [bp, C.c_int, C.c_int]
    L.etree_attn_diff_workspace_size.restype = C.c_size_t
    tail = [i64, C.c_int, C.c_int, C.c_int, f32, vp, vp, f32, f32, vp, vp, vp, C.c_size_t, vp]
    rows = [vp, i64, vp, i64, vp, i64, vp, vp]
    L.etree_verify_attn_diff.argtypes = [bp, *rows, *tail]
    L.etree_verify_attn_diff.restype = C.c_int
    L.etree_verify_attn_diff_paged.argtypes = [bp, vp, i32, i32, *rows, *tail]
    L.etree_verify_attn_diff_paged.restype = C.c_int
    L.etree_w4_workspace_size.argtypes = [C.c_int, C.c_int, C.c_int]
    L.etree_w4_workspace_size.restype = C.c_size_t
    L.etree_w4_linear.argtypes = [vp, i64, C.c_int, vp, vp, vp, C.c_int, C.c_int, C.c_int, vp, vp,
                                  i64, C.c_int, vp, C.c_size_t, vp]
    L.etree_w4_linear.restype = C.c_int
    L.etree_device_status.argtypes = [vp, vp, C.POINTER(i32)]
    L.etree_device_status.restype = C.c_int
    L.etree_selftest_timeout.argtypes = [vp, C.c_size_t, vp]
    L.etree_selftest_timeout.restype = C.c_int
    L.etree_strerror.argtypes = [C.c_int]
    L.etree_strerror.restype = C.c_char_p
    L.etree_last_error.argtypes = []
    L.etree_last_error.restype = C.c_char_p
    L.etree_version.argtypes = []
    L.etree_version.restype = C.c_int
    L.etree_verify_attn_noalloc.argtypes = [bp, vp, vp, vp, vp, vp, i64, C.c_int, C.c_int,
                                            C.c_int, f32, vp, vp, vp, vp]
    L.etree_verify_attn_noalloc.restype = C.c_int
    ip = C.POINTER(C.c_int32)
    L.etree_attn_plan.argtypes = [bp, C.c_int, C.c_int, ip, ip, ip, ip, ip, ip]
    L.etree_attn_plan.restype = C.c_int
    _lib = L
    return L


def _check(st: int) -> int:
    if st != 0:
        raise EtreeError(st, lib().etree_last_error().decode())
    return st


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        # the raw call gives the same handle without 3 us of wrapping, but torch keeps it private
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        return raw(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def etree_lowrank_workspace_size(M: int, hidden_dim: int, rank: int, vocab: int) -> int:
    return int(lib().etree_lowrank_workspace_size(int(M), int(hidden_dim), int(rank),
                                                  int(vocab)))


def etree_lowrank_candidates(hidden, D, U, W, k: int, out_ids, out_logit, workspace,
                             stream=None, check: bool = True) -> int:
    """hidden [M, H], D [r, H], U [V, r], W [V, H] bf16; out_ids int32 / out_logit fp32 [M, k]."""
    bf = torch.bfloat16
    M, H = hidden.shape
    r, V = D.shape[0], U.shape[0]
    st = lib().etree_lowrank_candidates(
        _ptr(hidden, bf, "hidden"), M, H, _ptr(D, bf, "D"), _ptr(U, bf, "U"), r,
        _ptr(W, bf, "W"), V, int(k), _ptr(out_ids, torch.int32, "out_ids"),
        _ptr(out_logit, torch.float32, "out_logit"), _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream))
    return _check(st) if check else st


class CostTable(C.Structure):
    _fields_ = [("nB", C.c_int32), ("nN", C.c_int32), ("nL", C.c_int32),
                ("B", C.POINTER(C.c_int32)), ("N", C.POINTER(C.c_int32)),
                ("L", C.POINTER(C.c_int32)), ("us", C.POINTER(C.c_float))]


class TreePlan(C.Structure):
    _fields_ = [("depth", C.c_int32), ("width", C.c_int32), ("nodes", C.c_int32),
                ("expected_accept", C.c_double), ("step_us", C.c_double),
                ("tokens_per_s", C.c_double)]


def cost_table(d: dict) -> CostTable:
    """An etree_cost_table over the dict {"B", "N", "L", "us"} (as calibrate.py writes it)."""
    import numpy as np
    arrs = [np.ascontiguousarray(d[k], dtype=np.int32) for k in ("B", "N", "L")]
    us = np.ascontiguousarray(d["us"], dtype=np.float32)
    if us.shape != (len(arrs[0]), len(arrs[1]), len(arrs[2])):
        raise ValueError(f"us has shape {us.shape}, want (|B|, |N|, |L|)")
    i32p, f32p = C.POINTER(C.c_int32), C.POINTER(C.c_float)
    t = CostTable(len(arrs[0]), len(arrs[1]), len(arrs[2]), arrs[0].ctypes.data_as(i32p),
                  arrs[1].ctypes.data_as(i32p), arrs[2].ctypes.data_as(i32p),
                  us.ctypes.data_as(f32p))
    t._keep = (arrs, us)
    return t


def load_cost_table(name: str = "b200_dense27b") -> dict:
    """A packaged calibration (cost_tables/<name>.json) or a path to one."""
    import json
    path = name if os.path.exists(name) else os.path.join(HERE, "cost_tables", name + ".json")
    with open(path) as f:
        return json.load(f)


def etree_verify_cost(table, B: float, N: float, L: float) -> float:
    t = table if isinstance(table, CostTable) else cost_table(table)
    out = C.c_double()
    _check(lib().etree_verify_cost(C.byref(t), float(B), float(N), float(L), C.byref(out)))
    return out.value


def etree_plan_tree(table, B: int, L: int, acc_rank, draft_us_per_level: float,
                    draft_us_fixed: float = 0.0, max_depth: int = 16, max_width: int = 16,
                    max_nodes: int = 64) -> dict:
    """The static (depth, width) draft tree with the most expected tokens/s (host only)."""
    t = table if isinstance(table, CostTable) else cost_table(table)
    acc = (C.c_float * len(acc_rank))(*[float(a) for a in acc_rank])
    out = TreePlan()
    _check(lib().etree_plan_tree(C.byref(t), int(B), int(L), acc, len(acc_rank),
                                 float(draft_us_per_level), float(draft_us_fixed),
                                 int(max_depth), int(max_width), int(max_nodes), C.byref(out)))
    return {k: getattr(out, k) for k, _ in TreePlan._fields_}


def make_batch(cu_nodes, parent, tokens, kv_len, slot_base, slot_cap, n_max: int,
               kv_len_max: int) -> Batch:
    """Wrap device int tensors as an etree_batch (keeps references to them)."""
    b = Batch()
    b.B = cu_nodes.numel() - 1
    b.n_total = parent.numel()
    b.n_max = int(n_max)
    b.kv_len_max = int(kv_len_max)
    b.cu_nodes = _ptr(cu_nodes, torch.int32, "cu_nodes")
    b.parent = _ptr(parent, torch.int32, "parent")
    b.tokens = _ptr(tokens, torch.int32, "tokens")
    b.kv_len = _ptr(kv_len, torch.int32, "kv_len")
    b.slot_base = _ptr(slot_base, torch.int64, "slot_base")
    b.slot_cap = _ptr(slot_cap, torch.int32, "slot_cap")
    b._keep = (cu_nodes, parent, tokens, kv_len, slot_base, slot_cap)
    return b


def etree_version() -> int:
    return int(lib().etree_version())


def etree_strerror(status: int) -> str:
    return lib().etree_strerror(int(status)).decode()


def etree_workspace_size(batch: Batch, hq: int, hkv: int, head_dim: int, hidden_dim: int,
                         vocab: int) -> int:
    return int(lib().etree_workspace_size(C.byref(batch), hq, hkv, head_dim, hidden_dim, vocab))


def etree_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _check(lib().etree_workspace_init(_ptr(workspace, torch.uint8, "workspace"),
                                      workspace.numel(), _stream(stream)))


def etree_verify_attn(batch: Batch, q, k_tree, v_tree, k_cache, v_cache, scale: float, out,
                      lse, workspace, stream=None, check: bool = True) -> int:
    bf = torch.bfloat16
    hq, d = q.shape[1], q.shape[2]
    hkv = k_tree.shape[1]
    st = lib().etree_verify_attn(
        C.byref(batch), _ptr(q, bf, "q"), _ptr(k_tree, bf, "k_tree"), _ptr(v_tree, bf, "v_tree"),
        _ptr(k_cache, bf, "k_cache"), _ptr(v_cache, bf, "v_cache"), k_cache.shape[0], hq, hkv,
        d, float(scale), _ptr(out, bf, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return _check(st) if check else st


def etree_verify_attn_noalloc(batch: Batch, q, k_tree, v_tree, k_cache, v_cache, scale: float,
                              out, lse, status_out=None, stream=None, check: bool = True) -> int:
    """Tree attention backed by the library's static scratch array: for callers that cannot
    allocate device memory (no workspace argument; see etree.h for the contract)."""
    bf = torch.bfloat16
    hq, d = q.shape[1], q.shape[2]
    hkv = k_tree.shape[1]
    st = lib().etree_verify_attn_noalloc(
        C.byref(batch), _ptr(q, bf, "q"), _ptr(k_tree, bf, "k_tree"), _ptr(v_tree, bf, "v_tree"),
        _ptr(k_cache, bf, "k_cache"), _ptr(v_cache, bf, "v_cache"), k_cache.shape[0], hq, hkv,
        d, float(scale), _ptr(out, bf, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(status_out, torch.int32, "status_out"), _stream(stream))
    return _check(st) if check else st


def etree_lmhead_accept(batch: Batch, hidden, w_lm, temperature: float, q_draft, seed: int,
                        step: int, accept_len, path, out_tokens, node_argmax, node_gap,
                        workspace, stream=None, check: bool = True) -> int:
    bf = torch.bfloat16
    st = lib().etree_lmhead_accept(
        C.byref(batch), _ptr(hidden, bf, "hidden"), _ptr(w_lm, bf, "w_lm"), hidden.shape[1],
        w_lm.shape[0], float(temperature), _ptr(q_draft, torch.float32, "q_draft"),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _ptr(accept_len, torch.int32, "accept_len"), _ptr(path, torch.int32, "path"),
        _ptr(out_tokens, torch.int32, "out_tokens"),
        _ptr(node_argmax, torch.int32, "node_argmax"), _ptr(node_gap, torch.float32, "node_gap"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return _check(st) if check else st


def etree_lmhead_accept_tree(batch: Batch, hidden, w_lm, temperature: float, q_draft, seed: int,
                             step: int, accept_len, path, out_tokens, zbuf, workspace,
                             stream=None, check: bool = True) -> int:
    """zbuf: fp32 [rows][vocab] device tensor (or None for no rows)."""
    bf = torch.bfloat16
    rows = 0 if zbuf is None else int(zbuf.shape[0])
    st = lib().etree_lmhead_accept_tree(
        C.byref(batch), _ptr(hidden, bf, "hidden"), _ptr(w_lm, bf, "w_lm"), hidden.shape[1],
        w_lm.shape[0], float(temperature), _ptr(q_draft, torch.float32, "q_draft"),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _ptr(accept_len, torch.int32, "accept_len"), _ptr(path, torch.int32, "path"),
        _ptr(out_tokens, torch.int32, "out_tokens"), _ptr(zbuf, torch.float32, "zbuf"), rows,
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return _check(st) if check else st


def etree_lmhead_accept_timed(batch: Batch, hidden, w_lm, temperature: float, q_draft, seed: int,
                              step: int, accept_len, path, out_tokens, node_argmax, node_gap,
                              zbuf, branching: bool, marks, workspace, stream=None,
                              check: bool = True) -> int:
    """etree_lmhead_accept(_tree) with phase marks: `marks` is a list of 4 torch.cuda.Event
    (or None entries) recorded after the set-up kernels, the first GEMM, the acceptance kernels
    and the draw GEMM.  torch creates an Event's CUDA event on its first record(): record each
    once before passing it, or its handle is NULL and the mark is skipped."""
    bf = torch.bfloat16
    rows = 0 if zbuf is None else int(zbuf.shape[0])
    arr = (C.c_void_p * 4)(*[None if m is None else m.cuda_event for m in marks])
    st = lib().etree_lmhead_accept_timed(
        C.byref(batch), _ptr(hidden, bf, "hidden"), _ptr(w_lm, bf, "w_lm"), hidden.shape[1],
        w_lm.shape[0], float(temperature), _ptr(q_draft, torch.float32, "q_draft"),
        int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
        _ptr(accept_len, torch.int32, "accept_len"), _ptr(path, torch.int32, "path"),
        _ptr(out_tokens, torch.int32, "out_tokens"),
        _ptr(node_argmax, torch.int32, "node_argmax"), _ptr(node_gap, torch.float32, "node_gap"),
        _ptr(zbuf, torch.float32, "zbuf"), rows, int(bool(branching)), arr,
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return _check(st) if check else st


def etree_verify_attn_paged(batch: Batch, block_table, page_size: int, q, k_tree, v_tree,
                            k_pool, v_pool, scale: float, out, lse, workspace, stream=None,
                            check: bool = True) -> int:
    """block_table: int32 [B, max_pages] device tensor; pools [num_pages * page_size, hkv, d]."""
    bf = torch.bfloat16
    hq, d = q.shape[1], q.shape[2]
    hkv = k_tree.shape[1]
    num_pages = k_pool.shape[0] // int(page_size)
    st = lib().etree_verify_attn_paged(
        C.byref(batch), _ptr(block_table, torch.int32, "block_table"), block_table.shape[1],
        int(page_size), _ptr(q, bf, "q"), _ptr(k_tree, bf, "k_tree"), _ptr(v_tree, bf, "v_tree"),
        _ptr(k_pool, bf, "k_pool"), _ptr(v_pool, bf, "v_pool"), num_pages, hq, hkv, d,
        float(scale), _ptr(out, bf, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream))
    return _check(st) if check else st


def _check_path(batch: Batch, path):
    # the library reads a full row of ETREE_PATH_STRIDE entries per request
    if isinstance(path, torch.Tensor) and path.numel() < batch.B * 64:
        raise ValueError(f"path must hold [B][64] entries, got {tuple(path.shape)}")


def etree_kv_compact_paged(batch: Batch, block_table, page_size: int, accept_len, path, k_tree,
                           v_tree, k_pool, v_pool, num_pages: int, n_layers: int,
                           tree_layer_stride: int, cache_layer_stride: int, kv_len_out,
                           workspace, stream=None, check: bool = True) -> int:
    bf = torch.bfloat16
    _check_path(batch, path)
    hkv, d = k_tree.shape[-2], k_tree.shape[-1]
    st = lib().etree_kv_compact_paged(
        C.byref(batch), _ptr(block_table, torch.int32, "block_table"), block_table.shape[1],
        int(page_size), _ptr(accept_len, torch.int32, "accept_len"),
        _ptr(path, torch.int32, "path"), _ptr(k_tree, bf, "k_tree"), _ptr(v_tree, bf, "v_tree"),
        _ptr(k_pool, bf, "k_pool"), _ptr(v_pool, bf, "v_pool"), int(num_pages), int(n_layers),
        int(tree_layer_stride), int(cache_layer_stride), hkv, d,
        _ptr(kv_len_out, torch.int32, "kv_len_out"), _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream))
    return _check(st) if check else st


def etree_kv_compact(batch: Batch, accept_len, path, k_tree, v_tree, k_cache, v_cache,
                     n_layers: int, tree_layer_stride: int, cache_layer_stride: int, kv_len_out,
                     workspace, stream=None, check: bool = True) -> int:
    bf = torch.bfloat16
    _check_path(batch, path)
    hkv, d = k_tree.shape[-2], k_tree.shape[-1]
    st = lib().etree_kv_compact(
        C.byref(batch), _ptr(accept_len, torch.int32, "accept_len"),
        _ptr(path, torch.int32, "path"), _ptr(k_tree, bf, "k_tree"), _ptr(v_tree, bf, "v_tree"),
        _ptr(k_cache, bf, "k_cache"), _ptr(v_cache, bf, "v_cache"), int(n_layers),
        int(tree_layer_stride), int(cache_layer_stride), hkv, d,
        _ptr(kv_len_out, torch.int32, "kv_len_out"), _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream))
    return _check(st) if check else st


def _arg(t, dtype, dev: int, n: int, name: str):
    """Pointer of a contiguous tensor of `n` entries on device `dev` (None stays None).  The checks
    of the serving calls: one short pass where all is well, since those calls take microseconds."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and t.numel() == n and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    _ptr(t, dtype, name)                    # raises for the type, the host or the layout
    _here(t)
    raise ValueError(f"{name} must hold {n} entries, got {tuple(t.shape)}")


def _here(*tensors):
    """Calls run on the current device's stream: tensors of another device are refused."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.is_cuda and t.device.index != dev:
            raise ValueError(f"a tensor lives on {t.device}, the current device is cuda:{dev}")


def etree_page_plan(cu_new, kv_len, page_size: int, num_pages: int, pages_held, free_ring,
                    ring_state, block_table, pages_held_out, ring_state_out, slot_cap, slot_map,
                    workspace, stream=None, check: bool = True) -> int:
    """Block tables and slot maps from request lengths.  cu_new int32 [B + 1], kv_len and
    pages_held int32 [B], free_ring int32 [num_pages], ring_state int64 [2], block_table int32
    [B, max_pages] (updated in place); slot_cap int32 [B] and slot_map int64 may be None."""
    i32, i64 = torch.int32, torch.int64
    B, max_pages, dev = kv_len.numel(), block_table.shape[-1], torch.cuda.current_device()
    page_size, num_pages = int(page_size), int(num_pages)
    tokens = 0 if slot_map is None else slot_map.numel()
    st = lib().etree_page_plan(
        B, tokens, _arg(cu_new, i32, dev, B + 1, "cu_new"), _arg(kv_len, i32, dev, B, "kv_len"),
        page_size, max_pages, num_pages, _arg(pages_held, i32, dev, B, "pages_held"),
        _arg(free_ring, i32, dev, num_pages, "free_ring"),
        _arg(ring_state, i64, dev, 2, "ring_state"),
        _arg(block_table, i32, dev, B * max_pages, "block_table"),
        _arg(pages_held_out, i32, dev, B, "pages_held_out"),
        _arg(ring_state_out, i64, dev, 2, "ring_state_out"), _arg(slot_cap, i32, dev, B, "slot_cap"),
        _arg(slot_map, i64, dev, tokens, "slot_map"), *_work(workspace, dev), _stream(stream))
    return _check(st) if check else st


def _work(workspace, dev: int):
    """Pointer and size of a workspace."""
    n = workspace.numel()
    return _arg(workspace, torch.uint8, dev, n, "workspace"), n


def _rows(t, name: str, dev: int):
    """Pointer and row stride of a [rows, heads, dims] bf16 tensor whose rows are dense inside."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    _, h, d = t.shape
    s0, s1, s2 = t.stride()
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != dev:
        _on_device(t, name)
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise ValueError(f"{name}: a row's heads must be contiguous")
    return t.data_ptr(), (s0 if t.shape[0] > 1 else h * d)


def _on_device(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    _here(t)


def etree_kv_store(slot_map, k, v, k_pool, v_pool, workspace, stream=None,
                   check: bool = True) -> int:
    """slot_map int64 [n]; k, v bf16 [n, hkv, 128], rows any stride apart (views of a fused
    projection, say); pools bf16 [slots, hkv, 128]."""
    bf, dev = torch.bfloat16, torch.cuda.current_device()
    n, hkv, d = k.shape
    slots = k_pool.shape[0]
    if v.shape != k.shape or k_pool.shape != (slots, hkv, d) or v_pool.shape != k_pool.shape:
        raise ValueError("k, v and the pools must have the same heads")
    (kp, ks), (vp, vs) = _rows(k, "k", dev), _rows(v, "v", dev)
    size = slots * hkv * d
    st = lib().etree_kv_store(
        _arg(slot_map, torch.int64, dev, n, "slot_map"), n, kp, ks, vp, vs,
        _arg(k_pool, bf, dev, size, "k_pool"), _arg(v_pool, bf, dev, size, "v_pool"), slots, hkv, d,
        *_work(workspace, dev), _stream(stream))
    return _check(st) if check else st


def etree_attn_diff_workspace_size(batch: Batch, hq: int, hkv: int) -> int:
    return int(lib().etree_attn_diff_workspace_size(C.byref(batch), int(hq), int(hkv)))


def _diff_args(batch, q, k_tree, v_tree, k_cache, v_cache, slots, scale, lam, norm_w, norm_eps,
               out_scale, out, lse, workspace):
    """The arguments that the contiguous and the paged call share, checked."""
    bf, f32, dev = torch.bfloat16, torch.float32, torch.cuda.current_device()
    n, hq, d = q.shape
    hkv = k_tree.shape[1]
    if n != batch.n_total or k_tree.shape != (n, hkv, d) or v_tree.shape != k_tree.shape:
        raise ValueError(f"q, k_tree and v_tree must hold {batch.n_total} nodes of {d} dims")
    if k_cache.shape[1:] != (hkv, d) or k_cache.shape != v_cache.shape:
        raise ValueError("the caches must have k_tree's heads")
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    size = k_cache.shape[0] * hkv * d
    return (*_rows(q, "q", dev), *_rows(k_tree, "k_tree", dev), *_rows(v_tree, "v_tree", dev),
            _arg(k_cache, bf, dev, size, "k_cache"), _arg(v_cache, bf, dev, size, "v_cache"), slots,
            hq, hkv, d, float(scale), _arg(lam, f32, dev, hq, "lam"),
            _arg(norm_w, bf, dev, d, "norm_w"), float(norm_eps), float(out_scale),
            _arg(out, bf, dev, n * hq * d, "out"), _arg(lse, f32, dev, n * hq * 2, "lse"),
            *_work(workspace, dev))


def etree_verify_attn_diff(batch: Batch, q, k_tree, v_tree, k_cache, v_cache, scale: float, lam,
                           norm_w, norm_eps: float, out_scale: float, out, lse, workspace,
                           stream=None, check: bool = True) -> int:
    """Differential tree attention.  q, k_tree, v_tree bf16 [n, heads, 128], rows any stride
    apart; lam fp32 [hq]; norm_w bf16 [128] or None; lse fp32 [n, hq, 2] or None."""
    st = lib().etree_verify_attn_diff(
        C.byref(batch), *_diff_args(batch, q, k_tree, v_tree, k_cache, v_cache, k_cache.shape[0],
                                    scale, lam, norm_w, norm_eps, out_scale, out, lse, workspace),
        _stream(stream))
    return _check(st) if check else st


def etree_verify_attn_diff_paged(batch: Batch, block_table, page_size: int, q, k_tree, v_tree,
                                 k_pool, v_pool, scale: float, lam, norm_w, norm_eps: float,
                                 out_scale: float, out, lse, workspace, stream=None,
                                 check: bool = True) -> int:
    """The same over pools [num_pages * page_size, hkv, 128]; block_table int32 [B, max_pages]."""
    max_pages, dev = block_table.shape[-1], torch.cuda.current_device()
    st = lib().etree_verify_attn_diff_paged(
        C.byref(batch), _arg(block_table, torch.int32, dev, batch.B * max_pages, "block_table"),
        max_pages, int(page_size), *_diff_args(batch, q, k_tree, v_tree, k_pool, v_pool,
                                    k_pool.shape[0] // max(1, int(page_size)), scale, lam, norm_w,
                                    norm_eps, out_scale, out, lse, workspace),
        _stream(stream))
    return _check(st) if check else st


def etree_w4_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().etree_w4_workspace_size(int(M), int(N), int(K)))


def etree_w4_linear(x, wq, scales, zeros, group: int, bias, out, workspace, stream=None,
                    check: bool = True) -> int:
    """x bf16 [M, K]; wq uint8 [N, K / 2], two weights a byte; scales bf16 [N, K / group]; zeros
    uint8 [N, K / group] or None; bias bf16 [N] or None; out bf16 or fp32 [M, N].  Rows of x and
    out may lie any stride apart."""
    bf, u8, dev = torch.bfloat16, torch.uint8, torch.cuda.current_device()
    M, K = x.shape
    N, group = wq.shape[0], int(group)
    f32 = out.dtype is torch.float32
    if not f32 and out.dtype is not bf:
        raise TypeError(f"out must be bfloat16 or float32, got {out.dtype}")
    if wq.shape != (N, K // 2) or out.shape != (M, N):
        raise ValueError(f"wq and out must be [N, {K // 2}] and [{M}, N]")
    groups = K // max(1, group)
    if scales.shape != (N, groups) or (zeros is not None and zeros.shape != (N, groups)):
        raise ValueError(f"scales and zeros must be {(N, groups)}")
    (xp, xs), (op, os_) = _matrix(x, bf, "x", dev), _matrix(out, out.dtype, "out", dev)
    st = lib().etree_w4_linear(
        xp, xs, M, _arg(wq, u8, dev, N * (K // 2), "wq"),
        _arg(scales, bf, dev, N * groups, "scales"), _arg(zeros, u8, dev, N * groups, "zeros"),
        group, N, K, _arg(bias, bf, dev, N, "bias"), op, os_, int(f32), *_work(workspace, dev),
        _stream(stream))
    return _check(st) if check else st


def _matrix(t, dtype, name: str, dev: int):
    """Pointer and row stride of a [rows, columns] tensor whose rows are dense inside."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        _on_device(t, name)
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.data_ptr(), (s0 if rows > 1 else cols)


def etree_attn_plan(batch: Batch, hq: int, hkv: int) -> dict:
    v = [C.c_int32(0) for _ in range(6)]
    _check(lib().etree_attn_plan(C.byref(batch), hq, hkv, *[C.byref(x) for x in v]))
    return dict(zip(["kernel", "rows_per_cta", "row_blocks", "splits", "tiles_per_split",
                     "launches"], [int(x.value) for x in v]))


def etree_selftest_timeout(workspace: torch.Tensor, stream=None, check: bool = True) -> int:
    """Enqueue the bounded-wait self-test; etree_device_status then reports ETREE_ETIMEOUT."""
    st = lib().etree_selftest_timeout(_ptr(workspace, torch.uint8, "workspace"),
                                      workspace.numel(), _stream(stream))
    return _check(st) if check else st


def etree_device_status(workspace: torch.Tensor, stream=None) -> tuple[int, int]:
    det = C.c_int32(0)
    st = lib().etree_device_status(_ptr(workspace, torch.uint8, "workspace"), _stream(stream),
                                   C.byref(det))
    return int(st), int(det.value)
