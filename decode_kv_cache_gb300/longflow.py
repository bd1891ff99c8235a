"""Thin Python binding of liblongflow.so (ctypes).

The functions below carry the C names and only marshal arguments: torch
tensors become device pointers, torch streams become ``cudaStream_t``.  Every
step of the decode path runs in the library's CUDA kernels; there is no
Python or CPU fallback, and a missing library raises immediately.

``LFCache`` is a convenience owner of one cache handle that checks tensor
shapes/dtypes before calling the C functions, and exposes the slab as torch
views (through ``__cuda_array_interface__``) for tests, snapshots and restores.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import torch

__all__ = [
    "LF_OK", "LF_ERR_ARG", "LF_ERR_OOM", "LF_ERR_CUDA", "LF_ERR_DEVICE", "LF_ERR_UNSUPPORTED",
    "LF_BF16", "LF_F32", "LF_KERNEL_AUTO", "LF_KERNEL_SIMT", "LF_KERNEL_TENSOR_CORE",
    "LF_DEVERR_NONFINITE", "LF_DEVERR_STATE", "LF_DEVERR_TIMEOUT",
    "LF_EVICT_OFF", "LF_EVICT_LONGFLOW", "LF_EVICT_RKV", "LF_SCORE_LONGFLOW", "LF_SCORE_H2O",
    "LF_SCOPE_KV_HEAD", "LF_SCOPE_LAYER",
    "LFError", "LFConfig", "LFLayout", "load_library", "library_path",
    "lf_cache_create", "lf_cache_create_ex", "lf_cache_destroy", "lf_prefill_fill",
    "lf_decode_step", "lf_cache_check", "lf_cache_layout", "lf_last_error", "lf_last_status",
    "lf_abi_version",
    "lf_prefill_fill_noalloc", "lf_rkv_compress", "lf_launch_plan", "lf_launch_plan_for",
    "LFCache",
    "LFPages", "lf_paged_append", "lf_paged_decode", "lf_paged_decode_workspace", "lf_paged_prompt",
    "lf_paged_prompt_workspace", "lf_paged_take_errors",
    "LFPagedCache",
    "LFRotaryTable", "LFRows", "lf_rotary_turns", "lf_rotate", "lf_paged_append_rotated",
    "LFRotary",
    "lf_paged_decode_shared", "lf_paged_decode_shared_workspace",
]

LF_OK, LF_ERR_ARG, LF_ERR_OOM, LF_ERR_CUDA, LF_ERR_DEVICE, LF_ERR_UNSUPPORTED = 0, -1, -2, -3, -5, -7
LF_BF16, LF_F32 = 0, 1
LF_KERNEL_AUTO, LF_KERNEL_SIMT, LF_KERNEL_TENSOR_CORE = 0, 1, 2
_KERNEL = {"auto": LF_KERNEL_AUTO, "simt": LF_KERNEL_SIMT, "tc": LF_KERNEL_TENSOR_CORE}
LF_EVICT_OFF, LF_EVICT_LONGFLOW, LF_EVICT_RKV = 0, 1, 2
_EVICT = {"off": LF_EVICT_OFF, "longflow": LF_EVICT_LONGFLOW, "rkv": LF_EVICT_RKV}
LF_SCORE_LONGFLOW, LF_SCORE_H2O = 0, 1
_SCORE = {"longflow": LF_SCORE_LONGFLOW, "h2o": LF_SCORE_H2O}
LF_SCOPE_KV_HEAD, LF_SCOPE_LAYER = 0, 1
_SCOPE = {"kv_head": LF_SCOPE_KV_HEAD, "layer": LF_SCOPE_LAYER}
LF_DEVERR_NONFINITE, LF_DEVERR_STATE, LF_DEVERR_TIMEOUT = 1, 2, 4

_MAX_AXES = 4           # LF_ROTARY_MAX_AXES
_INT_MAX = 2**31 - 1   # of the C calls' numbers, of which ctypes would take the low bits of larger ones

_DTYPE = {"bf16": LF_BF16, "f32": LF_F32}
_TORCH_DTYPE = {LF_BF16: torch.bfloat16, LF_F32: torch.float32}


class LFError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class LFConfig(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("evict", ctypes.c_int),
                ("budgets", ctypes.POINTER(ctypes.c_int32)), ("cluster", ctypes.c_int),
                ("stages", ctypes.c_int), ("kernel", ctypes.c_int),
                ("score", ctypes.c_int), ("norm", ctypes.c_int), ("sinks", ctypes.c_int),
                ("deferred", ctypes.c_int), ("scope", ctypes.c_int),
                ("rkv_buffer", ctypes.c_int), ("rkv_alpha", ctypes.c_int), ("rkv_beta", ctypes.c_int),
                ("rkv_lambda", ctypes.c_float), ("rkv_tau", ctypes.c_float)]


class LFLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "layers", "batch", "kv_heads", "q_heads", "head_dim", "capacity", "slot_stride",
        "window", "dtype", "evict", "cluster", "stages", "kernel")] + [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("vnorm", ctypes.c_void_p),
        ("pos", ctypes.c_void_p), ("count", ctypes.c_void_p), ("next_pos", ctypes.c_void_p),
        ("budget", ctypes.c_void_p), ("err", ctypes.c_void_p)] + [
        (n, ctypes.c_int) for n in ("score", "norm", "sinks", "deferred", "scope")] + [
        ("acc", ctypes.c_void_p), ("pending", ctypes.c_void_p)] + [
        (n, ctypes.c_int) for n in ("rkv_buffer", "rkv_alpha", "rkv_beta")] + [
        ("rkv_lambda", ctypes.c_float), ("rkv_tau", ctypes.c_float),
        ("split_units", ctypes.c_int), ("split_cnt", ctypes.c_void_p)]


class LFPages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "dtype", "kv_heads", "head_dim", "page_size", "num_pages")] + [
        (n, ctypes.c_int64) for n in ("page_stride", "head_stride", "token_stride")] + [
        (n, ctypes.c_void_p) for n in ("k", "v", "err")]


class LFRotaryTable(ctypes.Structure):
    """lf_rotary."""
    _fields_ = [(n, ctypes.c_int) for n in ("rotary_dim", "axes", "adjacent")] + [
        ("scale", ctypes.c_float), ("turns", ctypes.c_void_p), ("axis", ctypes.c_void_p)]


class LFRows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int)] + [
        (n, ctypes.c_int64) for n in ("x_seq", "x_token", "x_head", "y_seq", "y_token", "y_head")]


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return os.environ.get("LONGFLOW_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                          "liblongflow.so")


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load liblongflow.so once; raise if it is missing (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"liblongflow.so not found at {path}: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    P, I, VP = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    lib.lf_cache_create.restype = P
    lib.lf_cache_create.argtypes = [I] * 7
    lib.lf_cache_create_ex.restype = P
    lib.lf_cache_create_ex.argtypes = [I] * 7 + [ctypes.POINTER(LFConfig)]
    lib.lf_cache_destroy.restype = I
    lib.lf_cache_destroy.argtypes = [P]
    lib.lf_prefill_fill.restype = I
    lib.lf_prefill_fill.argtypes = [P, I, VP, VP, ctypes.POINTER(ctypes.c_int32), I, VP]
    lib.lf_decode_step.restype = I
    lib.lf_decode_step.argtypes = [P, I, VP, VP, VP, VP, VP, VP]
    lib.lf_cache_check.restype = I
    lib.lf_cache_check.argtypes = [P, VP, ctypes.POINTER(ctypes.c_int32)]
    lib.lf_cache_layout.restype = I
    lib.lf_cache_layout.argtypes = [P, ctypes.POINTER(LFLayout)]
    lib.lf_last_error.restype = ctypes.c_char_p
    lib.lf_last_error.argtypes = []
    lib.lf_abi_version.restype = I
    lib.lf_abi_version.argtypes = []
    lib.lf_last_status.restype = I
    lib.lf_last_status.argtypes = []
    lib.lf_rkv_compress.restype = I
    lib.lf_rkv_compress.argtypes = [P, I, VP, VP]
    lib.lf_launch_plan.restype = I
    lib.lf_launch_plan.argtypes = [P, I] + [ctypes.POINTER(ctypes.c_int32)] * 3 + [I]
    lib.lf_launch_plan_for.restype = I
    lib.lf_launch_plan_for.argtypes = ([ctypes.POINTER(ctypes.c_int32)] + [I] * 4 +
                                       [ctypes.POINTER(ctypes.c_int32)] * 3)
    lib.lf_prefill_fill_noalloc.restype = I
    lib.lf_prefill_fill_noalloc.argtypes = [ctypes.POINTER(LFLayout), I, VP, VP,
                                            ctypes.POINTER(ctypes.c_int32), I, VP]
    PG = ctypes.POINTER(LFPages)
    lib.lf_paged_append.restype = I
    lib.lf_paged_append.argtypes = [PG, I, VP, I, VP, VP, VP, VP, I, VP]
    lib.lf_paged_decode.restype = I
    lib.lf_paged_decode.argtypes = [PG, I, VP, I, VP, I, VP, VP, VP, VP, VP, I, I, VP,
                                    ctypes.c_size_t, VP]
    lib.lf_paged_decode_workspace.restype = I
    lib.lf_paged_decode_workspace.argtypes = [PG, I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
    lib.lf_paged_prompt.restype = I
    lib.lf_paged_prompt.argtypes = [PG, I, VP, I, VP, I, VP, VP, I, I, VP, VP, I, I, VP,
                                    ctypes.c_size_t, VP]
    lib.lf_paged_prompt_workspace.restype = I
    lib.lf_paged_prompt_workspace.argtypes = [PG, I, I, I, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
    lib.lf_paged_take_errors.restype = I
    lib.lf_paged_take_errors.argtypes = [PG, VP, VP]
    lib.lf_paged_decode_shared.restype = I
    lib.lf_paged_decode_shared.argtypes = [PG, I, VP, I, VP, I, VP, VP, I, VP, VP, VP, VP, VP, VP, ctypes.c_size_t, VP]
    lib.lf_paged_decode_shared_workspace.restype = I
    lib.lf_paged_decode_shared_workspace.argtypes = [PG, I, I, I, I, ctypes.POINTER(ctypes.c_size_t)]
    RT, RW, LL = ctypes.POINTER(LFRotaryTable), ctypes.POINTER(LFRows), ctypes.c_int64
    lib.lf_rotary_turns.restype = I
    lib.lf_rotary_turns.argtypes = [ctypes.POINTER(ctypes.c_double), I, ctypes.POINTER(ctypes.c_uint64)]
    lib.lf_rotate.restype = I
    lib.lf_rotate.argtypes = [RT, I, I, I, I, RW, RW, VP, LL, I, VP]
    lib.lf_paged_append_rotated.restype = I
    lib.lf_paged_append_rotated.argtypes = [PG, I, VP, I, VP, VP, VP, VP, I, RT, VP, LL, I, VP, VP, VP]
    _lib = lib
    return lib


# ---- C-named wrappers (argument marshalling only) ---------------------------

def lf_last_error() -> str:
    return (load_library().lf_last_error() or b"").decode()


def lf_last_status() -> int:
    return load_library().lf_last_status()


def _create_failed() -> "LFError":
    """The error of a create call that returned NULL, with the library's status."""
    return LFError(lf_last_status() or LF_ERR_ARG, lf_last_error())


def lf_abi_version() -> int:
    return load_library().lf_abi_version()


def _check(code: int) -> int:
    if code != LF_OK:
        raise LFError(code, lf_last_error())
    return code


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def lf_cache_create(layers, batch, kv_heads, q_heads, head_dim, budget, window) -> int:
    h = load_library().lf_cache_create(layers, batch, kv_heads, q_heads, head_dim, budget, window)
    if not h:
        raise _create_failed()
    return h


def lf_cache_create_ex(layers, batch, kv_heads, q_heads, head_dim, capacity, window,
                       dtype="bf16", evict=True, budgets: Optional[Sequence[int]] = None,
                       cluster=0, stages=0, kernel="auto", score="longflow", norm=1, sinks=0,
                       deferred=False, scope="kv_head", rkv_buffer=0, rkv_alpha=0, rkv_beta=0,
                       rkv_lambda=0.0, rkv_tau=0.0) -> int:
    cfg = LFConfig()
    cfg.dtype = _DTYPE[dtype] if isinstance(dtype, str) else int(dtype)
    cfg.evict = _EVICT[evict] if isinstance(evict, str) else int(evict)
    arr = None
    if budgets is not None:
        arr = (ctypes.c_int32 * len(budgets))(*[int(x) for x in budgets])
        cfg.budgets = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
    cfg.cluster = int(cluster)
    cfg.stages = int(stages)
    cfg.kernel = _KERNEL[kernel] if isinstance(kernel, str) else int(kernel)
    cfg.score = _SCORE[score] if isinstance(score, str) else int(score)
    cfg.norm = int(norm)
    cfg.sinks = int(sinks)
    cfg.deferred = int(bool(deferred))
    cfg.scope = _SCOPE[scope] if isinstance(scope, str) else int(scope)
    cfg.rkv_buffer, cfg.rkv_alpha, cfg.rkv_beta = int(rkv_buffer), int(rkv_alpha), int(rkv_beta)
    cfg.rkv_lambda, cfg.rkv_tau = float(rkv_lambda), float(rkv_tau)
    h = load_library().lf_cache_create_ex(layers, batch, kv_heads, q_heads, head_dim, capacity,
                                          window, ctypes.byref(cfg))
    if not h:
        raise _create_failed()
    return h


def lf_cache_destroy(handle) -> int:
    return _check(load_library().lf_cache_destroy(handle))


def lf_prefill_fill(handle, layer, k, v, prompt_len: Sequence[int], max_prompt, stream=None) -> int:
    arr = (ctypes.c_int32 * len(prompt_len))(*[int(x) for x in prompt_len])
    return _check(load_library().lf_prefill_fill(handle, layer, _ptr(k), _ptr(v), arr,
                                                 int(max_prompt), _stream(stream)))


def lf_decode_step(handle, layer, q, k_new, v_new, out, evicted_slot, stream=None) -> int:
    return _check(load_library().lf_decode_step(handle, layer, _ptr(q), _ptr(k_new), _ptr(v_new),
                                                _ptr(out), _ptr(evicted_slot), _stream(stream)))


def lf_cache_check(handle, stream=None) -> int:
    """Return the device error bits (0 when clean); raise on a CUDA failure."""
    bits = ctypes.c_int32(0)
    code = load_library().lf_cache_check(handle, _stream(stream), ctypes.byref(bits))
    if code not in (LF_OK, LF_ERR_DEVICE):
        raise LFError(code, lf_last_error())
    return int(bits.value)


def lf_prefill_fill_noalloc(dst: LFLayout, layer, k, v, prompt_len: Sequence[int], max_prompt,
                            stream=None) -> int:
    arr = (ctypes.c_int32 * len(prompt_len))(*[int(x) for x in prompt_len])
    return _check(load_library().lf_prefill_fill_noalloc(ctypes.byref(dst), layer, _ptr(k), _ptr(v),
                                                         arr, int(max_prompt), _stream(stream)))


def lf_rkv_compress(handle, layer, q_obs, stream=None) -> int:
    return _check(load_library().lf_rkv_compress(handle, layer, _ptr(q_obs), _stream(stream)))


def lf_launch_plan(handle, layer):
    """The next step's plan of `layer`: None (whole units j, j + nc, ... per
    cluster), or (rounds, cuts) with cuts[j] = (unit, slot) where cluster j's
    range of the units past the whole rounds starts (cuts[nc] = (units, 0))."""
    lib = load_library()
    n = 256
    rounds = ctypes.c_int32(0)
    cu, cs = ((ctypes.c_int32 * n)() for _ in range(2))
    nc = lib.lf_launch_plan(handle, layer, ctypes.byref(rounds), cu, cs, n)
    if nc < 0:
        raise LFError(nc, lf_last_error())
    if nc == 0:
        return None
    return int(rounds.value), [(int(cu[j]), int(cs[j])) for j in range(nc + 1)]


def lf_launch_plan_for(occupancy: Sequence[int], cluster: int, clusters: int, max_items: int):
    """The planner on given per-unit occupancies: None or (rounds, cuts), as
    lf_launch_plan returns them."""
    lib = load_library()
    occ = (ctypes.c_int32 * len(occupancy))(*[int(x) for x in occupancy])
    rounds = ctypes.c_int32(0)
    cu, cs = ((ctypes.c_int32 * (clusters + 1))() for _ in range(2))
    nc = lib.lf_launch_plan_for(occ, len(occupancy), cluster, clusters, max_items,
                                ctypes.byref(rounds), cu, cs)
    if nc < 0:
        raise LFError(nc, lf_last_error())
    if nc == 0:
        return None
    return int(rounds.value), [(int(cu[j]), int(cs[j])) for j in range(nc + 1)]


def lf_cache_layout(handle) -> LFLayout:
    lay = LFLayout()
    _check(load_library().lf_cache_layout(handle, ctypes.byref(lay)))
    return lay


def lf_paged_append(pages: LFPages, batch, page_table, max_pages, lens, k_new, v_new, new_start,
                    total_new, stream=None) -> int:
    return _check(load_library().lf_paged_append(
        ctypes.byref(pages), batch, _ptr(page_table), max_pages, _ptr(lens), _ptr(k_new), _ptr(v_new),
        _ptr(new_start), total_new, _stream(stream)))


def lf_paged_decode(pages: LFPages, batch, page_table, max_pages, lens, q_heads, q, k_new, v_new, out,
                    lse, window, sinks, workspace, workspace_bytes, stream=None) -> int:
    return _check(load_library().lf_paged_decode(
        ctypes.byref(pages), batch, _ptr(page_table), max_pages, _ptr(lens), q_heads, _ptr(q),
        _ptr(k_new), _ptr(v_new), _ptr(out), _ptr(lse), window, sinks, _ptr(workspace), workspace_bytes,
        _stream(stream)))


def lf_paged_decode_workspace(pages: LFPages, batch, max_pages, q_heads, window=0, sinks=0) -> int:
    """Bytes of the workspace that such lf_paged_decode calls need (0: none)."""
    n = ctypes.c_size_t(0)
    _check(load_library().lf_paged_decode_workspace(ctypes.byref(pages), batch, max_pages, q_heads,
                                                    window, sinks, ctypes.byref(n)))
    return int(n.value)


def lf_paged_decode_shared(pages: LFPages, batch, page_table, max_pages, lens, q_heads, q, group_start, groups,
                           prefix_lens, k_new, v_new, out, lse, workspace, workspace_bytes, stream=None) -> int:
    return _check(load_library().lf_paged_decode_shared(
        ctypes.byref(pages), batch, _ptr(page_table), max_pages, _ptr(lens), q_heads, _ptr(q), _ptr(group_start), groups,
        _ptr(prefix_lens), _ptr(k_new), _ptr(v_new), _ptr(out), _ptr(lse), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def lf_paged_decode_shared_workspace(pages: LFPages, batch, max_pages, q_heads, groups) -> int:
    """Bytes of the workspace that such lf_paged_decode_shared calls need."""
    n = ctypes.c_size_t(0)
    _check(load_library().lf_paged_decode_shared_workspace(ctypes.byref(pages), batch, max_pages, q_heads, groups,
                                                           ctypes.byref(n)))
    return int(n.value)


def lf_paged_prompt(pages: LFPages, batch, page_table, max_pages, lens, q_heads, q, q_start, total_q,
                    max_q, out, lse, window, sinks, workspace, workspace_bytes, stream=None) -> int:
    return _check(load_library().lf_paged_prompt(
        ctypes.byref(pages), batch, _ptr(page_table), max_pages, _ptr(lens), q_heads, _ptr(q),
        _ptr(q_start), total_q, max_q, _ptr(out), _ptr(lse), window, sinks, _ptr(workspace),
        workspace_bytes, _stream(stream)))


def lf_paged_prompt_workspace(pages: LFPages, batch, max_pages, q_heads, total_q, max_q, window=0,
                              sinks=0) -> int:
    """Bytes of the workspace that such lf_paged_prompt calls need (0: none)."""
    n = ctypes.c_size_t(0)
    _check(load_library().lf_paged_prompt_workspace(ctypes.byref(pages), batch, max_pages, q_heads,
                                                    total_q, max_q, window, sinks, ctypes.byref(n)))
    return int(n.value)


def lf_paged_take_errors(pages: LFPages, taken, stream=None) -> int:
    return _check(load_library().lf_paged_take_errors(ctypes.byref(pages), _ptr(taken), _stream(stream)))


def lf_rotary_turns(frequency: Sequence[float]) -> list:
    """Turns per position, in 2^-64 of a turn, of frequencies in radians per position."""
    n = len(frequency)
    turns = (ctypes.c_uint64 * n)()
    _check(load_library().lf_rotary_turns((ctypes.c_double * n)(*frequency), n, turns))
    return list(turns)


def lf_rotate(rotary: LFRotaryTable, dtype, row_dim, seqs, tokens, q: LFRows, k: Optional[LFRows], positions,
              axis_stride, inverse=False, stream=None) -> int:
    return _check(load_library().lf_rotate(
        ctypes.byref(rotary), _DTYPE[dtype] if isinstance(dtype, str) else int(dtype), row_dim, seqs, tokens,
        ctypes.byref(q), None if k is None else ctypes.byref(k), _ptr(positions), axis_stride, int(bool(inverse)),
        _stream(stream)))


def lf_paged_append_rotated(pages: LFPages, batch, page_table, max_pages, lens, k_new, v_new, new_start, total_new,
                            rotary: LFRotaryTable, positions, axis_stride, q_heads, q, q_out, stream=None) -> int:
    return _check(load_library().lf_paged_append_rotated(
        ctypes.byref(pages), batch, _ptr(page_table), max_pages, _ptr(lens), _ptr(k_new), _ptr(v_new),
        _ptr(new_start), total_new, ctypes.byref(rotary), _ptr(positions), axis_stride, q_heads, _ptr(q), _ptr(q_out),
        _stream(stream)))


# ---- convenience owner ------------------------------------------------------

class _DevArray:
    """Minimal __cuda_array_interface__ exporter for a raw device pointer."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"data": (int(ptr), False), "shape": tuple(shape),
                                         "typestr": typestr, "version": 3, "strides": None}


def _view(ptr, shape, dtype: torch.dtype, device) -> torch.Tensor:
    typestr = {torch.float32: "<f4", torch.int32: "<i4", torch.int16: "<i2"}[dtype]
    return torch.as_tensor(_DevArray(ptr, shape, typestr), device=device)


class LFCache:
    """One LongFlow cache (owns the C handle).  Sizes as in ``lf_cache_create_ex``."""

    def __init__(self, layers, batch, kv_heads, q_heads, head_dim, capacity, window,
                 dtype="bf16", evict=True, budgets=None, cluster=0, stages=0, kernel="auto",
                 device=None, score="longflow", norm=1, sinks=0, deferred=False,
                 scope="kv_head", **rkv):
        self.device = torch.device("cuda", torch.cuda.current_device() if device is None
                                   else torch.device(device).index or 0)
        with torch.cuda.device(self.device):
            self.handle = lf_cache_create_ex(layers, batch, kv_heads, q_heads, head_dim, capacity,
                                             window, dtype, evict, budgets, cluster, stages,
                                             kernel, score, norm, sinks, deferred, scope, **rkv)
        self.layout = lf_cache_layout(self.handle)
        self.dtype = _TORCH_DTYPE[self.layout.dtype]
        self.layers, self.batch = layers, batch
        self.kv_heads, self.q_heads, self.head_dim = kv_heads, q_heads, head_dim
        self.capacity, self.window = capacity, window
        self.evict = self.layout.evict != LF_EVICT_OFF

    def close(self):
        if getattr(self, "handle", None):
            lf_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _expect(self, t, shape, name, dtype=None):
        dtype = dtype or self.dtype
        if not isinstance(t, torch.Tensor) or t.device != self.device or t.dtype != dtype \
                or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            got = (tuple(t.shape), t.dtype, str(t.device)) if isinstance(t, torch.Tensor) else type(t)
            raise LFError(LF_ERR_ARG, f"{name}: expected contiguous {dtype} {tuple(shape)} on "
                                      f"{self.device}, got {got}")

    def prefill(self, layer, k, v, prompt_lens, stream=None):
        pmax = k.shape[2]
        self._expect(k, (self.batch, self.kv_heads, pmax, self.head_dim), "k")
        self._expect(v, (self.batch, self.kv_heads, pmax, self.head_dim), "v")
        lf_prefill_fill(self.handle, layer, k, v, list(prompt_lens), pmax, stream)

    def decode_step(self, layer, q, k_new, v_new, out=None, evicted=None, stream=None):
        b, hq, hkv, d = self.batch, self.q_heads, self.kv_heads, self.head_dim
        self._expect(q, (b, hq, d), "q")
        self._expect(k_new, (b, hkv, d), "k_new")
        self._expect(v_new, (b, hkv, d), "v_new")
        if out is None:
            out = torch.empty((b, hq, d), dtype=self.dtype, device=self.device)
        if evicted is None:
            evicted = torch.empty((b, hkv), dtype=torch.int32, device=self.device)
        self._expect(out, (b, hq, d), "out")
        self._expect(evicted, (b, hkv), "evicted", torch.int32)
        lf_decode_step(self.handle, layer, q, k_new, v_new, out, evicted, stream)
        return out, evicted

    def rkv_compress(self, layer, q_obs, stream=None):
        """R-KV compression of one layer; q_obs [batch][rkv_alpha][q_heads][head_dim]."""
        lay = self.layout
        self._expect(q_obs, (self.batch, lay.rkv_alpha, self.q_heads, self.head_dim), "q_obs")
        lf_rkv_compress(self.handle, layer, q_obs, stream)

    def plan(self, layer: int):
        """lf_launch_plan: None, or the (unit, slot) cuts of the next step of `layer`."""
        return lf_launch_plan(self.handle, layer)

    def check(self, stream=None) -> int:
        return lf_cache_check(self.handle, stream)

    def views(self):
        """Torch tensors aliasing the slab (no copy): k, v [L][b][H_kv][stride][d],
        vnorm, pos [L][b][H_kv][stride], count, next_pos [L][b][H_kv], budget [b];
        acc [L][b][H_kv][stride] (H2O) and pending [L][b][H_kv] (deferred), else None;
        split_cnt [split_units][2] (split launches), else None."""
        lay = self.layout
        L, b, g, s, d = lay.layers, lay.batch, lay.kv_heads, lay.slot_stride, lay.head_dim
        if self.dtype == torch.bfloat16:
            k = _view(lay.k, (L, b, g, s, d), torch.int16, self.device).view(torch.bfloat16)
            v = _view(lay.v, (L, b, g, s, d), torch.int16, self.device).view(torch.bfloat16)
        else:
            k = _view(lay.k, (L, b, g, s, d), torch.float32, self.device)
            v = _view(lay.v, (L, b, g, s, d), torch.float32, self.device)
        return {
            "k": k, "v": v,
            "vnorm": _view(lay.vnorm, (L, b, g, s), torch.float32, self.device),
            "pos": _view(lay.pos, (L, b, g, s), torch.int32, self.device),
            "count": _view(lay.count, (L, b, g), torch.int32, self.device),
            "next_pos": _view(lay.next_pos, (L, b, g), torch.int32, self.device),
            "budget": _view(lay.budget, (b,), torch.int32, self.device),
            "acc": (_view(lay.acc, (L, b, g, s), torch.float32, self.device)
                    if lay.acc else None),
            "pending": (_view(lay.pending, (L, b, g), torch.int32, self.device)
                        if lay.pending else None),
            "split_cnt": (_view(lay.split_cnt, (lay.split_units, 2), torch.int32, self.device)
                          if lay.split_cnt else None),
        }


def _run_on(device, index, stream, held, call, *args):
    """call(stream handle, *args) with the device and `stream` (None: the current one) current; a stream that the
    caller names is known to the allocator as one that reads held() and the tensors among args."""
    if stream is None and torch.cuda.current_device() == index:
        return call(torch._C._cuda_getCurrentRawStream(index), *args)
    if isinstance(stream, int):
        # 0, the default stream's handle, would make torch take a stream of its pool
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    if stream is not None and getattr(stream, "device", None) != device:
        raise LFError(LF_ERR_ARG, f"stream: expected a stream of {device}, got {stream}")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        if stream is not None:
            for t in (*held(), *args):
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
        return call(torch._C._cuda_getCurrentRawStream(index), *args)


def _cuda_device(device) -> torch.device:
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise LFError(LF_ERR_ARG, f"device: expected a CUDA device, got {device}")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


_ROW_TYPES = (torch.bfloat16, torch.float32)


def _rows(x, y) -> LFRows:
    """Rows of x, to be written to y of the same shape.  A size of one has no use for its stride."""
    shape, sx, sy = x.shape, x.stride(), y.stride()
    if 1 in shape:
        sx, sy = ([s if n > 1 else 0 for n, s in zip(shape, st)] for st in (sx, sy))
    if len(shape) == 3:
        return LFRows(x.data_ptr(), y.data_ptr(), shape[1], 0, sx[0], sx[1], 0, sy[0], sy[1])
    return LFRows(x.data_ptr(), y.data_ptr(), shape[2], *sx[:3], *sy[:3])


def _no_gradients(*tensors):
    """A call on raw memory gives its result no graph: a gradient would be lost unseen."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise LFError(LF_ERR_ARG, "a tensor requires a gradient, which rotations do not record: call them under "
                                          "torch.no_grad(), or in an autograd function whose backward turns back (inverse)")


def _will_change(*tensors):
    """A call writes to these tensors of the caller's: autograd, which may have saved one for a backward pass, has to know."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


class LFRotary:
    """Rotary positions of a model's heads: its frequencies, kept on the device, and the calls that rotate by them.

    Rotations record no gradients: tensors that require one are refused while gradients are recorded.

    The first ``rotary_dim`` columns of a row are ``rotary_dim / 2`` pairs, columns ``(i, i + rotary_dim / 2)``, or
    ``(2 i, 2 i + 1)`` if ``adjacent``.  Pair i turns by ``inv_freq[i]`` radians per position; without ``inv_freq`` by
    ``base ** (-2 i / rotary_dim)``.  ``scale`` multiplies the turned columns.

    Where tokens have a position on each of several axes (time, height, width), ``sections`` gives the number of
    consecutive pairs of every axis, or ``axis`` each pair's axis.
    """

    def __init__(self, rotary_dim, base=10000.0, inv_freq=None, sections=None, axis=None, adjacent=False, scale=1.0,
                 device=None):
        if not isinstance(rotary_dim, int) or rotary_dim < 16 or rotary_dim % 16 or rotary_dim > 512:
            raise LFError(LF_ERR_ARG, f"rotary_dim must be a multiple of 16 in [16, 512], got {rotary_dim}")
        pairs = rotary_dim // 2
        if inv_freq is None:
            if not base > 0:
                raise LFError(LF_ERR_ARG, f"base must be above 0, got {base}")
            inv_freq = [float(base) ** (-2.0 * i / rotary_dim) for i in range(pairs)]
        inv_freq = [float(f) for f in inv_freq]
        if sections is not None:
            if axis is not None:
                raise LFError(LF_ERR_ARG, "sections and axis: at most one of them")
            sections = [int(n) for n in sections]
            if not 1 <= len(sections) <= _MAX_AXES or min(sections) < 0 or sum(sections) != pairs:
                raise LFError(LF_ERR_ARG, f"sections: expected up to {_MAX_AXES} numbers of pairs that sum to {pairs}, "
                                          f"got {sections}")
            axis, self.axes = [a for a, n in enumerate(sections) for _ in range(n)], len(sections)
        elif axis is not None:
            axis = [int(a) for a in axis]
            if axis and not 0 <= min(axis) <= max(axis) < _MAX_AXES:
                raise LFError(LF_ERR_ARG, f"axis: expected axes in [0, {_MAX_AXES}), got {axis}")
            self.axes = max(axis, default=0) + 1
        else:
            axis, self.axes = [0] * pairs, 1
        if len(inv_freq) != pairs or len(axis) != pairs:
            raise LFError(LF_ERR_ARG, f"expected {pairs} frequencies and axes, got {len(inv_freq)} and {len(axis)}")
        if not math.isfinite(scale):
            raise LFError(LF_ERR_ARG, f"scale must be finite, got {scale}")
        turns = [t - 2**64 if t >= 2**63 else t for t in lf_rotary_turns(inv_freq)]
        self.rotary_dim, self.adjacent, self.scale = rotary_dim, bool(adjacent), float(scale)
        self.device = _cuda_device(device)
        self._index = self.device.index
        # copied from the host, which waits, so that no stream that uses them can come before it
        if torch.cuda.is_current_stream_capturing():
            raise LFError(LF_ERR_ARG, "make the rotary before the capture of a graph")
        self._turns = torch.tensor(turns, dtype=torch.int64).to(self.device)
        self._axis = torch.tensor(axis, dtype=torch.int32).to(self.device)
        self._held = (self._turns, self._axis)
        self._table = LFRotaryTable(rotary_dim, self.axes, int(self.adjacent), self.scale, self._turns.data_ptr(),
                                    self._axis.data_ptr())
        self._lib = load_library()

    def _positions(self, positions, lead):
        """The axis stride of positions [*lead], or [axes, *lead]."""
        if isinstance(positions, torch.Tensor) and positions.dtype == torch.int32 \
                and positions.get_device() == self._index and positions.is_contiguous():
            shape = positions.shape
            if shape == lead:
                return 0
            if shape[0] == self.axes and shape[1:] == lead:
                return positions.numel() // self.axes
        got = (tuple(positions.shape), positions.dtype, str(positions.device)) \
            if isinstance(positions, torch.Tensor) else type(positions)
        raise LFError(LF_ERR_ARG, f"positions: expected contiguous torch.int32 {tuple(lead)} or "
                                  f"{(self.axes, *lead)} on {self.device}, got {got}")

    def _expect(self, t, name, dtype=None, shape=None):
        """Rows of a call: with `dtype` and `shape`, of these; -> their shape."""
        if isinstance(t, torch.Tensor) and t.get_device() == self._index:
            mine = t.shape
            if (t.dtype == dtype if dtype else t.dtype in _ROW_TYPES) and (mine == shape if shape else 3 <= len(mine) <= 4) \
                    and (t.stride(-1) == 1 or mine[-1] <= 1):
                return mine
        got = (tuple(t.shape), t.dtype, str(t.device)) if isinstance(t, torch.Tensor) else type(t)
        raise LFError(LF_ERR_ARG, f"{name}: expected bf16 or fp32 rows [tokens][heads][dim] or [sequences][tokens][heads]"
                                  f"[dim], of the call's type and tokens, on {self.device}, got {got}")

    def rotate(self, q, positions, k=None, q_out=None, k_out=None, inverse=False, stream=None):
        """lf_rotate: rows q [tokens][heads][dim] or [sequences][tokens][heads][dim], in any order in memory with
        contiguous rows, and of k where it is given, by positions int32 [tokens] ([sequences][tokens]), or
        [axes][...].  Returns q_out (a new tensor if None; q rotates in place), or (q_out, k_out) with k.
        ``inverse`` turns back: the transpose, which takes a gradient of the result to that of the rows (the call
        itself records none)."""
        shape = self._expect(q, "q")
        if q_out is not None:
            self._expect(q_out, "q_out", q.dtype, shape)
        if k is not None:
            k_shape = self._expect(k, "k", q.dtype)
            if k_shape[:-2] != shape[:-2] or k_shape[-1] != shape[-1]:
                raise LFError(LF_ERR_ARG, f"k: expected q's {tuple(shape[:-2])} tokens and {shape[-1]} columns, got "
                                          f"{tuple(k_shape)}")
            if k_out is not None:
                self._expect(k_out, "k_out", q.dtype, k_shape)
        elif k_out is not None:
            raise LFError(LF_ERR_ARG, "k_out without k")
        step = self._positions(positions, shape[:-2])
        _no_gradients(q, k, q_out, k_out)
        if q_out is not None or k_out is not None:
            _will_change(q_out, k_out)
        return _run_on(self.device, self._index, stream, lambda: self._held, self._rotate, q, positions, k, q_out, k_out, step,
                       1 if inverse else 0)

    def _rotate(self, st, q, positions, k, q_out, k_out, step, inverse):
        shape = q.shape
        seqs, tokens = (1, shape[0]) if len(shape) == 3 else shape[:2]
        if max(shape) > _INT_MAX or (k is not None and k.shape[-2] > _INT_MAX):
            raise LFError(LF_ERR_ARG, f"no size may be above 2^31 - 1, got {tuple(shape)}")
        if q_out is None:
            q_out = torch.empty_like(q)
        k_rows = None
        if k is not None:
            if k_out is None:
                k_out = torch.empty_like(k)
            k_rows = _rows(k, k_out)
        _check(self._lib.lf_rotate(
            self._table, LF_BF16 if q.dtype == torch.bfloat16 else LF_F32, shape[-1], seqs, tokens, _rows(q, q_out),
            k_rows, positions.data_ptr(), step, inverse, st))
        return q_out if k is None else (q_out, k_out)


class LFPagedCache:
    """Paged K and V pools of a model's layers, and the calls that use them.

    ``LFPagedCache(layers, num_pages, page_size, kv_heads, head_dim)`` allocates pools
    ``[layers][num_pages][kv_heads][page_size][head_dim]`` (uninitialised); ``over(k, v)`` takes
    tensors that the caller owns, of that shape in any stride order with contiguous rows.  The
    caller hands out pages: ``page_table`` int32 ``[batch][max_pages]`` and ``lens`` int32
    ``[batch]`` (lengths including the call's own tokens) are contiguous tensors on the device.

    Calls run on the current stream, or on ``stream`` (a torch stream or a raw handle), which the
    caller orders behind the stream that made the inputs.  What a call returns belongs to the stream
    that it ran on.
    """

    def __init__(self, layers, num_pages, page_size, kv_heads, head_dim, dtype="bf16", device=None):
        device = _cuda_device(device)
        if min(layers, num_pages, page_size, kv_heads, head_dim) < 1:
            raise LFError(LF_ERR_ARG, "layers, num_pages, page_size, kv_heads and head_dim must be >= 1")
        if dtype not in _DTYPE:
            raise LFError(LF_ERR_ARG, f"dtype must be one of {sorted(_DTYPE)}")
        shape = (layers, num_pages, kv_heads, page_size, head_dim)
        t = _TORCH_DTYPE[_DTYPE[dtype]]
        self._take(torch.empty(shape, dtype=t, device=device), torch.empty(shape, dtype=t, device=device))

    @classmethod
    def over(cls, k: torch.Tensor, v: torch.Tensor) -> "LFPagedCache":
        """A cache on the caller's pools k, v [layers][num_pages][kv_heads][page_size][head_dim]."""
        self = cls.__new__(cls)
        self._take(k, v)
        return self

    def _take(self, k, v):
        types = {t: n for n, t in _TORCH_DTYPE.items()}
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or t.dim() != 5 or not t.is_cuda or t.dtype not in types:
                raise LFError(LF_ERR_ARG, f"{name}: expected a bf16 or fp32 CUDA tensor [layers][num_pages]"
                                          "[kv_heads][page_size][head_dim]")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device or k.stride() != v.stride():
            raise LFError(LF_ERR_ARG, "k and v must agree in shape, strides, dtype and device")
        strides = k.stride()
        if k.numel() == 0 or (k.shape[4] > 1 and strides[4] != 1):
            raise LFError(LF_ERR_ARG, "the pools must not be empty and their rows must be contiguous")
        if max(k.shape) > _INT_MAX:
            raise LFError(LF_ERR_ARG, f"pools {tuple(k.shape)}: no size may be above 2^31 - 1")
        self.k, self.v, self.dtype, self.device = k, v, k.dtype, k.device
        self.layers, self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self._index = k.get_device()
        self._row = (self.kv_heads, self.head_dim)
        # the device error word, as a tensor of one int32; copied from the host, which waits, so that
        # no stream that uses the cache can come before it (and which no graph can hold)
        if torch.cuda.is_current_stream_capturing():
            raise LFError(LF_ERR_ARG, "make the cache before the capture of a graph")
        self.err = torch.zeros(1, dtype=torch.int32).to(k.device)
        step, pk, pv = strides[0] * k.element_size(), k.data_ptr(), v.data_ptr()
        self._pages = [LFPages(types[k.dtype], self.kv_heads, self.head_dim, self.page_size, self.num_pages,
                               strides[1], strides[2], strides[3], pk + i * step, pv + i * step,
                               self.err.data_ptr()) for i in range(self.layers)]
        self._need = {}   # workspace bytes by the shape of a decode or prompt call
        self._lib = load_library()

    def _layer(self, layer) -> LFPages:
        if not 0 <= layer < self.layers:
            raise LFError(LF_ERR_ARG, f"layer {layer} outside [0, {self.layers})")
        return self._pages[layer]

    def _expect(self, t, name, dtype, shape):
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape \
                or t.get_device() != self._index or not t.is_contiguous():
            got = (tuple(t.shape), t.dtype, str(t.device)) if isinstance(t, torch.Tensor) else type(t)
            raise LFError(LF_ERR_ARG, f"{name}: expected contiguous {dtype} {tuple(shape)} on {self.device}, "
                                      f"got {got}")

    def _sizes(self, t, name, dims):
        """The shape of a tensor of so many dimensions; a wrong one fails the check that follows."""
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise LFError(LF_ERR_ARG, f"{name}: expected a tensor of {dims} dimensions, got "
                                      f"{tuple(t.shape) if isinstance(t, torch.Tensor) else type(t)}")
        return t.shape

    def _sequences(self, page_table, lens):
        shape = self._sizes(page_table, "page_table", 2)
        self._expect(page_table, "page_table", torch.int32, shape)
        self._expect(lens, "lens", torch.int32, shape[:1])
        return shape

    def _numbers(self, rows, window=0, sinks=0, max_q=0):
        if rows > _INT_MAX or max_q < 0:
            raise LFError(LF_ERR_ARG, f"need at most 2^31 - 1 tokens and max_q >= 0, got {rows} and {max_q}")
        if not 0 <= window <= _INT_MAX or not 0 <= sinks <= _INT_MAX:
            raise LFError(LF_ERR_ARG, f"window and sinks must be in [0, 2^31 - 1], got {window} and {sinks}")

    def _outputs(self, q, out, lse):
        if out is not None:
            self._expect(out, "out", self.dtype, q.shape)
        if lse is not None:
            self._expect(lse, "lse", torch.float32, q.shape[:2])
        if out is not None or lse is not None:
            _will_change(out, lse)

    def _run(self, stream, call, *args):
        """call(stream handle, *args) with this cache's device and `stream` current, so that
        what it allocates belongs to that stream.  The allocator is told that a stream which the caller
        names reads the tensors: they may be let go as soon as the call returns."""
        if stream is None and torch.cuda.current_device() == self._index:
            return call(torch._C._cuda_getCurrentRawStream(self._index), *args)
        return _run_on(self.device, self._index, stream, lambda: (self.k, self.v, self.err), call, *args)

    def _ask(self, call, pages, key):
        """The workspace that calls of this shape need, remembered (of the last few thousand shapes)."""
        if len(self._need) >= 4096:
            self._need.clear()
        need = self._need[key] = call(pages, *key)
        return need

    def append(self, layer, k_new, v_new, page_table, lens, new_start=None, stream=None):
        """lf_paged_append: k_new, v_new [tokens][kv_heads][head_dim] go to their pages;
        new_start int32 [batch + 1], or None: one token per sequence."""
        pages = self._layer(layer)
        batch, width = self._sequences(page_table, lens)
        n = batch if new_start is None else self._sizes(k_new, "k_new", 3)[0]
        self._expect(k_new, "k_new", self.dtype, (n, *self._row))
        self._expect(v_new, "v_new", self.dtype, (n, *self._row))
        if new_start is not None:
            self._expect(new_start, "new_start", torch.int32, (batch + 1,))
            self._numbers(n)
        self._run(stream, self._append, pages, batch, width, page_table, lens, k_new, v_new, new_start, n)

    def _append(self, st, pages, batch, width, page_table, lens, k_new, v_new, new_start, n):
        _check(self._lib.lf_paged_append(
            pages, batch, page_table.data_ptr(), width, lens.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
            None if new_start is None else new_start.data_ptr(), n, st))

    def append_rotated(self, layer, k_new, v_new, page_table, lens, rotary, new_start=None, positions=None, q=None,
                       q_out=None, stream=None):
        """lf_paged_append_rotated: ``append`` with the rows of k_new rotated by ``rotary`` (an LFRotary) on the way,
        and q [tokens][q_heads][head_dim] into q_out (a new tensor if None; q rotates in place), which is returned.
        positions int32 [tokens] or [axes][tokens], or None: each token's position in the cache."""
        pages = self._layer(layer)
        batch, width = self._sequences(page_table, lens)
        if not isinstance(rotary, LFRotary) or rotary._index != self._index:
            raise LFError(LF_ERR_ARG, f"rotary: expected an LFRotary on {self.device}, got {rotary}")
        n = batch if new_start is None else self._sizes(k_new, "k_new", 3)[0]
        self._expect(k_new, "k_new", self.dtype, (n, *self._row))
        self._expect(v_new, "v_new", self.dtype, (n, *self._row))
        if new_start is not None:
            self._expect(new_start, "new_start", torch.int32, (batch + 1,))
        self._numbers(n)
        step = 0 if positions is None else rotary._positions(positions, (n,))
        q_heads = 0
        if q is not None:
            q_heads = self._sizes(q, "q", 3)[1]
            self._expect(q, "q", self.dtype, (n, q_heads, self.head_dim))
            if q_out is not None:
                self._expect(q_out, "q_out", self.dtype, q.shape)
        elif q_out is not None:
            raise LFError(LF_ERR_ARG, "q_out without q")
        _no_gradients(k_new, v_new, q, q_out)
        if q_out is not None:
            _will_change(q_out)
        return self._run(stream, self._append_rotated, pages, batch, width, page_table, lens, k_new, v_new, new_start,
                         n, rotary, *rotary._held, positions, step, q_heads, q, q_out)

    def _append_rotated(self, st, pages, batch, width, page_table, lens, k_new, v_new, new_start, n, rotary, _turns,
                        _axis, positions, step, q_heads, q, q_out):
        if q is not None and q_out is None:
            q_out = torch.empty_like(q)
        _check(self._lib.lf_paged_append_rotated(
            pages, batch, page_table.data_ptr(), width, lens.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
            _ptr(new_start), n, rotary._table, _ptr(positions), step, q_heads, _ptr(q), _ptr(q_out), st))
        return q_out

    def decode(self, layer, q, page_table, lens, k_new=None, v_new=None, window=0, sinks=0, out=None,
               lse=None, stream=None):
        """lf_paged_decode: q [batch][q_heads][head_dim] -> out of that shape.  With k_new and v_new
        [batch][kv_heads][head_dim] the call stores the new token too."""
        pages = self._layer(layer)
        batch, width = self._sequences(page_table, lens)
        q_heads = self._sizes(q, "q", 3)[1]
        self._expect(q, "q", self.dtype, (batch, q_heads, self.head_dim))
        if k_new is not None or v_new is not None:
            self._expect(k_new, "k_new", self.dtype, (batch, *self._row))
            self._expect(v_new, "v_new", self.dtype, (batch, *self._row))
        self._numbers(batch, window, sinks)
        self._outputs(q, out, lse)
        return self._run(stream, self._decode, pages, batch, width, q_heads, page_table, lens, q, k_new,
                         v_new, out, lse, window, sinks)

    def _decode(self, st, pages, batch, width, q_heads, page_table, lens, q, k_new, v_new, out, lse, window,
                sinks):
        key = (batch, width, q_heads, window, sinks)
        need = self._need.get(key)
        if need is None:
            need = self._ask(lf_paged_decode_workspace, pages, key)
        if out is None:
            out = torch.empty_like(q)
        # a workspace of this call's own: calls on other streams and graphs cannot meet in it
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        _check(self._lib.lf_paged_decode(
            pages, batch, page_table.data_ptr(), width, lens.data_ptr(), q_heads, q.data_ptr(), _ptr(k_new),
            _ptr(v_new), out.data_ptr(), _ptr(lse), window, sinks, _ptr(ws), need, st))
        return out

    def decode_shared(self, layer, q, page_table, lens, group_start, prefix_lens, k_new=None, v_new=None, out=None,
                      lse=None, stream=None):
        """lf_paged_decode_shared: ``decode`` for sequences in groups that share prefixes, each read once.  group_start
        int32 [groups + 1]: sequences group_start[i] .. group_start[i + 1] - 1 are group i; prefix_lens int32 [batch]:
        sequence b's first prefix_lens[b] positions are those of its group's first sequence, in the pages that
        one's row of the page table lists, and no member's is longer than that one's."""
        pages = self._layer(layer)
        batch, width = self._sequences(page_table, lens)
        q_heads = self._sizes(q, "q", 3)[1]
        self._expect(q, "q", self.dtype, (batch, q_heads, self.head_dim))
        groups = self._sizes(group_start, "group_start", 1)[0] - 1
        self._expect(group_start, "group_start", torch.int32, (groups + 1,))
        self._expect(prefix_lens, "prefix_lens", torch.int32, (batch,))
        if not 1 <= groups <= batch:
            raise LFError(LF_ERR_ARG, f"group_start: expected 1 to {batch} groups, got {groups}")
        if k_new is not None or v_new is not None:
            self._expect(k_new, "k_new", self.dtype, (batch, *self._row))
            self._expect(v_new, "v_new", self.dtype, (batch, *self._row))
        self._numbers(batch)
        self._outputs(q, out, lse)
        return self._run(stream, self._decode_shared, pages, batch, width, q_heads, page_table, lens, q, group_start,
                         groups, prefix_lens, k_new, v_new, out, lse)

    def _decode_shared(self, st, pages, batch, width, q_heads, page_table, lens, q, group_start, groups, prefix_lens,
                       k_new, v_new, out, lse):
        key = (batch, width, q_heads, groups)
        need = self._need.get(key)
        if need is None:
            need = self._ask(lf_paged_decode_shared_workspace, pages, key)
        if out is None:
            out = torch.empty_like(q)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)   # of this call's own
        _check(self._lib.lf_paged_decode_shared(
            pages, batch, page_table.data_ptr(), width, lens.data_ptr(), q_heads, q.data_ptr(), group_start.data_ptr(),
            groups, prefix_lens.data_ptr(), _ptr(k_new), _ptr(v_new), out.data_ptr(), _ptr(lse), ws.data_ptr(), need, st))
        return out

    def prompt(self, layer, q, page_table, lens, q_start, max_q, window=0, sinks=0, out=None, lse=None,
               stream=None):
        """lf_paged_prompt: q [rows][q_heads][head_dim] -> out of that shape; q_start int32
        [batch + 1], max_q at least every sequence's number of rows (a chunk limit, say: what is
        larger than the call's rows counts as these)."""
        pages = self._layer(layer)
        batch, width = self._sequences(page_table, lens)
        rows, q_heads, _ = self._sizes(q, "q", 3)
        self._expect(q, "q", self.dtype, (rows, q_heads, self.head_dim))
        self._expect(q_start, "q_start", torch.int32, (batch + 1,))
        self._numbers(rows, window, sinks, max_q)
        self._outputs(q, out, lse)
        return self._run(stream, self._prompt, pages, batch, width, q_heads, page_table, lens, q, q_start,
                         rows, min(max_q, rows), out, lse, window, sinks)

    def _prompt(self, st, pages, batch, width, q_heads, page_table, lens, q, q_start, rows, max_q, out, lse,
                window, sinks):
        key = (batch, width, q_heads, rows, max_q, window, sinks)
        need = self._need.get(key)
        if need is None:
            need = self._ask(lf_paged_prompt_workspace, pages, key)
        if out is None:
            out = torch.empty_like(q)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        _check(self._lib.lf_paged_prompt(
            pages, batch, page_table.data_ptr(), width, lens.data_ptr(), q_heads, q.data_ptr(),
            q_start.data_ptr(), rows, max_q, out.data_ptr(), _ptr(lse), window, sinks, _ptr(ws), need, st))
        return out

    def check(self, stream=None) -> int:
        """The device error bits since the last check (0 when clean); synchronises the stream."""
        return self._run(stream, self._take_bits)

    def _take_bits(self, st):
        taken = torch.empty_like(self.err)
        _check(self._lib.lf_paged_take_errors(self._pages[0], taken.data_ptr(), st))
        return int(taken.item())
