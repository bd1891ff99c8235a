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
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise LFError(LF_ERR_ARG, f"device: expected a CUDA device, got {device}")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
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

    def _run(self, stream, call, *args):
        """call(stream handle, *args) with this cache's device and `stream` current, so that
        what it allocates belongs to that stream.  The allocator is told that a stream which the caller
        names reads the tensors: they may be let go as soon as the call returns."""
        if stream is None and torch.cuda.current_device() == self._index:
            return call(torch._C._cuda_getCurrentRawStream(self._index), *args)
        if isinstance(stream, int):
            # 0, the default stream's handle, would make torch take a stream of its pool
            stream = (torch.cuda.ExternalStream(stream, device=self.device) if stream
                      else torch.cuda.default_stream(self.device))
        if stream is not None and getattr(stream, "device", None) != self.device:
            raise LFError(LF_ERR_ARG, f"stream: expected a stream of {self.device}, got {stream}")
        with torch.cuda.device(self._index), torch.cuda.stream(stream):
            if stream is not None:
                for t in (self.k, self.v, self.err, *args):
                    if isinstance(t, torch.Tensor):
                        t.record_stream(stream)
            return call(torch._C._cuda_getCurrentRawStream(self._index), *args)

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
