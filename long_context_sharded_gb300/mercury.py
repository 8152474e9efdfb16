"""Thin ctypes binding of libmercury_attn.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module
only turns torch tensors into pointers and sizes and status codes into
exceptions.  It loads the in-tree library built by ``build.py`` and raises
immediately if it is missing: there is no CPU fallback.

The functions keep the C names:
  mercury_plan_shift(R, shift)                      -> [R, R] int32 numpy table
  mercury_attn_sharded(q, k, v, R, shift, causal, out=None, lse=None, stream=None)
  mercury_attn_partial(q, k, v, R, shift, causal, o_part=None, lse_part=None, stream=None)
  mercury_lse_merge(o_part, lse_part, out=None, lse=None, stream=None)
  mercury_sync_status(stream=None)
  mercury_plan_schedules(B, Hq, Hkv, Sq, Skv, d, causal, R, shift, budget_bytes, profile)
  mercury_choose_runs(B, Hq, Hkv, Sq, Skv, d, causal, R, shift, n_sms, scratch_cap=-1) -> int
  mercury_attn_run_schedule(q, k, v, causal, plan, out=None, lse=None, stream=None)
  mercury_tune_schedule(q, k, v, R, shift, causal, budget_bytes, top_k, ...)
  mercury_rope_init(rot_dim, base, interleaved, scaling, factor, ...) -> RopePlan
  mercury_rope(x, plan, positions=None, start=0, inverse=False, out=None, stream=None)
  PagedCache(k_cache, v_cache, block_table, k_scale=None, v_scale=None)
  mercury_kv_append(cache, k, v, past_lens, new_lens=None, rope=None, q=None, q_out=None, stream=None)
  mercury_attn_paged(q, cache, seq_lens, new_lens=None, causal=True, out=None, lse=None, stream=None)
  mercury_attn_paged_bf16(...) the same, O in bf16
Tensors: q [B,Hq,Sq,d], k/v [B,Hkv,Skv,d] bf16 CUDA tensors, contiguous.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

from . import build as _build

MERCURY_OK = 0
MERCURY_EINVAL = -1
MERCURY_EALIGN = -2
MERCURY_ECUDA = -3
MERCURY_ETIMEOUT = -4
MERCURY_ENOMEM = -5
MERCURY_EBUDGET = -6
MERCURY_EBOUNDS = -7
MERCURY_MAX_R = 128

_STATUS_NAMES = {
    MERCURY_EINVAL: "EINVAL", MERCURY_EALIGN: "EALIGN", MERCURY_ECUDA: "ECUDA",
    MERCURY_ETIMEOUT: "ETIMEOUT", MERCURY_ENOMEM: "ENOMEM", MERCURY_EBUDGET: "EBUDGET",
    MERCURY_EBOUNDS: "EBOUNDS",
}

# Every symbol include/mercury_attn.h declares.
EXPORTED = ("mercury_plan_shift", "mercury_attn_sharded", "mercury_attn_partial",
            "mercury_lse_merge", "mercury_sync_status", "mercury_last_error",
            "mercury_work_decomposition", "mercury_work_item_rows", "mercury_attn_split_noalloc",
            "mercury_gemm_shifted", "mercury_attn_decode", "mercury_attn_sharded_bf16",
            "mercury_default_cost_profile", "mercury_measure_cost_profile",
            "mercury_plan_schedules", "mercury_attn_run_schedule", "mercury_tune_schedule",
            "mercury_tune_cache_clear", "mercury_choose_runs", "mercury_rope_frequencies",
            "mercury_rope_init", "mercury_rope", "mercury_kv_append", "mercury_attn_paged",
            "mercury_attn_paged_bf16")

MERCURY_MAX_ROT = 256
ELEM_BF16, ELEM_E4M3, ELEM_FP32 = 0, 1, 2
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class CostProfile(ctypes.Structure):
    """mercury_cost_profile: kernel costs of one device (us, GB/s)."""
    _fields_ = [("tile_us", ctypes.c_double), ("tile1_us", ctypes.c_double),
                ("item_us", ctypes.c_double), ("launch_us", ctypes.c_double),
                ("merge_gbs", ctypes.c_double), ("hbm_gbs", ctypes.c_double),
                ("n_sms", ctypes.c_int), ("measured", ctypes.c_int)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class Schedule(ctypes.Structure):
    """mercury_schedule: one candidate schedule (R, Rq, n_runs, shift) and its costs."""
    _fields_ = [("R", ctypes.c_int), ("Rq", ctypes.c_int), ("n_runs", ctypes.c_int),
                ("shift", ctypes.c_int), ("work_items", ctypes.c_longlong),
                ("scratch_bytes", ctypes.c_longlong), ("hbm_bytes", ctypes.c_longlong),
                ("predicted_us", ctypes.c_double), ("measured_us", ctypes.c_double),
                ("pareto", ctypes.c_int)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class RopePlan(ctypes.Structure):
    """mercury_rope_plan: a rotation (plain host data, from mercury_rope_init)."""
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("magnitude", ctypes.c_float),
                ("turns", ctypes.c_ulonglong * (MERCURY_MAX_ROT // 2))]


class PagedCacheStruct(ctypes.Structure):
    """mercury_paged_cache: the device arrays of a paged cache and their sizes."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("page_stride", ctypes.c_longlong), ("table_stride", ctypes.c_longlong),
                ("elem", ctypes.c_int), ("Hkv", ctypes.c_int), ("d", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("B", ctypes.c_int)]


class MercuryError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s (%d): %s" % (_STATUS_NAMES.get(status, "?"), status, message))
        self.status = status


# MERCURY_CHECKED_BUILD=1 loads the bounds-checked variant (build(check=True)).
CHECKED = os.environ.get("MERCURY_CHECKED_BUILD", "") == "1"


def _load() -> ctypes.CDLL:
    path = _build.CHECK_LIB_PATH if CHECKED else _build.LIB_PATH
    if not os.path.exists(path):
        raise ImportError(
            "libmercury_attn.so is not built (%s); run long_context_sharded_gb300.build.build(%s) "
            "or __graft_entry__.build() first" % (path, "check=True" if CHECKED else ""))
    lib = ctypes.CDLL(path)
    i32, i64, p = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p
    attn_args = [p, p, p, i32, i32, i32, i32, i32, i32, i32, i32, i32, p, p, p]
    lib.mercury_plan_shift.argtypes = [i32, i32, p]
    lib.mercury_attn_sharded.argtypes = attn_args
    lib.mercury_attn_sharded_bf16.argtypes = attn_args
    lib.mercury_attn_partial.argtypes = attn_args
    lib.mercury_lse_merge.argtypes = [p, p, i32, i64, i32, p, p, p]
    lib.mercury_gemm_shifted.argtypes = [p, p, i32, i32, i32, i32, i32, p, p]
    lib.mercury_attn_decode.argtypes = [p, p, p, i32, i32, i32, i32, i32, i32, i32, i32, p, p, p]
    lib.mercury_attn_split_noalloc.argtypes = [p, p, p, i32, i32, i32, i32, i32, i32, i32, i32, i32,
                                               i32, p, p, p]
    lib.mercury_sync_status.argtypes = [p]
    lib.mercury_last_error.argtypes = []
    lib.mercury_last_error.restype = ctypes.c_char_p
    lib.mercury_work_decomposition.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, p]
    lib.mercury_work_item_rows.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i32,
                                           i64, p, p, p]
    lib.mercury_default_cost_profile.argtypes = [i32, p]
    lib.mercury_measure_cost_profile.argtypes = [p, p]
    lib.mercury_plan_schedules.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i64, p, p,
                                           i32, p]
    lib.mercury_attn_run_schedule.argtypes = [p, p, p, i32, i32, i32, i32, i32, i32, i32, p, p, p, p]
    lib.mercury_tune_schedule.argtypes = [p, p, p, i32, i32, i32, i32, i32, i32, i32, i32, i32, i64,
                                          i32, p, p, p, p, p]
    lib.mercury_tune_cache_clear.argtypes = []
    lib.mercury_choose_runs.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, i64, p]
    lib.mercury_rope_frequencies.argtypes = [i32, ctypes.c_double, i32, ctypes.c_double, ctypes.c_double,
                                             ctypes.c_double, ctypes.c_double, p, p]
    lib.mercury_rope_init.argtypes = [i32, i32, p, ctypes.c_double, p]
    lib.mercury_rope.argtypes = [p, p, p, i64, i64, i32, i32, i32, i32, i32, p, i32, p, p, p]
    lib.mercury_kv_append.argtypes = [p, p, p, p, i32, i32, p, p, p, p, p, p, i32, p, p, p]
    lib.mercury_attn_paged.argtypes = [p, p, p, p, p, i32, i32, i32, i32, p, p, p]
    lib.mercury_attn_paged_bf16.argtypes = lib.mercury_attn_paged.argtypes
    for name in EXPORTED:
        if name not in ("mercury_last_error", "mercury_tune_cache_clear"):
            getattr(lib, name).restype = i32
    lib.mercury_tune_cache_clear.restype = None
    return lib


lib = _load()


def _load_binding():
    """The C side of the serving calls' marshalling (csrc/binding.c)."""
    import importlib.machinery
    import importlib.util
    path = _build.BINDING_PATH
    if not os.path.exists(path):
        raise ImportError("the binding's extension is not built (%s); run long_context_sharded_gb300.build.build() first" % path)
    loader = importlib.machinery.ExtensionFileLoader("mercury_binding", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("mercury_binding", path, loader=loader))
    loader.exec_module(module)
    return module


_fast = _load_binding()


def _check(rc: int) -> None:
    if rc != MERCURY_OK:
        raise MercuryError(rc, lib.mercury_last_error().decode(errors="replace"))


def _stream_ptr(stream):
    """cudaStream_t of `stream`, or of the current stream of the current
    device.  The raw getter avoids building a torch Stream object, which costs
    more host time than the library's whole launch path on small calls; the
    public call is the fallback where the getter is absent."""
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_DTYPES = {}


def _dtype(name):
    """torch dtype object for "torch.bfloat16" / "torch.float32" (looked up once)."""
    dt = _DTYPES.get(name)
    if dt is None:
        import torch
        dt = _DTYPES[name] = getattr(torch, name.split(".", 1)[1])
    return dt


def _dev_ptr(t, dtype_name, what):
    """Device pointer of a contiguous CUDA tensor of the given dtype on the
    current device (the library runs on the current device, and a pointer
    into another device's memory would be read there).  Small calls are
    bound by this marshalling, so the checks use the cheapest tensor queries."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % what)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if t.dtype is not _dtype(dtype_name):
        raise TypeError("%s must be %s (got %s)" % (what, dtype_name, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    cur = torch.cuda.current_device()
    if t.get_device() != cur:
        raise ValueError("%s is on %s but the current device is cuda:%d" % (what, t.device, cur))
    return t.data_ptr()


def _check_shape(t, shape, what):
    """A caller-provided output must have exactly the shape the call writes:
    the kernels write every element of that shape, so a smaller buffer would
    be overrun."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % what)
    if t.shape != shape:  # torch.Size is a tuple
        raise ValueError("%s must have shape %s (got %s)" % (what, tuple(int(x) for x in shape),
                                                            tuple(t.shape)))


def mercury_plan_shift(R: int, shift: int) -> np.ndarray:
    out = np.zeros((R * R if R > 0 else 1,), dtype=np.int32)
    _check(lib.mercury_plan_shift(R, shift, out.ctypes.data_as(ctypes.c_void_p)))
    return out.reshape(R, R)


def _shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, H, S, d]")
    B, Hq, Sq, d = q.shape
    Bk, Hkv, Skv, dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Bk != B or dk != d:
        raise ValueError("shape mismatch: q %s k %s v %s" % (tuple(q.shape), tuple(k.shape),
                                                             tuple(v.shape)))
    return B, Hq, Hkv, Sq, Skv, d


def mercury_attn_sharded(q, k, v, R: int, shift: int, causal: bool, out=None, lse=None,
                         stream=None):
    """Attention through the shifted schedule; returns (out fp32, lse fp32)."""
    import torch
    B, Hq, Hkv, Sq, Skv, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty((B, Hq, Sq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    _check_shape(out, (B, Hq, Sq, d), "out")
    _check_shape(lse, (B, Hq, Sq), "lse")
    rc = lib.mercury_attn_sharded(
        _dev_ptr(q, "torch.bfloat16", "q"), _dev_ptr(k, "torch.bfloat16", "k"),
        _dev_ptr(v, "torch.bfloat16", "v"), B, Hq, Hkv, Sq, Skv, d, R, shift, int(bool(causal)),
        _dev_ptr(out, "torch.float32", "out"), _dev_ptr(lse, "torch.float32", "lse"),
        _stream_ptr(stream))
    _check(rc)
    return out, lse


def mercury_attn_sharded_bf16(q, k, v, R: int, shift: int, causal: bool, out=None, lse=None,
                              stream=None):
    """As mercury_attn_sharded, with O returned in bf16 (lse fp32)."""
    import torch
    B, Hq, Hkv, Sq, Skv, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty((B, Hq, Sq, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    _check_shape(out, (B, Hq, Sq, d), "out")
    _check_shape(lse, (B, Hq, Sq), "lse")
    rc = lib.mercury_attn_sharded_bf16(
        _dev_ptr(q, "torch.bfloat16", "q"), _dev_ptr(k, "torch.bfloat16", "k"),
        _dev_ptr(v, "torch.bfloat16", "v"), B, Hq, Hkv, Sq, Skv, d, R, shift, int(bool(causal)),
        _dev_ptr(out, "torch.bfloat16", "out"), _dev_ptr(lse, "torch.float32", "lse"),
        _stream_ptr(stream))
    _check(rc)
    return out, lse


def mercury_attn_partial(q, k, v, R: int, shift: int, causal: bool, o_part=None, lse_part=None,
                         stream=None):
    """Per-step partials; returns (o_part [R,B,Hq,Sq,d], lse_part [R,B,Hq,Sq])."""
    import torch
    B, Hq, Hkv, Sq, Skv, d = _shapes(q, k, v)
    if o_part is None:
        o_part = torch.empty((R, B, Hq, Sq, d), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((R, B, Hq, Sq), dtype=torch.float32, device=q.device)
    _check_shape(o_part, (R, B, Hq, Sq, d), "o_part")
    _check_shape(lse_part, (R, B, Hq, Sq), "lse_part")
    rc = lib.mercury_attn_partial(
        _dev_ptr(q, "torch.bfloat16", "q"), _dev_ptr(k, "torch.bfloat16", "k"),
        _dev_ptr(v, "torch.bfloat16", "v"), B, Hq, Hkv, Sq, Skv, d, R, shift, int(bool(causal)),
        _dev_ptr(o_part, "torch.float32", "o_part"), _dev_ptr(lse_part, "torch.float32", "lse_part"),
        _stream_ptr(stream))
    _check(rc)
    return o_part, lse_part


def mercury_lse_merge(o_part, lse_part, out=None, lse=None, stream=None):
    """Merge partials o_part [n, ..., d] / lse_part [n, ...] over the first axis."""
    import torch
    n_parts = o_part.shape[0]
    d = o_part.shape[-1]
    rows = o_part[0].numel() // d if n_parts else 0
    if lse_part.shape[0] != n_parts or lse_part[0].numel() != rows:
        raise ValueError("lse_part does not match o_part")
    if out is None:
        out = torch.empty(tuple(o_part.shape[1:]), dtype=torch.float32, device=o_part.device)
    if lse is None:
        lse = torch.empty(tuple(lse_part.shape[1:]), dtype=torch.float32, device=o_part.device)
    if out.numel() != rows * d or out.shape[-1] != d:
        raise ValueError("out must hold %d rows of %d (got shape %s)" % (rows, d, tuple(out.shape)))
    if lse.numel() != rows:
        raise ValueError("lse must hold %d rows (got shape %s)" % (rows, tuple(lse.shape)))
    rc = lib.mercury_lse_merge(
        _dev_ptr(o_part, "torch.float32", "o_part"), _dev_ptr(lse_part, "torch.float32", "lse_part"),
        n_parts, rows, d, _dev_ptr(out, "torch.float32", "out"),
        _dev_ptr(lse, "torch.float32", "lse"), _stream_ptr(stream))
    _check(rc)
    return out, lse


def mercury_attn_split_noalloc(q, k, v, R: int, shift: int, causal: bool, n_runs: int, out, lse,
                               stream=None):
    """Split-KV attention whose partials live in the library's fixed 64 MiB
    device array: no device memory is allocated (out and lse are the
    caller's).  Calls that may overlap on the GPU must not share a device."""
    B, Hq, Hkv, Sq, Skv, d = _shapes(q, k, v)
    _check_shape(out, (B, Hq, Sq, d), "out")
    _check_shape(lse, (B, Hq, Sq), "lse")
    rc = lib.mercury_attn_split_noalloc(
        _dev_ptr(q, "torch.bfloat16", "q"), _dev_ptr(k, "torch.bfloat16", "k"),
        _dev_ptr(v, "torch.bfloat16", "v"), B, Hq, Hkv, Sq, Skv, d, R, shift, int(bool(causal)),
        int(n_runs), _dev_ptr(out, "torch.float32", "out"), _dev_ptr(lse, "torch.float32", "lse"),
        _stream_ptr(stream))
    _check(rc)
    return out, lse


def mercury_attn_decode(q, k, v, n_splits: int = 0, causal: bool = False, out=None, lse=None, stream=None):
    """Short query side against a long KV, split over the KV and merged."""
    import torch
    B, Hq, Hkv, Sq, Skv, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty((B, Hq, Sq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    _check_shape(out, (B, Hq, Sq, d), "out")
    _check_shape(lse, (B, Hq, Sq), "lse")
    rc = lib.mercury_attn_decode(
        _dev_ptr(q, "torch.bfloat16", "q"), _dev_ptr(k, "torch.bfloat16", "k"),
        _dev_ptr(v, "torch.bfloat16", "v"), B, Hq, Hkv, Sq, Skv, d, int(n_splits), int(bool(causal)),
        _dev_ptr(out, "torch.float32", "out"), _dev_ptr(lse, "torch.float32", "lse"), _stream_ptr(stream))
    _check(rc)
    return out, lse


def mercury_gemm_shifted(a, b, R: int, shift: int, c=None, stream=None):
    """C = A @ B through the shifted schedule: a [M,K], b [K,N] bf16 -> c [M,N] fp32."""
    import torch
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError("a [M,K] and b [K,N] expected")
    M, K = a.shape
    N = b.shape[1]
    if c is None:
        c = torch.empty((M, N), dtype=torch.float32, device=a.device)
    _check_shape(c, (M, N), "c")
    rc = lib.mercury_gemm_shifted(_dev_ptr(a, "torch.bfloat16", "a"), _dev_ptr(b, "torch.bfloat16", "b"),
                                  M, N, K, R, shift, _dev_ptr(c, "torch.float32", "c"), _stream_ptr(stream))
    _check(rc)
    return c


def mercury_sync_status(stream=None) -> None:
    _check(lib.mercury_sync_status(_stream_ptr(stream)))


def mercury_work_decomposition(B, Hq, Hkv, Sq, Skv, d, R, causal, mode):
    """mode: 0 fused, 1 per-step partials, g >= 2 split into g runs of steps."""
    info = (ctypes.c_longlong * 8)()
    _check(lib.mercury_work_decomposition(B, Hq, Hkv, Sq, Skv, d, R, int(bool(causal)),
                                          int(mode), info))
    keys = ("Mq", "Gp", "head_mode", "T_h", "T_r", "items_per_group", "n_items", "slots")
    return {k: int(info[i]) for i, k in enumerate(keys)}


def mercury_work_item_rows(B, Hq, Hkv, Sq, Skv, d, R, shift, causal, mode, item):
    rows = (ctypes.c_longlong * 256)()
    n = ctypes.c_int(0)
    step = ctypes.c_int(0)
    _check(lib.mercury_work_item_rows(B, Hq, Hkv, Sq, Skv, d, R, shift, int(bool(causal)),
                                      int(mode), item, rows, ctypes.byref(n),
                                      ctypes.byref(step)))
    return [rows[i] for i in range(n.value)], step.value


def mercury_default_cost_profile(n_sms: int) -> CostProfile:
    prof = CostProfile()
    _check(lib.mercury_default_cost_profile(int(n_sms), ctypes.byref(prof)))
    return prof


def mercury_measure_cost_profile(stream=None) -> CostProfile:
    """Time the kernels on the current device (allocates ~2 GB, synchronises)."""
    prof = CostProfile()
    _check(lib.mercury_measure_cost_profile(ctypes.byref(prof), _stream_ptr(stream)))
    return prof


def mercury_plan_schedules(B, Hq, Hkv, Sq, Skv, d, causal, R, shift, budget_bytes, profile,
                           max_plans: int = 512):
    """Candidates within the budget, fastest predicted first: (list of Schedule, total count)."""
    plans = (Schedule * max(int(max_plans), 1))()
    n = ctypes.c_int(0)
    _check(lib.mercury_plan_schedules(B, Hq, Hkv, Sq, Skv, d, int(bool(causal)), R, shift,
                                      int(budget_bytes), ctypes.byref(profile), plans,
                                      int(max_plans), ctypes.byref(n)))
    return [plans[i] for i in range(min(n.value, int(max_plans)))], n.value


def mercury_choose_runs(B, Hq, Hkv, Sq, Skv, d, causal, R, shift, n_sms, scratch_cap=-1) -> int:
    """The run count mercury_attn_sharded uses for this shape on n_sms SMs (host only)."""
    n = ctypes.c_int(0)
    _check(lib.mercury_choose_runs(B, Hq, Hkv, Sq, Skv, d, int(bool(causal)), R, shift, int(n_sms),
                                   int(scratch_cap), ctypes.byref(n)))
    return n.value


def _schedule(plan):
    if isinstance(plan, Schedule):
        return plan
    s = Schedule()
    s.R, s.Rq, s.n_runs, s.shift = (int(x) for x in plan)
    s.measured_us = -1.0
    return s


def mercury_attn_run_schedule(q, k, v, causal: bool, plan, out=None, lse=None, stream=None):
    """Attention by the schedule `plan` (a Schedule or an (R, Rq, n_runs, shift) tuple)."""
    import torch
    B, Hq, Hkv, Sq, Skv, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty((B, Hq, Sq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    _check_shape(out, (B, Hq, Sq, d), "out")
    _check_shape(lse, (B, Hq, Sq), "lse")
    plan = _schedule(plan)
    rc = lib.mercury_attn_run_schedule(
        _dev_ptr(q, "torch.bfloat16", "q"), _dev_ptr(k, "torch.bfloat16", "k"),
        _dev_ptr(v, "torch.bfloat16", "v"), B, Hq, Hkv, Sq, Skv, d, int(bool(causal)),
        ctypes.byref(plan), _dev_ptr(out, "torch.float32", "out"),
        _dev_ptr(lse, "torch.float32", "lse"), _stream_ptr(stream))
    _check(rc)
    return out, lse


def mercury_tune_schedule(q, k, v, R: int, shift: int, causal: bool, budget_bytes: int = 0,
                          top_k: int = 4, out=None, lse=None, stream=None):
    """Tune by measurement (cached per process); returns (out, lse, Schedule, cache_hit)."""
    import torch
    B, Hq, Hkv, Sq, Skv, d = _shapes(q, k, v)
    if out is None:
        out = torch.empty((B, Hq, Sq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    _check_shape(out, (B, Hq, Sq, d), "out")
    _check_shape(lse, (B, Hq, Sq), "lse")
    best = Schedule()
    hit = ctypes.c_int(0)
    rc = lib.mercury_tune_schedule(
        _dev_ptr(q, "torch.bfloat16", "q"), _dev_ptr(k, "torch.bfloat16", "k"),
        _dev_ptr(v, "torch.bfloat16", "v"), B, Hq, Hkv, Sq, Skv, d, R, shift, int(bool(causal)),
        int(budget_bytes), int(top_k), _dev_ptr(out, "torch.float32", "out"),
        _dev_ptr(lse, "torch.float32", "lse"), _stream_ptr(stream), ctypes.byref(best),
        ctypes.byref(hit))
    _check(rc)
    return out, lse, best, bool(hit.value)


def mercury_tune_cache_clear() -> None:
    lib.mercury_tune_cache_clear()


_Strides = ctypes.c_longlong * 3


class _Torch:
    """The torch names that the serving calls use, looked up once.  Those calls
    are bound by their marshalling (a decode step's kernels take a few
    microseconds), so a call whose tensors are all as they should be goes
    through the C extension; the Python side allocates outputs, takes a given
    stream, and says what is wrong where something is."""

    def __init__(self):
        import torch
        self.Tensor, self.empty, self.zeros = torch.Tensor, torch.empty, torch.zeros
        self.stream_context, self.external_stream = torch.cuda.stream, torch.cuda.ExternalStream
        self.current_stream = torch.cuda.current_stream
        self.bf16, self.fp32, self.int32 = torch.bfloat16, torch.float32, torch.int32
        self.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.raw_stream = raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_torch_names = None


def _names():
    global _torch_names
    if _torch_names is None:
        T = _Torch()
        _fast.init(T.bf16, T.fp32, T.int32, T.current_device, T.raw_stream,
                   *(ctypes.cast(f, ctypes.c_void_p).value for f in (
                       lib.mercury_rope, lib.mercury_kv_append, lib.mercury_attn_paged, lib.mercury_attn_paged_bf16)))
        _torch_names = T
    return _torch_names


def _refuse(t, dtype, dev, what):
    """Says what is wrong with a tensor that a call cannot take."""
    if not isinstance(t, _names().Tensor):
        raise TypeError("%s must be a torch tensor" % what)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s (got %s)" % (what, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on %s but the call runs on cuda:%d" % (what, t.device, dev))
    raise ValueError("%s must be contiguous" % what)


def _flat(t, dtype, dev, shape, what):
    """Device pointer of a contiguous tensor of this dtype and shape on device `dev`."""
    try:
        ok = t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
    except AttributeError:
        ok = False
    if not ok:
        _refuse(t, dtype, dev, what)
    if t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (what, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _strides(t, dtype, dev, what):
    """Element strides of a 4-D tensor on device `dev` whose heads (last axis)
    are contiguous; None where all of it is."""
    if t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, dtype, dev, what)
    if t.is_contiguous():
        return None
    st = t.stride()
    if st[3] != 1 and t.shape[3] != 1:
        raise ValueError("the heads (last axis) of %s must be contiguous" % what)
    return st


def _shape4(t, what):
    """The shape of a 4-D tensor."""
    try:
        shape = t.shape
        if len(shape) == 4:
            return shape
    except AttributeError:
        pass
    raise ValueError("%s must be a 4-D tensor" % what)


def _on_current(dev, what):
    cur = _torch_names.current_device()
    if cur != dev:
        raise ValueError("%s is on cuda:%d but the current device is cuda:%d" % (what, dev, cur))


def _new_output(make, shape, dtype, like, dev, stream):
    """A call's own output beside `like`, made (and filled, where `make` fills) on the stream
    that the call runs on: on the caller's current stream a fill could land
    behind the kernel's rows, and a reused block still be in use.  The tensor
    stays out of reuse until what the caller's stream does with it is done."""
    T = _torch_names
    if stream is None or _stream_ptr(stream) == T.raw_stream(dev):
        return make(shape, dtype=dtype, device=like.device)
    with T.stream_context(T.external_stream(_stream_ptr(stream), device=like.device)):
        t = make(shape, dtype=dtype, device=like.device)
    t.record_stream(T.current_stream(dev))
    return t


def mercury_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                             original_length: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(radians per position of each pair as a float64 array, magnitude)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s (got %r)" % (sorted(ROPE_SCALINGS), scaling))
    freq = np.zeros(MERCURY_MAX_ROT // 2, dtype=np.float64)
    magnitude = ctypes.c_double(0.0)
    _check(lib.mercury_rope_frequencies(int(rot_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                        float(original_length), float(beta_fast), float(beta_slow),
                                        freq.ctypes.data_as(ctypes.c_void_p), ctypes.byref(magnitude)))
    return freq[:int(rot_dim) // 2].copy(), magnitude.value


def mercury_rope_init(rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                      factor: float = 1.0, original_length: float = 0.0, beta_fast: float = 32.0,
                      beta_slow: float = 1.0, freq=None, magnitude=None) -> RopePlan:
    """A rotation plan: the frequencies of mercury_rope_frequencies, or those
    given as `freq` (rot_dim/2 radians per position); `magnitude` replaces the
    scaling's own."""
    if freq is None:
        freq, own = mercury_rope_frequencies(rot_dim, base, scaling, factor, original_length, beta_fast, beta_slow)
    else:
        freq, own = np.ascontiguousarray(freq, dtype=np.float64), 1.0
        if freq.shape != (int(rot_dim) // 2,):
            raise ValueError("freq must hold rot_dim/2 = %d values (got shape %s)" % (int(rot_dim) // 2, freq.shape))
    plan = RopePlan()
    _check(lib.mercury_rope_init(int(rot_dim), int(bool(interleaved)), freq.ctypes.data_as(ctypes.c_void_p),
                                 float(own if magnitude is None else magnitude), ctypes.byref(plan)))
    return plan


def mercury_rope(x, plan: RopePlan, positions=None, start: int = 0, inverse: bool = False, out=None, stream=None):
    """Rotary positions on every head of x [B,H,S,d] (bf16 or fp32, any strides
    with contiguous heads).  positions: int32 [B,S] or [S]; None: start + s.
    inverse=True applies the transpose, the gradient of the forward call.
    out: a tensor of x's shape and dtype, or x itself; a new one by default."""
    if not isinstance(plan, RopePlan):
        raise TypeError("plan must be a RopePlan (mercury_rope_init)")
    T = _torch_names or _names()
    if out is not None and stream is None:
        rc = _fast.rope(x, ctypes.addressof(plan), positions, start, inverse, out)
        if rc is not None:
            if rc:
                _check(rc)
            return out
    shape = _shape4(x, "x")
    dtype = x.dtype
    if dtype is not T.bf16 and dtype is not T.fp32:
        raise TypeError("x must be torch.bfloat16 or torch.float32 (got %s)" % dtype)
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be a CUDA tensor")
    _on_current(dev, "x")
    B, H, S, d = shape
    sx = _strides(x, dtype, dev, "x")
    if sx is not None:
        sx = _Strides(sx[0], sx[1], sx[2])
    px = x.data_ptr()
    if out is None:
        out = _new_output(T.empty, shape, dtype, x, dev, stream)
        po, so = out.data_ptr(), None
    elif out is x:
        po, so = px, sx
    else:
        if _shape4(out, "out") != shape:
            raise ValueError("out must have shape %s (got %s)" % (tuple(shape), tuple(out.shape)))
        so = _strides(out, dtype, dev, "out")
        if so is not None:
            so = _Strides(so[0], so[1], so[2])
        po = out.data_ptr()
    pp, row = None, 0
    if positions is not None:
        if not isinstance(positions, T.Tensor):
            raise TypeError("positions must be a torch tensor")
        row = S if positions.dim() == 2 else 0
        pp = _flat(positions, T.int32, dev, (B, S) if row else (S,), "positions")
    rc = lib.mercury_rope(px, sx, pp, row, start, B, H, S, d, ELEM_BF16 if dtype is T.bf16 else ELEM_FP32,
                          ctypes.byref(plan), 1 if inverse else 0, po, so,
                          T.raw_stream(dev) if stream is None else _stream_ptr(stream))
    if rc:
        _check(rc)
    return out


class PagedCache:
    """A paged key-value cache over the caller's tensors, checked once.

    k_cache, v_cache: [num_pages, Hkv, page_size, d], bf16 or float8_e4m3fn,
    each page contiguous (pages may lie further apart, as slices of a larger
    allocation do, equally far in both); block_table: int32 [B, max_pages];
    k_scale, v_scale: fp32 [Hkv], for e4m3 only.  The object keeps the tensors
    alive; their contents (the block table's too) may change between calls."""

    def __init__(self, k_cache, v_cache, block_table, k_scale=None, v_scale=None):
        import torch
        for t, what in ((k_cache, "k_cache"), (v_cache, "v_cache"), (block_table, "block_table")):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch tensor" % what)
            if not t.is_cuda:
                raise ValueError("%s must be a CUDA tensor" % what)
            if t.get_device() != torch.cuda.current_device():
                raise ValueError("%s is on %s but the current device is cuda:%d"
                                 % (what, t.device, torch.cuda.current_device()))
        if k_cache.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError("k_cache must be torch.bfloat16 or torch.float8_e4m3fn (got %s)" % k_cache.dtype)
        if v_cache.dtype is not k_cache.dtype:
            raise TypeError("v_cache must be %s like k_cache (got %s)" % (k_cache.dtype, v_cache.dtype))
        if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
            raise ValueError("k_cache and v_cache must both be [num_pages, Hkv, page_size, d] (got %s and %s)"
                             % (tuple(k_cache.shape), tuple(v_cache.shape)))
        n, Hkv, page_size, d = k_cache.shape
        page = Hkv * page_size * d
        for t, what in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            if n and not t[0].is_contiguous():
                raise ValueError("the pages of %s must be contiguous" % what)
        stride = max(k_cache.stride(0), page) if n <= 1 else k_cache.stride(0)
        if n > 1 and (v_cache.stride(0) != stride or stride < page):
            raise ValueError("the pages of k_cache and v_cache must lie equally far apart, without overlap "
                             "(strides %d and %d)" % (k_cache.stride(0), v_cache.stride(0)))
        if block_table.dtype is not torch.int32:
            raise TypeError("block_table must be torch.int32 (got %s)" % block_table.dtype)
        if block_table.dim() != 2 or (block_table.shape[1] > 1 and block_table.stride(1) != 1) or (
                block_table.shape[0] > 1 and block_table.stride(0) < block_table.shape[1]):
            raise ValueError("block_table must be [B, max_pages] with contiguous rows")
        e4m3 = k_cache.dtype is torch.float8_e4m3fn
        scales = []
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if not e4m3 and t is not None:
                raise ValueError("%s is for e4m3 caches only" % what)
            if e4m3:
                if t is None:
                    raise ValueError("an e4m3 cache needs %s" % what)
                _check_shape(t, (Hkv,), what)
                scales.append(_dev_ptr(t, "torch.float32", what))
            else:
                scales.append(None)
        _names()
        self.k_cache, self.v_cache, self.block_table = k_cache, v_cache, block_table
        self.k_scale, self.v_scale = k_scale, v_scale
        self.device_index = k_cache.get_device()
        self.B, self.Hkv, self.d = block_table.shape[0], Hkv, d
        self.struct = PagedCacheStruct(
            k_cache.data_ptr(), v_cache.data_ptr(), scales[0], scales[1], block_table.data_ptr(), stride,
            max(block_table.stride(0), block_table.shape[1]), ELEM_E4M3 if e4m3 else ELEM_BF16, Hkv, d, page_size, n,
            block_table.shape[1], self.B)
        self._ref = ctypes.byref(self.struct)
        self.address = ctypes.addressof(self.struct)


def mercury_kv_append(cache: PagedCache, k, v, past_lens, new_lens=None, rope=None, q=None, q_out=None, stream=None):
    """New keys and values k, v [B,Hkv,S,d] bf16 into the cache at positions
    past_lens[b] + i, keys rotated by `rope` (a RopePlan) on the way; q
    [B,Hq,S,d], where given, is rotated into q_out (q itself is fine; a new
    tensor by default), which is returned."""
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    if rope is not None and not isinstance(rope, RopePlan):
        raise TypeError("rope must be a RopePlan (mercury_rope_init)")
    dev = cache.device_index
    if stream is None and (q is None or q_out is not None):
        rc = _fast.append(cache.address, dev, k, v, past_lens, new_lens, 0 if rope is None else ctypes.addressof(rope), q,
                          q_out)
        if rc is not None:
            if rc:
                _check(rc)
            return q_out
    T = _names()
    _on_current(dev, "the cache")
    shape = _shape4(k, "k")
    B, Hkv, S, d = shape
    if _shape4(v, "v") != shape or B != cache.B or Hkv != cache.Hkv or d != cache.d:
        raise ValueError("k and v must be [B=%d, Hkv=%d, S, d=%d] (got %s and %s)"
                         % (cache.B, cache.Hkv, cache.d, tuple(shape), tuple(v.shape)))
    bf16 = T.bf16
    sk, sv = _strides(k, bf16, dev, "k"), _strides(v, bf16, dev, "v")
    if sk is not None:
        sk = _Strides(sk[0], sk[1], sk[2])
    if sv is not None:
        sv = _Strides(sv[0], sv[1], sv[2])
    plan = None if rope is None else ctypes.byref(rope)
    pq = sq = po = so = None
    Hq = 0
    if q is not None:
        qshape = _shape4(q, "q")
        Bq, Hq, Sq, dq = qshape
        if Bq != B or Sq != S or dq != d:
            raise ValueError("q must be [B=%d, Hq, S=%d, d=%d] (got %s)" % (B, S, d, tuple(qshape)))
        sq = _strides(q, bf16, dev, "q")
        if sq is not None:
            sq = _Strides(sq[0], sq[1], sq[2])
        pq = q.data_ptr()
        if q_out is None:
            # rows behind new_lens are not written: zeros rather than whatever was there
            q_out = _new_output(T.empty if new_lens is None else T.zeros, qshape, bf16, q, dev, stream)
            po = q_out.data_ptr()
        elif q_out is q:
            po, so = pq, sq
        else:
            if _shape4(q_out, "q_out") != qshape:
                raise ValueError("q_out must have shape %s (got %s)" % (tuple(qshape), tuple(q_out.shape)))
            so = _strides(q_out, bf16, dev, "q_out")
            if so is not None:
                so = _Strides(so[0], so[1], so[2])
            po = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = lib.mercury_kv_append(k.data_ptr(), sk, v.data_ptr(), sv, B, S, cache._ref, _flat(past_lens, T.int32, dev, (B,), "past_lens"),
                               None if new_lens is None else _flat(new_lens, T.int32, dev, (B,), "new_lens"), plan,
                               pq, sq, Hq, po, so, T.raw_stream(dev) if stream is None else _stream_ptr(stream))
    if rc:
        _check(rc)
    return q_out


def _attn_paged(fn, out_dtype, q, cache, seq_lens, new_lens, causal, out, lse, stream):
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")
    T = _torch_names
    dev = cache.device_index
    if out is not None and lse is not None and stream is None:
        rc = _fast.attn(out_dtype is T.bf16, q, cache.address, dev, seq_lens, new_lens, causal, out, lse)
        if rc is not None:
            if rc:
                _check(rc)
            return out, lse
    _on_current(dev, "the cache")
    shape = _shape4(q, "q")
    B, Hq, Sq, d = shape
    if B != cache.B or d != cache.d:
        raise ValueError("q must be [B=%d, Hq, Sq, d=%d] (got %s)" % (cache.B, cache.d, tuple(shape)))
    sq = _strides(q, T.bf16, dev, "q")
    if sq is not None:
        sq = _Strides(sq[0], sq[1], sq[2])
    # rows behind new_lens are not written: zeros rather than whatever was there
    make = T.empty if new_lens is None else T.zeros
    if out is None:
        out = _new_output(make, shape, out_dtype, q, dev, stream)
    if lse is None:
        lse = _new_output(make, (B, Hq, Sq), T.fp32, q, dev, stream)
    rc = fn(q.data_ptr(), sq, cache._ref, _flat(seq_lens, T.int32, dev, (B,), "seq_lens"),
            None if new_lens is None else _flat(new_lens, T.int32, dev, (B,), "new_lens"), B, Hq, Sq,
            1 if causal else 0, _flat(out, out_dtype, dev, shape, "out"), _flat(lse, T.fp32, dev, (B, Hq, Sq), "lse"),
            T.raw_stream(dev) if stream is None else _stream_ptr(stream))
    if rc:
        _check(rc)
    return out, lse


def mercury_attn_paged(q, cache: PagedCache, seq_lens, new_lens=None, causal: bool = True, out=None, lse=None,
                       stream=None):
    """Attention of the newest tokens q [B,Hq,Sq,d] bf16 of every sequence over
    the cache's first seq_lens[b] tokens; returns (out fp32, lse fp32), made on
    the call's stream where they are not given (rows behind new_lens[b]: 0)."""
    return _attn_paged(lib.mercury_attn_paged, _names().fp32, q, cache, seq_lens, new_lens, causal, out, lse, stream)


def mercury_attn_paged_bf16(q, cache: PagedCache, seq_lens, new_lens=None, causal: bool = True, out=None, lse=None,
                            stream=None):
    """As mercury_attn_paged, with O returned in bf16 (lse fp32)."""
    return _attn_paged(lib.mercury_attn_paged_bf16, _names().bf16, q, cache, seq_lens, new_lens, causal, out, lse,
                       stream)
