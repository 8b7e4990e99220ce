"""ctypes binding of libdsa_decode.so (include/dsa_decode.h).

Argument marshalling only: torch tensors become device pointers, strides and
sizes; every step of the decode runs in the library's CUDA kernels. The calls
beyond the decode (cache, shared prefix, prompt) go through a small C extension
(csrc/marshal.c) that also checks the tensors, loaded with the first of them. The
functions keep the C names. Loading fails loudly when the library or the
extension is missing (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import sysconfig
from typing import Optional

import torch

from . import workloads as W

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libdsa_decode.so")
MARSHAL_PATH = os.path.join(_HERE, "lib", "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))

DSA_OK = 0
STATUS_NAMES = {0: "DSA_OK", -1: "DSA_ERR_INVALID_ARG", -2: "DSA_ERR_UNSUPPORTED",
                -3: "DSA_ERR_ALIGNMENT", -4: "DSA_ERR_WORKSPACE", -5: "DSA_ERR_CUDA",
                -6: "DSA_ERR_TIMEOUT", -7: "DSA_ERR_PLAN", -8: "DSA_ERR_BOUNDS"}
EXPORTED = ("dsa_decode_plan", "dsa_decode_plan_qk", "dsa_decode_run", "dsa_decode_combine", "dsa_decode_selection",
            "dsa_decode_read_status", "dsa_decode_status_string", "dsa_decode_abi_version",
            "dsa_decode_run_noalloc", "dsa_decode_run_v41", "dsa_decode_combine_v41")
EXPORTED_CACHE = ("dsa_cache_write", "dsa_cache_read")
EXPORTED_PREFIX = ("dsa_prefix_plan", "dsa_prefix_run")
EXPORTED_CHUNK = ("dsa_chunk_plan", "dsa_chunk_run")
EXPORTED_WEIGHTS = ("dsa_weights_plan", "dsa_weights_run")
EXPORTED_STEP = ("dsa_qk_norm", "dsa_evict")
DSA_ROPE_NEOX = 0
DSA_ROPE_GPTJ = 1
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


class DsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} -> {STATUS_NAMES.get(status, status)}")
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_stride_bytes", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("format", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "magic", "abi_version", "num_tokens", "num_heads", "swa_width", "extra_width",
        "num_sms", "head_groups", "heads_per_group", "tiles_swa", "tiles_extra",
        "tiles_per_token", "units_per_cta", "ctas_per_group", "split_tokens", "kernel")] + \
        [(n, ctypes.c_int64) for n in (
            "total_units", "ws_sel_offset", "ws_part_lse_offset", "ws_part_sel_offset",
            "ws_part_o_offset", "workspace_bytes", "ws_bounds_offset", "balance_live",
            "ws_stage_offset", "workspace_bytes_mx", "wait_budget_cycles", "d_qk",
            "producer_q", "merge_in_run", "ws_count_offset")] + \
        [("reserved", ctypes.c_int64 * 7)]


class PrefixPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "magic", "abi_version", "num_tokens", "num_heads", "width", "d_qk", "num_sms",
        "pairs", "row_tiles", "key_tiles")] + \
        [(n, ctypes.c_int64) for n in (
            "ws_info_offset", "ws_key_e_offset", "ws_image_offset", "ws_tile_offset",
            "ws_part_lse_offset", "ws_part_o_offset", "workspace_bytes", "wait_budget_cycles")] + \
        [("reserved", ctypes.c_int64 * 4)]


class ChunkPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "magic", "abi_version", "num_tokens", "num_seqs", "num_heads", "width", "d_qk", "num_sms",
        "pairs", "row_tiles", "seq_halves", "reserved0")] + \
        [(n, ctypes.c_int64) for n in (
            "ws_info_offset", "ws_key_e_offset", "ws_image_offset", "ws_row_tile_offset",
            "ws_seq_tile_offset", "ws_begin_offset", "ws_tile_offset", "ws_part_lse_offset",
            "ws_part_o_offset", "workspace_bytes", "wait_budget_cycles")] + \
        [("reserved", ctypes.c_int64 * 4)]


class WeightsPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "magic", "abi_version", "num_tokens", "num_seqs", "num_heads", "width", "d_qk", "num_sms",
        "pairs", "splits", "tiles", "wide_splits")] + \
        [(n, ctypes.c_int64) for n in (
            "ws_item_offset", "ws_image_offset", "ws_row_offset", "ws_part_offset",
            "workspace_bytes", "wait_budget_cycles")] + \
        [("reserved", ctypes.c_int64 * 4)]


_lib = None


class MxOutDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("data_stride_t", ctypes.c_int64), ("data_stride_g", ctypes.c_int64),
                ("scale_stride_t", ctypes.c_int64), ("scale_stride_g", ctypes.c_int64),
                ("scale_stride_w", ctypes.c_int64), ("group_size", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MxOut:
    """MXFP8 output buffers in the o-fused layout: data uint8 [T, H/G, G*512]
    (e4m3 codes), scale int32 [T, H/G, G*4] (ue8m0 bytes, four to a word)."""

    def __init__(self, T: int, H: int, group_size: int, device):
        assert H % group_size == 0
        G = group_size
        self.group_size = G
        self.data = torch.zeros((T, H // G, G * W.HEAD_DIM), dtype=torch.uint8, device=device)
        self.scale = torch.zeros((T, H // G, G * 4), dtype=torch.int32, device=device)

    def desc(self) -> MxOutDesc:
        d, s = self.data, self.scale
        return MxOutDesc(d.data_ptr(), s.data_ptr(), d.stride(0), d.stride(1), s.stride(0),
                         s.stride(1), s.stride(2), self.group_size, 0)

    def scale_bytes(self) -> torch.Tensor:
        """[T, H/G, G*16] uint8 (byte ka of a group's scales, little-endian words)."""
        return self.scale.contiguous().view(torch.uint8)


_marshal = None


def _load_marshal():
    """The marshalling extension of the cache and prefix calls (csrc/marshal.c)."""
    global _marshal
    if _marshal is None:
        if not os.path.exists(MARSHAL_PATH):
            raise RuntimeError(f"{MARSHAL_PATH} is missing: build it with `python -m swa_paged_decode_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_marshal", MARSHAL_PATH)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
        loader.exec_module(m)
        m.setup(torch.uint8, torch.int32, torch.int64, torch.bfloat16, torch.float16, torch.float32,
                _current_device, _raw_stream)
        _marshal = m
    return _marshal


LIB_DEBUG_PATH = os.path.join(_HERE, "lib", "libdsa_decode_debug.so")
_libs = {}


def use_checking_build(on: bool):
    """Route every call of this module through the checking build
    (libdsa_decode_debug.so: bounds checks on every global and tile access,
    reported as DSA_ERR_BOUNDS) or back to the release library."""
    global _lib
    _lib = _load_path(LIB_DEBUG_PATH if on else LIB_PATH)
    return _lib


def load(path: str = LIB_PATH):
    """Load libdsa_decode.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = _load_path(path)
    return _lib


def _load_path(path: str):
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m swa_paged_decode_gb300.build`"
                           " (the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.dsa_decode_plan.restype = ctypes.c_int
    lib.dsa_decode_plan.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(Plan),
                                    ctypes.POINTER(ctypes.c_size_t)]
    lib.dsa_decode_plan_qk.restype = ctypes.c_int
    lib.dsa_decode_plan_qk.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(Plan),
                                       ctypes.POINTER(ctypes.c_size_t)]
    lib.dsa_decode_run.restype = ctypes.c_int
    lib.dsa_decode_run.argtypes = [ctypes.POINTER(Plan), vp, ctypes.c_size_t, vp, i64, i64,
                                   ctypes.POINTER(CacheDesc), vp, i64, vp,
                                   ctypes.POINTER(CacheDesc), vp, i64, vp,
                                   vp, vp, vp, i64, ctypes.c_float, vp, vp, vp]
    lib.dsa_decode_combine.restype = ctypes.c_int
    lib.dsa_decode_combine.argtypes = [ctypes.POINTER(Plan), vp, ctypes.c_size_t, vp, vp, vp, vp]
    lib.dsa_decode_selection.restype = ctypes.c_int
    lib.dsa_decode_selection.argtypes = [ctypes.POINTER(Plan), vp, vp, vp, vp]
    lib.dsa_decode_read_status.restype = ctypes.c_int
    lib.dsa_decode_read_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int32)]
    lib.dsa_decode_run_noalloc.restype = ctypes.c_int
    lib.dsa_decode_run_noalloc.argtypes = [ctypes.POINTER(Plan), vp, i64, i64,
                                           ctypes.POINTER(CacheDesc), vp, i64, vp,
                                           ctypes.POINTER(CacheDesc), vp, i64, vp,
                                           vp, vp, vp, i64, ctypes.c_float, vp, vp, vp, vp]
    lib.dsa_decode_run_v41.restype = ctypes.c_int
    lib.dsa_decode_run_v41.argtypes = [ctypes.POINTER(Plan), vp, ctypes.c_size_t, vp, i64, i64,
                                       ctypes.POINTER(CacheDesc), vp, i64, vp,
                                       ctypes.POINTER(CacheDesc), vp, i64, vp,
                                       vp, vp, vp, i64, i32, ctypes.c_float, vp,
                                       ctypes.POINTER(MxOutDesc), vp, vp]
    lib.dsa_decode_combine_v41.restype = ctypes.c_int
    lib.dsa_decode_combine_v41.argtypes = [ctypes.POINTER(Plan), vp, ctypes.c_size_t, vp, vp, vp,
                                           i64, i32, vp, ctypes.POINTER(MxOutDesc), vp, vp]
    lib.dsa_cache_write.restype = ctypes.c_int
    lib.dsa_cache_write.argtypes = [ctypes.POINTER(CacheDesc), vp, i64, vp, i64, i32, vp,
                                    ctypes.c_float, vp, vp, i64, i32, vp, vp]
    lib.dsa_cache_read.restype = ctypes.c_int
    lib.dsa_cache_read.argtypes = [ctypes.POINTER(CacheDesc), vp, i64, vp, i64, i32, vp]
    lib.dsa_prefix_plan.restype = ctypes.c_int
    lib.dsa_prefix_plan.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(PrefixPlan),
                                    ctypes.POINTER(ctypes.c_size_t)]
    lib.dsa_prefix_run.restype = ctypes.c_int
    lib.dsa_prefix_run.argtypes = [ctypes.POINTER(PrefixPlan), vp, ctypes.c_size_t, vp, i64, i64,
                                   ctypes.POINTER(CacheDesc), vp, vp, vp, vp, vp, i64, i32,
                                   ctypes.c_float, vp, vp, vp, vp, vp]
    lib.dsa_chunk_plan.restype = ctypes.c_int
    lib.dsa_chunk_plan.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(ChunkPlan),
                                   ctypes.POINTER(ctypes.c_size_t)]
    lib.dsa_chunk_run.restype = ctypes.c_int
    lib.dsa_chunk_run.argtypes = [ctypes.POINTER(ChunkPlan), vp, ctypes.c_size_t, vp, i64, i64,
                                  ctypes.POINTER(CacheDesc), vp, i64, vp, vp, i32, vp, vp, vp, i64, i32,
                                  ctypes.c_float, vp, vp, vp, vp, vp]
    lib.dsa_weights_plan.restype = ctypes.c_int
    lib.dsa_weights_plan.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(WeightsPlan),
                                     ctypes.POINTER(ctypes.c_size_t)]
    lib.dsa_weights_run.restype = ctypes.c_int
    lib.dsa_weights_run.argtypes = [ctypes.POINTER(WeightsPlan), vp, ctypes.c_size_t, vp, i64, i64,
                                    ctypes.POINTER(CacheDesc), vp, i64, vp, vp, i32, ctypes.c_float, vp, vp, vp, i64,
                                    vp, i64, vp]
    lib.dsa_qk_norm.restype = ctypes.c_int
    lib.dsa_qk_norm.argtypes = [i32, i32, i32, i32, vp, i64, i64, vp, i64, vp, i64, i64, vp, i64, vp,
                                ctypes.POINTER(CacheDesc), vp, ctypes.c_float, vp, vp, i64, i32, vp, vp]
    lib.dsa_evict.restype = ctypes.c_int
    lib.dsa_evict.argtypes = [i32, i32, vp, i64, vp, vp, i64, i32, i32, i32, vp, i64, vp, i64, vp, vp, i64, vp, vp]
    lib.dsa_decode_status_string.restype = ctypes.c_char_p
    lib.dsa_decode_status_string.argtypes = [ctypes.c_int]
    lib.dsa_decode_abi_version.restype = ctypes.c_int32
    lib.dsa_decode_abi_version.argtypes = []
    lib.marshal = {}   # the calls of the marshalling extension, filled as they are used
    _libs[path] = lib
    return lib


def _check(fn: str, rc: int):
    if rc != DSA_OK:
        raise DsaError(fn, rc)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:   # the current stream of the current device
        return _raw_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def cache_desc(c: Optional[W.PagedCache]) -> Optional[CacheDesc]:
    if c is None:
        return None
    return CacheDesc(c.data.data_ptr(), c.num_pages, c.page_stride, c.page_size, c.fmt)


def dsa_decode_plan(num_tokens: int, num_heads: int, swa_width: int, extra_width: int = 0,
                    num_sms: int = 0):
    """-> (Plan, workspace_bytes)."""
    plan = Plan()
    ws = ctypes.c_size_t(0)
    _check("dsa_decode_plan", load().dsa_decode_plan(num_tokens, num_heads, swa_width,
                                                     extra_width, num_sms, ctypes.byref(plan),
                                                     ctypes.byref(ws)))
    return plan, int(ws.value)


def dsa_decode_plan_qk(num_tokens: int, num_heads: int, swa_width: int, extra_width: int = 0,
                       num_sms: int = 0, d_qk: int = 512):
    """-> (Plan, workspace_bytes) for key / query dims d_qk (512, or 576 for
    V3.2 records)."""
    plan = Plan()
    ws = ctypes.c_size_t(0)
    _check("dsa_decode_plan_qk", load().dsa_decode_plan_qk(num_tokens, num_heads, swa_width,
                                                           extra_width, num_sms, d_qk,
                                                           ctypes.byref(plan), ctypes.byref(ws)))
    return plan, int(ws.value)


def dsa_decode_run(plan: Plan, workspace: Optional[torch.Tensor], q: torch.Tensor,
                   swa_cache: W.PagedCache, swa_idx: torch.Tensor, swa_lens: torch.Tensor,
                   extra_cache: Optional[W.PagedCache], extra_idx: Optional[torch.Tensor],
                   extra_lens: Optional[torch.Tensor], sink: Optional[torch.Tensor],
                   positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
                   scale: float, out: torch.Tensor, lse: torch.Tensor, stream=None,
                   check: bool = True) -> int:
    sc, ec = cache_desc(swa_cache), cache_desc(extra_cache)
    rc = load().dsa_decode_run(
        ctypes.byref(plan), _ptr(workspace), 0 if workspace is None else workspace.numel(),
        q.data_ptr(), q.stride(0), q.stride(1),
        ctypes.byref(sc), swa_idx.data_ptr(), swa_idx.stride(0), swa_lens.data_ptr(),
        None if ec is None else ctypes.byref(ec), _ptr(extra_idx),
        0 if extra_idx is None else extra_idx.stride(0), _ptr(extra_lens),
        _ptr(sink), _ptr(positions), _ptr(cos_sin),
        0 if cos_sin is None else cos_sin.shape[0], float(scale),
        out.data_ptr(), lse.data_ptr(), _stream(stream))
    if check:
        _check("dsa_decode_run", rc)
    return rc


def dsa_decode_combine(plan: Plan, workspace: Optional[torch.Tensor], sink: Optional[torch.Tensor],
                       out: torch.Tensor, lse: torch.Tensor, stream=None, check: bool = True) -> int:
    rc = load().dsa_decode_combine(ctypes.byref(plan), _ptr(workspace),
                                   0 if workspace is None else workspace.numel(), _ptr(sink),
                                   out.data_ptr(), lse.data_ptr(), _stream(stream))
    if check:
        _check("dsa_decode_combine", rc)
    return rc


def dsa_decode_run_v41(plan: Plan, workspace: Optional[torch.Tensor], q: torch.Tensor,
                       swa_cache: W.PagedCache, swa_idx: torch.Tensor, swa_lens: torch.Tensor,
                       extra_cache: Optional[W.PagedCache], extra_idx: Optional[torch.Tensor],
                       extra_lens: Optional[torch.Tensor], sink: Optional[torch.Tensor],
                       positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
                       rope_style: int, scale: float, out: Optional[torch.Tensor],
                       mx: Optional[MxOut], lse: torch.Tensor, stream=None,
                       check: bool = True) -> int:
    sc, ec = cache_desc(swa_cache), cache_desc(extra_cache)
    md = None if mx is None else mx.desc()
    rc = load().dsa_decode_run_v41(
        ctypes.byref(plan), _ptr(workspace), 0 if workspace is None else workspace.numel(),
        q.data_ptr(), q.stride(0), q.stride(1),
        ctypes.byref(sc), swa_idx.data_ptr(), swa_idx.stride(0), swa_lens.data_ptr(),
        None if ec is None else ctypes.byref(ec), _ptr(extra_idx),
        0 if extra_idx is None else extra_idx.stride(0), _ptr(extra_lens),
        _ptr(sink), _ptr(positions), _ptr(cos_sin),
        0 if cos_sin is None else cos_sin.shape[0], int(rope_style), float(scale),
        _ptr(out), None if md is None else ctypes.byref(md), lse.data_ptr(), _stream(stream))
    if check:
        _check("dsa_decode_run_v41", rc)
    return rc


def dsa_decode_combine_v41(plan: Plan, workspace: Optional[torch.Tensor],
                           sink: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                           cos_sin: Optional[torch.Tensor], rope_style: int,
                           out: Optional[torch.Tensor], mx: Optional[MxOut], lse: torch.Tensor,
                           stream=None, check: bool = True) -> int:
    md = None if mx is None else mx.desc()
    rc = load().dsa_decode_combine_v41(
        ctypes.byref(plan), _ptr(workspace), 0 if workspace is None else workspace.numel(),
        _ptr(sink), _ptr(positions), _ptr(cos_sin), 0 if cos_sin is None else cos_sin.shape[0],
        int(rope_style), _ptr(out), None if md is None else ctypes.byref(md), lse.data_ptr(),
        _stream(stream))
    if check:
        _check("dsa_decode_combine_v41", rc)
    return rc


def dsa_decode_selection(plan: Plan, workspace: torch.Tensor, kept: torch.Tensor,
                         checksum: torch.Tensor, stream=None):
    _check("dsa_decode_selection", load().dsa_decode_selection(
        ctypes.byref(plan), workspace.data_ptr(), kept.data_ptr(), checksum.data_ptr(),
        _stream(stream)))


def dsa_decode_read_status(workspace: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check("dsa_decode_read_status", load().dsa_decode_read_status(
        workspace.data_ptr(), _stream(stream), ctypes.byref(v)))
    return int(v.value)


def dsa_decode_run_noalloc(plan: Plan, q: torch.Tensor, swa_cache: W.PagedCache,
                           swa_idx: torch.Tensor, swa_lens: torch.Tensor,
                           extra_cache: Optional[W.PagedCache], extra_idx: Optional[torch.Tensor],
                           extra_lens: Optional[torch.Tensor], sink: Optional[torch.Tensor],
                           positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
                           scale: float, out: torch.Tensor, lse: torch.Tensor,
                           device_status: Optional[torch.Tensor] = None, stream=None,
                           check: bool = True) -> int:
    """run + combine on the library's own device scratch (no workspace)."""
    sc, ec = cache_desc(swa_cache), cache_desc(extra_cache)
    rc = load().dsa_decode_run_noalloc(
        ctypes.byref(plan), q.data_ptr(), q.stride(0), q.stride(1),
        ctypes.byref(sc), swa_idx.data_ptr(), swa_idx.stride(0), swa_lens.data_ptr(),
        None if ec is None else ctypes.byref(ec), _ptr(extra_idx),
        0 if extra_idx is None else extra_idx.stride(0), _ptr(extra_lens),
        _ptr(sink), _ptr(positions), _ptr(cos_sin),
        0 if cos_sin is None else cos_sin.shape[0], float(scale),
        out.data_ptr(), lse.data_ptr(), _ptr(device_status), _stream(stream))
    if check:
        _check("dsa_decode_run_noalloc", rc)
    return rc


def _marshalled(fn: str, check: bool, *args) -> int:
    """Call ``fn`` through the marshalling extension. A tensor of another
    device than the current one, dtype, shape or layout than the call takes
    raises DSA_ERR_INVALID_ARG before the library is called."""
    lib = load()
    entry = lib.marshal.get(fn)
    if entry is None:
        entry = lib.marshal[fn] = (getattr(_load_marshal(), fn[4:]), ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value)
    rc = entry[0](entry[1], *args)
    if rc == -1000:                      # BAD_TENSOR
        raise DsaError(fn, -1)
    if check and rc != DSA_OK:
        raise DsaError(fn, rc)
    return rc


def dsa_cache_write(cache: W.PagedCache, slots: torch.Tensor, rows: torch.Tensor,
                    norm_weight: Optional[torch.Tensor] = None, norm_eps: float = 0.0,
                    positions: Optional[torch.Tensor] = None,
                    cos_sin: Optional[torch.Tensor] = None, rope_style: int = DSA_ROPE_NEOX,
                    device_status: Optional[torch.Tensor] = None, stream=None,
                    check: bool = True) -> int:
    """Quantize rows [n, 512] (576 for V3.2 records; bf16, f16 or fp32, any
    row stride) into the records of ``slots`` [n] int32 (-1: not written),
    after an optional RMS norm (weight fp32 [512]) and RoPE of their last 64
    dims (positions int64 [n], cos_sin fp32 [rows, 64])."""
    return _marshalled("dsa_cache_write", check, cache.data, cache.page_size, cache.fmt, slots, rows,
                       norm_weight, norm_eps, positions, cos_sin, rope_style, device_status,
                       None if stream is None else _stream(stream))


def dsa_cache_read(cache: W.PagedCache, slots: torch.Tensor, rows: torch.Tensor, stream=None,
                   check: bool = True) -> int:
    """Fill rows [n, 512] (576 for V3.2 records; bf16, f16 or fp32, any row
    stride) with the values of the records of ``slots`` [n] int32; a slot
    outside the cache gives zeros."""
    return _marshalled("dsa_cache_read", check, cache.data, cache.page_size, cache.fmt, slots, rows,
                       None if stream is None else _stream(stream))


def dsa_prefix_plan(num_tokens: int, num_heads: int, width: int, num_sms: int = 0,
                    d_qk: int = 512):
    """-> (PrefixPlan, workspace_bytes)."""
    plan = PrefixPlan()
    ws = ctypes.c_size_t(0)
    _check("dsa_prefix_plan", load().dsa_prefix_plan(num_tokens, num_heads, width, num_sms, d_qk,
                                                     ctypes.byref(plan), ctypes.byref(ws)))
    return plan, int(ws.value)


def dsa_prefix_run(plan: PrefixPlan, workspace: torch.Tensor, q: torch.Tensor, cache: W.PagedCache,
                   slots: torch.Tensor, length: torch.Tensor, sink: Optional[torch.Tensor],
                   positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
                   rope_style: int, scale: float, tail_out: Optional[torch.Tensor],
                   tail_lse: Optional[torch.Tensor], out: torch.Tensor, lse: torch.Tensor,
                   stream=None, check: bool = True) -> int:
    """Attention of every token over the shared list ``slots`` [width] int32
    of ``length`` [1] int32 (on the device), merged with the tail state."""
    return _marshalled("dsa_prefix_run", check, ctypes.addressof(plan), workspace, q, cache.data,
                       cache.page_size, cache.fmt, slots, length, sink, positions, cos_sin, rope_style,
                       scale, tail_out, tail_lse, out, lse, None if stream is None else _stream(stream))


class PrefixAttention:
    """Plan + workspace for T tokens of H heads behind one shared list of up
    to ``width`` records; ``__call__`` runs on the current stream and returns
    (``self.out``, ``self.lse``). Behind each token's own list: a ``Decoder``
    of a workload without a sink gives ``tail_out`` and ``tail_lse``, and the
    sink goes here."""

    def __init__(self, T: int, H: int, width: int, device, d_qk: int = 512, num_sms: int = 0):
        self.plan, nbytes = dsa_prefix_plan(T, H, width, num_sms, d_qk)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        self.out = torch.empty((T, H, W.HEAD_DIM), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((T, H), dtype=torch.float32, device=device)

    def __call__(self, q: torch.Tensor, cache: W.PagedCache, slots: torch.Tensor,
                 length: torch.Tensor, scale: float, sink: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
                 rope_style: int = DSA_ROPE_NEOX, tail_out: Optional[torch.Tensor] = None,
                 tail_lse: Optional[torch.Tensor] = None, stream=None):
        dsa_prefix_run(self.plan, self.workspace, q, cache, slots, length, sink, positions, cos_sin,
                       rope_style, scale, tail_out, tail_lse, self.out, self.lse, stream)
        return self.out, self.lse


def dsa_chunk_plan(num_tokens: int, num_seqs: int, num_heads: int, width: int, num_sms: int = 0,
                   d_qk: int = 512):
    """-> (ChunkPlan, workspace_bytes)."""
    plan = ChunkPlan()
    ws = ctypes.c_size_t(0)
    _check("dsa_chunk_plan", load().dsa_chunk_plan(num_tokens, num_seqs, num_heads, width, num_sms, d_qk,
                                                   ctypes.byref(plan), ctypes.byref(ws)))
    return plan, int(ws.value)


def dsa_chunk_run(plan: ChunkPlan, workspace: torch.Tensor, q: torch.Tensor, cache: W.PagedCache,
                  slots: torch.Tensor, lengths: torch.Tensor, starts: torch.Tensor, window: int,
                  sink: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                  cos_sin: Optional[torch.Tensor], rope_style: int, scale: float,
                  tail_out: Optional[torch.Tensor], tail_lse: Optional[torch.Tensor],
                  out: torch.Tensor, lse: torch.Tensor, stream=None, check: bool = True) -> int:
    """Causal attention of the new tokens of every sequence b (``starts``
    [B + 1] int32) over its list ``slots[b]`` [B, width] int32 of
    ``lengths[b]`` records, the new tokens' own last; ``window`` > 0: over the
    last that many of them."""
    return _marshalled("dsa_chunk_run", check, ctypes.addressof(plan), workspace, q, cache.data,
                       cache.page_size, cache.fmt, slots, lengths, starts, window, sink, positions,
                       cos_sin, rope_style, scale, tail_out, tail_lse, out, lse,
                       None if stream is None else _stream(stream))


class ChunkAttention:
    """Plan + workspace for up to T new tokens of ``num_seqs`` sequences whose
    lists have up to ``width`` records; ``__call__`` runs on the current stream
    and returns (``self.out``, ``self.lse``). ``q`` has T tokens; those outside
    every sequence are left as they were."""

    def __init__(self, T: int, num_seqs: int, H: int, width: int, device, d_qk: int = 512, num_sms: int = 0):
        self.plan, nbytes = dsa_chunk_plan(T, num_seqs, H, width, num_sms, d_qk)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        self.out = torch.empty((T, H, W.HEAD_DIM), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((T, H), dtype=torch.float32, device=device)

    def __call__(self, q: torch.Tensor, cache: W.PagedCache, slots: torch.Tensor, lengths: torch.Tensor,
                 starts: torch.Tensor, scale: float, window: int = 0, sink: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, cos_sin: Optional[torch.Tensor] = None,
                 rope_style: int = DSA_ROPE_NEOX, tail_out: Optional[torch.Tensor] = None,
                 tail_lse: Optional[torch.Tensor] = None, stream=None):
        dsa_chunk_run(self.plan, self.workspace, q, cache, slots, lengths, starts, window, sink, positions,
                      cos_sin, rope_style, scale, tail_out, tail_lse, self.out, self.lse, stream)
        return self.out, self.lse


def dsa_qk_norm(q: torch.Tensor, out: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                keys: Optional[torch.Tensor] = None, key_weight: Optional[torch.Tensor] = None,
                cache: Optional[W.PagedCache] = None, slots: Optional[torch.Tensor] = None,
                eps: float = 0.0, positions: Optional[torch.Tensor] = None,
                cos_sin: Optional[torch.Tensor] = None, rope_style: int = DSA_ROPE_NEOX,
                device_status: Optional[torch.Tensor] = None, stream=None, check: bool = True) -> int:
    """Queries [T, H, 512] (576 for V3.2; bf16, f16 or fp32, any token and head
    strides) normed per head (weight fp32 [512], or [H, 512]) and rotated into
    ``out`` bf16 (which may be ``q``), and with ``cache`` the tokens' keys [T,
    512] of the same type into the records of ``slots`` [T] int32, as
    ``dsa_cache_write`` does."""
    data, page, fmt = (None, 0, 0) if cache is None else (cache.data, cache.page_size, cache.fmt)
    return _marshalled("dsa_qk_norm", check, q, out, q_weight, keys, key_weight, data, page, fmt, slots, eps,
                       positions, cos_sin, rope_style, device_status, None if stream is None else _stream(stream))


def dsa_weights_plan(num_tokens: int, num_seqs: int, num_heads: int, width: int, num_sms: int = 0,
                     d_qk: int = 512):
    """-> (WeightsPlan, workspace_bytes)."""
    plan = WeightsPlan()
    ws = ctypes.c_size_t(0)
    _check("dsa_weights_plan", load().dsa_weights_plan(num_tokens, num_seqs, num_heads, width, num_sms, d_qk,
                                                       ctypes.byref(plan), ctypes.byref(ws)))
    return plan, int(ws.value)


def dsa_weights_run(plan: WeightsPlan, workspace: torch.Tensor, q: torch.Tensor, cache: W.PagedCache,
                    slots: torch.Tensor, lengths: torch.Tensor, starts: torch.Tensor, window: int, scale: float,
                    sink: Optional[torch.Tensor], lse: torch.Tensor, scores_in: Optional[torch.Tensor],
                    scores_out: torch.Tensor, stream=None, check: bool = True) -> int:
    """``scores_out`` [B, width] fp32 = ``scores_in`` + the attention weight
    that every entry of the lists received from the new tokens and all heads;
    ``q`` rotated already, ``lse`` [T, H] as their attention left it."""
    return _marshalled("dsa_weights_run", check, ctypes.addressof(plan), workspace, q, cache.data,
                       cache.page_size, cache.fmt, slots, lengths, starts, window, scale, sink, lse, scores_in,
                       scores_out, None if stream is None else _stream(stream))


class AttentionWeights:
    """Plan + workspace for the weights that records receive from up to T new
    tokens of ``num_seqs`` sequences whose lists have up to ``width`` records;
    ``__call__`` runs on the current stream and returns ``scores_out`` (which may be
    ``scores_in``)."""

    def __init__(self, T: int, num_seqs: int, H: int, width: int, device, d_qk: int = 512, num_sms: int = 0):
        self.plan, nbytes = dsa_weights_plan(T, num_seqs, H, width, num_sms, d_qk)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)

    def __call__(self, q: torch.Tensor, cache: W.PagedCache, slots: torch.Tensor, lengths: torch.Tensor,
                 starts: torch.Tensor, lse: torch.Tensor, scores_in: Optional[torch.Tensor],
                 scores_out: torch.Tensor, scale: float, window: int = 0, sink: Optional[torch.Tensor] = None,
                 stream=None):
        dsa_weights_run(self.plan, self.workspace, q, cache, slots, lengths, starts, window, scale, sink, lse,
                        scores_in, scores_out, stream)
        return scores_out


def dsa_evict(slots: torch.Tensor, lengths: torch.Tensor, scores: torch.Tensor, budget: int,
              kept_slots: torch.Tensor, kept_scores: torch.Tensor, kept_lengths: torch.Tensor,
              freed: Optional[torch.Tensor] = None, freed_counts: Optional[torch.Tensor] = None,
              keep_first: int = 0, keep_last: int = 0, stream=None, check: bool = True) -> int:
    """Lists ``slots`` [B, width] int32 of ``lengths`` [B] entries cut to
    ``budget`` each: the first ``keep_first``, the last ``keep_last`` and of the
    rest those with the largest ``scores`` [B, width] fp32, in order, into
    ``kept_slots`` and ``kept_scores`` [B, >= budget]; the others' slots into
    ``freed`` [B, >= width - budget]."""
    return _marshalled("dsa_evict", check, slots, lengths, scores, budget, keep_first, keep_last, kept_slots,
                       kept_scores, kept_lengths, freed, freed_counts, None if stream is None else _stream(stream))


class Decoder:
    """Plan + workspace for one workload shape; ``__call__`` runs run+combine
    on the current stream. Allocation uses torch; compute is the library's.
    With ``mx_group`` the output is MXFP8 (``self.mx``, o-fused with that many
    heads per group) instead of bf16 ``self.out``; a GPT-J workload or an
    MXFP8 output goes through the V4.1 entry points."""

    def __init__(self, w: W.Workload, num_sms: int = 0, mx_group: Optional[int] = None):
        self.plan, nbytes = dsa_decode_plan_qk(w.T, w.H, w.swa.width,
                                               0 if w.extra is None else w.extra.width, num_sms,
                                               int(w.q.shape[-1]))
        dev = w.q.device
        if mx_group is not None:
            nbytes = self.plan.workspace_bytes_mx
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        self.mx = None if mx_group is None else MxOut(w.T, w.H, mx_group, dev)
        self.out = (torch.empty((w.T, w.H, W.HEAD_DIM), dtype=torch.bfloat16, device=dev)
                    if self.mx is None else None)
        self.lse = torch.empty((w.T, w.H), dtype=torch.float32, device=dev)

    def __call__(self, w: W.Workload, stream=None):
        ei = None if w.extra is None else w.extra.ids
        el = None if w.extra is None else w.extra.lens
        if self.mx is None and w.rope_style == DSA_ROPE_NEOX:
            dsa_decode_run(self.plan, self.workspace, w.q, w.swa_cache, w.swa.ids, w.swa.lens,
                           w.extra_cache, ei, el, w.sink, w.positions, w.cos_sin, w.scale,
                           self.out, self.lse, stream)
            dsa_decode_combine(self.plan, self.workspace, w.sink, self.out, self.lse, stream)
            return self.out, self.lse
        dsa_decode_run_v41(self.plan, self.workspace, w.q, w.swa_cache, w.swa.ids, w.swa.lens,
                           w.extra_cache, ei, el, w.sink, w.positions, w.cos_sin, w.rope_style,
                           w.scale, self.out, self.mx, self.lse, stream)
        dsa_decode_combine_v41(self.plan, self.workspace, w.sink, w.positions, w.cos_sin,
                               w.rope_style, self.out, self.mx, self.lse, stream)
        return (self.out if self.mx is None else self.mx), self.lse

    def selection(self, stream=None):
        dev = self.lse.device
        kept = torch.empty(self.plan.num_tokens, dtype=torch.int32, device=dev)
        chk = torch.empty(self.plan.num_tokens, dtype=torch.int32, device=dev)
        dsa_decode_selection(self.plan, self.workspace, kept, chk, stream)
        return kept, chk
