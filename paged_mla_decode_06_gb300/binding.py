"""Thin ctypes binding over the C ABI of ``include/mla_decode.h``.

Argument marshalling only: tensors become raw device pointers, the current
PyTorch stream becomes the ``cudaStream_t``, and a non-OK status raises
``MLAError``. Every step of the decode runs in the library's kernels; there
is no fallback. Names match the C entry points.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

MLA_OK = 0
MLA_ERR_INVALID_ARG = 1
MLA_ERR_UNSUPPORTED = 2
MLA_ERR_WORKSPACE = 3
MLA_ERR_CUDA = 4
MLA_ERR_DEVICE_STATUS = 5

MLA_DTYPE_BF16 = 0
MLA_DTYPE_FP8_E4M3 = 1

MLA_KERNEL_AUTO = 0
MLA_KERNEL_WARP_MMA = 1
MLA_KERNEL_TCGEN05 = 2
MLA_KERNEL_TCGEN05_ROWS_N = 3

MLA_ROPE_INTERLEAVED = 0
MLA_ROPE_HALF = 1
MLA_ROPE_SCALING_NONE = 0
MLA_ROPE_SCALING_LINEAR = 1
MLA_ROPE_SCALING_YARN = 2

HEAD_DIM = 576
KV_LORA_RANK = 512


class MLAError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        name = _status_name(status)
        msg = f"{fn} failed: {name}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "num_reqs", "num_heads", "head_dim", "kv_lora_rank", "block_size",
        "max_blocks_per_req", "num_blocks", "max_seq_len", "max_qlen", "topk", "q_dtype",
        "kv_dtype", "has_sinks", "num_segments", "num_sms", "kernel")]


class Plan(ctypes.Structure):
    _fields_ = [("prob", Problem)] + [(n, ctypes.c_int32) for n in (
        "num_segments", "tile_size", "kernel", "rows_per_cta", "row_tiles", "grid_x", "grid_y",
        "grid_z", "num_sms", "schedule", "max_items", "split_items", "wait_limit_us", "tile_rows")] + [
        ("workspace_bytes", ctypes.c_size_t), ("status_offset", ctypes.c_size_t),
        ("segm_output_offset", ctypes.c_size_t), ("segm_max_offset", ctypes.c_size_t),
        ("segm_expsum_offset", ctypes.c_size_t)]


class SharedPlan(ctypes.Structure):
    _fields_ = [("plan", Plan)] + [(n, ctypes.c_int32) for n in (
        "num_groups", "workers", "max_items", "unit_tiles", "prefix_tiles", "partial_rows")] + [
        ("workspace_bytes", ctypes.c_size_t)]


class RopeProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dim", "layout", "scaling", "original_max_position")] + [
        (n, ctypes.c_double) for n in ("base", "factor", "beta_fast", "beta_slow", "mscale", "mscale_all_dim")]


class Rope(ctypes.Structure):
    _fields_ = [("prob", RopeProblem), ("mscale", ctypes.c_float), ("turns", ctypes.c_double * 32)]


_lib = None
_lock = threading.Lock()
_vp = ctypes.c_void_p


def library_path() -> str:
    return _build.LIB_PATH


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load the compiled library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _build.LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"CUDA library not found at {p}; build it with "
                "`python -m paged_mla_decode_06_gb300.build`")
        lib = ctypes.CDLL(p)
        st = ctypes.c_int32
        lib.mla_decode_plan.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(Plan)]
        lib.mla_decode_plan.restype = st
        common = [ctypes.POINTER(Plan), _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, _vp, _vp,
                  ctypes.c_float, ctypes.c_float, ctypes.c_float]
        lib.mla_decode_fwd.argtypes = common + [_vp, _vp, ctypes.c_size_t, _vp, _vp, _vp]
        lib.mla_decode_fwd.restype = st
        lib.mla_decode_fwd_static.argtypes = common + [_vp, _vp, _vp, _vp, _vp]
        lib.mla_decode_fwd_static.restype = st
        lib.mla_decode_segments.argtypes = common + [_vp, _vp, _vp, _vp]
        lib.mla_decode_segments.restype = st
        lib.mla_decode_schedule.argtypes = [ctypes.POINTER(Plan), _vp, _vp, _vp, _vp,
                                            ctypes.c_size_t, _vp]
        lib.mla_decode_schedule.restype = st
        lib.mla_decode_items.argtypes = common + [_vp, _vp, ctypes.c_size_t, _vp, _vp, _vp]
        lib.mla_decode_items.restype = st
        lib.mla_merge_items.argtypes = [ctypes.POINTER(Plan), _vp, _vp, _vp, ctypes.c_size_t,
                                        _vp, _vp, _vp]
        lib.mla_merge_items.restype = st

        lib.mla_merge_segments.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _vp,
                                           ctypes.c_int32, _vp, _vp, _vp]
        lib.mla_merge_segments.restype = st
        lib.mla_sparse_index_convert.argtypes = [_vp, _vp, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_int64, _vp, ctypes.c_int64,
                                                 ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 _vp, _vp, _vp]
        lib.mla_sparse_index_convert.restype = st
        lib.mla_sparse_seqlen.argtypes = [_vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                          _vp, _vp, _vp]
        lib.mla_sparse_seqlen.restype = st
        lib.mla_fit_kpool_indices.argtypes = [_vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                              ctypes.c_int32, _vp, ctypes.c_int64, _vp]
        lib.mla_fit_kpool_indices.restype = st
        lib.mla_merge_lse.argtypes = [_vp, _vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_int32, _vp, _vp, _vp, _vp]
        lib.mla_merge_lse.restype = st
        lib.mla_concat_quant_q.argtypes = [_vp, ctypes.c_int64, ctypes.c_int64, _vp,
                                           ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_float, _vp,
                                           _vp]
        lib.mla_concat_quant_q.restype = st
        i32, i64, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        scaled = [ctypes.POINTER(Plan), _vp, _vp, _vp, i32, _vp, i64, _vp, _vp, _vp, _vp, f32, f32,
                  _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp]
        lib.mla_decode_fwd_scaled.argtypes = scaled
        lib.mla_decode_fwd_scaled.restype = st
        lib.mla_decode_items_scaled.argtypes = scaled
        lib.mla_decode_items_scaled.restype = st
        lib.mla_decode_schedule_scaled.argtypes = lib.mla_decode_schedule.argtypes
        lib.mla_decode_schedule_scaled.restype = st
        lib.mla_decode_scaled_kernel.argtypes = [ctypes.POINTER(Plan), ctypes.POINTER(i32)]
        lib.mla_decode_scaled_kernel.restype = st
        lib.mla_block_tables.argtypes = [_vp, _vp, i32, i32, i32, _vp, i32, _vp, i64, i32, _vp, _vp,
                                         _vp, _vp, _vp]
        lib.mla_block_tables.restype = st
        lib.mla_cache_append.argtypes = [_vp, i64, _vp, i64, _vp, i32, i32, i32, i32, _vp, _vp, _vp]
        lib.mla_cache_append.restype = st
        lib.mla_decode_shared_plan.argtypes = [ctypes.POINTER(Problem), i32, ctypes.POINTER(SharedPlan)]
        lib.mla_decode_shared_plan.restype = st
        lib.mla_decode_fwd_shared.argtypes = [ctypes.POINTER(SharedPlan), _vp, _vp, _vp, i32, _vp, i64, _vp, _vp, _vp,
                                              _vp, f32, f32, f32, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp]
        lib.mla_decode_fwd_shared.restype = st
        lib.mla_rope_plan.argtypes = [ctypes.POINTER(RopeProblem), ctypes.POINTER(Rope)]
        lib.mla_rope_plan.restype = st
        lib.mla_rope_qk.argtypes = [ctypes.POINTER(Rope), _vp, i32, i32, _vp, i64, i64, _vp, i64, i64, i32, f32,
                                    _vp, _vp, i64, _vp, i64, _vp]
        lib.mla_rope_qk.restype = st
        lib.mla_cache_fork.argtypes = [_vp, _vp, _vp, i32, _vp, i32, _vp, i64, i32, i32, _vp, i32, i32, i32, i32,
                                       _vp, _vp, _vp, _vp]
        lib.mla_cache_fork.restype = st
        lib.mla_cache_copy_blocks.argtypes = [_vp, _vp, i32, i32, i32, i32, i32, _vp, _vp, _vp]
        lib.mla_cache_copy_blocks.restype = st
        lib.mla_cache_workspace.argtypes = [i32]
        lib.mla_cache_workspace.restype = ctypes.c_size_t
        lib.mla_cache_free.argtypes = [_vp, _vp, i32, _vp, i64, i32, i32, _vp, i32, i32, _vp, i32, _vp, _vp,
                                       ctypes.c_size_t, _vp]
        lib.mla_cache_free.restype = st
        lib.mla_cache_compact.argtypes = [_vp, _vp, _vp, i64, _vp, i64, i32, i32, i32, i32, i32, i32, _vp, _vp, _vp,
                                          _vp, ctypes.c_size_t, _vp]
        lib.mla_cache_compact.restype = st
        lib.mla_workspace_status.argtypes = [ctypes.POINTER(Plan), _vp, ctypes.POINTER(ctypes.c_int32),
                                             ctypes.c_int32, _vp]
        lib.mla_workspace_status.restype = st
        lib.mla_status_string.argtypes = [ctypes.c_int32]
        lib.mla_status_string.restype = ctypes.c_char_p
        lib.mla_last_cuda_error.argtypes = []
        lib.mla_last_cuda_error.restype = ctypes.c_char_p
        lib.mla_version.argtypes = []
        lib.mla_version.restype = ctypes.c_int32
        _lib = lib
        return lib


def _status_name(status: int) -> str:
    names = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
             3: "MLA_ERR_WORKSPACE", 4: "MLA_ERR_CUDA", 5: "MLA_ERR_DEVICE_STATUS"}
    return names.get(int(status), f"status {status}")


def _check(fn: str, status: int):
    if status != MLA_OK:
        detail = ""
        if status == MLA_ERR_CUDA and _lib is not None:
            detail = _lib.mla_last_cuda_error().decode()
        raise MLAError(fn, status, detail)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(name: str) -> int:
    return {"bf16": MLA_DTYPE_BF16, "fp8": MLA_DTYPE_FP8_E4M3}[name]


def make_problem(*, num_tokens: int, num_heads: int, block_size: int, num_blocks: int,
                 num_reqs: int = 0, max_blocks_per_req: int = 0, max_seq_len: int = 0,
                 max_qlen: int = 1, topk: int = 0, dtype: str = "bf16",
                 has_sinks: bool = False, num_segments: int = 0, num_sms: int = 0,
                 kernel: int = MLA_KERNEL_AUTO) -> Problem:
    return Problem(num_tokens=num_tokens, num_reqs=num_reqs, num_heads=num_heads,
                   head_dim=HEAD_DIM, kv_lora_rank=KV_LORA_RANK, block_size=block_size,
                   max_blocks_per_req=max_blocks_per_req, num_blocks=num_blocks,
                   max_seq_len=max_seq_len, max_qlen=max_qlen, topk=topk,
                   q_dtype=_dtype_code(dtype), kv_dtype=_dtype_code(dtype),
                   has_sinks=int(bool(has_sinks)), num_segments=num_segments, num_sms=num_sms,
                   kernel=kernel)


def mla_decode_plan(problem: Problem) -> Plan:
    lib = load_library()
    plan = Plan()
    _check("mla_decode_plan", lib.mla_decode_plan(ctypes.byref(problem), ctypes.byref(plan)))
    return plan


def mla_decode_fwd(plan: Plan, q, kv_cache, *, block_table=None, block_table_stride=None,
                   seq_lens=None, qo_indptr=None, sparse_slots=None, sparse_indptr=None,
                   softmax_scale: float, q_scale: float = 1.0, kv_scale: float = 1.0,
                   sinks=None, workspace=None, out, lse, stream=None) -> None:
    lib = load_library()
    if block_table_stride is None:
        block_table_stride = block_table.stride(0) if block_table is not None else 0
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
    _check("mla_decode_fwd", lib.mla_decode_fwd(
        ctypes.byref(plan), _ptr(q), _ptr(kv_cache), _ptr(block_table), int(block_table_stride),
        _ptr(seq_lens), _ptr(qo_indptr), _ptr(sparse_slots), _ptr(sparse_indptr),
        float(softmax_scale), float(q_scale), float(kv_scale), _ptr(sinks), _ptr(workspace),
        ws_bytes, _ptr(out), _ptr(lse), _stream(stream)))


def mla_decode_fwd_static(plan: Plan, q, kv_cache, *, block_table=None,
                          block_table_stride=None, seq_lens=None, qo_indptr=None,
                          sparse_slots=None, sparse_indptr=None, softmax_scale: float,
                          q_scale: float = 1.0, kv_scale: float = 1.0, sinks=None, out, lse,
                          status_out=None, stream=None) -> None:
    """mla_decode_fwd on the library's own static device scratch (no workspace)."""
    lib = load_library()
    if block_table_stride is None:
        block_table_stride = block_table.stride(0) if block_table is not None else 0
    _check("mla_decode_fwd_static", lib.mla_decode_fwd_static(
        ctypes.byref(plan), _ptr(q), _ptr(kv_cache), _ptr(block_table), int(block_table_stride),
        _ptr(seq_lens), _ptr(qo_indptr), _ptr(sparse_slots), _ptr(sparse_indptr),
        float(softmax_scale), float(q_scale), float(kv_scale), _ptr(sinks), _ptr(out), _ptr(lse),
        _ptr(status_out), _stream(stream)))


def mla_workspace_status(plan: Plan, workspace, *, clear: bool = False, stream=None) -> int:
    """The workspace's device status word after the stream's work so far
    (0: no kernel reported a timed-out wait); with ``clear`` a nonzero word
    is reset. Returns the word instead of raising on MLA_ERR_DEVICE_STATUS."""
    lib = load_library()
    code = ctypes.c_int32(0)
    st = lib.mla_workspace_status(ctypes.byref(plan), _ptr(workspace), ctypes.byref(code),
                                  1 if clear else 0, _stream(stream))
    if st not in (MLA_OK, MLA_ERR_DEVICE_STATUS):
        _check("mla_workspace_status", st)
    return int(code.value)


def _ws_bytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def mla_decode_schedule(plan: Plan, *, seq_lens=None, qo_indptr=None, sparse_indptr=None,
                        workspace, stream=None) -> None:
    """Balanced plans: the work list into ``workspace``."""
    lib = load_library()
    _check("mla_decode_schedule", lib.mla_decode_schedule(
        ctypes.byref(plan), _ptr(seq_lens), _ptr(qo_indptr), _ptr(sparse_indptr),
        _ptr(workspace), _ws_bytes(workspace), _stream(stream)))


def mla_decode_items(plan: Plan, q, kv_cache, *, block_table=None, block_table_stride=None,
                     seq_lens=None, qo_indptr=None, sparse_slots=None, sparse_indptr=None,
                     softmax_scale: float, q_scale: float = 1.0, kv_scale: float = 1.0,
                     sinks=None, workspace, out, lse, stream=None) -> None:
    """Balanced plans: the decode kernel over the work list in ``workspace``."""
    lib = load_library()
    if block_table_stride is None:
        block_table_stride = block_table.stride(0) if block_table is not None else 0
    _check("mla_decode_items", lib.mla_decode_items(
        ctypes.byref(plan), _ptr(q), _ptr(kv_cache), _ptr(block_table), int(block_table_stride),
        _ptr(seq_lens), _ptr(qo_indptr), _ptr(sparse_slots), _ptr(sparse_indptr),
        float(softmax_scale), float(q_scale), float(kv_scale), _ptr(sinks), _ptr(workspace),
        _ws_bytes(workspace), _ptr(out), _ptr(lse), _stream(stream)))


def mla_merge_items(plan: Plan, *, qo_indptr=None, sinks=None, workspace, out, lse,
                    stream=None) -> None:
    """Balanced plans: out and lse of the split rows from their partials."""
    lib = load_library()
    _check("mla_merge_items", lib.mla_merge_items(
        ctypes.byref(plan), _ptr(qo_indptr), _ptr(sinks), _ptr(workspace), _ws_bytes(workspace),
        _ptr(out), _ptr(lse), _stream(stream)))


def mla_decode_segments(plan: Plan, q, kv_cache, *, block_table=None, block_table_stride=None,
                        seq_lens=None, qo_indptr=None, sparse_slots=None, sparse_indptr=None,
                        softmax_scale: float, q_scale: float = 1.0, kv_scale: float = 1.0,
                        segm_output, segm_max, segm_expsum, stream=None) -> None:
    lib = load_library()
    if block_table_stride is None:
        block_table_stride = block_table.stride(0) if block_table is not None else 0
    _check("mla_decode_segments", lib.mla_decode_segments(
        ctypes.byref(plan), _ptr(q), _ptr(kv_cache), _ptr(block_table), int(block_table_stride),
        _ptr(seq_lens), _ptr(qo_indptr), _ptr(sparse_slots), _ptr(sparse_indptr),
        float(softmax_scale), float(q_scale), float(kv_scale), _ptr(segm_output),
        _ptr(segm_max), _ptr(segm_expsum), _stream(stream)))


def mla_merge_segments(segm_output, segm_max, segm_expsum, part_lens, *, tile_size: int,
                       sinks=None, out, lse, stream=None) -> None:
    lib = load_library()
    T, H, NS, rank = segm_output.shape
    _check("mla_merge_segments", lib.mla_merge_segments(
        _ptr(segm_output), _ptr(segm_max), _ptr(segm_expsum), _ptr(part_lens), T, H, NS, rank,
        int(tile_size), _ptr(sinks), MLA_DTYPE_BF16, _ptr(out), _ptr(lse), _stream(stream)))


def mla_merge_lse(shard_out, shard_lse, *, sinks=None, out, lse, stream=None) -> None:
    lib = load_library()
    W, T, H, rank = shard_out.shape
    _check("mla_merge_lse", lib.mla_merge_lse(
        _ptr(shard_out), _ptr(shard_lse), W, T, H, rank, _ptr(sinks), _ptr(out), _ptr(lse),
        _stream(stream)))


def mla_concat_quant_q(ql_nope, q_pe, *, out, q_scale: float | None = None, stream=None) -> None:
    """q = ql_nope || q_pe into ``out`` (bf16), or e4m3 codes of q / q_scale
    when ``q_scale`` is given (``out`` then holds uint8 codes)."""
    lib = load_library()
    T, H, _ = ql_nope.shape
    fp8 = q_scale is not None
    _check("mla_concat_quant_q", lib.mla_concat_quant_q(
        _ptr(ql_nope), ql_nope.stride(0), ql_nope.stride(1), _ptr(q_pe), q_pe.stride(0),
        q_pe.stride(1), T, H, MLA_DTYPE_FP8_E4M3 if fp8 else MLA_DTYPE_BF16,
        float(q_scale) if fp8 else 1.0, _ptr(out), _stream(stream)))


def mla_sparse_seqlen(query_start_loc, seq_lens, *, topk: int, indptr, lens=None,
                      stream=None) -> None:
    """Per-token sparse list lengths (``lens``, optional) and their exclusive
    prefix sum (``indptr``, ``[T + 1]``)."""
    lib = load_library()
    num_reqs = query_start_loc.numel() - 1
    num_tokens = indptr.numel() - 1
    _check("mla_sparse_seqlen", lib.mla_sparse_seqlen(
        _ptr(query_start_loc), _ptr(seq_lens), num_reqs, num_tokens, int(topk), _ptr(lens),
        _ptr(indptr), _stream(stream)))


# The calls over a cache with group scales check what their pointers cannot
# tell the library: element type, shape, device and density of each tensor.
# Each check is one chain of cheap reads (a call costs the host about as much
# as its launch); only a call that fails it works out which tensor is at fault.

_torch = None


def _load_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _refuse(fn: str, device: int, tensors, rules):
    """Raise for the first tensor or rule that does not hold: ``tensors`` is
    [(name, tensor, dtypes)], ``rules`` [(holds, what)]."""
    def need(cond, what):
        if not cond:
            raise MLAError(fn, MLA_ERR_INVALID_ARG, what)

    need(device >= 0, "the tensors must be on a CUDA device")
    need(device == _torch.cuda.current_device(), f"cuda:{device} is not the current device")
    for name, t, dtypes in tensors:
        if t is not None:
            need(t.get_device() == device, f"{name} is on {t.device}, not cuda:{device}")
            need(t.dtype in dtypes, f"{name} must be {' or '.join(str(d) for d in dtypes)}")
    for holds, what in rules:
        need(holds, what)
    need(False, "bad arguments")


def _dense_rows(shape, strides, min_cols: int) -> bool:
    """A matrix's rows are dense and do not overlap."""
    rows, cols = shape
    return cols >= min_cols and (rows == 0 or ((strides[1] == 1 or cols == 1)
                                               and (rows == 1 or strides[0] >= cols)))


def _scaled_args(fn: str, plan: Plan, q, kv_cache, kv_scales, scale_group, block_table,
                 block_table_stride, seq_lens, qo_indptr, sparse_slots, sparse_indptr,
                 softmax_scale, q_scale, sinks, workspace, out, lse, stream):
    torch = _torch or _load_torch()
    dev = q.get_device()
    pr = plan.prob
    T, H, R, nb, bs, topk = pr.num_tokens, pr.num_heads, pr.num_reqs, pr.num_blocks, pr.block_size, pr.topk
    i32, f32, codes = torch.int32, torch.float32, (torch.float8_e4m3fn, torch.uint8)
    ok = (pr.kv_dtype == MLA_DTYPE_FP8_E4M3 and dev >= 0 and dev == torch._C._cuda_getDevice()
          and q.dtype in codes and q.shape == (T, H, HEAD_DIM) and q.is_contiguous()
          and kv_cache.dtype in codes and kv_cache.get_device() == dev
          and kv_cache.shape == (nb, bs, HEAD_DIM) and kv_cache.is_contiguous()
          and scale_group > 0 and bs % scale_group == 0
          and kv_scales.dtype is f32 and kv_scales.get_device() == dev
          and kv_scales.numel() == nb * bs // scale_group and kv_scales.is_contiguous()
          and out.dtype is torch.bfloat16 and out.get_device() == dev
          and out.shape == (T, H, KV_LORA_RANK) and out.is_contiguous()
          and lse.dtype is f32 and lse.get_device() == dev and lse.shape == (T, H) and lse.is_contiguous()
          and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous()))
          and (sinks is None or (sinks.dtype is f32 and sinks.get_device() == dev
                                 and sinks.numel() == H and sinks.is_contiguous())))
    if ok and topk > 0:
        ok = (sparse_slots is None
              or (sparse_slots.dtype is i32 and sparse_slots.get_device() == dev and sparse_slots.is_contiguous()
                  and (sparse_indptr is not None or sparse_slots.numel() == T * topk)))
        ok = ok and (sparse_indptr is None
                     or (sparse_indptr.dtype is i32 and sparse_indptr.get_device() == dev
                         and sparse_indptr.numel() == T + 1 and sparse_indptr.is_contiguous()))
    elif ok:
        ok = (seq_lens is None or (seq_lens.dtype is i32 and seq_lens.get_device() == dev
                                   and seq_lens.numel() == R and seq_lens.is_contiguous()))
        ok = ok and (qo_indptr is None or (qo_indptr.dtype is i32 and qo_indptr.get_device() == dev
                                           and qo_indptr.numel() == R + 1 and qo_indptr.is_contiguous()))
        ok = ok and (block_table is None
                     or (block_table.dtype is i32 and block_table.get_device() == dev and block_table.dim() == 2
                         and block_table.shape[0] == R
                         and _dense_rows(block_table.shape, block_table.stride(), pr.max_blocks_per_req)))
    if not ok:
        if pr.kv_dtype != MLA_DTYPE_FP8_E4M3:
            raise MLAError(fn, MLA_ERR_UNSUPPORTED, "the plan's cache is not e4m3")
        dense = [("q", q), ("kv_cache", kv_cache), ("kv_scales", kv_scales), ("out", out), ("lse", lse),
                 ("workspace", workspace), ("sinks", sinks), ("seq_lens", seq_lens), ("qo_indptr", qo_indptr),
                 ("sparse_slots", sparse_slots), ("sparse_indptr", sparse_indptr)]
        _refuse(fn, dev, [("q", q, codes), ("kv_cache", kv_cache, codes), ("kv_scales", kv_scales, (f32,)),
                          ("out", out, (torch.bfloat16,)), ("lse", lse, (f32,)), ("sinks", sinks, (f32,)),
                          ("seq_lens", seq_lens, (i32,)), ("qo_indptr", qo_indptr, (i32,)),
                          ("sparse_slots", sparse_slots, (i32,)), ("sparse_indptr", sparse_indptr, (i32,)),
                          ("block_table", block_table, (i32,))],
                [(t is None or t.is_contiguous(), f"{name} must be contiguous") for name, t in dense] +
                [(q.shape == (T, H, HEAD_DIM), f"q must be [{T}, {H}, {HEAD_DIM}] for this plan"),
                 (kv_cache.shape == (nb, bs, HEAD_DIM), f"kv_cache must be [{nb}, {bs}, {HEAD_DIM}] for this plan"),
                 (scale_group > 0 and bs % scale_group == 0, "scale_group must divide the block size"),
                 (scale_group > 0 and kv_scales.numel() == nb * bs // scale_group,
                  "kv_scales must hold num_blocks * block_size / scale_group scales"),
                 (out.shape == (T, H, KV_LORA_RANK), f"out must be [{T}, {H}, {KV_LORA_RANK}]"),
                 (lse.shape == (T, H), f"lse must be [{T}, {H}]"),
                 (False, "sinks, seq_lens, qo_indptr, block_table or the slot lists do not have the plan's sizes")])
    if block_table_stride is None:
        block_table_stride = 0 if block_table is None else max(block_table.stride(0), block_table.size(1))
    return (ctypes.byref(plan), q.data_ptr(), kv_cache.data_ptr(), kv_scales.data_ptr(), scale_group,
            _ptr(block_table), block_table_stride, _ptr(seq_lens), _ptr(qo_indptr),
            _ptr(sparse_slots), _ptr(sparse_indptr), softmax_scale, q_scale,
            _ptr(sinks), _ptr(workspace), _ws_bytes(workspace), out.data_ptr(), lse.data_ptr(),
            torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))


def mla_decode_fwd_scaled(plan: Plan, q, kv_cache, kv_scales, *, scale_group: int, block_table=None,
                          block_table_stride=None, seq_lens=None, qo_indptr=None,
                          sparse_slots=None, sparse_indptr=None, softmax_scale: float,
                          q_scale: float = 1.0, sinks=None, workspace=None, out, lse,
                          stream=None) -> None:
    """mla_decode_fwd over an e4m3 cache with one fp32 scale per ``scale_group``
    slots of a block (``kv_scales``)."""
    lib = _lib or load_library()
    fn = "mla_decode_fwd_scaled"
    _check(fn, lib.mla_decode_fwd_scaled(*_scaled_args(
        fn, plan, q, kv_cache, kv_scales, scale_group, block_table, block_table_stride, seq_lens,
        qo_indptr, sparse_slots, sparse_indptr, softmax_scale, q_scale, sinks, workspace, out, lse,
        stream)))


def mla_decode_schedule_scaled(plan: Plan, *, seq_lens=None, qo_indptr=None, sparse_indptr=None,
                               workspace, stream=None) -> None:
    """Balanced plans: the work list of mla_decode_items_scaled into ``workspace``."""
    lib = _lib or load_library()
    _check("mla_decode_schedule_scaled", lib.mla_decode_schedule_scaled(
        ctypes.byref(plan), _ptr(seq_lens), _ptr(qo_indptr), _ptr(sparse_indptr),
        _ptr(workspace), _ws_bytes(workspace), _stream(stream)))


def mla_decode_items_scaled(plan: Plan, q, kv_cache, kv_scales, *, scale_group: int,
                            block_table=None, block_table_stride=None, seq_lens=None,
                            qo_indptr=None, sparse_slots=None, sparse_indptr=None,
                            softmax_scale: float, q_scale: float = 1.0, sinks=None, workspace,
                            out, lse, stream=None) -> None:
    """Balanced plans: the decode kernel of mla_decode_fwd_scaled over the work
    list in ``workspace`` (mla_decode_schedule_scaled's)."""
    lib = _lib or load_library()
    fn = "mla_decode_items_scaled"
    _check(fn, lib.mla_decode_items_scaled(*_scaled_args(
        fn, plan, q, kv_cache, kv_scales, scale_group, block_table, block_table_stride, seq_lens,
        qo_indptr, sparse_slots, sparse_indptr, softmax_scale, q_scale, sinks, workspace, out, lse,
        stream)))


def mla_decode_scaled_kernel(plan: Plan) -> int:
    """The decode kernel that the scaled calls of ``plan`` run on (``plan.kernel``,
    or 6 for the kernel of their own)."""
    lib = _lib or load_library()
    kernel = ctypes.c_int32(0)
    _check("mla_decode_scaled_kernel", lib.mla_decode_scaled_kernel(ctypes.byref(plan), ctypes.byref(kernel)))
    return kernel.value


def mla_block_tables(query_start_loc, seq_lens, free_blocks, block_table, *, block_size: int,
                     slot_mapping, req_id=None, positions=None, taken, stream=None) -> None:
    """The step's new columns of ``block_table [R, C]`` from ``free_blocks``
    (None: no free block), and ``slot_mapping``, ``req_id`` and ``positions``
    (``[T]``) of its tokens; ``taken`` (``[1]``) receives the number of blocks
    the step takes."""
    lib = _lib or load_library()
    torch = _torch or _load_torch()
    i32 = torch.int32
    dev = query_start_loc.get_device()
    R, T, shape = seq_lens.numel(), slot_mapping.numel(), block_table.shape
    ok = (dev >= 0 and dev == torch._C._cuda_getDevice()
          and query_start_loc.dtype is i32 and query_start_loc.numel() == R + 1 and query_start_loc.is_contiguous()
          and seq_lens.dtype is i32 and seq_lens.get_device() == dev and seq_lens.is_contiguous()
          and slot_mapping.dtype is i32 and slot_mapping.get_device() == dev and slot_mapping.is_contiguous()
          and taken.dtype is i32 and taken.get_device() == dev and taken.numel() == 1
          and block_table.dtype is i32 and block_table.get_device() == dev and len(shape) == 2 and shape[0] == R
          and _dense_rows(shape, block_table.stride(), 1))
    free = reqs = pos = None
    num_free = 0
    if free_blocks is not None:
        ok = ok and free_blocks.dtype is i32 and free_blocks.get_device() == dev and free_blocks.is_contiguous()
        free, num_free = free_blocks.data_ptr(), free_blocks.numel()
    if req_id is not None:
        ok = (ok and req_id.dtype is i32 and req_id.get_device() == dev and req_id.numel() == T
              and req_id.is_contiguous())
        reqs = req_id.data_ptr()
    if positions is not None:
        ok = (ok and positions.dtype is i32 and positions.get_device() == dev and positions.numel() == T
              and positions.is_contiguous())
        pos = positions.data_ptr()
    if not ok:
        fn = "mla_block_tables"
        named = [("query_start_loc", query_start_loc), ("seq_lens", seq_lens), ("slot_mapping", slot_mapping),
                 ("free_blocks", free_blocks), ("req_id", req_id), ("positions", positions)]
        _refuse(fn, dev, [(n, t, (i32,)) for n, t in named + [("taken", taken), ("block_table", block_table)]],
                [(t is None or t.is_contiguous(), f"{n} must be contiguous") for n, t in named] +
                [(query_start_loc.numel() == R + 1, "query_start_loc must be [num_reqs + 1]"),
                 (taken.numel() == 1, "taken must be [1]"),
                 (req_id is None or req_id.numel() == T, "req_id must be [num_tokens]"),
                 (positions is None or positions.numel() == T, "positions must be [num_tokens]"),
                 (False, "block_table must be [num_reqs, columns] with dense rows that do not overlap")])
    cols = shape[1]
    status = lib.mla_block_tables(
        query_start_loc.data_ptr(), seq_lens.data_ptr(), R, T, block_size, free, num_free, block_table.data_ptr(),
        block_table.stride()[0] if R > 1 else cols, cols, slot_mapping.data_ptr(), reqs, pos, taken.data_ptr(),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check("mla_block_tables", status)


def mla_cache_append(c_kv, k_pe, slot_mapping, kv_cache, kv_scales, *, scale_group: int,
                     stream=None) -> None:
    """The rows ``c_kv [T, 512] || k_pe [T, 64]`` (bf16) into the slots of
    ``slot_mapping``, as e4m3 codes under their groups' scales."""
    lib = _lib or load_library()
    torch = _torch or _load_torch()
    i32, f32, b16 = torch.int32, torch.float32, torch.bfloat16
    dev, T, shape, code = kv_cache.get_device(), slot_mapping.numel(), kv_cache.shape, kv_cache.dtype
    nb, bs, width = shape if len(shape) == 3 else (0, 0, 0)
    rope = HEAD_DIM - KV_LORA_RANK
    c_shape, p_shape = c_kv.shape, k_pe.shape
    c_stride, p_stride = c_kv.stride(), k_pe.stride()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and (code is torch.uint8 or code is torch.float8_e4m3fn)
            and width == HEAD_DIM and kv_cache.is_contiguous()
            and scale_group > 0 and bs % scale_group == 0
            and kv_scales.dtype is f32 and kv_scales.get_device() == dev and kv_scales.is_contiguous()
            and kv_scales.numel() == nb * bs // scale_group
            and slot_mapping.dtype is i32 and slot_mapping.get_device() == dev and slot_mapping.is_contiguous()
            and c_kv.dtype is b16 and c_kv.get_device() == dev and c_shape == (T, KV_LORA_RANK)
            and k_pe.dtype is b16 and k_pe.get_device() == dev and p_shape == (T, rope)
            and _dense_rows(c_shape, c_stride, 1) and _dense_rows(p_shape, p_stride, 1)):
        fn, codes = "mla_cache_append", (torch.float8_e4m3fn, torch.uint8)
        _refuse(fn, dev, [("kv_cache", kv_cache, codes), ("kv_scales", kv_scales, (f32,)),
                          ("slot_mapping", slot_mapping, (i32,)), ("c_kv", c_kv, (b16,)), ("k_pe", k_pe, (b16,))],
                [(t.is_contiguous(), f"{n} must be contiguous") for n, t in
                 (("kv_cache", kv_cache), ("kv_scales", kv_scales), ("slot_mapping", slot_mapping))] +
                [(width == HEAD_DIM, f"kv_cache must be [num_blocks, block_size, {HEAD_DIM}]"),
                 (c_kv.shape == (T, KV_LORA_RANK), f"c_kv must be [num_tokens, {KV_LORA_RANK}]"),
                 (k_pe.shape == (T, rope), f"k_pe must be [num_tokens, {rope}]"),
                 (scale_group > 0 and bs % scale_group == 0, "scale_group must divide the block size"),
                 (scale_group > 0 and kv_scales.numel() == nb * bs // scale_group,
                  "kv_scales must hold num_blocks * block_size / scale_group scales"),
                 (False, "the rows of c_kv and k_pe must be dense and must not overlap")])
    many = T > 1
    status = lib.mla_cache_append(
        c_kv.data_ptr(), c_stride[0] if many else KV_LORA_RANK, k_pe.data_ptr(), p_stride[0] if many else rope,
        slot_mapping.data_ptr(), T, nb, bs, scale_group, kv_cache.data_ptr(), kv_scales.data_ptr(),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check("mla_cache_append", status)


def mla_decode_shared_plan(problem: Problem, *, num_groups: int = 1) -> SharedPlan:
    """The plan of mla_decode_fwd_shared calls for up to ``num_groups`` groups."""
    lib = _lib or load_library()
    plan = SharedPlan()
    _check("mla_decode_shared_plan",
           lib.mla_decode_shared_plan(ctypes.byref(problem), num_groups, ctypes.byref(plan)))
    return plan


def mla_decode_fwd_shared(plan: SharedPlan, q, kv_cache, *, kv_scales=None, scale_group: int = 0, block_table,
                          seq_lens, qo_indptr=None, prefix_lens, group_indptr=None, softmax_scale: float,
                          q_scale: float = 1.0, kv_scale: float = 1.0, sinks=None, workspace, out, lse,
                          stream=None) -> None:
    """The decode of a batch whose requests share prefixes: ``prefix_lens [G]`` tokens
    in common among the requests ``group_indptr[g]`` to ``group_indptr[g + 1]``."""
    lib, fn = _lib or load_library(), "mla_decode_fwd_shared"
    torch = _torch or _load_torch()
    pr, G = plan.plan.prob, plan.num_groups
    dev, T, H, R, nb, bs = q.get_device(), pr.num_tokens, pr.num_heads, pr.num_reqs, pr.num_blocks, pr.block_size
    i32, f32 = torch.int32, torch.float32
    kinds = (torch.float8_e4m3fn, torch.uint8) if pr.kv_dtype == MLA_DTYPE_FP8_E4M3 else (torch.bfloat16,)
    lists = (("seq_lens", seq_lens, R), ("qo_indptr", qo_indptr, R + 1), ("prefix_lens", prefix_lens, G),
             ("group_indptr", group_indptr, G + 1))
    ok = (dev >= 0 and dev == torch._C._cuda_getDevice() and q.dtype in kinds and q.shape == (T, H, HEAD_DIM)
          and q.is_contiguous() and kv_cache.dtype in kinds and kv_cache.get_device() == dev
          and kv_cache.shape == (nb, bs, HEAD_DIM) and kv_cache.is_contiguous()
          and (kv_scales is None) == (scale_group == 0)
          and (kv_scales is None
               or (scale_group > 0 and bs % scale_group == 0 and kv_scales.dtype is f32
                   and kv_scales.get_device() == dev and kv_scales.numel() == nb * bs // scale_group
                   and kv_scales.is_contiguous()))
          and out.dtype is torch.bfloat16 and out.get_device() == dev and out.shape == (T, H, KV_LORA_RANK)
          and out.is_contiguous() and lse.dtype is f32 and lse.get_device() == dev and lse.shape == (T, H)
          and lse.is_contiguous() and workspace.get_device() == dev and workspace.is_contiguous()
          and (sinks is None or (sinks.dtype is f32 and sinks.get_device() == dev and sinks.numel() == H
                                 and sinks.is_contiguous()))
          and block_table.dtype is i32 and block_table.get_device() == dev and block_table.dim() == 2
          and block_table.shape[0] == R
          and _dense_rows(block_table.shape, block_table.stride(), pr.max_blocks_per_req))
    for _, t, n in lists:
        ok = ok and (t is None or (t.dtype is i32 and t.get_device() == dev and t.numel() == n and t.is_contiguous()))
    if not ok:
        if kv_scales is not None and pr.kv_dtype != MLA_DTYPE_FP8_E4M3:
            raise MLAError(fn, MLA_ERR_UNSUPPORTED, "the plan's cache is not e4m3")
        dense = [("q", q), ("kv_cache", kv_cache), ("kv_scales", kv_scales), ("out", out), ("lse", lse),
                 ("workspace", workspace), ("sinks", sinks)] + [(n, t) for n, t, _ in lists]
        _refuse(fn, dev, [("q", q, kinds), ("kv_cache", kv_cache, kinds), ("kv_scales", kv_scales, (f32,)),
                          ("out", out, (torch.bfloat16,)), ("lse", lse, (f32,)), ("sinks", sinks, (f32,)),
                          ("block_table", block_table, (i32,)), ("workspace", workspace, (workspace.dtype,))] +
                [(n, t, (i32,)) for n, t, _ in lists],
                [(t is None or t.is_contiguous(), f"{n} must be contiguous") for n, t in dense] +
                [(t is None or t.numel() == k, f"{n} must hold {k} numbers") for n, t, k in lists] +
                [(q.shape == (T, H, HEAD_DIM), f"q must be [{T}, {H}, {HEAD_DIM}] for this plan"),
                 (kv_cache.shape == (nb, bs, HEAD_DIM), f"kv_cache must be [{nb}, {bs}, {HEAD_DIM}] for this plan"),
                 ((kv_scales is None) == (scale_group == 0), "kv_scales and scale_group go together"),
                 (scale_group >= 0 and (scale_group == 0 or bs % scale_group == 0), "scale_group must divide the block size"),
                 (out.shape == (T, H, KV_LORA_RANK), f"out must be [{T}, {H}, {KV_LORA_RANK}]"),
                 (lse.shape == (T, H), f"lse must be [{T}, {H}]"),
                 (False, "kv_scales, sinks or block_table do not have the plan's sizes")])
    status = lib.mla_decode_fwd_shared(
        ctypes.byref(plan), q.data_ptr(), kv_cache.data_ptr(), _ptr(kv_scales), scale_group, block_table.data_ptr(),
        max(block_table.stride(0), block_table.size(1)), _ptr(seq_lens), _ptr(qo_indptr), _ptr(prefix_lens),
        _ptr(group_indptr), softmax_scale, q_scale, kv_scale, _ptr(sinks), workspace.data_ptr(), _ws_bytes(workspace),
        out.data_ptr(), lse.data_ptr(), torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check(fn, status)


def mla_rope_plan(*, dim: int = 64, layout: str = "interleaved", base: float = 10000.0, scaling: str = "none",
                  factor: float = 1.0, original_max_position: int = 4096, beta_fast: float = 32.0,
                  beta_slow: float = 1.0, mscale: float = 0.0, mscale_all_dim: float = 0.0) -> Rope:
    """The rotary frequencies of a model: ``layout`` "interleaved" or "half",
    ``scaling`` "none", "linear" or "yarn"."""
    lib = _lib or load_library()
    layouts = {"interleaved": MLA_ROPE_INTERLEAVED, "half": MLA_ROPE_HALF}
    scalings = {"none": MLA_ROPE_SCALING_NONE, "linear": MLA_ROPE_SCALING_LINEAR, "yarn": MLA_ROPE_SCALING_YARN}
    for value, known in ((layout, layouts), (scaling, scalings)):
        if value not in known:
            raise MLAError("mla_rope_plan", MLA_ERR_INVALID_ARG, f"{value!r} is none of {sorted(known)}")
    prob = RopeProblem(dim=dim, layout=layouts[layout], scaling=scalings[scaling],
                       original_max_position=original_max_position, base=base, factor=factor,
                       beta_fast=beta_fast, beta_slow=beta_slow, mscale=mscale, mscale_all_dim=mscale_all_dim)
    rope = Rope()
    _check("mla_rope_plan", lib.mla_rope_plan(ctypes.byref(prob), ctypes.byref(rope)))
    return rope


def _last_dense(t) -> bool:
    return t.shape[-1] <= 1 or t.stride(-1) == 1


def mla_rope_qk(rope: Rope, positions, *, ql_nope=None, q_pe=None, q_out=None, q_scale: float | None = None,
                k_pe=None, k_out=None, stream=None) -> None:
    """``q_out [T, H, 576]`` = ``ql_nope || rotated q_pe`` (bf16, or e4m3 codes of
    q / ``q_scale`` when that is given), and ``k_out [T, 64]`` = rotated ``k_pe``
    (which may be ``k_out`` itself); either may be left out."""
    lib = _lib or load_library()
    torch = _torch or _load_torch()
    i32, b16 = torch.int32, torch.bfloat16
    codes = (b16,) if q_scale is None else (torch.float8_e4m3fn, torch.uint8)
    dev, T, H = positions.get_device(), positions.numel(), 0
    ok = (dev >= 0 and dev == torch._C._cuda_getDevice() and positions.dtype is i32 and positions.is_contiguous()
          and (ql_nope is not None or k_pe is not None))
    nope = pe = out = keys = kout = None
    n_st = p_st = (0, 0, 0)
    k_st = ko_st = (64, 1)
    if ql_nope is None:
        ok = ok and q_pe is None and q_out is None
    elif ok:
        ok = False
        if q_pe is not None and q_out is not None and ql_nope.dim() == 3:
            n_st, p_st, H = ql_nope.stride(), q_pe.stride(), ql_nope.size(1)
            ok = (H > 0 and ql_nope.shape == (T, H, 512) and ql_nope.dtype is b16 and ql_nope.get_device() == dev
                  and n_st[2] == 1 and q_pe.shape == (T, H, 64) and q_pe.dtype is b16 and q_pe.get_device() == dev
                  and p_st[2] == 1 and q_out.shape == (T, H, 576) and q_out.dtype in codes
                  and q_out.get_device() == dev and q_out.is_contiguous())
            nope, pe, out = ql_nope.data_ptr(), q_pe.data_ptr(), q_out.data_ptr()
    if k_pe is None:
        ok = ok and k_out is None
    elif ok:
        ok = False
        if k_out is not None and k_pe.shape == (T, 64) and k_out.shape == (T, 64):
            k_st, ko_st = k_pe.stride(), k_out.stride()
            ok = (k_pe.dtype is b16 and k_pe.get_device() == dev and k_st[1] == 1 and k_out.dtype is b16
                  and k_out.get_device() == dev and ko_st[1] == 1 and (T < 2 or ko_st[0] >= 64))
            keys, kout = k_pe.data_ptr(), k_out.data_ptr()
    fn = "mla_rope_qk"
    if not ok:
        named = [("ql_nope", ql_nope, (b16,)), ("q_pe", q_pe, (b16,)), ("q_out", q_out, codes), ("k_pe", k_pe, (b16,)),
                 ("k_out", k_out, (b16,))]
        given = [t is not None for _, t, _ in named]
        _refuse(fn, dev, [("positions", positions, (i32,))] + named,
                [(positions.is_contiguous(), "positions must be contiguous"),
                 (given[0] == given[1] == given[2], "ql_nope, q_pe and q_out go together"),
                 (given[3] == given[4], "k_pe and k_out go together"),
                 (given[0] or given[3], "neither queries nor keys")] +
                [(t is None or _last_dense(t), f"the last dimension of {n} must be contiguous") for n, t, _ in named] +
                [(False, f"the shapes must be [{T}, H, 512], [{T}, H, 64] and contiguous [{T}, H, 576]; [{T}, 64] with "
                         "rows of k_out that do not overlap")])
    if T < 2 or H < 2:  # (strides of dimensions of one element say nothing)
        n_st, p_st = ((st[0] if T > 1 else 0, st[1] if H > 1 else 0) for st in (n_st, p_st))
        if T < 2:
            k_st = ko_st = (64, 1)
    status = lib.mla_rope_qk(
        ctypes.byref(rope), positions.data_ptr(), T, H, nope, n_st[0], n_st[1], pe, p_st[0], p_st[1],
        MLA_DTYPE_BF16 if q_scale is None else MLA_DTYPE_FP8_E4M3, 1.0 if q_scale is None else q_scale, out, keys,
        k_st[0], kout, max(ko_st[0], 64), torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check(fn, status)


# The calls on the pages of a cache.

def _pages_args(fn: str, kv_cache, kv_scales, scale_group):
    """(device, num_blocks, block_size, dtype code) of a cache, checked."""
    torch = _torch or _load_torch()
    dev, shape, kind = kv_cache.get_device(), kv_cache.shape, kv_cache.dtype
    fp8 = kind is torch.uint8 or kind is torch.float8_e4m3fn
    nb, bs, width = shape if len(shape) == 3 else (0, 0, 0)
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and (fp8 or kind is torch.bfloat16) and width == HEAD_DIM
            and kv_cache.is_contiguous() and (kv_scales is not None) == (scale_group > 0)
            and (kv_scales is None
                 or (fp8 and bs % scale_group == 0 and kv_scales.dtype is torch.float32
                     and kv_scales.get_device() == dev and kv_scales.is_contiguous()
                     and kv_scales.numel() == nb * bs // scale_group))):
        _refuse(fn, dev, [("kv_cache", kv_cache, (torch.bfloat16, torch.float8_e4m3fn, torch.uint8)),
                          ("kv_scales", kv_scales, (torch.float32,))],
                [(width == HEAD_DIM, f"kv_cache must be [num_blocks, block_size, {HEAD_DIM}]"),
                 (kv_cache.is_contiguous(), "kv_cache must be contiguous"),
                 ((kv_scales is not None) == (scale_group > 0), "kv_scales and scale_group go together"),
                 (kv_scales is None or fp8, "a cache with group scales is e4m3"),
                 (scale_group <= 0 or bs % scale_group == 0, "scale_group must divide the block size"),
                 (False, "kv_scales must be contiguous and hold num_blocks * block_size / scale_group scales")])
    return dev, nb, bs, MLA_DTYPE_FP8_E4M3 if fp8 else MLA_DTYPE_BF16


def _int_lists(fn: str, dev: int, tables, lists):
    """``tables`` [(name, 2-D int32 tensor)], ``lists`` [(name, contiguous int32
    tensor or None, size or None)] on device ``dev``."""
    i32 = _torch.int32
    for name, t, n in lists:
        if t is None or (t.dtype is i32 and t.get_device() == dev and t.is_contiguous()
                         and (n is None or t.numel() == n)):
            continue
        _refuse(fn, dev, [(name, t, (i32,))], [(t.is_contiguous(), f"{name} must be contiguous"),
                                               (False, f"{name} must hold {n} numbers")])
    for name, t in tables:
        if t.dtype is i32 and t.get_device() == dev and t.dim() == 2:
            rows, cols = t.shape
            st = t.stride()
            if cols > 0 and (rows == 0 or ((st[1] == 1 or cols == 1) and (rows == 1 or st[0] >= cols))):
                continue
        _refuse(fn, dev, [(name, t, (i32,))],
                [(False, f"{name} must be [rows, columns] with dense rows that do not overlap")])


def _table(t, i32, dev: int):
    """(rows, columns, row stride) of a 2-D int32 tensor with dense rows that do not
    overlap, on device ``dev``; no columns of another one."""
    shape = t.shape
    if t.dtype is not i32 or t.get_device() != dev or len(shape) != 2:
        return 0, 0, 0
    (rows, cols), (across, along) = shape, t.stride()
    if rows > 0 and not ((along == 1 or cols == 1) and (rows == 1 or across >= cols)):
        return 0, 0, 0
    return rows, cols, across if rows > 1 else cols


def _table_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def mla_cache_workspace(num_blocks: int) -> int:
    """Workspace bytes (zeroed once) of mla_cache_free and mla_cache_compact."""
    return (_lib or load_library()).mla_cache_workspace(num_blocks)


def mla_cache_fork(parent, child, lens, free_blocks, block_table, ref_counts, kv_cache, kv_scales=None, *,
                   scale_group: int = 0, taken, stream=None) -> None:
    """Table rows ``child`` as copies of rows ``parent`` for the first ``lens`` tokens:
    whole blocks shared, a partly filled last one copied into the next entry of
    ``free_blocks`` (None: no free block)."""
    lib, fn = _lib or load_library(), "mla_cache_fork"
    dev, nb, bs, code = _pages_args(fn, kv_cache, kv_scales, scale_group)
    n, i32, free, num_free = parent.numel(), _torch.int32, None, 0
    rows, cols, stride = _table(block_table, i32, dev)
    ok = (cols > 0 and parent.dtype is i32 and parent.get_device() == dev and parent.is_contiguous()
          and child.dtype is i32 and child.get_device() == dev and child.is_contiguous() and child.numel() == n
          and lens.dtype is i32 and lens.get_device() == dev and lens.is_contiguous() and lens.numel() == n
          and ref_counts.dtype is i32 and ref_counts.get_device() == dev and ref_counts.is_contiguous()
          and ref_counts.numel() == nb
          and taken.dtype is i32 and taken.get_device() == dev and taken.numel() == 1)
    if free_blocks is not None:
        ok = ok and free_blocks.dtype is i32 and free_blocks.get_device() == dev and free_blocks.is_contiguous()
        free, num_free = free_blocks.data_ptr(), free_blocks.numel()
    if not ok:
        _int_lists(fn, dev, [("block_table", block_table)],
                   [("parent", parent, n), ("child", child, n), ("lens", lens, n), ("free_blocks", free_blocks, None),
                    ("ref_counts", ref_counts, nb), ("taken", taken, 1)])
    status = lib.mla_cache_fork(
        parent.data_ptr(), child.data_ptr(), lens.data_ptr(), n, free, num_free, block_table.data_ptr(), stride, rows, cols,
        ref_counts.data_ptr(), nb, bs, code, scale_group, kv_cache.data_ptr(),
        None if kv_scales is None else kv_scales.data_ptr(), taken.data_ptr(),
        _torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check(fn, status)


def mla_cache_copy_blocks(src, dst, kv_cache, kv_scales=None, *, scale_group: int = 0, stream=None) -> None:
    """Blocks ``src`` of the cache, with their scales, to blocks ``dst``."""
    lib, fn = _lib or load_library(), "mla_cache_copy_blocks"
    dev, nb, bs, code = _pages_args(fn, kv_cache, kv_scales, scale_group)
    n = src.numel()
    _int_lists(fn, dev, [], [("src", src, n), ("dst", dst, n)])
    status = lib.mla_cache_copy_blocks(
        src.data_ptr(), dst.data_ptr(), n, nb, bs, code, scale_group, kv_cache.data_ptr(), _ptr(kv_scales),
        _torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check(fn, status)


def mla_cache_free(rows, block_table, ref_counts, *, lens=None, block_size: int | None = None, freed, num_freed,
                   workspace, stream=None) -> None:
    """Gives up the table rows ``rows``, all their columns or those of ``lens`` tokens
    in blocks of ``block_size``; the blocks that no row holds any more go to
    ``freed``, in ascending order, their number to ``num_freed``."""
    lib, fn = _lib or load_library(), "mla_cache_free"
    torch = _torch or _load_torch()
    if block_size is None:
        if lens is not None:
            raise MLAError(fn, MLA_ERR_INVALID_ARG, "lens are in tokens: they need a block_size")
        block_size = 1
    dev, n = block_table.get_device(), rows.numel()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and workspace.get_device() == dev
            and workspace.is_contiguous()):
        _refuse(fn, dev, [("workspace", workspace, (workspace.dtype,))], [(False, "workspace must be contiguous")])
    i32 = torch.int32
    num_rows, cols, stride = _table(block_table, i32, dev)
    if not (cols > 0 and rows.dtype is i32 and rows.get_device() == dev and rows.is_contiguous()
            and (lens is None or (lens.dtype is i32 and lens.get_device() == dev and lens.is_contiguous()
                                  and lens.numel() == n))
            and ref_counts.dtype is i32 and ref_counts.get_device() == dev and ref_counts.is_contiguous()
            and freed.dtype is i32 and freed.get_device() == dev and freed.is_contiguous()
            and num_freed.dtype is i32 and num_freed.get_device() == dev and num_freed.numel() == 1):
        _int_lists(fn, dev, [("block_table", block_table)],
                   [("rows", rows, n), ("lens", lens, n), ("ref_counts", ref_counts, None), ("freed", freed, None),
                    ("num_freed", num_freed, 1)])
    status = lib.mla_cache_free(
        rows.data_ptr(), None if lens is None else lens.data_ptr(), n, block_table.data_ptr(), stride, num_rows, cols,
        ref_counts.data_ptr(), ref_counts.numel(), block_size, freed.data_ptr(), freed.numel(), num_freed.data_ptr(),
        workspace.data_ptr(), _ws_bytes(workspace),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check(fn, status)


def mla_cache_compact(ref_counts, block_table, kv_cache, kv_scales=None, *, scale_group: int = 0, refs_out=None,
                      table_out=None, num_live, workspace, stream=None) -> None:
    """Moves the blocks in use to the front of the pool. ``refs_out`` and
    ``table_out`` receive the counts and the tables (None: in place), ``num_live``
    the number of blocks in use."""
    lib, fn = _lib or load_library(), "mla_cache_compact"
    dev, nb, bs, code = _pages_args(fn, kv_cache, kv_scales, scale_group)
    refs_out = ref_counts if refs_out is None else refs_out
    table_out = block_table if table_out is None else table_out
    if not (workspace.get_device() == dev and workspace.is_contiguous() and block_table.shape == table_out.shape):
        _refuse(fn, dev, [("workspace", workspace, (workspace.dtype,))],
                [(workspace.is_contiguous(), "workspace must be contiguous"),
                 (False, "table_out must have block_table's shape")])
    _int_lists(fn, dev, [("block_table", block_table), ("table_out", table_out)],
               [("ref_counts", ref_counts, nb), ("refs_out", refs_out, nb), ("num_live", num_live, 1)])
    rows, cols = block_table.shape
    status = lib.mla_cache_compact(
        ref_counts.data_ptr(), refs_out.data_ptr(), block_table.data_ptr(), _table_stride(block_table),
        table_out.data_ptr(), _table_stride(table_out), rows, cols, nb, bs, code, scale_group, kv_cache.data_ptr(),
        _ptr(kv_scales), num_live.data_ptr(), workspace.data_ptr(), _ws_bytes(workspace),
        _torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream))
    if status:
        _check(fn, status)


def mla_fit_kpool_indices(token_indices, *, topk: int, out, stream=None) -> None:
    """``[T, W]`` top-k rows fitted to width ``topk`` into ``out [T, topk]``."""
    lib = load_library()
    T, W = token_indices.shape
    _check("mla_fit_kpool_indices", lib.mla_fit_kpool_indices(
        _ptr(token_indices), token_indices.stride(0), T, W, int(topk), _ptr(out), out.stride(0),
        _stream(stream)))


def mla_sparse_index_convert(req_id, block_table, token_indices, *, block_size: int,
                             cu_seqlens=None, out, stream=None) -> None:
    lib = load_library()
    bt_rows, bt_cols = block_table.shape
    T, topk = token_indices.shape
    _check("mla_sparse_index_convert", lib.mla_sparse_index_convert(
        _ptr(req_id), _ptr(block_table), bt_rows, bt_cols, block_table.stride(0),
        _ptr(token_indices), token_indices.stride(0), T, topk, int(block_size),
        _ptr(cu_seqlens), _ptr(out), _stream(stream)))


# ---------------------------------------------------------------------------
# convenience: one decode call on a Workload whose tensors live on a device
# ---------------------------------------------------------------------------

class DeviceWorkload:
    """Device copies of an ``inputs.Workload`` plus a plan and output buffers."""

    def __init__(self, w, device="cuda", num_segments=None, num_sms=0, plan=True,
                 kernel=MLA_KERNEL_AUTO):
        import torch

        self.w = w
        dev = torch.device(device)
        self.device = dev
        self.q = torch.from_numpy(w.q.view(_np_view(w.q_dtype))).to(dev)
        self.cache = torch.from_numpy(w.cache.view(_np_view(w.kv_dtype))).to(dev)
        self.block_table = torch.from_numpy(w.block_table).to(dev)
        self.seq_lens = torch.from_numpy(w.seq_lens).to(dev)
        self.qo_indptr = None if w.qo_indptr is None else torch.from_numpy(w.qo_indptr).to(dev)
        self.sinks = None if w.sinks is None else torch.from_numpy(w.sinks).to(dev)
        self.slots = None
        if w.sparse:
            self.req_id = torch.from_numpy(w.req_id_per_token).to(dev)
            self.topk_indices = torch.from_numpy(w.topk_indices).to(dev)
            self.slots = torch.empty_like(self.topk_indices)
        T, H = w.num_tokens, w.num_heads
        self.out = torch.empty((T, H, KV_LORA_RANK), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((T, H), dtype=torch.float32, device=dev)
        ns = w.num_segments if num_segments is None else num_segments
        self.problem = make_problem(
            num_tokens=T, num_heads=H, block_size=w.block_size, num_blocks=w.num_blocks,
            num_reqs=w.num_reqs if not w.sparse else 0,
            max_blocks_per_req=w.max_blocks_per_req,
            max_seq_len=int(w.seq_lens.max()) if w.num_reqs else 0,
            max_qlen=w.max_qlen, topk=w.topk, dtype=w.kv_dtype, has_sinks=w.sinks is not None,
            num_segments=ns, num_sms=num_sms, kernel=kernel)
        self.plan = mla_decode_plan(self.problem) if plan else None
        self.workspace = None
        if self.plan is not None and self.plan.workspace_bytes:
            # zeroed once: its first int32 is the device status word
            self.workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=dev)

    def status(self) -> int:
        """Device status word of the workspace (0 = no kernel reported a timeout)."""
        import torch

        if self.workspace is None:
            return 0
        return int(self.workspace[:4].view(torch.int32).item())

    def convert(self, stream=None):
        """Top-k positions -> global slots (sparse workloads)."""
        mla_sparse_index_convert(self.req_id, self.block_table, self.topk_indices,
                                 block_size=self.w.block_size, out=self.slots, stream=stream)

    def forward(self, stream=None, convert=True):
        w = self.w
        if w.sparse and convert:
            self.convert(stream)
        mla_decode_fwd(self.plan, self.q, self.cache,
                       block_table=None if w.sparse else self.block_table,
                       seq_lens=None if w.sparse else self.seq_lens, qo_indptr=self.qo_indptr,
                       sparse_slots=self.slots, softmax_scale=w.softmax_scale,
                       q_scale=w.q_scale, kv_scale=w.kv_scale, sinks=self.sinks,
                       workspace=self.workspace, out=self.out, lse=self.lse, stream=stream)
        return self.out, self.lse


def _np_view(dtype_name: str):
    import numpy as np
    return np.int16 if dtype_name == "bf16" else np.uint8
