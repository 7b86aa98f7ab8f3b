"""Python binding of libmla_gb300.so (paged MLA latent-cache decode, sm_103a).

Argument marshalling only: every step of the decode runs in the library's
CUDA kernels.  Functions mirror the C ABI in include/mla_decode.h,
include/mla_layer.h and include/mla_chunk.h and take
device addresses as ints (or any object with ``data_ptr()``, e.g. a torch
tensor) and CUDA streams as ints (``torch.cuda.current_stream().cuda_stream``)
or None for the default stream.  There is no fallback: if the library cannot
be loaded every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_gb300.so")

MLA_OK = 0
MLA_ERR_INVALID_ARGUMENT = -1
MLA_ERR_UNSUPPORTED = -2
MLA_ERR_MISALIGNED = -3
MLA_ERR_WORKSPACE_TOO_SMALL = -4
MLA_ERR_CUDA = -5

MLA_KV_BF16 = 0
MLA_KV_FP8_E4M3_E8M0 = 1
MLA_KV_FP4_E2M1_E8M0 = 2

MLA_STATUS_BAD_PAGE = 0x1
MLA_STATUS_BAD_INDEX = 0x2
MLA_STATUS_TIMEOUT = 0x4

MLA_TILE_TOKENS = 64

MLA_DTYPE_BF16 = 0
MLA_DTYPE_F16 = 1
MLA_DTYPE_F32 = 2

MLA_NORM_OUT_SAME = 0
MLA_NORM_OUT_E4M3_E8M0 = 1
MLA_NORM_OUT_E4M3_ROW = 2
MLA_NORM_MAX_COLS = 32768

MLA_ROPE_INTERLEAVED = 0
MLA_ROPE_HALVES = 1
MLA_ROPE_SCALING_NONE = 0
MLA_ROPE_SCALING_LINEAR = 1
MLA_ROPE_SCALING_PARTS = 2
MLA_ROPE_SCALING_YARN = 3
MLA_ROPE_MAX_DIM = 256

MLA_CHUNK_MAX_HEADS = 128
MLA_CHUNK_MAX_REQUESTS = 8192

EXPORTED = (
    "mla_decode_plan", "mla_q_absorb", "mla_decode_run", "mla_combine", "mla_uv_proj",
    "mla_get_status", "mla_clear_status", "mla_strerror", "mla_version",
    "mla_decode_run_static", "mla_cache_append", "mla_selftest_bounded_wait", "mla_decode_step",
    "mla_rms_norm", "mla_rope_make_plan", "mla_rope", "mla_cache_append_tokens", "mla_cache_gather",
    "mla_chunk_make_plan", "mla_chunk_attend", "mla_cache_weights", "mla_evict_make_plan",
    "mla_cache_evict",
)


class MlaProblem(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("q_len", ctypes.c_int32), ("num_heads", ctypes.c_int32),
        ("kv_lora_rank", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
        ("nope_dim", ctypes.c_int32), ("v_head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("max_pages_per_seq", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
        ("topk_width", ctypes.c_int32), ("causal", ctypes.c_int32), ("sm_scale", ctypes.c_float),
    ]


class MlaPlan(ctypes.Structure):
    _fields_ = [
        ("problem", MlaProblem), ("num_streams", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
        ("num_slots", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
        ("ws_partial_o", ctypes.c_int64), ("ws_partial_lse", ctypes.c_int64),
        ("ws_prefix", ctypes.c_int64), ("ws_status", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
        ("planned_tiles", ctypes.c_int64), ("ws_q_hat", ctypes.c_int64),
        ("split_tokens", ctypes.c_int32), ("sm_count", ctypes.c_int32),
        ("prefix_pass", ctypes.c_int32), ("reserved", ctypes.c_int32 * 3),
    ]


class MlaNormProblem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("out_format", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
        ("residual_out_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
        ("scale_stride", ctypes.c_int64),
    ]


class MlaRopeConfig(ctypes.Structure):
    _fields_ = [
        ("layout", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("original_positions", ctypes.c_int32), ("theta", ctypes.c_double),
        ("factor", ctypes.c_double), ("fast_rotations", ctypes.c_double),
        ("slow_rotations", ctypes.c_double), ("amplitude", ctypes.c_double),
    ]


class MlaRopePlan(ctypes.Structure):
    _fields_ = [
        ("config", MlaRopeConfig), ("amplitude", ctypes.c_float), ("reserved", ctypes.c_int32),
        ("turns", ctypes.c_uint64 * (MLA_ROPE_MAX_DIM // 2)),
    ]


class MlaRopeProblem(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rope_offset", ctypes.c_int32), ("dtype", ctypes.c_int32), ("transposed", ctypes.c_int32),
        ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
        ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
    ]


class MlaChunkPlan(ctypes.Structure):
    _fields_ = [
        ("problem", MlaProblem), ("tokens", ctypes.c_int32), ("sm_count", ctypes.c_int32),
        ("context_tokens", ctypes.c_int64), ("clusters", ctypes.c_int32), ("mark", ctypes.c_int32),
        ("ws_partial_o", ctypes.c_int64), ("ws_partial_lse", ctypes.c_int64),
        ("ws_segments", ctypes.c_int64), ("ws_starts", ctypes.c_int64), ("ws_rows", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
    ]


class MlaEvictPlan(ctypes.Structure):
    _fields_ = [
        ("problem", MlaProblem), ("budget", ctypes.c_int32), ("sinks", ctypes.c_int32),
        ("recent", ctypes.c_int32), ("mark", ctypes.c_int32), ("most_moves", ctypes.c_int64),
        ("ws_counts", ctypes.c_int64), ("ws_moves", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_int64),
    ]


class MlaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {code} ({strerror(code)})")


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the shared library (once).  Raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    P = ctypes.POINTER
    sz = ctypes.c_size_t
    lib.mla_decode_plan.argtypes = [P(MlaProblem), P(ctypes.c_int32), i32, i32, P(MlaPlan), P(sz)]
    lib.mla_q_absorb.argtypes = [P(MlaPlan), vp, vp, vp, vp]
    lib.mla_decode_run.argtypes = [P(MlaPlan), vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    lib.mla_combine.argtypes = [P(MlaPlan), vp, vp, sz, vp, vp, vp, vp, vp]
    lib.mla_decode_step.argtypes = [P(MlaPlan), vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp, vp]
    lib.mla_decode_run_static.argtypes = [P(MlaPlan), vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.mla_uv_proj.argtypes = [vp, vp, vp, i32, i32, vp]
    lib.mla_cache_append.argtypes = [P(MlaProblem), vp, vp, vp, ctypes.c_float, vp, vp, vp]
    lib.mla_rms_norm.argtypes = [P(MlaNormProblem), vp, vp, vp, vp, vp, vp, vp]
    lib.mla_rope_make_plan.argtypes = [P(MlaRopeConfig), P(MlaRopePlan)]
    lib.mla_rope.argtypes = [P(MlaRopeProblem), P(MlaRopePlan), vp, vp, vp, vp]
    lib.mla_cache_append_tokens.argtypes = [P(MlaProblem), i32, vp, i64, vp, vp, vp, vp,
                                            ctypes.c_float, P(MlaRopePlan), vp, vp, vp]
    lib.mla_cache_gather.argtypes = [P(MlaProblem), i32, vp, vp, vp, vp, vp, i64, vp, vp]
    lib.mla_chunk_make_plan.argtypes = [P(MlaProblem), i32, i64, i32, P(MlaChunkPlan), P(sz)]
    lib.mla_chunk_attend.argtypes = [P(MlaChunkPlan), vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp]
    lib.mla_cache_weights.argtypes = [P(MlaChunkPlan), vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, i64, vp, vp]
    lib.mla_evict_make_plan.argtypes = [P(MlaProblem), i32, i32, i32, P(MlaEvictPlan), P(sz)]
    lib.mla_cache_evict.argtypes = [P(MlaEvictPlan), vp, vp, vp, vp, vp, i64, vp, sz, vp, vp, vp, vp, vp]
    lib.mla_selftest_bounded_wait.argtypes = [vp, i64, vp, vp]
    lib.mla_get_status.argtypes = [P(MlaPlan), vp, P(ctypes.c_uint32), vp]
    lib.mla_clear_status.argtypes = [P(MlaPlan), vp, vp]
    lib.mla_strerror.argtypes = [ctypes.c_int]
    lib.mla_strerror.restype = ctypes.c_char_p
    lib.mla_version.argtypes = []
    for name in EXPORTED:
        if name not in ("mla_strerror",):
            getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    return int(x)


def _stream(s) -> Optional[int]:
    if s is None:
        return None
    if hasattr(s, "cuda_stream"):
        return int(s.cuda_stream)
    return int(s)


def _check(fn: str, rc: int) -> None:
    if rc != MLA_OK:
        raise MlaError(fn, rc)


def strerror(code: int) -> str:
    return load().mla_strerror(code).decode()


def version() -> int:
    return load().mla_version()


def make_problem(batch, q_len, num_heads, page_size, num_pages, max_pages_per_seq,
                 kv_dtype=MLA_KV_BF16, topk_width=0, causal=1, sm_scale=1.0 / 16.0,
                 kv_lora_rank=512, rope_dim=64, nope_dim=192, v_head_dim=256) -> MlaProblem:
    return MlaProblem(batch, q_len, num_heads, kv_lora_rank, rope_dim, nope_dim, v_head_dim,
                      page_size, num_pages, max_pages_per_seq, kv_dtype, topk_width, causal,
                      sm_scale)


def _nbytes(buf, given, plan) -> int:
    """Byte size of a device buffer: as given, else a tensor's size, else the
    plan's workspace size (a bare address carries no size)."""
    if given is not None:
        return int(given)
    if hasattr(buf, "numel") and hasattr(buf, "element_size"):
        return int(buf.numel()) * int(buf.element_size())
    return int(plan.workspace_bytes)


def _rows_stride(given, *rows) -> int:
    """Elements between two requests' entries of [batch][stride] arrays: as given, else
    the tensors' last dimension, which it is only where all are packed and equally wide."""
    if given is not None:
        return given
    stride = int(rows[0].shape[-1])
    for t in rows:
        if hasattr(t, "is_contiguous") and (int(t.shape[-1]) != stride or not t.is_contiguous()):
            raise ValueError(f"arrays that are not packed rows of {stride} elements need their stride given")
    return stride


def mla_decode_plan(problem: MlaProblem, seq_lens_host=None, sm_count: int = 152,
                    split_tokens: int = 0) -> MlaPlan:
    plan = MlaPlan()
    ws = ctypes.c_size_t(0)
    arr = None
    if seq_lens_host is not None:
        arr = np.ascontiguousarray(seq_lens_host, dtype=np.int32)
        ptr = arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    else:
        ptr = None
    _check("mla_decode_plan", load().mla_decode_plan(ctypes.byref(problem), ptr, int(sm_count),
                                                     int(split_tokens), ctypes.byref(plan),
                                                     ctypes.byref(ws)))
    assert ws.value == plan.workspace_bytes
    return plan


def mla_q_absorb(plan: MlaPlan, q, w_uk, q_hat, stream=None) -> None:
    """q_hat = [W_UK[h] q[..., :192] || q[..., 192:]] (q bf16 [B*Q][H][256])."""
    _check("mla_q_absorb", load().mla_q_absorb(ctypes.byref(plan), _ptr(q), _ptr(w_uk),
                                               _ptr(q_hat), _stream(stream)))


def mla_decode_run(plan: MlaPlan, q, w_uk, kv_cache, block_table, seq_lens, topk_idx, workspace,
                   o_lat, lse, stream=None, workspace_bytes=None) -> None:
    """The attention pass.  q is the absorbed q_hat (w_uk None) or the
    un-absorbed [q_nope || q_rope] with w_uk.  Split row sets are completed
    by mla_combine."""
    _check("mla_decode_run", load().mla_decode_run(
        ctypes.byref(plan), _ptr(q), _ptr(w_uk), _ptr(kv_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(topk_idx), _ptr(workspace), _nbytes(workspace, workspace_bytes, plan),
        _ptr(o_lat), _ptr(lse), _stream(stream)))


def mla_decode_run_static(plan: MlaPlan, q_hat, kv_cache, block_table, seq_lens, topk_idx,
                          o_lat, lse, status=None, stream=None) -> None:
    """mla_decode_run and the merge without a caller workspace: the scratch is
    the library's fixed 16 MiB device array (for callers that cannot
    allocate)."""
    _check("mla_decode_run_static", load().mla_decode_run_static(
        ctypes.byref(plan), _ptr(q_hat), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
        _ptr(topk_idx), _ptr(o_lat), _ptr(lse), _ptr(status), _stream(stream)))


def mla_combine(plan: MlaPlan, seq_lens, workspace, o_lat, lse, w_uv=None, out=None,
                stream=None, workspace_bytes=None) -> None:
    """Merge split row sets into o_lat / lse; with w_uv also out = W_UV^T o_lat
    (bf16 [B*Q][H][256]) in the same kernel."""
    _check("mla_combine", load().mla_combine(
        ctypes.byref(plan), _ptr(seq_lens), _ptr(workspace),
        _nbytes(workspace, workspace_bytes, plan), _ptr(w_uv), _ptr(o_lat), _ptr(lse), _ptr(out),
        _stream(stream)))


def mla_decode_step(plan: MlaPlan, q, w_uk, kv_cache, block_table, seq_lens, topk_idx, workspace,
                    w_uv, o_lat, lse, out, stream=None, workspace_bytes=None) -> None:
    """A whole decode step, mla_decode_run then mla_combine with W_UV: two
    kernels, the attention pass and then the merge of split row sets inside
    the W_UV projection (a programmatic dependent of the first)."""
    _check("mla_decode_step", load().mla_decode_step(
        ctypes.byref(plan), _ptr(q), _ptr(w_uk), _ptr(kv_cache), _ptr(block_table),
        _ptr(seq_lens), _ptr(topk_idx), _ptr(workspace), _nbytes(workspace, workspace_bytes, plan),
        _ptr(w_uv), _ptr(o_lat), _ptr(lse), _ptr(out), _stream(stream)))


def mla_cache_append(problem: MlaProblem, new_rows, positions, block_table, kv_cache,
                     status=None, stream=None, rope_theta: float = 0.0) -> None:
    """Write row b of new_rows (bf16 [batch][576]) at logical position
    positions[b] of request b (bf16 copy or on-GPU FP8 / FP4 quantisation);
    with rope_theta > 0 its RoPE key is rotated to that position first."""
    _check("mla_cache_append", load().mla_cache_append(
        ctypes.byref(problem), _ptr(new_rows), _ptr(positions), _ptr(block_table),
        float(rope_theta), _ptr(kv_cache), _ptr(status), _stream(stream)))


def mla_selftest_bounded_wait(status, limit_ns: int, waited_ns=None, stream=None) -> None:
    """Launch the bounded-wait self-test: a wait that nothing completes gives
    up after limit_ns and ORs MLA_STATUS_TIMEOUT into the device word status."""
    _check("mla_selftest_bounded_wait", load().mla_selftest_bounded_wait(
        _ptr(status), int(limit_ns), _ptr(waited_ns), _stream(stream)))


def mla_uv_proj(o_lat, w_uv, out, rows: int, num_heads: int, stream=None) -> None:
    _check("mla_uv_proj", load().mla_uv_proj(_ptr(o_lat), _ptr(w_uv), _ptr(out), int(rows),
                                             int(num_heads), _stream(stream)))


def make_norm_problem(rows, cols, dtype=MLA_DTYPE_BF16, out_format=MLA_NORM_OUT_SAME, eps=1e-6,
                      x_stride=None, residual_stride=None, residual_out_stride=None,
                      out_stride=None, scale_stride=None) -> MlaNormProblem:
    """Strides are in elements (scale_stride in bytes) and default to packed rows."""
    s = [cols if v is None else v for v in (x_stride, residual_stride, residual_out_stride,
                                            out_stride)]
    return MlaNormProblem(rows, cols, dtype, out_format, eps, 0, *s,
                          (cols + 31) // 32 if scale_stride is None else scale_stride)


# The layer calls below take a few microseconds on the device for a decode
# step's sizes, less than a call per argument costs here: tensors and torch
# streams are read in place, and anything else (addresses, stream handles, the
# library not yet loaded) goes through _ptr and _stream.  A call falls back
# before it is made: the attribute that is missing is one of its arguments'.
def mla_rms_norm(problem: MlaNormProblem, x, weight, out, residual=None, residual_out=None,
                 scales=None, stream=None) -> None:
    """out = h / sqrt(mean(h^2) + eps) * weight for each row, h = x + residual
    (residual_out receives h); weight None is ones.  An 8-bit out_format writes
    e4m3 codes to out and the scales to scales."""
    try:
        rc = _lib.mla_rms_norm(
            problem, x.data_ptr(), None if residual is None else residual.data_ptr(),
            None if weight is None else weight.data_ptr(),
            None if residual_out is None else residual_out.data_ptr(), out.data_ptr(),
            None if scales is None else scales.data_ptr(),
            None if stream is None else stream.cuda_stream)
    except AttributeError:
        rc = load().mla_rms_norm(problem, _ptr(x), _ptr(residual), _ptr(weight),
                                 _ptr(residual_out), _ptr(out), _ptr(scales), _stream(stream))
    if rc:
        raise MlaError("mla_rms_norm", rc)


def mla_rope_make_plan(config: MlaRopeConfig) -> MlaRopePlan:
    plan = MlaRopePlan()
    _check("mla_rope_make_plan", load().mla_rope_make_plan(ctypes.byref(config), ctypes.byref(plan)))
    return plan


def mla_rope_plan(layout=MLA_ROPE_INTERLEAVED, rope_dim=64, theta=1.0e6,
                  scaling=MLA_ROPE_SCALING_NONE, factor=1.0, original_positions=0,
                  fast_rotations=32.0, slow_rotations=1.0, amplitude=0.0) -> MlaRopePlan:
    """The plan of a rotation: layout, theta and long-context scaling."""
    return mla_rope_make_plan(MlaRopeConfig(layout, rope_dim, scaling, original_positions, theta,
                                            factor, fast_rotations, slow_rotations, amplitude))


def make_rope_problem(tokens, num_heads, head_dim, rope_offset=0, dtype=MLA_DTYPE_BF16,
                      transposed=0, x_token_stride=None, x_head_stride=None,
                      out_token_stride=None, out_head_stride=None) -> MlaRopeProblem:
    """Strides are in elements; x defaults to packed [tokens][num_heads][head_dim]
    and out to x's strides."""
    xh = head_dim if x_head_stride is None else x_head_stride
    xt = num_heads * xh if x_token_stride is None else x_token_stride
    return MlaRopeProblem(tokens, num_heads, head_dim, rope_offset, dtype, transposed, xt, xh,
                          xt if out_token_stride is None else out_token_stride,
                          xh if out_head_stride is None else out_head_stride)


def mla_rope(problem: MlaRopeProblem, plan: MlaRopePlan, x, positions, out=None,
             stream=None) -> None:
    """Rotate part of every head of token t to positions[t] (in place without
    an out); a negative position leaves the token's out as it was."""
    try:
        x = x.data_ptr()
        rc = _lib.mla_rope(problem, plan, x, positions.data_ptr(),
                           x if out is None else out.data_ptr(),
                           None if stream is None else stream.cuda_stream)
    except AttributeError:
        x = _ptr(x)
        rc = load().mla_rope(problem, plan, x, _ptr(positions), x if out is None else _ptr(out),
                             _stream(stream))
    if rc:
        raise MlaError("mla_rope", rc)


def mla_cache_append_tokens(problem: MlaProblem, tokens: int, rows, positions, block_table,
                            kv_cache, requests=None, row_stride: int = 576, norm_weight=None,
                            norm_eps: float = 1e-6, rope: Optional[MlaRopePlan] = None,
                            status=None, stream=None) -> None:
    """Write row t of rows (bf16, row_stride elements apart) at position
    positions[t] of request requests[t] (None: tokens / batch consecutive rows
    per request), its latent normed with norm_weight and its key rotated by
    rope where given."""
    try:
        rc = _lib.mla_cache_append_tokens(
            problem, tokens, rows.data_ptr(), row_stride, positions.data_ptr(),
            None if requests is None else requests.data_ptr(), block_table.data_ptr(),
            None if norm_weight is None else norm_weight.data_ptr(), norm_eps, rope,
            kv_cache.data_ptr(), None if status is None else status.data_ptr(),
            None if stream is None else stream.cuda_stream)
    except AttributeError:
        rc = load().mla_cache_append_tokens(
            problem, tokens, _ptr(rows), row_stride, _ptr(positions), _ptr(requests),
            _ptr(block_table), _ptr(norm_weight), norm_eps, rope, _ptr(kv_cache), _ptr(status),
            _stream(stream))
    if rc:
        raise MlaError("mla_cache_append_tokens", rc)


def mla_cache_gather(problem: MlaProblem, tokens: int, kv_cache, positions, block_table, out,
                     requests=None, out_stride: int = 576, status=None, stream=None) -> None:
    """The cached row at position positions[t] of request requests[t] as bf16
    row t of out (out_stride elements apart)."""
    try:
        rc = _lib.mla_cache_gather(
            problem, tokens, kv_cache.data_ptr(), positions.data_ptr(),
            None if requests is None else requests.data_ptr(), block_table.data_ptr(),
            out.data_ptr(), out_stride, None if status is None else status.data_ptr(),
            None if stream is None else stream.cuda_stream)
    except AttributeError:
        rc = load().mla_cache_gather(
            problem, tokens, _ptr(kv_cache), _ptr(positions), _ptr(requests), _ptr(block_table),
            _ptr(out), out_stride, _ptr(status), _stream(stream))
    if rc:
        raise MlaError("mla_cache_gather", rc)


def mla_chunk_make_plan(problem: MlaProblem, tokens: int, context_tokens: int = 0,
                        sm_count: int = 152) -> MlaChunkPlan:
    """The plan of mla_chunk_attend and mla_cache_weights for `tokens` query
    tokens; context_tokens: the most cached rows of one call (quantised caches)."""
    plan, ws = MlaChunkPlan(), ctypes.c_size_t(0)
    _check("mla_chunk_make_plan", load().mla_chunk_make_plan(
        ctypes.byref(problem), int(tokens), int(context_tokens), int(sm_count), ctypes.byref(plan),
        ctypes.byref(ws)))
    return plan


def mla_chunk_attend(plan: MlaChunkPlan, q_hat, query_starts, kv_cache, block_table, seq_lens,
                     workspace, o_lat, lse, status=None, stream=None, workspace_bytes=None) -> None:
    """Causal attention of the new tokens query_starts[b] .. query_starts[b + 1]
    of each request over its cached rows (its own among them): o_lat bf16
    [tokens][H][512], lse f32 [tokens][H]."""
    size = _nbytes(workspace, workspace_bytes, plan)
    try:
        rc = _lib.mla_chunk_attend(
            plan, q_hat.data_ptr(), query_starts.data_ptr(), kv_cache.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), workspace.data_ptr(), size,
            o_lat.data_ptr(), lse.data_ptr(), None if status is None else status.data_ptr(),
            None if stream is None else stream.cuda_stream)
    except AttributeError:
        rc = load().mla_chunk_attend(
            plan, _ptr(q_hat), _ptr(query_starts), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
            _ptr(workspace), size, _ptr(o_lat), _ptr(lse), _ptr(status), _stream(stream))
    if rc:
        raise MlaError("mla_chunk_attend", rc)


def mla_cache_weights(plan: MlaChunkPlan, q_hat, lse, query_starts, kv_cache, block_table, seq_lens,
                      workspace, weights_out, weights_in=None, stride=None, status=None, stream=None,
                      workspace_bytes=None) -> None:
    """weights_out[b][t] = weights_in[b][t] (None: 0) + the weight that request
    b's queries give to its cached row t, f32 [batch][stride] (stride None: packed
    tensors', their last dimension)."""
    size = _nbytes(workspace, workspace_bytes, plan)
    stride = _rows_stride(stride, weights_out, weights_in)
    try:
        rc = _lib.mla_cache_weights(
            plan, q_hat.data_ptr(), lse.data_ptr(), query_starts.data_ptr(), kv_cache.data_ptr(),
            block_table.data_ptr(), seq_lens.data_ptr(), workspace.data_ptr(), size,
            None if weights_in is None else weights_in.data_ptr(), weights_out.data_ptr(), stride,
            None if status is None else status.data_ptr(),
            None if stream is None else stream.cuda_stream)
    except AttributeError:
        rc = load().mla_cache_weights(
            plan, _ptr(q_hat), _ptr(lse), _ptr(query_starts), _ptr(kv_cache), _ptr(block_table),
            _ptr(seq_lens), _ptr(workspace), size, _ptr(weights_in), _ptr(weights_out), stride,
            _ptr(status), _stream(stream))
    if rc:
        raise MlaError("mla_cache_weights", rc)


def mla_evict_make_plan(problem: MlaProblem, budget: int, sinks: int = 0, recent: int = 0) -> MlaEvictPlan:
    """The plan of mla_cache_evict: rows that a request keeps, and which positions
    are kept before all others (the first `sinks`, the last `recent`)."""
    plan, ws = MlaEvictPlan(), ctypes.c_size_t(0)
    _check("mla_evict_make_plan", load().mla_evict_make_plan(
        ctypes.byref(problem), int(budget), int(sinks), int(recent), ctypes.byref(plan), ctypes.byref(ws)))
    return plan


def mla_cache_evict(plan: MlaEvictPlan, kv_cache, block_table, seq_lens, weights, positions,
                    workspace, seq_lens_out=None, weights_out=None, positions_out=None, stride=None,
                    status=None, stream=None, workspace_bytes=None) -> None:
    """Cut each request's cache to the plan's budget: kept rows behind it move
    into the slots below that became free.  Outputs that are not given are their
    inputs; weights and positions are [batch][stride] (stride None: as in
    mla_cache_weights)."""
    size = _nbytes(workspace, workspace_bytes, plan)
    stride = _rows_stride(stride, weights, positions, weights_out, positions_out)
    seq_lens_out = seq_lens if seq_lens_out is None else seq_lens_out
    weights_out = weights if weights_out is None else weights_out
    positions_out = positions if positions_out is None else positions_out
    try:
        rc = _lib.mla_cache_evict(
            plan, kv_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), weights.data_ptr(),
            positions.data_ptr(), stride, workspace.data_ptr(), size, seq_lens_out.data_ptr(),
            weights_out.data_ptr(), positions_out.data_ptr(),
            None if status is None else status.data_ptr(),
            None if stream is None else stream.cuda_stream)
    except AttributeError:
        rc = load().mla_cache_evict(
            plan, _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), _ptr(weights), _ptr(positions),
            stride, _ptr(workspace), size, _ptr(seq_lens_out), _ptr(weights_out),
            _ptr(positions_out), _ptr(status), _stream(stream))
    if rc:
        raise MlaError("mla_cache_evict", rc)


def mla_get_status(plan: MlaPlan, workspace, stream=None) -> int:
    bits = ctypes.c_uint32(0)
    _check("mla_get_status", load().mla_get_status(ctypes.byref(plan), _ptr(workspace),
                                                   ctypes.byref(bits), _stream(stream)))
    return int(bits.value)


def mla_clear_status(plan: MlaPlan, workspace, stream=None) -> None:
    _check("mla_clear_status", load().mla_clear_status(ctypes.byref(plan), _ptr(workspace),
                                                       _stream(stream)))
