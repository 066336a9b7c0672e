"""libql Python binding: q4_0 dense-transformer decode on one GB300.

Thin wrappers with the names of the C entry points (``include/ql.h``). Device buffers are
``torch`` CUDA tensors (PyTorch provides memory and streams only); every computation runs in
the CUDA library ``_build/libql.so``. Each wrapper raises :class:`QLError` on a non-zero
status.
"""
from __future__ import annotations

import ctypes

from ._lib import (QLError, QL_OK, QL_EINVAL, QL_ENOMEM, QL_ECUDA, QL_EPOOL, QL_ERANGE,
                   QL_EDEVICE, QL_ESTATE, QL_DTYPE_F32, QL_DTYPE_F16, QL_EPI_NONE,
                   QL_EPI_ADD_RESIDUAL, QL_EPI_SILU_MUL, QL_STEP_AUTO, QL_STEP_LAUNCHES,
                   QL_STEP_PERSISTENT, QL_OPT_STEP_KERNEL, QL_OPT_BARRIER_TIMEOUT_NS,
                   QL_OPT_TEST_BARRIER_EXTRA, QL_OPT_STEP_TRACE, QL_OPT_MERGE_TRACE, QL_BATCHED_MMA_SYNC, QL_BATCHED_TCGEN05,
                   QL_GEMV_ACT_INT16, QL_GEMV_ACT_INT8, QL_KV_F16, QL_KV_Q8_0_Q5_1, QL_KV_Q4_1,
                   QL_ATTN_MERGE_TICKET, QL_ATTN_MERGE_CLUSTER,
                   Q4Matrix, LayerDesc, ModelDesc,
                   StepArgs, Sampling, SIGNATURES, LIB_PATH, lib, check, check_array, check_device, check_pool, device_index,
                   check_sampling, ptr, stream_ptr)

__all__ = [
    "QLError", "lib", "ql_q4_0_pack", "ql_q4_0_unpack", "ql_q4_0_pack_device", "ql_gemv_q4_0",
    "ql_q4_0_stream_bytes", "ql_q4_0_stream_pack", "ql_gemv_q4_0_stream",
    "ql_gemv_q4_0_stream_workspace_bytes", "ql_gemm_q4_0_stream", "ql_set_batched_gemv_form", "ql_set_gemv_activation_form",
    "ql_paged_attn_workspace_bytes", "ql_paged_attn_decode", "ql_paged_attn_decode_noalloc",
    "ql_paged_attn_chunk_workspace_bytes", "ql_paged_attn_chunk",
    "ql_kvq_record_bytes", "ql_kvq_write", "ql_paged_attn_decode_kvq",
    "ql_kv4_record_bytes", "ql_kv4_write", "ql_kv4_read", "ql_paged_attn_kv4_workspace_bytes",
    "ql_paged_attn_decode_kv4", "ql_mla_append", "ql_mla_decode_workspace_bytes", "ql_mla_attn_decode",
    "ql_mla_chunk_workspace_bytes", "ql_mla_attn_chunk", "ql_sample",
    "ql_set_attn_merge_form", "ql_paged_attn_merge_form",
    "ql_kv_q8_0_row_bytes", "ql_kv_q5_1_row_bytes", "ql_kv_quantize_q8_0", "ql_kv_dequantize_q8_0",
    "ql_kv_quantize_q5_1", "ql_kv_dequantize_q5_1", "ql_kv_quantize_device", "ql_kv_dequantize_device",
    "ql_fused_norm_rope",
    "ql_rope_tables", "ql_check_device_error", "BlockPool", "SIGNATURES",
]


def ql_q4_0_pack(w, scales, quants):
    """Host codec: ``w`` f32 [rows, cols] numpy -> ``scales`` u16 [rows, cols/32], ``quants`` u8."""
    rows, cols = w.shape
    check(lib().ql_q4_0_pack(w.ctypes.data, rows, cols, scales.ctypes.data, quants.ctypes.data))


def ql_q4_0_unpack(scales, quants, w):
    rows, cols = w.shape
    check(lib().ql_q4_0_unpack(scales.ctypes.data, quants.ctypes.data, rows, cols, w.ctypes.data))


def ql_q4_0_pack_device(w, scales, quants, stream=None):
    rows, cols = w.shape
    check(lib().ql_q4_0_pack_device(ptr(w), rows, cols, ptr(scales), ptr(quants), stream_ptr(stream)))


def ql_gemv_q4_0(scales, quants, rows, cols, x, batch, y, y_dtype=QL_DTYPE_F32,
                 epilogue=QL_EPI_NONE, residual=None, stream=None):
    check(lib().ql_gemv_q4_0(ptr(scales), ptr(quants), rows, cols, ptr(x), batch, ptr(y), y_dtype,
                             epilogue, ptr(residual), stream_ptr(stream)))


def ql_q4_0_stream_bytes(rows, cols, silu=0):
    return int(lib().ql_q4_0_stream_bytes(rows, cols, silu))


def ql_q4_0_stream_pack(scales, quants, rows, cols, silu, out, stream=None):
    check(lib().ql_q4_0_stream_pack(ptr(scales), ptr(quants), rows, cols, silu, ptr(out), stream_ptr(stream)))


def ql_gemv_q4_0_stream_workspace_bytes(rows, cols, silu=0):
    return int(lib().ql_gemv_q4_0_stream_workspace_bytes(rows, cols, silu))


def ql_set_batched_gemv_form(form):
    """Tensor-core form of the batch 3-32 GEMV for this process; returns the previous form."""
    rc = int(lib().ql_set_batched_gemv_form(form))
    if rc < 0:
        check(rc)
    return rc


def ql_set_gemv_activation_form(form):
    """Activation form of the batch 1-2 GEMV for this process; returns the previous form."""
    rc = int(lib().ql_set_gemv_activation_form(form))
    if rc < 0:
        check(rc)
    return rc


def ql_set_attn_merge_form(form):
    """How attention merges its context splits, for this process; returns the previous form."""
    rc = int(lib().ql_set_attn_merge_form(form))
    if rc < 0:
        check(rc)
    return rc


def ql_paged_attn_merge_form(batch, n_heads, n_kv_heads, head_dim, max_blocks_per_seq):
    """The merge form an attention launch of this shape takes on the current device."""
    rc = int(lib().ql_paged_attn_merge_form(batch, n_heads, n_kv_heads, head_dim, max_blocks_per_seq))
    if rc < 0:
        check(rc)
    return rc


def ql_kv_q8_0_row_bytes(dim):
    return int(lib().ql_kv_q8_0_row_bytes(dim))


def ql_kv_q5_1_row_bytes(dim):
    return int(lib().ql_kv_q5_1_row_bytes(dim))


def _kv_quantize(fn, row_bytes, x):
    import numpy as np
    x = np.ascontiguousarray(x, dtype=np.float32)
    rows, dim = x.shape
    out = np.zeros((rows, row_bytes(dim)), dtype=np.uint8)
    check(fn(x.ctypes.data, rows, dim, out.ctypes.data))
    return out


def _kv_dequantize(fn, data, dim):
    import numpy as np
    data = np.ascontiguousarray(data, dtype=np.uint8)
    x = np.zeros((data.shape[0], dim), dtype=np.float32)
    check(fn(data.ctypes.data, data.shape[0], dim, x.ctypes.data))
    return x


def ql_kv_quantize_q8_0(x):
    """Host codec: f32 rows [n, dim] numpy -> q8_0 bytes [n, ql_kv_q8_0_row_bytes(dim)]."""
    return _kv_quantize(lib().ql_kv_quantize_q8_0, ql_kv_q8_0_row_bytes, x)


def ql_kv_dequantize_q8_0(data, dim):
    return _kv_dequantize(lib().ql_kv_dequantize_q8_0, data, dim)


def ql_kv_quantize_q5_1(x):
    """Host codec: f32 rows [n, dim] numpy -> q5_1 bytes [n, ql_kv_q5_1_row_bytes(dim)]."""
    return _kv_quantize(lib().ql_kv_quantize_q5_1, ql_kv_q5_1_row_bytes, x)


def ql_kv_dequantize_q5_1(data, dim):
    return _kv_dequantize(lib().ql_kv_dequantize_q5_1, data, dim)


def ql_kv_quantize_device(x, out, fmt="q8_0", stream=None):
    """Device codec: ``x`` f32 [rows, dim] CUDA tensor -> ``out`` uint8 [rows, row bytes]."""
    fn = lib().ql_kv_quantize_q8_0_device if fmt == "q8_0" else lib().ql_kv_quantize_q5_1_device
    check(fn(ptr(x), x.shape[0], x.shape[1], ptr(out), stream_ptr(stream)))


def ql_kv_dequantize_device(data, x, fmt="q8_0", stream=None):
    """Device codec: ``data`` uint8 [rows, row bytes] -> ``x`` f32 [rows, dim] CUDA tensor."""
    fn = lib().ql_kv_dequantize_q8_0_device if fmt == "q8_0" else lib().ql_kv_dequantize_q5_1_device
    check(fn(ptr(data), x.shape[0], x.shape[1], ptr(x), stream_ptr(stream)))


def ql_gemv_q4_0_stream(w_stream, rows, cols, x, batch, y, epilogue=QL_EPI_NONE, workspace=None, stream=None):
    """``workspace``: a zero-filled device byte tensor of ql_gemv_q4_0_stream_workspace_bytes
    (batch 3-32; None at batch 1-2)."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(lib().ql_gemv_q4_0_stream(ptr(w_stream), rows, cols, ptr(x), batch, ptr(y), epilogue,
                                    ptr(workspace), nbytes, stream_ptr(stream)))


def ql_gemm_q4_0_stream(w_stream, rows, cols, x, n_tokens, y, epilogue=QL_EPI_NONE, stream=None):
    """The prompt-chunk GEMM over the tile stream copy: ``x`` f16 [n_tokens, cols]."""
    check(lib().ql_gemm_q4_0_stream(ptr(w_stream), rows, cols, ptr(x), n_tokens, ptr(y), epilogue,
                                    stream_ptr(stream)))


def ql_paged_attn_chunk_workspace_bytes(n_tokens, n_heads, n_kv_heads, head_dim):
    return int(lib().ql_paged_attn_chunk_workspace_bytes(n_tokens, n_heads, n_kv_heads, head_dim))


def ql_paged_attn_chunk(q, k_pool, v_pool, block_table, position, n_tokens, n_heads, n_kv_heads, head_dim,
                        block_size, max_blocks_per_seq, num_blocks, scale, out, workspace, stream=None):
    """Causal attention of a prefill chunk: ``q`` f16 [n_tokens][n_heads][head_dim] at positions
    ``position[0] + t`` (int32 [1] device) over the sequence's ``block_table``."""
    check(lib().ql_paged_attn_chunk(ptr(q), ptr(k_pool), ptr(v_pool), ptr(block_table), ptr(position), n_tokens,
                                    n_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                                    scale, ptr(out), ptr(workspace), workspace.numel() * workspace.element_size(),
                                    stream_ptr(stream)))


def ql_paged_attn_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq):
    return int(lib().ql_paged_attn_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, block_size,
                                                   max_blocks_per_seq))


def ql_paged_attn_decode(q, k_pool, v_pool, block_tables, context_lens, batch, n_heads, n_kv_heads,
                         head_dim, block_size, max_blocks_per_seq, num_blocks, scale, out,
                         workspace, stream=None):
    check(lib().ql_paged_attn_decode(ptr(q), ptr(k_pool), ptr(v_pool), ptr(block_tables),
                                     ptr(context_lens), batch, n_heads, n_kv_heads, head_dim,
                                     block_size, max_blocks_per_seq, num_blocks, scale, ptr(out),
                                     ptr(workspace), workspace.numel() * workspace.element_size(),
                                     stream_ptr(stream)))


def ql_kvq_record_bytes(head_dim):
    return int(lib().ql_kvq_record_bytes(head_dim))


def ql_kvq_write(k, v, slots, n_kv_heads, head_dim, pool, num_blocks, stream=None):
    """Quantise f32 rows ``k``, ``v`` [n, n_kv, hd] into one layer's pool at physical ``slots``
    (int64 [n], block * 16 + offset)."""
    check(lib().ql_kvq_write(ptr(k), ptr(v), ptr(slots), slots.numel(), n_kv_heads, head_dim, ptr(pool),
                             num_blocks, stream_ptr(stream)))


def ql_paged_attn_decode_kvq(q, pool, block_tables, context_lens, batch, n_heads, n_kv_heads, head_dim,
                             block_size, max_blocks_per_seq, num_blocks, scale, out, workspace, stream=None):
    check(lib().ql_paged_attn_decode_kvq(ptr(q), ptr(pool), ptr(block_tables), ptr(context_lens), batch, n_heads,
                                         n_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks, scale,
                                         ptr(out), ptr(workspace), workspace.numel() * workspace.element_size(),
                                         stream_ptr(stream)))


def _dtype_of(name, a, b=None):
    """QL_DTYPE_* of tensors that have to share one type."""
    t = a.dtype
    if b is None or b.dtype == t:
        code = _CODES.get(t)
        if code is None:
            code = _DTYPES.get(str(t))
        if code is not None:
            _CODES[t] = code
            return code
    raise QLError(QL_EINVAL, f"{name}: tensors must be all float32 or all float16")


_DTYPES = {"torch.float32": QL_DTYPE_F32, "torch.float16": QL_DTYPE_F16}
_CODES = {}   # by the type itself, as they come


def _row_stride(name, t, n, n_kv_heads, head_dim):
    """Row stride in elements of a [n, n_kv_heads, head_dim] (or [n, n_kv_heads * head_dim]) tensor whose rows are
    contiguous."""
    shape, strides = t.shape, t.stride()
    if shape == (n, n_kv_heads, head_dim):
        ok = strides[2] == 1 and (strides[1] == head_dim or n_kv_heads == 1)
    else:
        ok = shape == (n, n_kv_heads * head_dim) and strides[1] == 1
    if not ok:
        raise QLError(QL_EINVAL, f"{name}: need {n} rows of {n_kv_heads} x {head_dim} with contiguous heads, got "
                                 f"{tuple(shape)} with strides {tuple(strides)}")
    return strides[0]


def ql_kv4_record_bytes(head_dim):
    return int(lib().ql_kv4_record_bytes(head_dim))


_types = None   # float16, int32, int64


def _torch_types():
    global _types
    import torch
    _types = (torch.float16, torch.int32, torch.int64)
    return _types


def _kv4_rows(name, k, v, slots, n_kv_heads, head_dim, pool, num_blocks):
    """The tensors of a write or a read checked: the number of rows, k's and v's type and row strides, the pool's address."""
    here, size = device_index(), num_blocks * n_kv_heads * 20 * head_dim
    address = pool
    if pool.__class__ is not int:
        if pool is None or pool.get_device() != here or pool.nbytes < size or not pool.is_contiguous():
            check_pool(name, pool, size)
            check_device(name, pool)
        address = pool.data_ptr()
    n = slots.numel()
    if (k.get_device() != here or v.get_device() != here or slots.get_device() != here
            or slots.dtype is not (_types or _torch_types())[2] or not slots.is_contiguous()):
        check_array(name, "slots", slots, "torch.int64", 0)
        check_device(name, k, v, slots)
    return (n, _dtype_of(name, k, v), _row_stride(name, k, n, n_kv_heads, head_dim), _row_stride(name, v, n, n_kv_heads, head_dim),
            address)


def ql_kv4_write(k, v, slots, n_kv_heads, head_dim, pool, num_blocks, stream=None):
    """Quantise rows ``k``, ``v`` (f32 or f16 [n, n_kv, hd], rows may be strided) into one layer's 4-bit
    pool at physical ``slots`` (int64 [n], block * 16 + offset; -1: leave the row out)."""
    n, kind, ks, vs, address = _kv4_rows("ql_kv4_write", k, v, slots, n_kv_heads, head_dim, pool, num_blocks)
    status = lib().ql_kv4_write(k.data_ptr(), v.data_ptr(), kind, ks, vs, slots.data_ptr(), n, n_kv_heads, head_dim, address,
                                num_blocks, stream_ptr(stream))
    if status:
        check(status)


def ql_kv4_read(pool, slots, n_kv_heads, head_dim, num_blocks, k, v, stream=None):
    """The values of ``slots`` read back into ``k``, ``v`` (f32 or f16 [n, n_kv, hd], rows may be strided)."""
    n, kind, ks, vs, address = _kv4_rows("ql_kv4_read", k, v, slots, n_kv_heads, head_dim, pool, num_blocks)
    status = lib().ql_kv4_read(address, slots.data_ptr(), n, n_kv_heads, head_dim, num_blocks, k.data_ptr(), v.data_ptr(), kind,
                               ks, vs, stream_ptr(stream))
    if status:
        check(status)


def ql_paged_attn_kv4_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_blocks_per_seq):
    return int(lib().ql_paged_attn_kv4_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_blocks_per_seq))


def ql_paged_attn_decode_kv4(q, pool, block_tables, context_lens, batch, n_heads, n_kv_heads, head_dim,
                             block_size, max_blocks_per_seq, num_blocks, scale, out, workspace, stream=None):
    """Single-token attention over a 4-bit pool: ``q``, ``out`` f16 [batch, n_heads, head_dim], ``block_tables`` int32
    [batch, max_blocks_per_seq], ``context_lens`` int32 [batch], all contiguous; ``workspace``: a zero-filled byte tensor."""
    name = "ql_paged_attn_decode_kv4"
    half, whole, _ = _types or _torch_types()
    here, rows, size = device_index(), batch * n_heads * head_dim, num_blocks * n_kv_heads * 20 * head_dim
    entries = batch * max_blocks_per_seq
    for t, kind, n in ((q, half, rows), (out, half, rows), (block_tables, whole, entries), (context_lens, whole, batch)):
        if t.__class__ is not int and (t is None or t.dtype is not kind or t.numel() < n or t.get_device() != here
                                       or not t.is_contiguous()):
            for what, x, dtype, m in (("q", q, "torch.float16", rows), ("out", out, "torch.float16", rows),
                                      ("block_tables", block_tables, "torch.int32", entries),
                                      ("context_lens", context_lens, "torch.int32", batch)):
                if not isinstance(x, int):
                    check_array(name, what, x, dtype, m)
            check_device(name, q, out, block_tables, context_lens)
            break
    if pool.__class__ is not int and (pool is None or pool.nbytes < size or pool.get_device() != here or not pool.is_contiguous()):
        check_pool(name, pool, size)
        check_device(name, pool)
    if workspace.get_device() != here or not workspace.is_contiguous():
        check_device(name, workspace)
        raise QLError(QL_EINVAL, f"{name}: the workspace must be contiguous")
    status = lib().ql_paged_attn_decode_kv4(ptr(q), ptr(pool), ptr(block_tables), ptr(context_lens), batch, n_heads, n_kv_heads,
                                            head_dim, block_size, max_blocks_per_seq, num_blocks, scale, ptr(out),
                                            workspace.data_ptr(), workspace.nbytes, stream_ptr(stream))
    if status:
        check(status)


def ql_mla_append(q, kv, norm_w, cos_t, sin_t, positions, slots, eps, n_heads, head_dim, rank, rope_dim, q_out, pool, num_blocks,
                  max_position, stream=None):
    """Latent rows ``kv`` (f32 or f16 [n, rank + rope_dim], rows may be strided) normalised and rotated into the paged ``pool`` (f16) at
    physical ``slots`` (int64 [n], block * 16 + offset; -1: leave the row out), queries ``q`` ([n, n_heads, head_dim + rope_dim] of the same
    type, or None) rotated into ``q_out`` (f16, contiguous); ``positions`` int32 [n], the tables f32 [max_position, rope_dim / 2]. Pairs of the
    rotation are (j, j + rope_dim / 2): projections whose pairs lie next to each other have their rows reordered first."""
    name = "ql_mla_append"
    half, whole, long = _types or _torch_types()
    here, row, width = device_index(), rank + rope_dim, head_dim + rope_dim
    n, turns, kind = slots.numel(), max_position * rope_dim // 2, norm_w.dtype
    if not (norm_w.get_device() == cos_t.get_device() == sin_t.get_device() == positions.get_device() == slots.get_device()
            == pool.get_device() == kv.get_device() == here and _DTYPES.get(str(kind)) == QL_DTYPE_F32
            and cos_t.dtype is kind and sin_t.dtype is kind and positions.dtype is whole and slots.dtype is long and pool.dtype is half
            and norm_w.numel() >= rank and cos_t.numel() >= turns and sin_t.numel() >= turns and positions.numel() >= n
            and pool.numel() >= num_blocks * 16 * row and norm_w.is_contiguous() and cos_t.is_contiguous() and sin_t.is_contiguous()
            and positions.is_contiguous() and slots.is_contiguous() and pool.is_contiguous()):
        for what, t, dtype, size in (("norm_w", norm_w, "torch.float32", rank), ("cos_t", cos_t, "torch.float32", turns),
                                     ("sin_t", sin_t, "torch.float32", turns), ("positions", positions, "torch.int32", n),
                                     ("slots", slots, "torch.int64", n), ("pool", pool, "torch.float16", num_blocks * 16 * row)):
            check_array(name, what, t, dtype, size)
        check_device(name, norm_w, cos_t, sin_t, positions, slots, pool, kv)
    q_at = out_at = None
    q_stride = 0
    if q is not None and q_out is not None:
        if not (q.get_device() == q_out.get_device() == here and q_out.dtype is half and q_out.numel() >= n * n_heads * width
                and q_out.is_contiguous()):
            check_array(name, "q_out", q_out, "torch.float16", n * n_heads * width)
            check_device(name, q, q_out)
        q_at, out_at, q_stride = q.data_ptr(), q_out.data_ptr(), _row_stride(name, q, n, n_heads, width)
    elif q is not q_out:
        raise QLError(QL_EINVAL, f"{name}: q and q_out come together")
    dtype, kv_stride = _dtype_of(name, kv, q), _row_stride(name, kv, n, 1, row)
    status = lib().ql_mla_append(q_at, kv.data_ptr(), dtype, q_stride, kv_stride, norm_w.data_ptr(), cos_t.data_ptr(), sin_t.data_ptr(),
                                 positions.data_ptr(), slots.data_ptr(), eps, n, n_heads, head_dim, rank, rope_dim, out_at, pool.data_ptr(),
                                 num_blocks, max_position, stream_ptr(stream))
    if status:
        check(status)


def _mla_tensors(name, q, w_kv, pool, table, lens, rows, tables, n_lens, n_heads, head_dim, rank, rope_dim, max_blocks_per_seq,
                 num_blocks, out, workspace):
    """The tensors of a latent attention checked."""
    half, whole, _ = _types or _torch_types()
    here = device_index()
    n_q, n_w, n_pool = rows * n_heads * (head_dim + rope_dim), n_heads * 2 * head_dim * rank, num_blocks * 16 * (rank + rope_dim)
    n_table, n_out = tables * max_blocks_per_seq, rows * n_heads * head_dim
    if not (q.get_device() == w_kv.get_device() == pool.get_device() == table.get_device() == lens.get_device() == out.get_device()
            == workspace.get_device() == here and q.dtype is half and w_kv.dtype is half and pool.dtype is half and out.dtype is half
            and table.dtype is whole and lens.dtype is whole and q.numel() >= n_q and w_kv.numel() >= n_w and pool.numel() >= n_pool
            and table.numel() >= n_table and lens.numel() >= n_lens and out.numel() >= n_out and q.is_contiguous() and w_kv.is_contiguous()
            and pool.is_contiguous() and table.is_contiguous() and lens.is_contiguous() and out.is_contiguous() and workspace.is_contiguous()):
        for what, t, dtype, size in (("q", q, "torch.float16", n_q), ("w_kv", w_kv, "torch.float16", n_w), ("pool", pool, "torch.float16", n_pool),
                                     ("the table", table, "torch.int32", n_table), ("the lengths", lens, "torch.int32", n_lens),
                                     ("out", out, "torch.float16", n_out)):
            check_array(name, what, t, dtype, size)
        check_device(name, q, w_kv, pool, table, lens, out, workspace)
        raise QLError(QL_EINVAL, f"{name}: the workspace must be contiguous")


def ql_mla_decode_workspace_bytes(batch, n_heads, head_dim, rank, max_blocks_per_seq):
    return int(lib().ql_mla_decode_workspace_bytes(batch, n_heads, head_dim, rank, max_blocks_per_seq))


def ql_mla_attn_decode(q, w_kv, pool, block_tables, context_lens, batch, n_heads, head_dim, rank, rope_dim, block_size,
                       max_blocks_per_seq, num_blocks, scale, out, workspace, stream=None):
    """Single-token latent attention over the paged pool of ql_mla_append: ``q`` f16 [batch, n_heads, head_dim + rope_dim], ``w_kv`` f16
    [n_heads, 2 head_dim, rank], ``block_tables`` int32 [batch, max_blocks_per_seq], ``context_lens`` int32 [batch], ``out`` f16
    [batch, n_heads, head_dim], all contiguous; ``workspace``: a byte tensor of ql_mla_decode_workspace_bytes, any contents."""
    _mla_tensors("ql_mla_attn_decode", q, w_kv, pool, block_tables, context_lens, batch, batch, batch, n_heads, head_dim, rank, rope_dim,
                 max_blocks_per_seq, num_blocks, out, workspace)
    status = lib().ql_mla_attn_decode(q.data_ptr(), w_kv.data_ptr(), pool.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
                                      batch, n_heads, head_dim, rank, rope_dim, block_size, max_blocks_per_seq, num_blocks, scale,
                                      out.data_ptr(), workspace.data_ptr(), workspace.nbytes, stream_ptr(stream))
    if status:
        check(status)


def ql_mla_chunk_workspace_bytes(n_tokens, n_heads, head_dim, rank, max_blocks_per_seq):
    return int(lib().ql_mla_chunk_workspace_bytes(n_tokens, n_heads, head_dim, rank, max_blocks_per_seq))


def ql_mla_attn_chunk(q, w_kv, pool, block_table, position, n_tokens, n_heads, head_dim, rank, rope_dim, block_size,
                      max_blocks_per_seq, num_blocks, scale, out, workspace, stream=None):
    """Causal latent attention of a prompt chunk at positions ``position[0] + i`` (int32 [1] device) over the sequence's ``block_table``:
    ``q`` f16 [n_tokens, n_heads, head_dim + rope_dim], ``out`` f16 [n_tokens, n_heads, head_dim]; the rest as for ql_mla_attn_decode,
    ``workspace`` of ql_mla_chunk_workspace_bytes."""
    _mla_tensors("ql_mla_attn_chunk", q, w_kv, pool, block_table, position, n_tokens, 1, 1, n_heads, head_dim, rank, rope_dim,
                 max_blocks_per_seq, num_blocks, out, workspace)
    status = lib().ql_mla_attn_chunk(q.data_ptr(), w_kv.data_ptr(), pool.data_ptr(), block_table.data_ptr(), position.data_ptr(),
                                     n_tokens, n_heads, head_dim, rank, rope_dim, block_size, max_blocks_per_seq, num_blocks, scale,
                                     out.data_ptr(), workspace.data_ptr(), workspace.nbytes, stream_ptr(stream))
    if status:
        check(status)


def ql_sample(logits, uniform, tokens, temperature=None, top_k=None, top_p=None, min_p=None, probs=None,
              active=None, stream=None):
    """Draw ``tokens`` (int32 [batch]) from ``logits`` (f32 or f16 [batch, vocab], rows may be strided) with one
    ``uniform`` number (f32 [batch]) a row; the filters are device tensors [batch] (``top_k`` int32, the others
    f32) or None. ``probs`` (f32 [batch]): the drawn tokens' probabilities."""
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise QLError(QL_EINVAL, "ql_sample: logits must be [batch, vocab] with contiguous rows")
    B, V = logits.shape
    check_array("ql_sample", "uniform", uniform, "torch.float32", B)
    check_array("ql_sample", "tokens", tokens, "torch.int32", B)
    real, whole = uniform.dtype, tokens.dtype
    for t, kind in ((temperature, real), (top_k, whole), (top_p, real), (min_p, real), (probs, real), (active, whole)):
        if t is not None and (t.dtype is not kind or t.numel() < B or not t.is_contiguous()):
            check_sampling("ql_sample", B, uniform, temperature, top_k, top_p, min_p)
            check_array("ql_sample", "probs", probs, "torch.float32", B)
            check_array("ql_sample", "active", active, "torch.int32", B)
    check_device("ql_sample", logits, uniform, tokens, temperature, top_k, top_p, min_p, probs, active)
    status = lib().ql_sample(logits.data_ptr(), _dtype_of("ql_sample", logits), logits.stride(0), B, V, ptr(temperature),
                             ptr(top_k), ptr(top_p), ptr(min_p), uniform.data_ptr(), ptr(active), tokens.data_ptr(),
                             ptr(probs), stream_ptr(stream))
    if status:
        check(status)


def ql_paged_attn_decode_noalloc(q, k_pool, v_pool, block_tables, context_lens, batch, n_heads,
                                 n_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks,
                                 scale, out, stream=None):
    """Attention whose split-K scratch is the library's fixed 8 MiB device array (no workspace
    argument, no device allocation); see include/ql.h for its limits."""
    check(lib().ql_paged_attn_decode_noalloc(ptr(q), ptr(k_pool), ptr(v_pool), ptr(block_tables),
                                             ptr(context_lens), batch, n_heads, n_kv_heads,
                                             head_dim, block_size, max_blocks_per_seq, num_blocks,
                                             scale, ptr(out), stream_ptr(stream)))


def ql_fused_norm_rope(qkv, q_norm, k_norm, cos_t, sin_t, positions, active, eps, batch, n_heads,
                       n_kv_heads, head_dim, q_out, k_pool, v_pool, block_tables,
                       max_blocks_per_seq, block_size, num_blocks, max_position, stream=None):
    check(lib().ql_fused_norm_rope(ptr(qkv), ptr(q_norm), ptr(k_norm), ptr(cos_t), ptr(sin_t),
                                   ptr(positions), ptr(active), eps, batch, n_heads, n_kv_heads,
                                   head_dim, ptr(q_out), ptr(k_pool), ptr(v_pool), ptr(block_tables),
                                   max_blocks_per_seq, block_size, num_blocks, max_position,
                                   stream_ptr(stream)))


def ql_rope_tables(cos_t, sin_t, theta):
    """Host: fill numpy f32 ``cos_t``, ``sin_t`` [max_position, head_dim/2]."""
    n, half = cos_t.shape
    check(lib().ql_rope_tables(cos_t.ctypes.data, sin_t.ctypes.data, n, 2 * half, theta))


def ql_check_device_error(model=None):
    h = model.handle if model is not None else None
    check(lib().ql_check_device_error(h))


class BlockPool:
    """Host KV block allocator (free list first, then bump; QL_EPOOL when exhausted)."""

    def __init__(self, num_blocks: int):
        h = ctypes.c_void_p()
        check(lib().ql_block_pool_create(num_blocks, ctypes.byref(h)))
        self.handle = h.value

    def alloc(self) -> int:
        out = ctypes.c_int32()
        check(lib().ql_block_pool_alloc(self.handle, ctypes.byref(out)))
        return int(out.value)

    def free(self, ids):
        arr = (ctypes.c_int32 * len(ids))(*[int(i) for i in ids])
        check(lib().ql_block_pool_free(self.handle, arr, len(ids)))

    def in_use(self) -> int:
        return int(lib().ql_block_pool_in_use(self.handle))

    def close(self):
        if self.handle:
            lib().ql_block_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
