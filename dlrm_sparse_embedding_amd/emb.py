"""Thin ctypes binding of libemb.so (C ABI declared in include/emb.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels. PyTorch supplies device memory and the current HIP stream. The
functions carry the C names; ``EmbeddingTables`` bundles a context with the
tensors that back it.

``torch`` is imported before the library is loaded so that the library's
``libamdhip64.so.7`` resolves to the HIP runtime torch already holds (one
runtime per process). If ``libemb.so`` has not been built, loading raises --
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libemb.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "emb.h")

EMB_OK = 0
EMB_E_INVAL = -1
EMB_E_DTYPE = -2
EMB_E_WORKSPACE = -3
EMB_E_HIP = -4
EMB_E_BOUNDS = -5
EMB_E_STATE = -6

EMB_F32, EMB_BF16, EMB_F16 = 0, 1, 2
EMB_I32, EMB_I64 = 0, 1
EMB_POOL_SUM, EMB_POOL_MEAN = 0, 1
EMB_OPT_SGD, EMB_OPT_ADAGRAD = 0, 1
EMB_MAX_SLICES = 4

KERNELS = ["init", "forward", "keys", "sort_hist", "sort_scan", "sort_scatter", "rle", "reduce",
           "combine", "apply", "atomic", "pack", "gather", "hash"]

DTYPE_CODE = {"f32": EMB_F32, "bf16": EMB_BF16, "f16": EMB_F16}
TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
POOL_CODE = {"sum": EMB_POOL_SUM, "mean": EMB_POOL_MEAN}
OPT_CODE = {"sgd": EMB_OPT_SGD, "adagrad": EMB_OPT_ADAGRAD}


class EmbError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"emb error {code}: {msg}")
        self.code = code


EMB_SHARD_TABLE = 0
EMB_SHARD_ROW_CYCLIC = 1
EMB_SHARD_ROW_BLOCK = 2
EMB_MAX_SHARDS = 4096
SHARD_KIND = {"table": EMB_SHARD_TABLE, "row_cyclic": EMB_SHARD_ROW_CYCLIC, "row_block": EMB_SHARD_ROW_BLOCK}


class emb_shard_rule(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("shard", ctypes.c_int32)]


class emb_table_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int32), ("col_slices", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("weights", ctypes.c_void_p * EMB_MAX_SLICES),
                ("state", ctypes.c_void_p * EMB_MAX_SLICES),
                ("master", ctypes.c_void_p * EMB_MAX_SLICES)]


EMB_ROT_HALF, EMB_ROT_INTERLEAVED = 0, 1
EMB_ROT_NONE, EMB_ROT_LINEAR, EMB_ROT_BASE, EMB_ROT_PARTS, EMB_ROT_BANDS = 0, 1, 2, 3, 4
EMB_MAX_ROT = 256
EMB_MAX_HEAD_DIM = 1024
ROT_LAYOUT = {"half": EMB_ROT_HALF, "interleaved": EMB_ROT_INTERLEAVED}
ROT_SCALING = {"none": EMB_ROT_NONE, "linear": EMB_ROT_LINEAR, "base": EMB_ROT_BASE, "parts": EMB_ROT_PARTS,
               "bands": EMB_ROT_BANDS}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_HEADS_DTYPE = {torch.float32: EMB_F32, torch.bfloat16: EMB_BF16, torch.float16: EMB_F16}


class emb_rotary_desc(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("turns_low", ctypes.c_double), ("turns_high", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


class emb_kv_desc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_page_stride", ctypes.c_int64), ("k_slot_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_page_stride", ctypes.c_int64), ("v_slot_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("page", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("error", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libemb.so once (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m dlrm_sparse_embedding_amd.build` (no CPU fallback exists)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.emb_create_tables.argtypes = [ctypes.POINTER(emb_table_desc), i32, ctypes.POINTER(vp)]
    L.emb_create_tables.restype = ctypes.c_int
    L.emb_destroy_tables.argtypes = [vp]
    L.emb_destroy_tables.restype = None
    L.emb_row_offsets.argtypes = [vp, ctypes.POINTER(i64)]
    L.emb_row_offsets.restype = ctypes.c_int
    L.emb_init_uniform.argtypes = [vp, ctypes.c_uint64, vp]
    L.emb_init_uniform.restype = ctypes.c_int
    L.emb_forward_pooled.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, vp]
    L.emb_forward_pooled.restype = ctypes.c_int
    L.emb_backward_workspace_bytes.argtypes = [vp, i64, i32]
    L.emb_backward_workspace_bytes.restype = sz
    L.emb_backward_unique_reduce.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, vp, sz, vp, vp, vp,
                                             vp, vp, vp]
    L.emb_backward_unique_reduce.restype = ctypes.c_int
    L.emb_backward_dedup.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, sz, vp, vp, vp, vp, vp]
    L.emb_backward_dedup.restype = ctypes.c_int
    L.emb_backward_atomic_reduce.argtypes = [vp, vp, i32, i64, i32, i32, vp, vp, vp, vp, vp]
    L.emb_backward_atomic_reduce.restype = ctypes.c_int
    L.emb_sparse_update.argtypes = [vp, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp, vp]
    L.emb_sparse_update.restype = ctypes.c_int
    L.emb_forward_pooled_unique.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, vp, sz, vp, vp]
    L.emb_forward_pooled_unique.restype = ctypes.c_int
    L.emb_hash_bytes.argtypes = [vp]
    L.emb_hash_bytes.restype = sz
    L.emb_hash_attach.argtypes = [vp, vp, sz, vp]
    L.emb_hash_attach.restype = ctypes.c_int
    L.emb_hash_workspace_bytes.argtypes = [vp, i64]
    L.emb_hash_workspace_bytes.restype = sz
    L.emb_hash_translate.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, sz, vp, vp]
    L.emb_hash_translate.restype = ctypes.c_int
    L.emb_hash_translate_noalloc.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, vp]
    L.emb_hash_translate_noalloc.restype = ctypes.c_int
    L.emb_forward_pooled_hashed.argtypes = [vp, vp, vp, i32, i64, i32, i32, vp, vp]
    L.emb_forward_pooled_hashed.restype = ctypes.c_int
    L.emb_hash_rows_used.argtypes = [vp, vp, vp]
    L.emb_hash_rows_used.restype = ctypes.c_int
    L.emb_set_shard_map.argtypes = [vp, ctypes.POINTER(emb_shard_rule), i32]
    L.emb_set_shard_map.restype = ctypes.c_int
    L.emb_pack_by_shard.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    L.emb_pack_by_shard.restype = ctypes.c_int
    L.emb_last_error.argtypes = []
    L.emb_last_error.restype = ctypes.c_char_p
    L.emb_check_device_error.argtypes = [vp, vp]
    L.emb_check_device_error.restype = ctypes.c_int
    L.emb_set_kernel_timing.argtypes = [vp, i32]
    L.emb_set_kernel_timing.restype = ctypes.c_int
    L.emb_kernel_times.argtypes = [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(i64)]
    L.emb_kernel_times.restype = ctypes.c_int
    L.emb_probe_blocks.argtypes = []
    L.emb_probe_blocks.restype = i32
    L.emb_probe_reads.argtypes = [vp, i64, i64, i32, i32, i32, vp, vp]
    L.emb_probe_reads.restype = ctypes.c_int
    L.emb_probe_update.argtypes = [vp, i64, vp, vp, i64, i32, vp]
    L.emb_probe_update.restype = ctypes.c_int
    f32 = ctypes.c_float
    heads_io = [vp, i64, i64]
    L.emb_create_rotary.argtypes = [ctypes.POINTER(emb_rotary_desc), ctypes.POINTER(vp)]
    L.emb_create_rotary.restype = ctypes.c_int
    L.emb_destroy_rotary.argtypes = [vp]
    L.emb_destroy_rotary.restype = None
    both = (heads_io * 2 + [i32]) * 2
    L.emb_rotary_apply.argtypes = [vp, vp, i32, i64, i32, i32] + both + [i32, vp]
    L.emb_rotary_apply.restype = ctypes.c_int
    L.emb_qk_norm_rotary.argtypes = [vp, vp, i32, i64, i32, i32] + both + [vp, vp, f32, vp]
    L.emb_qk_norm_rotary.restype = ctypes.c_int
    L.emb_qk_norm_rotary_workspace_bytes.argtypes = [i64, i32, i32, i32]
    L.emb_qk_norm_rotary_workspace_bytes.restype = sz
    L.emb_qk_norm_rotary_backward.argtypes = ([vp, vp, i32, i64, i32, i32] + (heads_io * 3 + [i32]) * 2 +
                                              [vp, vp, f32, vp, sz, vp, vp, vp])
    L.emb_qk_norm_rotary_backward.restype = ctypes.c_int
    L.emb_create_kv.argtypes = [ctypes.POINTER(emb_kv_desc), ctypes.POINTER(vp)]
    L.emb_create_kv.restype = ctypes.c_int
    L.emb_destroy_kv.argtypes = [vp]
    L.emb_destroy_kv.restype = None
    L.emb_check_kv_error.argtypes = [vp, vp]
    L.emb_check_kv_error.restype = ctypes.c_int
    L.emb_kv_append.argtypes = [vp, vp, i64, i32, i32, i32] + heads_io * 2 + [vp, i32, vp, vp, i32, vp, i32, i32, vp, f32, vp]
    L.emb_kv_append.restype = ctypes.c_int
    L.emb_prefix_attention_workspace_bytes.argtypes = [vp, i64, i32, i32, i32, i32]
    L.emb_prefix_attention_workspace_bytes.restype = sz
    L.emb_prefix_attention.argtypes = [vp, i64, i32, i32] + heads_io * 2 + [i32, f32, vp, i32, vp, vp, i32, vp, i32, vp, vp, i32,
                                                                  vp, sz, vp, vp]
    L.emb_prefix_attention.restype = ctypes.c_int
    _lib = L
    return L


def _check(rc: int) -> None:
    if rc != EMB_OK:
        raise EmbError(rc, lib().emb_last_error().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _itype(t: torch.Tensor) -> int:
    if t.dtype == torch.int32:
        return EMB_I32
    if t.dtype == torch.int64:
        return EMB_I64
    raise ValueError(f"indices/offsets must be int32 or int64, not {t.dtype}")


# ---- C entry points, same names --------------------------------------------

def emb_create_tables(descs) -> int:
    """descs: sequence of emb_table_desc. Returns the context handle."""
    arr = (emb_table_desc * len(descs))(*descs)
    out = ctypes.c_void_p()
    _check(lib().emb_create_tables(arr, len(descs), ctypes.byref(out)))
    return out.value


def emb_destroy_tables(ctx: int) -> None:
    lib().emb_destroy_tables(ctx)


def emb_row_offsets(ctx: int, T: int) -> list:
    buf = (ctypes.c_int64 * (T + 1))()
    _check(lib().emb_row_offsets(ctx, buf))
    return list(buf)


def emb_init_uniform(ctx: int, seed: int, stream=None) -> None:
    _check(lib().emb_init_uniform(ctx, int(seed), _stream(stream)))


def emb_forward_pooled(ctx: int, indices: torch.Tensor, offsets: torch.Tensor, B: int, pool: str,
                       out: torch.Tensor, stream=None) -> None:
    if offsets.dtype != indices.dtype:
        raise ValueError("indices and offsets must share one integer type")
    if out.dtype != torch.float32:
        raise ValueError("out must be fp32")
    _check(lib().emb_forward_pooled(ctx, _ptr(indices), _ptr(offsets), _itype(indices),
                                    int(indices.numel()), int(B), POOL_CODE[pool], _ptr(out),
                                    _stream(stream)))


def emb_backward_workspace_bytes(ctx: int, N: int, B: int) -> int:
    return int(lib().emb_backward_workspace_bytes(ctx, int(N), int(B)))


def emb_backward_unique_reduce(ctx: int, indices, offsets, B: int, pool: str, dY, ws, unique_keys,
                               counts, inverse, num_unique, reduced_grad=None, stream=None) -> None:
    if offsets.dtype != indices.dtype:
        raise ValueError("indices and offsets must share one integer type")
    _check(lib().emb_backward_unique_reduce(
        ctx, _ptr(indices), _ptr(offsets), _itype(indices), int(indices.numel()), int(B),
        POOL_CODE[pool], _ptr(dY), _ptr(ws), int(ws.numel() * ws.element_size()), _ptr(unique_keys),
        _ptr(counts), _ptr(inverse), _ptr(num_unique), _ptr(reduced_grad), _stream(stream)))


def emb_backward_dedup(ctx: int, indices, offsets, B: int, pool: str, ws, unique_keys, counts, inverse,
                       num_unique, stream=None) -> None:
    if offsets.dtype != indices.dtype:
        raise ValueError("indices and offsets must share one integer type")
    _check(lib().emb_backward_dedup(
        ctx, _ptr(indices), _ptr(offsets), _itype(indices), int(indices.numel()), int(B),
        POOL_CODE[pool], _ptr(ws), int(ws.numel() * ws.element_size()), _ptr(unique_keys),
        _ptr(counts), _ptr(inverse), _ptr(num_unique), _stream(stream)))


def emb_backward_atomic_reduce(ctx: int, offsets, N: int, B: int, pool: str, dY, inverse, num_unique,
                               reduced_grad, stream=None) -> None:
    _check(lib().emb_backward_atomic_reduce(
        ctx, _ptr(offsets), _itype(offsets), int(N), int(B), POOL_CODE[pool], _ptr(dY), _ptr(inverse),
        _ptr(num_unique), _ptr(reduced_grad), _stream(stream)))


def emb_sparse_update(ctx: int, opt: str, lr: float, eps: float, ws, dY=None, reduced_grad=None,
                      stream=None) -> None:
    _check(lib().emb_sparse_update(ctx, OPT_CODE[opt], float(lr), float(eps), _ptr(ws), _ptr(dY),
                                   _ptr(reduced_grad), _stream(stream)))


def emb_check_device_error(ctx: int, stream=None) -> None:
    _check(lib().emb_check_device_error(ctx, _stream(stream)))


def emb_set_kernel_timing(ctx: int, enable: bool) -> None:
    _check(lib().emb_set_kernel_timing(ctx, 1 if enable else 0))


def emb_forward_pooled_unique(ctx: int, indices, offsets, B: int, pool: str, ws, rows_buf, out,
                              stream=None) -> None:
    if offsets.dtype != indices.dtype:
        raise ValueError("indices and offsets must share one integer type")
    _check(lib().emb_forward_pooled_unique(
        ctx, _ptr(indices), _ptr(offsets), _itype(indices), int(indices.numel()), int(B), POOL_CODE[pool],
        _ptr(ws), _ptr(rows_buf), int(rows_buf.numel() * rows_buf.element_size()) if rows_buf is not None else 0,
        _ptr(out), _stream(stream)))


def emb_hash_bytes(ctx: int) -> int:
    return int(lib().emb_hash_bytes(ctx))


def emb_hash_attach(ctx: int, mem, stream=None) -> None:
    _check(lib().emb_hash_attach(ctx, _ptr(mem), int(mem.numel() * mem.element_size()), _stream(stream)))


def emb_hash_workspace_bytes(ctx: int, N: int) -> int:
    return int(lib().emb_hash_workspace_bytes(ctx, int(N)))


def emb_hash_translate(ctx: int, ids, offsets, B: int, insert: bool, ws, rows_out, stream=None) -> None:
    """ids: int64 [N]; rows_out: [N] of the offsets' integer type."""
    if ids.dtype != torch.int64:
        raise ValueError("ids must be int64")
    if rows_out.dtype != offsets.dtype:
        raise ValueError("rows_out must have the offsets' integer type")
    _check(lib().emb_hash_translate(ctx, _ptr(ids), _ptr(offsets), _itype(offsets), int(ids.numel()), int(B),
                                    1 if insert else 0, _ptr(ws), int(ws.numel() * ws.element_size()),
                                    _ptr(rows_out), _stream(stream)))


def emb_hash_translate_noalloc(ctx: int, ids, offsets, B: int, insert: bool, rows_out, stream=None) -> None:
    """emb_hash_translate without a workspace (the library's fixed scratch)."""
    if ids.dtype != torch.int64:
        raise ValueError("ids must be int64")
    if rows_out.dtype != offsets.dtype:
        raise ValueError("rows_out must have the offsets' integer type")
    _check(lib().emb_hash_translate_noalloc(ctx, _ptr(ids), _ptr(offsets), _itype(offsets), int(ids.numel()),
                                            int(B), 1 if insert else 0, _ptr(rows_out), _stream(stream)))


def emb_forward_pooled_hashed(ctx: int, ids, offsets, B: int, pool: str, out, stream=None) -> None:
    if ids.dtype != torch.int64:
        raise ValueError("ids must be int64")
    _check(lib().emb_forward_pooled_hashed(ctx, _ptr(ids), _ptr(offsets), _itype(offsets), int(ids.numel()),
                                           int(B), POOL_CODE[pool], _ptr(out), _stream(stream)))


def emb_hash_rows_used(ctx: int, used, stream=None) -> None:
    _check(lib().emb_hash_rows_used(ctx, _ptr(used), _stream(stream)))


def emb_set_shard_map(ctx: int, rules, num_shards: int) -> None:
    """rules: one (kind, shard) per table, kind an EMB_SHARD_* code or a
    SHARD_KIND name."""
    arr = (emb_shard_rule * len(rules))()
    for t, (kind, shard) in enumerate(rules):
        arr[t].kind = SHARD_KIND.get(kind, kind) if isinstance(kind, str) else int(kind)
        arr[t].shard = int(shard)
    _check(lib().emb_set_shard_map(ctx, arr, int(num_shards)))


def emb_pack_by_shard(ctx: int, ws, dY, send_keys, send_offsets, slot_of_unique, send_grad,
                      stream=None) -> None:
    _check(lib().emb_pack_by_shard(ctx, _ptr(ws), _ptr(dY), _ptr(send_keys), _ptr(send_offsets),
                                   _ptr(slot_of_unique), _ptr(send_grad), _stream(stream)))


def emb_probe_blocks() -> int:
    return int(lib().emb_probe_blocks())


def emb_probe_reads(buf, nrows: int, stride: int, xcd_local: bool, reads: int, sink, stream=None,
                    row_bytes: int = 512) -> None:
    """Measurement aid: random 256- or 512-byte row reads (see include/emb.h)."""
    _check(lib().emb_probe_reads(_ptr(buf), int(nrows), int(stride), 1 if xcd_local else 0, int(reads),
                                 int(row_bytes), _ptr(sink), _stream(stream)))


def emb_probe_update(src, nsrc: int, a, b, nrows: int, items: int, stream=None) -> None:
    """Measurement aid: the fused update's random row read/write mix (see include/emb.h)."""
    _check(lib().emb_probe_update(_ptr(src), int(nsrc), _ptr(a), _ptr(b), int(nrows), int(items), _stream(stream)))


def emb_probe_update_bytes(items: int) -> int:
    """Bytes one emb_probe_update launch moves (include/emb.h)."""
    n3 = 34 * (items // 50) + min(items % 50, 34)
    return 512 * (3 * n3 + 2 * (items - n3) + 4 * items)


def emb_kernel_times(ctx: int) -> dict:
    ms = (ctypes.c_double * len(KERNELS))()
    n = (ctypes.c_int64 * len(KERNELS))()
    _check(lib().emb_kernel_times(ctx, ms, n))
    return {k: (ms[i], int(n[i])) for i, k in enumerate(KERNELS)}


# ---- sequence operators --------------------------------------------------------

def _dtype_code(name: str, t: torch.Tensor) -> int:
    code = _HEADS_DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} is {t.dtype}: fp32, bf16 or fp16")
    return code


def _heads(name: str, t: torch.Tensor, tokens: int, dim: int, dtype: torch.dtype):
    """Checks a [tokens, heads, dim] operand; its (pointer, token stride, head stride)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != tokens or shape[2] != dim:
        raise ValueError(f"{name} has shape {tuple(shape)}, not [{tokens}, heads, {dim}]")
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} is not in device memory")
    ts, hs, es = t.stride()
    if es != 1 and dim > 1:
        raise ValueError(f"the elements of one head of {name} must be contiguous")
    return t.data_ptr(), ts, hs


def _dense(name: str, t: torch.Tensor, dtype, shape):
    """Checks a contiguous device tensor of known type and shape; its pointer."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous device memory")
    return t.data_ptr()


def _stream_for(t: torch.Tensor, stream) -> int | None:
    """The stream to launch on: the given one, or the current one of t's device (its handle alone is ten times
    cheaper to ask for than a Stream object, 0.1 against 2.7 us)."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _stream(stream)


def _weight(name: str, w, dim: int):
    return None if w is None else _dense(name, w, torch.float32, (dim,))


def _positions(positions: torch.Tensor, tokens: int):
    return _dense("positions", positions, positions.dtype, (tokens,)), _itype(positions)


def _workspace(ws: torch.Tensor):
    if not ws.is_cuda:
        raise ValueError("ws is not in device memory")
    return _ptr(ws), ws.numel() * ws.element_size()


def _io(q, q_out, k, k_out):
    """The operands of a call over queries and, where given, keys."""
    T, hq, D = q.shape
    code = _dtype_code("q", q)
    args = [*_heads("q", q, T, D, q.dtype), *_heads("q_out", q_out, T, D, q.dtype), hq]
    if q_out.shape[1] != hq:
        raise ValueError(f"q_out has {q_out.shape[1]} heads, q {hq}")
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        args += [None, 0, 0, None, 0, 0, 0]
    else:
        if k_out is None or k_out.shape[1] != k.shape[1]:
            raise ValueError("k_out must have k's heads")
        args += [*_heads("k", k, T, D, q.dtype), *_heads("k_out", k_out, T, D, q.dtype), k.shape[1]]
    return T, D, code, args


def emb_create_rotary(desc: emb_rotary_desc) -> int:
    out = ctypes.c_void_p()
    _check(lib().emb_create_rotary(ctypes.byref(desc), ctypes.byref(out)))
    return out.value


def emb_destroy_rotary(rot: int) -> None:
    lib().emb_destroy_rotary(rot)


def emb_rotary_apply(rot: int, positions, q, q_out, k=None, k_out=None, inverse: bool = False, stream=None) -> None:
    """q, k: [tokens, heads, dim], any strides over tokens and heads; positions: int32 or int64 [tokens].
    q_out may be q, k_out k."""
    T, D, code, args = _io(q, q_out, k, k_out)
    pos, itype = _positions(positions, T)
    _check(lib().emb_rotary_apply(rot, pos, itype, T, code, D, *args, 1 if inverse else 0, _stream_for(q, stream)))


def emb_qk_norm_rotary(rot: int, positions, q, q_out, k, k_out, wq, wk, eps: float, stream=None) -> None:
    """wq, wk: fp32 [dim] or None; k and k_out may be None."""
    T, D, code, args = _io(q, q_out, k, k_out)
    pos, itype = _positions(positions, T)
    _check(lib().emb_qk_norm_rotary(rot, pos, itype, T, code, D, *args, _weight("wq", wq, D), _weight("wk", wk, D),
                                    float(eps), _stream_for(q, stream)))


def emb_qk_norm_rotary_workspace_bytes(tokens: int, q_heads: int, k_heads: int, dim: int) -> int:
    return int(lib().emb_qk_norm_rotary_workspace_bytes(int(tokens), int(q_heads), int(k_heads), int(dim)))


def emb_qk_norm_rotary_backward(rot: int, positions, q, dyq, dq, k, dyk, dk, wq, wk, eps: float, ws, dwq=None,
                                dwk=None, stream=None) -> None:
    """Gradients of emb_qk_norm_rotary: dq, dk (may be dyq, dyk) and, where given, dwq and dwk (fp32 [dim])."""
    T, D, code, args = _io(q, dq, k, dk)
    hq, hk = args[6], args[13]
    if dyq.shape[1] != hq or (k is not None and (dyk is None or dyk.shape[1] != hk)):
        raise ValueError("dyq and dyk must have the heads of q and k")
    gq = _heads("dyq", dyq, T, D, q.dtype)
    gk = _heads("dyk", dyk, T, D, q.dtype) if k is not None else (None, 0, 0)
    pos, itype = _positions(positions, T)
    ws_p, ws_n = _workspace(ws)
    _check(lib().emb_qk_norm_rotary_backward(
        rot, pos, itype, T, code, D, *args[0:3], *gq, *args[3:7], *args[7:10], *gk, *args[10:14],
        _weight("wq", wq, D), _weight("wk", wk, D), float(eps), ws_p, ws_n, _weight("dwq", dwq, D),
        _weight("dwk", dwk, D), _stream_for(q, stream)))


def emb_create_kv(desc: emb_kv_desc) -> int:
    out = ctypes.c_void_p()
    _check(lib().emb_create_kv(ctypes.byref(desc), ctypes.byref(out)))
    return out.value


def emb_destroy_kv(kv: int) -> None:
    lib().emb_destroy_kv(kv)


def emb_check_kv_error(kv: int, stream=None) -> None:
    _check(lib().emb_check_kv_error(kv, _stream(stream)))


def _sequences(T: int, offsets, lens, table):
    B = lens.shape[0]
    if table.dim() != 2:
        raise ValueError("table must be [seqs, pages]")
    width = table.shape[1]
    return (None if offsets is None else _dense("offsets", offsets, torch.int32, (B + 1,)), B,
            _dense("lens", lens, torch.int32, (B,)), _dense("table", table, torch.int32, (B, width)), width)


def emb_kv_append(kv: int, rot, k, v, offsets, lens, table, wk=None, eps=None, positions=None, stream=None) -> None:
    """Appends k, v [tokens, heads, dim] to their sequences' pages. offsets: int32 [seqs + 1], or None for one token
    each; lens: int32 [seqs], with the new tokens; table: int32 [seqs, pages]. rot: a rotation's handle or None;
    positions: int32 or int64 [tokens], or None for the slots. Keys are normed where wk is given, or where eps is
    given and not 0."""
    T, D = k.shape[0], k.shape[2]
    if v.shape[1] != k.shape[1]:
        raise ValueError("k and v must have the same heads")
    pos, itype = (None, EMB_I64) if positions is None else _positions(positions, T)
    norm = wk is not None or bool(eps)
    _check(lib().emb_kv_append(kv, rot, T, _dtype_code("k", k), k.shape[1], D, *_heads("k", k, T, D, k.dtype), *_heads("v", v, T, D, k.dtype),
                               *_sequences(T, offsets, lens, table), pos, itype, 1 if norm else 0,
                               _weight("wk", wk, D), float(eps or 0.0), _stream_for(k, stream)))


def emb_prefix_attention_workspace_bytes(kv: int, tokens: int, q_heads: int, groups: int, prefix_width: int,
                                         table_width: int) -> int:
    return int(lib().emb_prefix_attention_workspace_bytes(kv, int(tokens), int(q_heads), int(groups),
                                                          int(prefix_width), int(table_width)))


def emb_prefix_attention(kv: int, q, out, scale: float, offsets, lens, table, group_offsets, prefix_lens,
                         prefix_table, ws, lse=None, stream=None) -> None:
    """q, out: [tokens, q_heads, dim] of the cache's type. offsets, lens, table: as emb_kv_append; group_offsets
    (int32 [groups + 1], over sequences), prefix_lens (int32 [groups]) and prefix_table (int32 [groups, pages]), or
    all None. lse: fp32 [tokens, q_heads] or None."""
    T, hq, D = q.shape
    if out.shape[1] != hq:
        raise ValueError(f"out has {out.shape[1]} heads, q {hq}")
    if prefix_lens is None:
        if group_offsets is not None or prefix_table is not None:
            raise ValueError("group_offsets, prefix_lens and prefix_table go together")
        groups = (None, 0, None, None, 0)
    else:
        G = prefix_lens.shape[0]
        if prefix_table.dim() != 2:
            raise ValueError("prefix_table must be [groups, pages]")
        width = prefix_table.shape[1]
        groups = (_dense("group_offsets", group_offsets, torch.int32, (G + 1,)), G,
                  _dense("prefix_lens", prefix_lens, torch.int32, (G,)),
                  _dense("prefix_table", prefix_table, torch.int32, (G, width)), width)
    ws_p, ws_n = _workspace(ws)
    _check(lib().emb_prefix_attention(
        kv, T, _dtype_code("q", q), D, *_heads("q", q, T, D, q.dtype), *_heads("out", out, T, D, q.dtype), hq, float(scale),
        *_sequences(T, offsets, lens, table), *groups, ws_p, ws_n,
        None if lse is None else _dense("lse", lse, torch.float32, (T, hq)), _stream_for(q, stream)))


class Rotary:
    """A rotation: the first `rot` elements of each head, in the "half" or "interleaved" layout, with the
    frequencies of `base`, scaled by one of "none", "linear", "base", "parts" and "bands" (include/emb.h)."""

    def __init__(self, rot: int, layout: str = "half", base: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, original_len: float = 0.0, turns_low: float = 0.0, turns_high: float = 0.0,
                 magnitude: float = 1.0):
        self.handle = None
        self.rot, self.layout, self.scaling = rot, layout, scaling
        self.handle = emb_create_rotary(emb_rotary_desc(rot, ROT_LAYOUT[layout], ROT_SCALING[scaling], 0, base, factor,
                                                        original_len, turns_low, turns_high, magnitude))

    def close(self) -> None:
        if self.handle:
            emb_destroy_rotary(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    """A paged cache over the caller's tensors k and v, indexed [page, slot, head, dim] (any strides, the dim
    elements of a head contiguous)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        self.handle = None
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages, slots, heads, dim] of one shape and type")
        code = _dtype_code("the cache", k)
        if not k.is_cuda or not v.is_cuda:
            raise ValueError("the cache is not in device memory")
        if k.shape[3] > 1 and (k.stride(3) != 1 or v.stride(3) != 1):
            raise ValueError("the elements of one head must be contiguous")
        self.k, self.v = k, v
        self.pages, self.page, self.heads, self.dim = k.shape
        self.error = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.handle = emb_create_kv(emb_kv_desc(k.data_ptr(), v.data_ptr(), *k.stride()[:3], *v.stride()[:3],
                                                self.pages, self.page, self.heads, self.dim, code,
                                                self.error.data_ptr()))

    def close(self) -> None:
        if self.handle:
            emb_destroy_kv(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def check_error(self, stream=None) -> None:
        """Waits for the stream; raises if a call met a bad page, length or offset since the last check."""
        emb_check_kv_error(self.handle, stream)


# ---- convenience: a context with the tensors behind it ---------------------

@dataclass
class TableSpec:
    rows: int
    dim: int
    dtype: str = "f32"
    col_slices: int = 1


class EmbeddingTables:
    """Allocates this GPU's tables (and Adagrad state, and fp32 master weights
    for low-precision tables if asked) as torch tensors, registers them with
    emb_create_tables and forwards the calls."""

    def __init__(self, specs, with_state: bool, device="cuda", with_master: bool = False):
        specs = list(specs)
        self.specs = specs
        self.T = len(specs)
        self.dim = specs[0].dim
        self.dtype = specs[0].dtype
        self.col_slices = specs[0].col_slices
        self.weights = []   # [t][s] tensors [rows, dim/col_slices]
        self.state = []     # [t][s] fp32 tensors or None
        self.master = []    # [t][s] fp32 tensors or None
        descs = []
        for sp in specs:
            dsl = sp.dim // sp.col_slices
            ws = [torch.empty((sp.rows, dsl), dtype=TORCH_DTYPE[sp.dtype], device=device)
                  for _ in range(sp.col_slices)]
            ss = ([torch.empty((sp.rows, dsl), dtype=torch.float32, device=device)
                   for _ in range(sp.col_slices)] if with_state else None)
            ms = ([torch.empty((sp.rows, dsl), dtype=torch.float32, device=device)
                   for _ in range(sp.col_slices)] if with_master else None)
            self.weights.append(ws)
            self.state.append(ss)
            self.master.append(ms)
            d = emb_table_desc()
            d.rows, d.dim, d.col_slices, d.dtype, d.reserved = sp.rows, sp.dim, sp.col_slices, DTYPE_CODE[sp.dtype], 0
            for s in range(sp.col_slices):
                d.weights[s] = ws[s].data_ptr()
                d.state[s] = ss[s].data_ptr() if ss else None
                d.master[s] = ms[s].data_ptr() if ms else None
            descs.append(d)
        self.ctx = emb_create_tables(descs)
        self.row_offset = emb_row_offsets(self.ctx, self.T)

    def close(self) -> None:
        if self.ctx:
            emb_destroy_tables(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def init_uniform(self, seed: int, stream=None) -> None:
        emb_init_uniform(self.ctx, seed, stream)

    def forward(self, indices, offsets, B: int, pool: str, out=None, stream=None):
        if out is None:
            out = torch.empty((B, self.T * self.dim), dtype=torch.float32, device=indices.device)
        emb_forward_pooled(self.ctx, indices, offsets, B, pool, out, stream)
        return out

    def workspace(self, N: int, B: int, device="cuda"):
        nbytes = emb_backward_workspace_bytes(self.ctx, N, B)
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)

    def backward_buffers(self, N: int, B: int, with_grad: bool, device="cuda"):
        """Device outputs of emb_backward_unique_reduce sized by N."""
        cap = max(N, 1)
        return dict(
            ws=self.workspace(N, B, device),
            unique_keys=torch.empty(cap, dtype=torch.int32, device=device),  # uint32 bits
            counts=torch.empty(cap, dtype=torch.int32, device=device),
            inverse=torch.empty(cap, dtype=torch.int32, device=device),
            num_unique=torch.empty(1, dtype=torch.int32, device=device),
            reduced_grad=(torch.empty((cap, self.dim), dtype=torch.float32, device=device)
                          if with_grad else None),
        )

    def backward(self, indices, offsets, B: int, pool: str, dY, bufs, stream=None) -> None:
        emb_backward_unique_reduce(self.ctx, indices, offsets, B, pool, dY, bufs["ws"],
                                   bufs["unique_keys"], bufs["counts"], bufs["inverse"],
                                   bufs["num_unique"], bufs["reduced_grad"], stream)

    def dedup(self, indices, offsets, B: int, pool: str, bufs, stream=None) -> None:
        emb_backward_dedup(self.ctx, indices, offsets, B, pool, bufs["ws"], bufs["unique_keys"],
                           bufs["counts"], bufs["inverse"], bufs["num_unique"], stream)

    def atomic_reduce(self, offsets, N: int, B: int, pool: str, dY, bufs, stream=None) -> None:
        emb_backward_atomic_reduce(self.ctx, offsets, N, B, pool, dY, bufs["inverse"], bufs["num_unique"],
                                   bufs["reduced_grad"], stream)

    def update(self, opt: str, lr: float, eps: float, bufs, dY=None, stream=None) -> None:
        emb_sparse_update(self.ctx, opt, lr, eps, bufs["ws"], dY, bufs["reduced_grad"], stream)

    def check_device_error(self, stream=None) -> None:
        emb_check_device_error(self.ctx, stream)

    def logical_rows(self, t: int, rows) -> torch.Tensor:
        """Rows of table t gathered from its column slices, [len(rows), dim]
        in the storage dtype (a read-back helper for checks)."""
        r = torch.as_tensor(rows, dtype=torch.int64, device=self.weights[t][0].device)
        return torch.cat([w.index_select(0, r) for w in self.weights[t]], dim=1)

    def logical_state(self, t: int, rows) -> torch.Tensor:
        r = torch.as_tensor(rows, dtype=torch.int64, device=self.weights[t][0].device)
        return torch.cat([s.index_select(0, r) for s in self.state[t]], dim=1)

    def unique_rows_buffer(self, N: int, device="cuda") -> torch.Tensor:
        """Capacity for emb_forward_pooled_unique: N rows of the storage type."""
        return torch.empty((max(N, 1), self.dim), dtype=TORCH_DTYPE[self.dtype], device=device)

    def forward_unique(self, indices, offsets, B: int, pool: str, bufs, rows_buf, out=None, stream=None):
        """Unique-first forward; needs self.dedup(...) of the same lookups first."""
        if out is None:
            out = torch.empty((B, self.T * self.dim), dtype=torch.float32, device=indices.device)
        emb_forward_pooled_unique(self.ctx, indices, offsets, B, pool, bufs["ws"], rows_buf, out, stream)
        return out

    def hash_attach(self, device="cuda", stream=None) -> None:
        """Allocates the id -> row maps of every table and empties them."""
        self.hash_mem = torch.empty(emb_hash_bytes(self.ctx), dtype=torch.uint8, device=device)
        emb_hash_attach(self.ctx, self.hash_mem, stream)

    def hash_translate(self, ids, offsets, B: int, insert: bool, stream=None):
        rows = torch.empty(max(ids.numel(), 1), dtype=offsets.dtype, device=ids.device)[:ids.numel()]
        ws = torch.empty(max(emb_hash_workspace_bytes(self.ctx, ids.numel()), 256), dtype=torch.uint8,
                         device=ids.device)
        emb_hash_translate(self.ctx, ids, offsets, B, insert, ws, rows, stream)
        if stream is not None:
            # the allocator must not hand ws (or rows) to another tensor while
            # the translation still runs on a stream other than the current one
            st = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            if st != torch.cuda.current_stream(ids.device):
                ws.record_stream(st)
                rows.record_stream(st)
        return rows

    def forward_hashed(self, ids, offsets, B: int, pool: str, out=None, stream=None):
        if out is None:
            out = torch.empty((B, self.T * self.dim), dtype=torch.float32, device=ids.device)
        emb_forward_pooled_hashed(self.ctx, ids, offsets, B, pool, out, stream)
        return out

    def hash_rows_used(self, stream=None):
        used = torch.empty(self.T, dtype=torch.int32, device=self.weights[0][0].device)
        emb_hash_rows_used(self.ctx, used, stream)
        return used

    def set_shard_map(self, rules, num_shards: int) -> None:
        emb_set_shard_map(self.ctx, rules, num_shards)

    def pack_buffers(self, N: int, num_shards: int, with_grad: bool, device="cuda"):
        cap = max(N, 1)
        return dict(
            send_keys=torch.empty(cap, dtype=torch.int32, device=device),   # uint32 bits
            send_offsets=torch.empty(num_shards + 1, dtype=torch.int32, device=device),
            slot_of_unique=torch.empty(cap, dtype=torch.int32, device=device),
            send_grad=(torch.empty((cap, self.dim), dtype=torch.float32, device=device)
                       if with_grad else None),
        )

    def pack(self, bufs, pbufs, dY=None, stream=None) -> None:
        emb_pack_by_shard(self.ctx, bufs["ws"], dY, pbufs["send_keys"], pbufs["send_offsets"],
                          pbufs["slot_of_unique"], pbufs["send_grad"] if dY is not None else None, stream)

    def logical_master(self, t: int, rows) -> torch.Tensor:
        r = torch.as_tensor(rows, dtype=torch.int64, device=self.weights[t][0].device)
        return torch.cat([m.index_select(0, r) for m in self.master[t]], dim=1)
