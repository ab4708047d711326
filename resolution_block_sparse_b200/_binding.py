"""ctypes binding of the C ABI in include/mra.h (argument marshalling only).

Every function here forwards to ``libmra_b200.so``; none computes any step of
the method itself.  Loading fails loudly when the library is missing: there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmra_b200.so")

(MRA_OK, MRA_ERR_INVALID_ARG, MRA_ERR_UNSUPPORTED, MRA_ERR_CUDA, MRA_ERR_ALLOC,
 MRA_ERR_DEVICE_TIMEOUT, MRA_ERR_TOO_LARGE) = range(7)
MRA_NOALLOC_SCRATCH_BYTES = 16 << 20
MRA_FULL, MRA_SPARSE = 0, 1
MRA_DTYPE_BF16, MRA_DTYPE_F32 = 0, 1
MRA_LAYER_NORM, MRA_RMS_NORM = 0, 1
MRA_NORM_POST, MRA_NORM_PRE = 1, 2
MRA_DEV_KEY_RANGE, MRA_DEV_COUNT, MRA_DEV_TIMEOUT = 1, 2, 4

EXPORTED = (
    "mra_attention_fwd", "mra_attention_fwd_f32", "mra_attention_fwd_ex", "mra_attention_fwd_host",
    "mra_num_block", "mra_status_string", "mra_get_device_status", "mra_profile_enable",
    "mra_profile_read", "mra_last_launch_count", "mra_attention_fwd_noalloc", "mra_attention_bwd",
    "mra_attention_bwd_f32", "mra_blocksparse_attention_fwd", "mra_bigbird_block_list",
    "mra_self_attention_fwd", "mra_qkv_projection", "mra_get_noalloc_status", "mra_status_from_device",
    "mra_blocksparse_attention_bias_workspace", "mra_blocksparse_attention_bias_fwd",
    "mra_blocksparse_attention_bias_bwd", "mra_relative_buckets", "mra_residual_norm_workspace",
    "mra_residual_norm_fwd", "mra_residual_norm_bwd",
)

_lock = threading.Lock()
_lib = None


class MraError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load libmra_b200.so and declare its signatures (raises if missing)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    with _lock:
        if _lib is not None and path == LIB_PATH:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library not built: {path} is missing "
                "(run `python -m resolution_block_sparse_b200.build`)")
        lib = ctypes.CDLL(path)
        vp, ip, c_int = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
        fwd_args = [vp, vp, vp, vp, vp] + [c_int] * 8 + [vp]
        lib.mra_attention_fwd.argtypes = fwd_args
        lib.mra_attention_fwd.restype = c_int
        lib.mra_attention_fwd_f32.argtypes = fwd_args
        lib.mra_attention_fwd_f32.restype = c_int
        lib.mra_attention_fwd_noalloc.argtypes = fwd_args
        lib.mra_attention_fwd_noalloc.restype = c_int
        lib.mra_attention_fwd_ex.argtypes = [vp, vp, vp, vp, vp] + [c_int] * 9 + [vp, vp, vp, vp]
        lib.mra_attention_fwd_ex.restype = c_int
        lib.mra_attention_fwd_host.argtypes = [vp, vp, vp, vp, vp] + [c_int] * 9 + [vp]
        lib.mra_attention_fwd_host.restype = c_int
        for name in ("mra_attention_bwd", "mra_attention_bwd_f32"):
            fn = getattr(lib, name)
            fn.argtypes = [vp] * 8 + [c_int] * 8 + [vp]
            fn.restype = c_int
        lib.mra_blocksparse_attention_fwd.argtypes = [vp] * 5 + [c_int] * 4 + [vp, c_int, c_int, vp]
        lib.mra_blocksparse_attention_fwd.restype = c_int
        lib.mra_bigbird_block_list.argtypes = [c_int, c_int, c_int, vp, vp, c_int, ctypes.POINTER(c_int)]
        lib.mra_bigbird_block_list.restype = c_int
        lib.mra_self_attention_fwd.argtypes = [vp] * 5 + [c_int] * 8 + [vp]
        lib.mra_self_attention_fwd.restype = c_int
        lib.mra_qkv_projection.argtypes = [vp] * 4 + [c_int] * 4 + [vp]
        lib.mra_qkv_projection.restype = c_int
        lib.mra_num_block.argtypes = [c_int, c_int]
        lib.mra_num_block.restype = ctypes.c_size_t
        lib.mra_status_string.argtypes = [c_int]
        lib.mra_status_string.restype = ctypes.c_char_p
        lib.mra_get_device_status.argtypes = [vp]
        lib.mra_get_noalloc_status.argtypes = [vp]
        lib.mra_get_noalloc_status.restype = c_int
        lib.mra_status_from_device.argtypes = [c_int]
        lib.mra_status_from_device.restype = c_int
        lib.mra_get_device_status.restype = c_int
        lib.mra_profile_enable.argtypes = [c_int]
        lib.mra_profile_enable.restype = None
        lib.mra_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(c_int),
                                         ctypes.POINTER(ctypes.c_double), c_int]
        lib.mra_profile_read.restype = c_int
        lib.mra_last_launch_count.argtypes = []
        lib.mra_last_launch_count.restype = c_int
        c_size, c_float, c_ll = ctypes.c_size_t, ctypes.c_float, ctypes.c_longlong
        lib.mra_blocksparse_attention_bias_workspace.argtypes = [c_int] * 8
        lib.mra_blocksparse_attention_bias_workspace.restype = c_size
        lib.mra_blocksparse_attention_bias_fwd.argtypes = (
            [vp] * 6 + [c_int, c_float, vp, vp] + [c_int] * 4 + [vp, c_int, c_int, vp, c_size, vp])
        lib.mra_blocksparse_attention_bias_fwd.restype = c_int
        lib.mra_blocksparse_attention_bias_bwd.argtypes = (
            [vp] * 6 + [c_int, c_float] + [vp] * 6 + [c_int] * 4 + [vp, c_int, c_int, vp, c_size, vp])
        lib.mra_blocksparse_attention_bias_bwd.restype = c_int
        lib.mra_relative_buckets.argtypes = [c_int] * 4 + [vp]
        lib.mra_relative_buckets.restype = c_int
        lib.mra_residual_norm_workspace.argtypes = [c_ll, c_int]
        lib.mra_residual_norm_workspace.restype = c_size
        norm_tail = [c_ll, c_int, c_int, c_int, c_float, c_float, c_int]
        lib.mra_residual_norm_fwd.argtypes = [vp] * 3 + [c_ll] + [vp] * 7 + norm_tail + [vp]
        lib.mra_residual_norm_fwd.restype = c_int
        lib.mra_residual_norm_bwd.argtypes = [vp] * 3 + [c_ll] + [vp] * 14 + norm_tail + [vp, c_size, vp]
        lib.mra_residual_norm_bwd.restype = c_int
        if path == LIB_PATH:
            _lib = lib
        return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(status: int, where: str):
    if status != MRA_OK:
        raise MraError(status, where)


def _shape(q):
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, D]")
    return tuple(int(x) for x in q.shape)


def _mode(approx_mode):
    if isinstance(approx_mode, str):
        return {"full": MRA_FULL, "sparse": MRA_SPARSE}[approx_mode]
    return int(approx_mode)


def mra_attention_fwd(q, k, v, key_mask, out, block_per_row, approx_mode, first_n, diag_n,
                      stream=None):
    """bf16 forward on device tensors [B,H,N,D]; key_mask float32 [B,N] or None."""
    B, H, N, D = _shape(q)
    st = load_library().mra_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(out),
                                          B, H, N, D, block_per_row, _mode(approx_mode), first_n,
                                          diag_n, _stream(stream))
    _check(st, "mra_attention_fwd")
    return out


def mra_attention_fwd_f32(q, k, v, key_mask, out, block_per_row, approx_mode, first_n, diag_n,
                          stream=None):
    """fp32 forward on device tensors [B,H,N,D]."""
    B, H, N, D = _shape(q)
    st = load_library().mra_attention_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(out),
                                              B, H, N, D, block_per_row, _mode(approx_mode),
                                              first_n, diag_n, _stream(stream))
    _check(st, "mra_attention_fwd_f32")
    return out


def mra_attention_fwd_noalloc(q, k, v, key_mask, out, block_per_row, approx_mode, first_n,
                              diag_n, stream=None):
    """bf16 forward that allocates no device memory (static 16 MiB scratch);
    raises MraError(MRA_ERR_TOO_LARGE) when the problem does not fit."""
    B, H, N, D = _shape(q)
    st = load_library().mra_attention_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(key_mask),
                                                  _ptr(out), B, H, N, D, block_per_row,
                                                  _mode(approx_mode), first_n, diag_n,
                                                  _stream(stream))
    _check(st, "mra_attention_fwd_noalloc")
    return out


def mra_attention_bwd(q, k, v, key_mask, dout, dq, dk, dv, block_per_row, approx_mode, first_n, diag_n,
                      stream=None):
    """Backward on device tensors: q, k, v, dout [B,H,N,D] (bf16 or fp32);
    dq, dk, dv fp32 [B,H,N,D] are written."""
    B, H, N, D = _shape(q)
    lib = load_library()
    fn = lib.mra_attention_bwd if q.dtype == torch.bfloat16 else lib.mra_attention_bwd_f32
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, D,
            block_per_row, _mode(approx_mode), first_n, diag_n, _stream(stream))
    _check(st, "mra_attention_bwd")
    return dq, dk, dv


def mra_attention_fwd_ex(q, k, v, key_mask, out, block_per_row, approx_mode, first_n, diag_n,
                         sel_idx=None, lowres_logit=None, pooled=None, stream=None):
    """Forward that also fills the optional intermediate tensors (device)."""
    B, H, N, D = _shape(q)
    dtype = MRA_DTYPE_BF16 if q.dtype == torch.bfloat16 else MRA_DTYPE_F32
    st = load_library().mra_attention_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(out),
                                             B, H, N, D, block_per_row, _mode(approx_mode), first_n,
                                             diag_n, dtype, _ptr(sel_idx), _ptr(lowres_logit),
                                             _ptr(pooled), _stream(stream))
    _check(st, "mra_attention_fwd_ex")
    return out


def mra_attention_fwd_host(q, k, v, key_mask, out, block_per_row, approx_mode, first_n, diag_n,
                           stream=None):
    """Forward on HOST tensors (pinned for asynchronous copies); synchronises."""
    B, H, N, D = _shape(q)
    dtype = MRA_DTYPE_BF16 if q.dtype == torch.bfloat16 else MRA_DTYPE_F32
    st = load_library().mra_attention_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(out),
                                               B, H, N, D, block_per_row, _mode(approx_mode),
                                               first_n, diag_n, dtype, _stream(stream))
    _check(st, "mra_attention_fwd_host")
    return out


def mra_blocksparse_attention_fwd(q, k, v, key_mask, out, block_idx, stream=None):
    """Attention on given 32x32 blocks: block_idx int32 [B*H, cap_sel] on the
    device, ascending flat indices r * (N/32) + c per head, -1 padded."""
    B, H, N, D = _shape(q)
    if block_idx.dtype != torch.int32 or block_idx.dim() != 2 or block_idx.shape[0] != B * H:
        raise ValueError("block_idx must be int32 [B*H, cap_sel]")
    if not block_idx.is_contiguous():
        raise ValueError("block_idx must be contiguous")
    dtype = MRA_DTYPE_BF16 if q.dtype == torch.bfloat16 else MRA_DTYPE_F32
    st = load_library().mra_blocksparse_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(out),
                                                      B, H, N, D, _ptr(block_idx), int(block_idx.shape[1]),
                                                      dtype, _stream(stream))
    _check(st, "mra_blocksparse_attention_fwd")
    return out


def mra_bigbird_block_list(N: int, block_size: int, rand_blocks):
    """The BigBird pattern of one head (host): rand_blocks int [nb, r] ->
    int32 numpy array of ascending flat 32-token block indices."""
    import numpy as np

    rb = np.ascontiguousarray(np.asarray(rand_blocks), dtype=np.int32)
    if rb.ndim != 2:
        raise ValueError("rand_blocks must be [nb, r]")
    nbr = N // 32 if N > 0 else 0
    out = np.empty(max(1, nbr * nbr), dtype=np.int32)
    count = ctypes.c_int(0)
    st = load_library().mra_bigbird_block_list(N, block_size, int(rb.shape[1]), rb.ctypes.data_as(ctypes.c_void_p),
                                               out.ctypes.data_as(ctypes.c_void_p), int(out.size), ctypes.byref(count))
    _check(st, "mra_bigbird_block_list")
    return out[:count.value].copy()


_NORMS = {"layer": MRA_LAYER_NORM, "rms": MRA_RMS_NORM}
_DTYPES = {torch.bfloat16: MRA_DTYPE_BF16, torch.float32: MRA_DTYPE_F32}


def _expect(where, index, dtype, shape, **tensors):
    """Raises ValueError for a tensor (None is skipped) that is not contiguous,
    of that dtype and shape, on CUDA device `index`."""
    for name, t in tensors.items():
        if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()):
            continue
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{where}: {name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
        if t.get_device() != index:
            raise ValueError(f"{where}: {name} is on {t.device}, not on cuda:{index}")
        raise ValueError(f"{where}: {name} must be contiguous")


def _expect_all(where, index, dtype, shape, names, *tensors):
    """_expect for tensors with their names in one string: no dictionary is
    built for a call that is right (a microsecond of ten for a small one)."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous()):
            _expect(where, index, dtype, shape, **dict(zip(names.split(), tensors)))


def _expect_each(where, index, dtype, shape, names, *tensors):
    """_expect_all for tensors that must be given."""
    for t in tensors:
        if t is None:
            missing = [n for n, x in zip(names.split(), tensors) if x is None]
            raise ValueError(f"{where}: {missing[0]} must be given")
        if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
            _expect(where, index, dtype, shape, **dict(zip(names.split(), tensors)))


def _cuda_index(where, name, t):
    if t is None:
        raise ValueError(f"{where}: {name} must be given")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{where}: tensors must be on a CUDA device")
    return index


def _addr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=64)
def _device(index):
    return torch.device("cuda", index)


def _call_on(index, stream, workspace_bytes, call):
    """Runs call(workspace address, stream handle) with device `index` current,
    on the given stream (None: the device's current one), with a workspace from
    torch's allocator that is not reused before the call's work is done."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _call_on(index, stream, workspace_bytes, call)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
        if not workspace_bytes:
            return call(None, handle)
        ws = torch.empty(workspace_bytes, dtype=torch.uint8, device=_device(index))
        return call(ws.data_ptr(), handle)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    if stream.device_index != index:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors are on cuda:{index}")
    with torch.cuda.stream(stream):
        return _call_on(index, None, workspace_bytes, call)


# Sizes of workspaces go by the SMs of the device that is current (kept per device).
@functools.lru_cache(maxsize=256)
def _bias_workspace(index, B, H, N, D, cap, nb, dtype, backward):
    with torch.cuda.device(index):
        return load_library().mra_blocksparse_attention_bias_workspace(B, H, N, D, cap, nb, dtype, backward)


def _bias_checks(where, q, k, v, key_mask, bias_table, bucket, lse, block_idx, scale, names, *like_q):
    index = _cuda_index(where, "q", q)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 4 or 0 in shape:
        raise ValueError(f"{where}: q, k, v must be [B, H, N, D], none of them 0")
    if dtype not in _DTYPES:
        raise ValueError(f"{where}: q must be bf16 or fp32")
    B, H, N, D = shape
    if bias_table is None or bias_table.dim() != 2:
        raise ValueError(f"{where}: bias_table must be [num_buckets, H]")
    nb, cap = bias_table.shape[0], 0
    _expect_each(where, index, dtype, shape, names, q, k, v, *like_q)
    _expect_each(where, index, dtype, (nb, H), "bias_table", bias_table)
    _expect_each(where, index, torch.int32, (2 * N - 1,), "bucket", bucket)
    if key_mask is not None:
        _expect_all(where, index, torch.float32, (B, N), "key_mask", key_mask)
    if lse is not None:
        _expect_all(where, index, torch.float32, (B, H, N), "lse", lse)
    if block_idx is not None:
        if block_idx.dim() != 2 or block_idx.shape[1] == 0:
            raise ValueError(f"{where}: block_idx must be int32 [B*H, cap_sel], cap_sel at least 1 (-1: no block)")
        cap = block_idx.shape[1]
        _expect_all(where, index, torch.int32, (B * H, cap), "block_idx", block_idx)
    return index, B, H, N, D, nb, cap, _DTYPES[dtype], D ** -0.5 if scale is None else float(scale)


def mra_blocksparse_attention_bias_fwd(q, k, v, key_mask, bias_table, bucket, out, lse=None, block_idx=None,
                                       scale=None, stream=None):
    """Block-sparse attention with a learned bias per bucket of the relative
    position: q, k, v, out [B, H, N, D] (bf16 or fp32, any N), bias_table
    [num_buckets, H] in their type, bucket int32 [2N-1] (the bucket of key -
    query from -(N-1) to N-1; outside [0, num_buckets): the pair is excluded),
    key_mask fp32 [B, N] or None, block_idx as in
    mra_blocksparse_attention_fwd or None (every block), scale by default
    1/sqrt(D).  Writes out and, where given, lse fp32 [B, H, N]."""
    where = "mra_blocksparse_attention_bias_fwd"
    index, B, H, N, D, nb, cap, dtype, scale = _bias_checks(where, q, k, v, key_mask, bias_table, bucket, lse, block_idx,
                                                            scale, "q k v out", out)
    size = _bias_workspace(index, B, H, N, D, cap, nb, dtype, 0)
    st = _call_on(index, stream, size, lambda ws, s: load_library().mra_blocksparse_attention_bias_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(key_mask), bias_table.data_ptr(), bucket.data_ptr(), nb, scale,
        out.data_ptr(), _addr(lse), B, H, N, D, _addr(block_idx), cap, dtype, ws, size, s))
    if st != MRA_OK:
        raise MraError(st, where)
    return out


def mra_blocksparse_attention_bias_bwd(q, k, v, key_mask, bias_table, bucket, lse, dout, dq, dk, dv, dbias_table,
                                       block_idx=None, scale=None, stream=None):
    """Gradients of mra_blocksparse_attention_bias_fwd for the gradient dout of
    its output, from its lse: writes dq, dk, dv (like q) and dbias_table (like
    bias_table)."""
    where = "mra_blocksparse_attention_bias_bwd"
    if lse is None:
        raise ValueError(f"{where}: lse of the forward pass is needed")
    index, B, H, N, D, nb, cap, dtype, scale = _bias_checks(where, q, k, v, key_mask, bias_table, bucket, lse, block_idx,
                                                            scale, "q k v dout dq dk dv", dout, dq, dk, dv)
    _expect_each(where, index, q.dtype, bias_table.shape, "dbias_table", dbias_table)
    size = _bias_workspace(index, B, H, N, D, cap, nb, dtype, 1)
    st = _call_on(index, stream, size, lambda ws, s: load_library().mra_blocksparse_attention_bias_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(key_mask), bias_table.data_ptr(), bucket.data_ptr(), nb, scale,
        lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dbias_table.data_ptr(), B, H, N,
        D, _addr(block_idx), cap, dtype, ws, size, s))
    if st != MRA_OK:
        raise MraError(st, where)
    return dq, dk, dv, dbias_table


def mra_relative_buckets(N: int, num_buckets: int, max_distance: int, bidirectional: bool = True):
    """The bucket of every relative position key - query from -(N-1) to N-1
    (host): int32 numpy array [2N-1] for the calls above."""
    import numpy as np

    out = np.empty(max(1, 2 * N - 1), dtype=np.int32)
    st = load_library().mra_relative_buckets(N, num_buckets, max_distance, 1 if bidirectional else 0,
                                             out.ctypes.data_as(ctypes.c_void_p))
    _check(st, "mra_relative_buckets")
    return out


@functools.lru_cache(maxsize=256)
def _norm_workspace(index, rows, hidden):
    with torch.cuda.device(index):
        return load_library().mra_residual_norm_workspace(rows, hidden)


def _norm_checks(where, x, rows_names, rows_like, gate, names, weights, stats, norm, dgate=None):
    index = _cuda_index(where, "x", x)
    shape, dtype = x.shape, x.dtype
    if dtype not in _DTYPES or len(shape) < 1 or shape[-1] == 0:
        raise ValueError(f"{where}: x must be bf16 or fp32 [..., hidden]")
    if norm not in _NORMS:
        raise ValueError(f"{where}: norm must be 'layer' or 'rms'")
    hidden = shape[-1]
    rows, per = x.numel() // hidden, 1
    _expect_all(where, index, dtype, shape, rows_names, x, *rows_like)
    _expect_all(where, index, dtype, (hidden,), names, *weights)
    if gate is not None:
        gates = gate.shape[0] if gate.dim() == 2 else -1
        if gates < 0 or (rows and (gates == 0 or rows % gates)):
            raise ValueError(f"{where}: gate must be [rows, hidden] with a number of rows that divides x's")
        per = max(1, rows // max(1, gates))
        _expect_all(where, index, dtype, (gates, hidden), "gate dgate", gate, dgate)
    elif dgate is not None:
        raise ValueError(f"{where}: dgate without a gate")
    if stats is not None:
        _expect_all(where, index, torch.float32, (4, rows), "stats", stats)
    return index, rows, hidden, per, _NORMS[norm], _DTYPES[dtype]


def mra_residual_norm_fwd(x, h, x_out, y, *, gate=None, post_norm=False, post_w=None, post_b=None, pre_norm=True,
                          pre_w=None, pre_b=None, stats=None, residual_scale=1.0, norm="layer", eps=1e-5, stream=None):
    """x' = residual_scale x + gate * post-norm(h) and y = pre-norm(x'): x, h,
    x_out, y [..., hidden] (h, x_out or y may be None), gate [G, hidden] with G
    dividing the rows (1: per channel, the batch: per sequence) or None, the
    weights [hidden] or None, stats fp32 [4, rows] or None.  norm 'layer' or
    'rms'.  Writes x_out, y and stats."""
    where = "mra_residual_norm_fwd"
    index, rows, hidden, per, kind, dtype = _norm_checks(
        where, x, "x h x_out y", (h, x_out, y), gate, "post_w post_b pre_w pre_b", (post_w, post_b, pre_w, pre_b), stats, norm)
    norms = (MRA_NORM_POST if post_norm else 0) | (MRA_NORM_PRE if pre_norm else 0)
    st = _call_on(index, stream, 0, lambda ws, s: load_library().mra_residual_norm_fwd(
        x.data_ptr(), _addr(h), _addr(gate), per, _addr(post_w), _addr(post_b), _addr(pre_w), _addr(pre_b), _addr(x_out),
        _addr(y), _addr(stats), rows, hidden, kind, norms, residual_scale, eps, dtype, s))
    if st != MRA_OK:
        raise MraError(st, where)
    return x_out, y


def mra_residual_norm_bwd(x, h, stats, dx_out, dy, dx, dh, *, gate=None, post_norm=False, post_w=None, post_b=None,
                          pre_norm=True, pre_w=None, pre_b=None, dgate=None, dpost_w=None, dpost_b=None, dpre_w=None,
                          dpre_b=None, residual_scale=1.0, norm="layer", eps=1e-5, stream=None):
    """Gradients of mra_residual_norm_fwd for the gradients dx_out of x' and dy
    of y (one of them may be None), from its inputs and stats: writes dx, dh
    and those of dgate, dpost_w, dpost_b, dpre_w, dpre_b that are given."""
    where = "mra_residual_norm_bwd"
    index, rows, hidden, per, kind, dtype = _norm_checks(
        where, x, "x h dx_out dy dx dh", (h, dx_out, dy, dx, dh), gate,
        "post_w post_b pre_w pre_b dpost_w dpost_b dpre_w dpre_b",
        (post_w, post_b, pre_w, pre_b, dpost_w, dpost_b, dpre_w, dpre_b), stats, norm, dgate)
    norms = (MRA_NORM_POST if post_norm else 0) | (MRA_NORM_PRE if pre_norm else 0)
    size = _norm_workspace(index, rows, hidden)
    st = _call_on(index, stream, size, lambda ws, s: load_library().mra_residual_norm_bwd(
        x.data_ptr(), _addr(h), _addr(gate), per, _addr(post_w), _addr(post_b), _addr(pre_w), _addr(pre_b), _addr(stats),
        _addr(dx_out), _addr(dy), _addr(dx), _addr(dh), _addr(dgate), _addr(dpost_w), _addr(dpost_b), _addr(dpre_w),
        _addr(dpre_b), rows, hidden, kind, norms, residual_scale, eps, dtype, ws, size, s))
    if st != MRA_OK:
        raise MraError(st, where)
    if rows == 0 and dgate is not None:
        _call_on(index, stream, 0, lambda ws, s: dgate.zero_())     # an empty sum
    return dx, dh


def _layer_shape(x, w_qkv, H):
    if x.dim() != 3 or x.dtype != torch.bfloat16 or w_qkv.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 [B, N, hidden] and w_qkv bf16 [3*hidden, hidden]")
    B, N, hidden = (int(s) for s in x.shape)
    if tuple(w_qkv.shape) != (3 * hidden, hidden):
        raise ValueError("w_qkv must be [3*hidden, hidden]")
    return B, N, hidden


def mra_self_attention_fwd(x, w_qkv, b_qkv, key_mask, out, H, block_per_row, approx_mode, first_n, diag_n,
                           stream=None):
    """The MraSelfAttention layer on device tensors: x bf16 [B, N, hidden],
    w_qkv bf16 [3*hidden, hidden], b_qkv fp32 [3*hidden] or None, key_mask
    fp32 [B, N] or None; out bf16 [B, N, hidden] is written."""
    B, N, hidden = _layer_shape(x, w_qkv, H)
    st = load_library().mra_self_attention_fwd(_ptr(x), _ptr(w_qkv), _ptr(b_qkv), _ptr(key_mask), _ptr(out), B,
                                               N, hidden, H, block_per_row, _mode(approx_mode), first_n, diag_n,
                                               _stream(stream))
    _check(st, "mra_self_attention_fwd")
    return out


def mra_qkv_projection(x, w_qkv, b_qkv, qkv, H, stream=None):
    """The layer's projection alone: qkv bf16 [3, B, H, N, Dp] (Dp = 32 if
    hidden/H <= 32 else 64) gets the head-split, zero-padded Q (scaled by
    sqrt(Dp/d)), K and V."""
    B, N, hidden = _layer_shape(x, w_qkv, H)
    st = load_library().mra_qkv_projection(_ptr(x), _ptr(w_qkv), _ptr(b_qkv), _ptr(qkv), B, N, hidden, H,
                                           _stream(stream))
    _check(st, "mra_qkv_projection")
    return qkv


def mra_num_block(N: int, block_per_row: int) -> int:
    return int(load_library().mra_num_block(N, block_per_row))


def status_string(status: int) -> str:
    try:
        return load_library().mra_status_string(status).decode()
    except RuntimeError:
        return f"status {status}"


mra_status_string = status_string


def mra_get_device_status(stream=None) -> int:
    return int(load_library().mra_get_device_status(_stream(stream)))


def mra_get_noalloc_status(stream=None) -> int:
    """Reads and clears the status word of the no-allocation entry point."""
    return int(load_library().mra_get_noalloc_status(_stream(stream)))


def mra_status_from_device(word: int) -> int:
    """mra_status for a device status word (host-side mapping)."""
    return int(load_library().mra_status_from_device(int(word)))


def mra_profile_enable(enable: bool) -> None:
    load_library().mra_profile_enable(1 if enable else 0)


def mra_profile_read(max_phases: int = 16):
    """{phase: (launches, total_ms)} since the previous read."""
    names = (ctypes.c_char_p * max_phases)()
    launches = (ctypes.c_int * max_phases)()
    ms = (ctypes.c_double * max_phases)()
    n = load_library().mra_profile_read(names, launches, ms, max_phases)
    return {names[i].decode(): (launches[i], ms[i]) for i in range(n)}


def mra_last_launch_count() -> int:
    return int(load_library().mra_last_launch_count())


def mra2_attention(q, k, v, key_mask=None, *, block_per_row: int = 4, approx_mode="full",
                   first_n: int = 0, diag_n: int = 0, stream=None):
    """Allocate the output and run the forward pass on device tensors."""
    out = torch.empty_like(q)
    fn = mra_attention_fwd if q.dtype == torch.bfloat16 else mra_attention_fwd_f32
    return fn(q, k, v, key_mask, out, block_per_row, approx_mode, first_n, diag_n, stream)
