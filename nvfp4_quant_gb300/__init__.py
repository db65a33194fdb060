"""nvfp4_quant_gb300: Python binding of librq, the GB300 (sm_103a) library of
fused residual add + RMSNorm + FP8 / NVFP4 quantisation kernels, the per-head
Q/K RMSNorm + RoPE + FP8 store, and the paged NVFP4 KV cache: its append and
the attention that reads it.

This module only marshals arguments: it turns torch CUDA tensors into device
pointers and sizes, calls the C ABI (include/rq.h) through ctypes, and raises
RQError when a call returns a non-OK status.  Every step of the computation
runs in the CUDA kernels of librq.so; there is no other code path.  If the
library has not been built, importing works but the first call raises.
"""
import ctypes
import functools
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "librq.so")

RQ_BF16, RQ_FP16 = 0, 1
RQ_MAX_HIDDEN = 262144
RQ_QK_HEAD_DIM = 128
RQ_QK_MAX_HEADS = 65536
RQ_KV_MAX_PAGE = 65536
RQ_ATTN_MAX_KEYS = 1073741824
RQ_ATTN_MAX_TOKENS = 16777216
RQ_ATTN_MAX_SEQS = 1048576
STATUS = {0: "RQ_OK", 1: "RQ_ERR_NULL", 2: "RQ_ERR_SHAPE", 3: "RQ_ERR_DTYPE",
          4: "RQ_ERR_MISALIGNED", 5: "RQ_ERR_ALIAS", 6: "RQ_ERR_UNSUPPORTED", 7: "RQ_ERR_CUDA"}

# exported symbol -> (restype, argtypes)
_vp, _i64, _f32, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
_size = ctypes.c_size_t
SIGNATURES = {
    "rq_add_rmsnorm_fp8": (_int, [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _i64, _i64, _int, _vp]),
    "rq_add_rmsnorm_nvfp4": (_int, [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _i64, _i64,
                                    _int, _vp]),
    "rq_qk_rmsnorm_rope_fp8": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp, _vp,
                                      _f32, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _int, _vp]),
    "rq_qk_rmsnorm_rope_fp8_kv_store": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp,
                                               _vp, _f32, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                               _vp, _i64, _int, _vp]),
    "rq_qk_rmsnorm_rope_fp8_kv_store_mixed": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _int, _int,
                                                     _int, _vp, _vp, _f32, _vp, _vp, _i64, _vp,
                                                     _vp, _vp, _vp, _vp, _i64, _int, _vp]),
    "rq_qk_rmsnorm_rope_amax": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp, _vp,
                                       _f32, _vp, _vp, _i64, _vp, _vp, _int, _vp]),
    "rq_qk_rmsnorm_rope_fp8_dynamic": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp,
                                              _vp, _f32, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _int,
                                              _vp]),
    "rq_add_rmsnorm_amax": (_int, [_vp, _vp, _vp, _f32, _vp, _i64, _i64, _int, _vp]),
    "rq_add_rmsnorm_fp8_per_token": (_int, [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _i64, _i64,
                                            _int, _vp]),
    "rq_add_rmsnorm_fp8_dynamic": (_int, [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _i64, _i64,
                                          _int, _vp]),
    "rq_add_rmsnorm_nvfp4_dynamic": (_int, [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _i64,
                                            _i64, _int, _vp]),
    "rq_fp8_scale_from_amax": (_int, [_vp, _vp, _vp]),
    "rq_nvfp4_global_scale_from_amax": (_int, [_vp, _vp, _vp]),
    "rq_nvfp4_packed_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "rq_nvfp4_scale_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "rq_add_rmsnorm_nvfp4_swizzled": (_int, [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _i64,
                                             _i64, _int, _vp]),
    "rq_add_rmsnorm_nvfp4_dynamic_swizzled": (_int, [_vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp,
                                                     _i64, _i64, _int, _vp]),
    "rq_nvfp4_swizzled_scale_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "rq_gated_rmsnorm_nvfp4": (_int, [_vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _i64, _i64, _int,
                                      _vp]),
    "rq_gated_rmsnorm_nvfp4_swizzled": (_int, [_vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _i64, _i64,
                                               _int, _vp]),
    "rq_qkv_rope_nvfp4_kv_append": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int, _int,
                                           _vp, _vp, _f32, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                           _i64, _int, _vp, _int, _vp]),
    "rq_paged_decode_attn_nvfp4": (_int, [_vp, _i64, _i64, _int, _int, _int, _vp, _i64, _int, _vp,
                                          _i64, _i64, _vp, _f32, _int, _vp, _vp, _vp, _vp, _vp,
                                          _size, _int, _vp]),
    "rq_paged_extend_attn_nvfp4": (_int, [_vp, _i64, _i64, _vp, _i64, _i64, _int, _int, _int, _vp,
                                          _i64, _int, _vp, _i64, _i64, _vp, _f32, _int, _vp, _vp,
                                          _vp, _vp, _vp, _size, _int, _vp]),
    "rq_paged_attn_nvfp4_workspace_bytes": (_size, [_int, _int]),
    "rq_nvfp4_kv_page_bytes": (_size, [_int]),
    "rq_status_string": (ctypes.c_char_p, [_int]),
    "rq_last_error": (ctypes.c_char_p, []),
    "rq_version": (_int, []),
}

_lib = None


class RQError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(message)
        self.status = status


def lib():
    """The loaded librq.so (ctypes); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("librq.so is not built (%s); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        L = lib()
        msg = L.rq_status_string(status).decode()
        if status == 7:
            msg += " (" + L.rq_last_error().decode() + ")"
        raise RQError(status, msg)


def _dt(t):
    if t.dtype == torch.bfloat16:
        return RQ_BF16
    if t.dtype == torch.float16:
        return RQ_FP16
    raise ValueError("tensors must be bfloat16 or float16, got %s" % t.dtype)


def _ptr(t):
    """Device pointer of a CUDA tensor (None for None).  A host tensor is
    refused here: its address would reach the kernels as a device pointer."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("every tensor argument must be a CUDA tensor (got one on %s)" % t.device)
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _out(t, nbytes, name):
    """An output buffer: contiguous, on x's device, and at least nbytes long
    (the kernels write exactly the sizes include/rq.h gives)."""
    if t is None or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise ValueError("%s must be a contiguous tensor of at least %d bytes" % (name, nbytes))


def _rows(x, *others):
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [rows, hidden] tensor")
    for o in others:
        if o is not None and (o.shape != x.shape or o.dtype != x.dtype or not o.is_contiguous()):
            raise ValueError("residual / norm_out must match x in shape, dtype and be contiguous")
    return x.shape[0], x.shape[1]


def rq_add_rmsnorm_fp8(x, residual_in, residual_out, weight, eps, scale, q_out,
                       norm_out=None, stream=None):
    """Residual add + RMSNorm + per-tensor FP8 E4M3 (include/rq.h).
    scale: 1-element float32 CUDA tensor (dequant scale); q_out: uint8 [rows, hidden]."""
    rows, hidden = _rows(x, residual_in, residual_out, norm_out)
    if weight.dtype != x.dtype:
        raise ValueError("weight dtype must match x")
    _out(q_out, rows * hidden, "q_out")
    _check(lib().rq_add_rmsnorm_fp8(_ptr(x), _ptr(residual_in), _ptr(residual_out), _ptr(weight),
                                    float(eps), _ptr(scale), _ptr(q_out), _ptr(norm_out),
                                    rows, hidden, _dt(x), _stream(stream)))


def rq_add_rmsnorm_nvfp4(x, residual_in, residual_out, weight, eps, global_scale, q_packed,
                         block_scales, norm_out=None, stream=None):
    """Residual add + RMSNorm (+ norm out) + NVFP4 (include/rq.h).
    q_packed: uint8 [rows, hidden/2]; block_scales: uint8 [rows, hidden/16]."""
    rows, hidden = _rows(x, residual_in, residual_out, norm_out)
    if weight.dtype != x.dtype:
        raise ValueError("weight dtype must match x")
    _out(q_packed, rows * hidden // 2, "q_packed")
    _out(block_scales, rows * (hidden // 16), "block_scales")
    _check(lib().rq_add_rmsnorm_nvfp4(_ptr(x), _ptr(residual_in), _ptr(residual_out),
                                      _ptr(weight), float(eps), _ptr(global_scale),
                                      _ptr(q_packed), _ptr(block_scales), _ptr(norm_out),
                                      rows, hidden, _dt(x), _stream(stream)))


def rq_gated_rmsnorm_nvfp4(x, z, weight, eps, global_scale, q_packed, block_scales,
                           norm_out=None, stream=None):
    """Gated RMSNorm + NVFP4 (include/rq.h): g = dt(x * dt(silu(z))), RMSNorm,
    NVFP4.  q_packed: uint8 [rows, hidden/2]; block_scales: uint8 [rows, hidden/16]."""
    rows, hidden = _rows(x, z, norm_out)
    if weight.dtype != x.dtype:
        raise ValueError("weight dtype must match x")
    _out(q_packed, rows * hidden // 2, "q_packed")
    _out(block_scales, rows * (hidden // 16), "block_scales")
    _check(lib().rq_gated_rmsnorm_nvfp4(_ptr(x), _ptr(z), _ptr(weight), float(eps),
                                        _ptr(global_scale), _ptr(q_packed), _ptr(block_scales),
                                        _ptr(norm_out), rows, hidden, _dt(x), _stream(stream)))


def rq_gated_rmsnorm_nvfp4_swizzled(x, z, weight, eps, global_scale, q_packed, block_scales,
                                    norm_out=None, stream=None):
    """rq_gated_rmsnorm_nvfp4 with swizzled block scales (include/rq.h);
    block_scales: uint8 of rq_nvfp4_swizzled_scale_bytes(rows, hidden) bytes."""
    rows, hidden = _rows(x, z, norm_out)
    if weight.dtype != x.dtype:
        raise ValueError("weight dtype must match x")
    _out(q_packed, rows * hidden // 2, "q_packed")
    _out(block_scales, rq_nvfp4_swizzled_scale_bytes(rows, hidden), "block_scales")
    _check(lib().rq_gated_rmsnorm_nvfp4_swizzled(
        _ptr(x), _ptr(z), _ptr(weight), float(eps), _ptr(global_scale), _ptr(q_packed),
        _ptr(block_scales), _ptr(norm_out), rows, hidden, _dt(x), _stream(stream)))


def rq_add_rmsnorm_amax(x, residual_in, weight, eps, amax_out, stream=None):
    """amax_out[0] = max |RMSNorm(x + residual) * weight| (include/rq.h)."""
    rows, hidden = _rows(x, residual_in)
    _out(amax_out, 4, "amax_out")
    _check(lib().rq_add_rmsnorm_amax(_ptr(x), _ptr(residual_in), _ptr(weight), float(eps),
                                     _ptr(amax_out), rows, hidden, _dt(x), _stream(stream)))


def rq_add_rmsnorm_fp8_per_token(x, residual_in, residual_out, weight, eps, q_out, row_scales,
                                 norm_out=None, stream=None):
    """Residual add + RMSNorm + FP8 with per-row dynamic scales (include/rq.h).
    row_scales: float32 [rows], written."""
    rows, hidden = _rows(x, residual_in, residual_out, norm_out)
    _out(q_out, rows * hidden, "q_out")
    _out(row_scales, rows * 4, "row_scales")
    _check(lib().rq_add_rmsnorm_fp8_per_token(_ptr(x), _ptr(residual_in), _ptr(residual_out),
                                              _ptr(weight), float(eps), _ptr(q_out),
                                              _ptr(row_scales), _ptr(norm_out), rows, hidden,
                                              _dt(x), _stream(stream)))


def rq_add_rmsnorm_fp8_dynamic(x, residual_in, residual_out, weight, eps, scale_out, q_out,
                               norm_out=None, stream=None):
    """Residual add + RMSNorm + FP8 with the per-tensor scale amax/448 computed
    on the device (include/rq.h); scale_out: 1-element float32, written."""
    rows, hidden = _rows(x, residual_in, residual_out, norm_out)
    _out(q_out, rows * hidden, "q_out")
    _out(scale_out, 4, "scale_out")
    _check(lib().rq_add_rmsnorm_fp8_dynamic(_ptr(x), _ptr(residual_in), _ptr(residual_out),
                                            _ptr(weight), float(eps), _ptr(scale_out), _ptr(q_out),
                                            _ptr(norm_out), rows, hidden, _dt(x), _stream(stream)))


def rq_add_rmsnorm_nvfp4_dynamic(x, residual_in, residual_out, weight, eps, global_scale_out,
                                 q_packed, block_scales, norm_out=None, stream=None):
    """Residual add + RMSNorm + NVFP4 with the global scale 2688/amax computed
    on the device (include/rq.h); global_scale_out: 1-element float32, written."""
    rows, hidden = _rows(x, residual_in, residual_out, norm_out)
    _out(q_packed, rows * hidden // 2, "q_packed")
    _out(block_scales, rows * (hidden // 16), "block_scales")
    _out(global_scale_out, 4, "global_scale_out")
    _check(lib().rq_add_rmsnorm_nvfp4_dynamic(_ptr(x), _ptr(residual_in), _ptr(residual_out),
                                              _ptr(weight), float(eps), _ptr(global_scale_out),
                                              _ptr(q_packed), _ptr(block_scales), _ptr(norm_out),
                                              rows, hidden, _dt(x), _stream(stream)))


def rq_add_rmsnorm_nvfp4_swizzled(x, residual_in, residual_out, weight, eps, global_scale,
                                  q_packed, block_scales, norm_out=None, stream=None):
    """rq_add_rmsnorm_nvfp4 with the block scales in the 128 x 4-tile layout a
    block-scaled NVFP4 GEMM reads (include/rq.h); block_scales: uint8 of
    rq_nvfp4_swizzled_scale_bytes(rows, hidden) bytes, every byte written."""
    rows, hidden = _rows(x, residual_in, residual_out, norm_out)
    if weight.dtype != x.dtype:
        raise ValueError("weight dtype must match x")
    _out(q_packed, rows * hidden // 2, "q_packed")
    _out(block_scales, rq_nvfp4_swizzled_scale_bytes(rows, hidden), "block_scales")
    _check(lib().rq_add_rmsnorm_nvfp4_swizzled(_ptr(x), _ptr(residual_in), _ptr(residual_out),
                                               _ptr(weight), float(eps), _ptr(global_scale),
                                               _ptr(q_packed), _ptr(block_scales), _ptr(norm_out),
                                               rows, hidden, _dt(x), _stream(stream)))


def rq_add_rmsnorm_nvfp4_dynamic_swizzled(x, residual_in, residual_out, weight, eps,
                                          global_scale_out, q_packed, block_scales,
                                          norm_out=None, stream=None):
    """rq_add_rmsnorm_nvfp4_dynamic with swizzled block scales (include/rq.h)."""
    rows, hidden = _rows(x, residual_in, residual_out, norm_out)
    _out(q_packed, rows * hidden // 2, "q_packed")
    _out(block_scales, rq_nvfp4_swizzled_scale_bytes(rows, hidden), "block_scales")
    _out(global_scale_out, 4, "global_scale_out")
    _check(lib().rq_add_rmsnorm_nvfp4_dynamic_swizzled(
        _ptr(x), _ptr(residual_in), _ptr(residual_out), _ptr(weight), float(eps),
        _ptr(global_scale_out), _ptr(q_packed), _ptr(block_scales), _ptr(norm_out), rows, hidden,
        _dt(x), _stream(stream)))


def rq_fp8_scale_from_amax(amax, scale_out, stream=None):
    _check(lib().rq_fp8_scale_from_amax(_ptr(amax), _ptr(scale_out), _stream(stream)))


def rq_nvfp4_global_scale_from_amax(amax, gs_out, stream=None):
    _check(lib().rq_nvfp4_global_scale_from_amax(_ptr(amax), _ptr(gs_out), _stream(stream)))


def _heads(t):
    """(n_tokens, n_heads, token_stride) of a [T, H, 128] view with dense heads."""
    if t is None:
        return 0, 0, 0
    if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
        raise ValueError("q / k must be [tokens, heads, head_dim] views with contiguous heads")
    return t.shape[0], t.shape[1], t.stride(0)


def _qk_buffers(ref, hq, hk, positions, cos_sin_cache, q_out, k_out, rope_dim=None, outs=True):
    """Sizes of the Q/K call's side inputs and dense outputs (k_out None: pool;
    outs False: a call without code outputs)."""
    t, d = ref.shape[0], ref.shape[2]
    if t == 0:
        return
    if positions is None or positions.numel() < t:
        raise ValueError("positions must hold one int32 per token")
    cols = d if rope_dim is None else rope_dim
    if cos_sin_cache is None or cos_sin_cache.dim() != 2 or cos_sin_cache.shape[1] != cols:
        raise ValueError("cos_sin_cache must be a [max_pos, %d] float32 tensor" % cols)
    if not outs:
        return
    if hq > 0:
        _out(q_out, t * hq * d, "q_out")
    if hk > 0 and k_out is not None:
        _out(k_out, t * hk * d, "k_out")


def rq_qk_rmsnorm_rope_fp8(q, k, q_weight, k_weight, eps, positions, cos_sin_cache,
                           q_scale, k_scale, q_out, k_out, stream=None):
    """Per-head Q/K RMSNorm + NeoX RoPE + FP8 E4M3 store (include/rq.h).
    q / k may be token-strided views into a fused QKV buffer."""
    tq, hq, sq = _heads(q)
    tk, hk, sk = _heads(k)
    ref = q if q is not None else k
    if q is not None and k is not None and (tq != tk or q.dtype != k.dtype):
        raise ValueError("q and k must have the same token count and dtype")
    head_dim = ref.shape[2]
    _qk_buffers(ref, hq, hk, positions, cos_sin_cache, q_out, k_out)
    _check(lib().rq_qk_rmsnorm_rope_fp8(
        _ptr(q), _ptr(k), sq, sk, ref.shape[0], hq, hk, head_dim, _ptr(q_weight),
        _ptr(k_weight), float(eps), _ptr(positions), _ptr(cos_sin_cache),
        cos_sin_cache.shape[0], _ptr(q_scale), _ptr(k_scale), _ptr(q_out), _ptr(k_out),
        _dt(ref), _stream(stream)))


def rq_qk_rmsnorm_rope_fp8_kv_store(q, k, q_weight, k_weight, eps, positions, cos_sin_cache,
                                    q_scale, k_scale, q_out, k_pool, k_slots, stream=None):
    """Q/K RMSNorm + RoPE + FP8 with K stored into a KV pool (include/rq.h):
    k_pool uint8 [num_slots, n_k_heads, 128]; k_slots int64 [n_tokens]."""
    tq, hq, sq = _heads(q)
    tk, hk, sk = _heads(k)
    ref = q if q is not None else k
    if q is not None and k is not None and (tq != tk or q.dtype != k.dtype):
        raise ValueError("q and k must have the same token count and dtype")
    _qk_buffers(ref, hq, hk, positions, cos_sin_cache, q_out, None)
    if hk > 0 and ref.shape[0] > 0:
        if k_pool is None or k_pool.dim() != 3 or k_pool.shape[1:] != (hk, ref.shape[2]) \
                or not k_pool.is_contiguous():
            raise ValueError("k_pool must be a contiguous [num_slots, n_k_heads, head_dim] tensor")
        if k_slots is None or k_slots.dtype != torch.int64 or k_slots.numel() < ref.shape[0]:
            raise ValueError("k_slots must hold one int64 slot per token")
    _check(lib().rq_qk_rmsnorm_rope_fp8_kv_store(
        _ptr(q), _ptr(k), sq, sk, ref.shape[0], hq, hk, ref.shape[2], _ptr(q_weight),
        _ptr(k_weight), float(eps), _ptr(positions), _ptr(cos_sin_cache), cos_sin_cache.shape[0],
        _ptr(q_scale), _ptr(k_scale), _ptr(q_out), _ptr(k_pool), _ptr(k_slots),
        0 if k_pool is None else k_pool.shape[0], _dt(ref), _stream(stream)))


def _qk_pair(q, k):
    tq, hq, sq = _heads(q)
    tk, hk, sk = _heads(k)
    ref = q if q is not None else k
    if q is not None and k is not None and (tq != tk or q.dtype != k.dtype):
        raise ValueError("q and k must have the same token count and dtype")
    return ref, hq, sq, hk, sk


def rq_qk_rmsnorm_rope_fp8_kv_store_mixed(q, k, q_weight, k_weight, eps, positions,
                                          cos_sin_cache, q_scale, k_scale, q_out, k_pool, k_slots,
                                          rope_dim, stream=None):
    """Q/K RMSNorm + NeoX RoPE on the last rope_dim elements of each head; Q's
    FP8 codes dense, K into a mixed KV pool (include/rq.h): k_pool uint8
    [num_slots, n_k_heads, head_dim + rope_dim] (E4M3 of the first head_dim -
    rope_dim elements, then rope_dim dtype values); cos_sin_cache float32
    [max_pos, rope_dim]; k_slots int64 [n_tokens]."""
    ref, hq, sq, hk, sk = _qk_pair(q, k)
    _qk_buffers(ref, hq, hk, positions, cos_sin_cache, q_out, None, rope_dim)
    if hk > 0 and ref.shape[0] > 0:
        row = ref.shape[2] + rope_dim
        if k_pool is None or k_pool.dim() != 3 or k_pool.shape[1:] != (hk, row) \
                or not k_pool.is_contiguous():
            raise ValueError("k_pool must be a contiguous [num_slots, n_k_heads, %d] tensor" % row)
        if k_slots is None or k_slots.dtype != torch.int64 or k_slots.numel() < ref.shape[0]:
            raise ValueError("k_slots must hold one int64 slot per token")
    _check(lib().rq_qk_rmsnorm_rope_fp8_kv_store_mixed(
        _ptr(q), _ptr(k), sq, sk, ref.shape[0], hq, hk, ref.shape[2], int(rope_dim),
        _ptr(q_weight), _ptr(k_weight), float(eps), _ptr(positions), _ptr(cos_sin_cache),
        cos_sin_cache.shape[0], _ptr(q_scale), _ptr(k_scale), _ptr(q_out), _ptr(k_pool),
        _ptr(k_slots), 0 if k_pool is None else k_pool.shape[0], _dt(ref), _stream(stream)))


def rq_qk_rmsnorm_rope_amax(q, k, q_weight, k_weight, eps, positions, cos_sin_cache, q_amax,
                            k_amax, stream=None):
    """q_amax[0] / k_amax[0] = max |o| over Q / K, o the dtype-rounded output of
    the Q/K RMSNorm + RoPE (include/rq.h); they may be the same tensor."""
    ref, hq, sq, hk, sk = _qk_pair(q, k)
    _qk_buffers(ref, hq, hk, positions, cos_sin_cache, None, None, outs=False)
    if hq > 0:
        _out(q_amax, 4, "q_amax")
    if hk > 0:
        _out(k_amax, 4, "k_amax")
    _check(lib().rq_qk_rmsnorm_rope_amax(
        _ptr(q), _ptr(k), sq, sk, ref.shape[0], hq, hk, ref.shape[2], _ptr(q_weight),
        _ptr(k_weight), float(eps), _ptr(positions), _ptr(cos_sin_cache), cos_sin_cache.shape[0],
        _ptr(q_amax), _ptr(k_amax), _dt(ref), _stream(stream)))


def rq_qk_rmsnorm_rope_fp8_dynamic(q, k, q_weight, k_weight, eps, positions, cos_sin_cache,
                                   q_scale_out, k_scale_out, q_out, k_out, stream=None):
    """The Q/K call with per-tensor scales amax(o) / 448 computed on the device
    (include/rq.h); q_scale_out / k_scale_out: 1-element float32, written."""
    ref, hq, sq, hk, sk = _qk_pair(q, k)
    _qk_buffers(ref, hq, hk, positions, cos_sin_cache, q_out, k_out)
    if hq > 0:
        _out(q_scale_out, 4, "q_scale_out")
    if hk > 0:
        _out(k_scale_out, 4, "k_scale_out")
    _check(lib().rq_qk_rmsnorm_rope_fp8_dynamic(
        _ptr(q), _ptr(k), sq, sk, ref.shape[0], hq, hk, ref.shape[2], _ptr(q_weight),
        _ptr(k_weight), float(eps), _ptr(positions), _ptr(cos_sin_cache), cos_sin_cache.shape[0],
        _ptr(q_scale_out), _ptr(k_scale_out), _ptr(q_out), _ptr(k_out), _dt(ref),
        _stream(stream)))


# ------------------------------------------------------- paged NVFP4 KV cache
# These calls are short (a decode step's append runs for 4 us on the GPU), so
# their checks are kept to the cheapest torch queries.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_I32, _I64, _F32, _U8 = torch.int32, torch.int64, torch.float32, torch.uint8


def _same_device(tensors):
    """The index of the device that every given tensor lies on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            break
    else:
        if dev >= 0:
            return dev
        t = tensors[0]
    raise ValueError("every tensor argument must be a CUDA tensor on one device (got %s and %s)"
                     % (tensors[0].device, t.device))


def _call_on(dev, fn, args, stream):
    """fn(*args, stream) with the tensors' device current; stream None is that
    device's current stream."""
    if stream is None:
        stream = _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    else:
        stream = getattr(stream, "cuda_stream", stream)
    if _current_device() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status)


def _typed(t, dtype, numel, name):
    """A contiguous tensor of at least numel elements of a type."""
    if t is None or t.dtype is not dtype or t.numel() < numel or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of at least %d elements"
                         % (name, str(dtype).replace("torch.", ""), numel))
    return t.data_ptr()


def _cache(kv_pool, page_size, heads):
    shape = kv_pool.shape
    if len(shape) != 3 or kv_pool.dtype is not _U8 or shape[1] != heads or \
            shape[2] != page_size * 144 or not kv_pool.is_contiguous():
        raise ValueError("kv_pool must be a contiguous uint8 [num_pages, n_kv_heads, page_size * 144] "
                         "tensor with %d heads" % heads)
    return kv_pool.data_ptr(), shape[0], int(page_size)


def _head_rows(t, name, like=None):
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or stride[2] != 1 or stride[1] != shape[2]:
        raise ValueError("%s must be a [tokens, heads, head_dim] view with contiguous heads" % name)
    if like is not None and (shape[0] != like.shape[0] or t.dtype != like.dtype
                             or shape[2] != like.shape[2]):
        raise ValueError("%s must match q in token count, head_dim and dtype" % name)
    # a single token's stride says nothing (torch leaves any value there)
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1] * shape[2]


def rq_qkv_rope_nvfp4_kv_append(q, k, v, q_weight, k_weight, eps, positions, cos_sin_cache,
                                k_global_scale, v_global_scale, q_out, kv_pool, slots, page_size,
                                stream=None):
    """Append K and V to a paged NVFP4 cache with the per-head norm (a None
    weight: no norm) and RoPE on the way, and write the rotated queries
    (include/rq.h).  q [T, Hq, 128], k, v [T, Hk, 128] may be token-strided
    views; q_out [T, Hq, 128]; kv_pool uint8 [pages, Hk, page_size * 144];
    slots int64 [T] (page * page_size + index; outside the cache: not stored)."""
    _append(q, k, v, q_weight, k_weight, eps, positions, cos_sin_cache, k_global_scale, v_global_scale,
            q_out, kv_pool, slots, page_size, stream, False)


def _append(q, k, v, q_weight, k_weight, eps, positions, cos_sin_cache, k_global_scale, v_global_scale,
            q_out, kv_pool, slots, page_size, stream, made):
    # made: q_out was allocated here for q, and needs no check
    dev = _same_device((q, k, v, q_weight, k_weight, positions, cos_sin_cache, k_global_scale,
                        v_global_scale, kv_pool, slots, None if made else q_out))
    qp, qs = _head_rows(q, "q")
    kp, ks = _head_rows(k, "k", q)
    vp, vs = _head_rows(v, "v", q)
    t, hq, d = q.shape
    hk = k.shape[1]
    if v.shape[1] != hk:
        raise ValueError("k and v must have the same heads")
    dtype = q.dtype
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not dtype or w.numel() != d or not w.is_contiguous()):
            raise ValueError("weights must be [head_dim] of q's dtype")
    table = cos_sin_cache.shape
    if cos_sin_cache.dtype is not _F32 or len(table) != 2 or table[1] != d or \
            not cos_sin_cache.is_contiguous():
        raise ValueError("cos_sin_cache must be a contiguous [max_pos, %d] float32 tensor" % d)
    pool, pages, page = _cache(kv_pool, page_size, hk)
    _call_on(dev, lib().rq_qkv_rope_nvfp4_kv_append, (
        qp, kp, vp, qs, ks, vs, t, hq, hk, d, None if q_weight is None else q_weight.data_ptr(),
        None if k_weight is None else k_weight.data_ptr(), eps, _typed(positions, _I32, t, "positions"),
        cos_sin_cache.data_ptr(), table[0], _typed(k_global_scale, _F32, 1, "k_global_scale"),
        _typed(v_global_scale, _F32, 1, "v_global_scale"),
        q_out.data_ptr() if made else _typed(q_out, dtype, t * hq * d, "q_out"),
        pool, pages, page, _typed(slots, _I64, t, "slots"), _dt(q)), stream)


def _paged_attn(q, kv_pool, page_size, block_table, q_starts, max_q_len, kv_lens, k_gs, v_gs,
                sm_scale, out, workspace, window, lse, stream, made=False):
    # made: out and lse were allocated here for q, and need no check
    dev = _same_device((q, kv_pool, block_table, q_starts, kv_lens, k_gs, v_gs, workspace) if made else
                       (q, kv_pool, block_table, q_starts, kv_lens, k_gs, v_gs, workspace, out, lse))
    qp, qs = _head_rows(q, "q")
    t, hq, d = q.shape
    hk = kv_pool.shape[1] if kv_pool.dim() == 3 else 0
    if hk < 1 or hq % hk != 0:
        raise ValueError("q's heads must be a multiple of the cache's")
    pool, pages, page = _cache(kv_pool, page_size, hk)
    if block_table.dtype is not _I32 or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 [n_seqs, pages_per_seq] tensor")
    n, per = block_table.shape
    row, col = block_table.stride()
    if col != 1 and per > 1:
        raise ValueError("block_table's rows must be contiguous")
    if n < 2:
        row = per
    if workspace is None or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    tail = (_typed(kv_lens, _I32, n, "kv_lens"), sm_scale, window, _typed(k_gs, _F32, 1, "k_global_scale"),
            _typed(v_gs, _F32, 1, "v_global_scale"),
            out.data_ptr() if made else _typed(out, q.dtype, t * hq * d, "out"),
            None if lse is None else lse.data_ptr() if made else _typed(lse, _F32, t * hq, "lse"), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _dt(q))
    if q_starts is None:
        if t != n:
            raise ValueError("q must hold one query per sequence")
        _call_on(dev, lib().rq_paged_decode_attn_nvfp4, (
            qp, qs, n, hq, hk, d, pool, pages, page, block_table.data_ptr(), row, per) + tail, stream)
    else:
        _call_on(dev, lib().rq_paged_extend_attn_nvfp4, (
            qp, qs, t, _typed(q_starts, _I32, n + 1, "q_starts"), n, max_q_len, hq, hk, d, pool, pages,
            page, block_table.data_ptr(), row, per) + tail, stream)


def rq_paged_decode_attn_nvfp4(q, kv_pool, page_size, block_table, kv_lens, k_global_scale,
                               v_global_scale, sm_scale, out, workspace, window=0, lse=None,
                               stream=None):
    """Attention of one query per sequence over a paged NVFP4 cache
    (include/rq.h).  q, out [n_seqs, Hq, 128]; block_table int32 [n_seqs,
    pages_per_seq]; kv_lens int32 [n_seqs]; lse float32 [n_seqs, Hq] or None;
    workspace: rq_paged_attn_nvfp4_workspace_bytes(Hq, Hk) bytes, not shared by
    calls that may run at the same time."""
    _paged_attn(q, kv_pool, page_size, block_table, None, 1, kv_lens, k_global_scale,
                v_global_scale, sm_scale, out, workspace, window, lse, stream)


def rq_paged_extend_attn_nvfp4(q, kv_pool, page_size, block_table, q_starts, kv_lens, max_q_len,
                               k_global_scale, v_global_scale, sm_scale, out, workspace, window=0,
                               lse=None, stream=None):
    """Causal attention of each sequence's last queries over a paged NVFP4
    cache (include/rq.h).  q, out [tokens, Hq, 128], sequence b's rows
    q_starts[b] .. q_starts[b + 1] - 1 (int32 [n_seqs + 1]); kv_lens counts the
    new tokens too; max_q_len: the longest run of queries (a bound)."""
    if q_starts is None:
        raise ValueError("q_starts must be an int32 [n_seqs + 1] tensor")
    _paged_attn(q, kv_pool, page_size, block_table, q_starts, max_q_len, kv_lens, k_global_scale,
                v_global_scale, sm_scale, out, workspace, window, lse, stream)


@functools.lru_cache(maxsize=None)
def rq_paged_attn_nvfp4_workspace_bytes(n_q_heads, n_kv_heads):
    return int(lib().rq_paged_attn_nvfp4_workspace_bytes(n_q_heads, n_kv_heads))


def rq_nvfp4_kv_page_bytes(page_size):
    return int(lib().rq_nvfp4_kv_page_bytes(page_size))


def rq_nvfp4_packed_bytes(rows, hidden):
    return int(lib().rq_nvfp4_packed_bytes(rows, hidden))


def rq_nvfp4_scale_bytes(rows, hidden):
    return int(lib().rq_nvfp4_scale_bytes(rows, hidden))


def rq_nvfp4_swizzled_scale_bytes(rows, hidden):
    return int(lib().rq_nvfp4_swizzled_scale_bytes(rows, hidden))


# ---------------------------------------------------------------- conveniences
def _nvfp4_outputs(x, rows, hidden, swizzled):
    q = torch.empty((rows, hidden // 2), dtype=torch.uint8, device=x.device)
    if swizzled:
        sf = torch.empty((rq_nvfp4_swizzled_scale_bytes(rows, hidden),), dtype=torch.uint8,
                         device=x.device)
    else:
        sf = torch.empty((rows, hidden // 16), dtype=torch.uint8, device=x.device)
    return q, sf


def add_rmsnorm_nvfp4(x, residual, weight, eps, global_scale, with_norm_out=False,
                      in_place=True, swizzled=False, stream=None):
    """Allocate the outputs (torch) and run rq_add_rmsnorm_nvfp4 (or, with
    swizzled, rq_add_rmsnorm_nvfp4_swizzled: block_scales then is the flat
    buffer in the GEMM's tile layout).  Returns (residual_out, q_packed,
    block_scales, norm_out or None)."""
    rows, hidden = _rows(x, residual)
    res_out = residual if in_place else torch.empty_like(x)
    q, sf = _nvfp4_outputs(x, rows, hidden, swizzled)
    y = torch.empty_like(x) if with_norm_out else None
    call = rq_add_rmsnorm_nvfp4_swizzled if swizzled else rq_add_rmsnorm_nvfp4
    call(x, residual, res_out, weight, eps, global_scale, q, sf, y, stream)
    return res_out, q, sf, y


def gated_rmsnorm_nvfp4(x, z, weight, eps, global_scale, with_norm_out=False, swizzled=False,
                        stream=None):
    """Allocate the outputs (torch) and run rq_gated_rmsnorm_nvfp4 (or its
    swizzled form).  Returns (q_packed, block_scales, norm_out or None)."""
    rows, hidden = _rows(x, z)
    q, sf = _nvfp4_outputs(x, rows, hidden, swizzled)
    y = torch.empty_like(x) if with_norm_out else None
    call = rq_gated_rmsnorm_nvfp4_swizzled if swizzled else rq_gated_rmsnorm_nvfp4
    call(x, z, weight, eps, global_scale, q, sf, y, stream)
    return q, sf, y


def qk_rmsnorm_rope_fp8(q, k, q_weight, k_weight, eps, positions, cos_sin_cache, q_scale,
                        k_scale, stream=None):
    """Allocate dense FP8 outputs (torch) and run rq_qk_rmsnorm_rope_fp8.
    Returns (q_out [T, Hq, 128], k_out [T, Hk, 128]); either is None when its
    input is None."""
    q_out = None if q is None else torch.empty(tuple(q.shape), dtype=torch.uint8, device=q.device)
    k_out = None if k is None else torch.empty(tuple(k.shape), dtype=torch.uint8, device=k.device)
    rq_qk_rmsnorm_rope_fp8(q, k, q_weight, k_weight, eps, positions, cos_sin_cache, q_scale,
                           k_scale, q_out, k_out, stream)
    return q_out, k_out


def add_rmsnorm_fp8(x, residual, weight, eps, scale, with_norm_out=False, in_place=True,
                    stream=None):
    """Allocate the outputs (torch) and run rq_add_rmsnorm_fp8.  Returns
    (residual_out, q, norm_out or None)."""
    rows, hidden = _rows(x, residual)
    res_out = residual if in_place else torch.empty_like(x)
    q = torch.empty((rows, hidden), dtype=torch.uint8, device=x.device)
    y = torch.empty_like(x) if with_norm_out else None
    rq_add_rmsnorm_fp8(x, residual, res_out, weight, eps, scale, q, y, stream)
    return res_out, q, y


def _on_stream(stream, device):
    """A context in which allocations come from `stream`'s pool, so that a
    buffer's memory is not handed out again while that stream still uses it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def nvfp4_kv_pool(num_pages, n_kv_heads, page_size, device="cuda"):
    """An empty paged NVFP4 KV cache: zeroed uint8 [pages, heads, page_size * 144]."""
    nbytes = rq_nvfp4_kv_page_bytes(page_size)
    if nbytes == 0:
        raise ValueError("page_size must be a positive multiple of 16, at most %d" % RQ_KV_MAX_PAGE)
    return torch.zeros((num_pages, n_kv_heads, nbytes), dtype=torch.uint8, device=device)


def qkv_rope_nvfp4_kv_append(q, k, v, q_weight, k_weight, eps, positions, cos_sin_cache,
                             k_global_scale, v_global_scale, kv_pool, slots, page_size, stream=None):
    """Allocate q_out (torch) and run rq_qkv_rope_nvfp4_kv_append.  Returns
    q_out [T, Hq, 128]."""
    if stream is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        with _on_stream(stream, q.device):
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    _append(q, k, v, q_weight, k_weight, eps, positions, cos_sin_cache, k_global_scale, v_global_scale,
            q_out, kv_pool, slots, page_size, stream, True)
    return q_out


def _attn_buffers(q, kv_pool, with_lse, workspace, stream):
    if q.dim() != 3 or kv_pool.dim() != 3:
        raise ValueError("q and kv_pool must have three dimensions")
    if stream is not None:
        with _on_stream(stream, q.device):
            return _attn_buffers(q, kv_pool, with_lse, workspace, None)
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = q.new_empty(q.shape[:2], dtype=_F32) if with_lse else None
    if workspace is None:
        workspace = q.new_empty((rq_paged_attn_nvfp4_workspace_bytes(q.shape[1], kv_pool.shape[1]),), dtype=_U8)
    return out, lse, workspace


def paged_decode_attn_nvfp4(q, kv_pool, page_size, block_table, kv_lens, k_global_scale,
                            v_global_scale, sm_scale, window=0, with_lse=False, workspace=None,
                            stream=None):
    """Allocate the outputs (and, unless given, the workspace) and run
    rq_paged_decode_attn_nvfp4.  Returns (out, lse or None)."""
    out, lse, workspace = _attn_buffers(q, kv_pool, with_lse, workspace, stream)
    _paged_attn(q, kv_pool, page_size, block_table, None, 1, kv_lens, k_global_scale,
                v_global_scale, sm_scale, out, workspace, window, lse, stream, True)
    return out, lse


def paged_extend_attn_nvfp4(q, kv_pool, page_size, block_table, q_starts, kv_lens, max_q_len,
                            k_global_scale, v_global_scale, sm_scale, window=0, with_lse=False,
                            workspace=None, stream=None):
    """Allocate the outputs (and, unless given, the workspace) and run
    rq_paged_extend_attn_nvfp4.  Returns (out, lse or None); rows of out behind
    the last sequence are not written."""
    if q_starts is None:
        raise ValueError("q_starts must be an int32 [n_seqs + 1] tensor")
    out, lse, workspace = _attn_buffers(q, kv_pool, with_lse, workspace, stream)
    _paged_attn(q, kv_pool, page_size, block_table, q_starts, max_q_len, kv_lens, k_global_scale,
                v_global_scale, sm_scale, out, workspace, window, lse, stream, True)
    return out, lse
