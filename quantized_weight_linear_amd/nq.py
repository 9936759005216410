"""ctypes binding of libnq.so, with the C function names.

Argument marshalling only: each wrapper checks that tensors are contiguous,
passes their device pointers and sizes to the C entry point of the same name
on the current HIP stream, and raises NQError on a non-zero status.  Every
step of the computation runs in the library's HIP kernels; there is no
fallback.  BF16 / FP16 tensors may be passed as torch.bfloat16 / float16 or as
16-bit integer bit patterns.
"""

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnq.so")

NQ_OK, NQ_ERR_NULL, NQ_ERR_SHAPE, NQ_ERR_ALIGN, NQ_ERR_FORMAT, NQ_ERR_RANGE, NQ_ERR_HIP, NQ_ERR_SCRATCH = range(8)
NQ_GEMV_STATIC_SCRATCH_BYTES = 8 << 20
NQ_OUT_F32, NQ_OUT_BF16 = 0, 1
NQ_W_Q4G64_F16S, NQ_W_Q8G32_F16S, NQ_W_Q8G64_F16S, NQ_W_MXFP8_G32, NQ_W_BF16 = range(5)
NQ_W_Q3G64_F16S, NQ_W_Q5G64_F16S, NQ_W_Q6G64_F16S = 5, 6, 7
NQ_ROUTE_BF16, NQ_ROUTE_A8, NQ_ROUTE_A8_DECODE = 0, 1, 2
NQ_A8_PREFILL, NQ_A8_DECODE = 1, 2
NQ_KV_BF16, NQ_KV_E4M3, NQ_KV_E4M3_TOKEN = 0, 1, 3
NQ_ACT_BF16, NQ_ACT_INT8_G64, NQ_ACT_E4M3_B128 = 0, 1, 2
NQ_ROPE_HALVES, NQ_ROPE_PAIRS = 0, 1

# every entry point the header declares: name -> (restype, argtypes)
_P, _I64, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "nq_abi_version": (ctypes.c_int, []),
    "nq_status_string": (ctypes.c_char_p, [_I]),
    "nq_decode_mxfp8": (_I, [_P, _P, _I64, _I64, _I, _P, _P]),
    "nq_decode_mlx_affine_int8": (_I, [_P, _P, _P, _I64, _I64, _I, _P, _P]),
    "nq_reencode_block128_to_row": (_I, [_P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _P]),
    "nq_encode_fp8row_bf16": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "nq_quantize_act_int8_g64": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "nq_quantize_act_fp8_row": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "nq_gemv_workspace_bytes": (_I64, [_I, _I64, _I64, _I64]),
    "nq_gemv_fp8row": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _I64, _P]),
    "nq_gemv_qgroup": (_I, [_I, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _I64, _P]),
    "nq_gemm_w8a8_g64": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P]),
    "nq_gemm_fp8row": (_I, [_P, _P, _P, _I64, _I64, _I64, _P, _P, _I, _P, _P]),
    "nq_route": (_I, [_I64, _I]),
    "nq_packed_weight_bytes": (_I64, [_I, _I64, _I64]),
    "nq_pack_weights": (_I, [_I, _P, _I64, _I64, _P, _P]),
    "nq_gemv_fp8row_packed": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _I64, _P]),
    "nq_gemv_qgroup_packed": (_I, [_I, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _I64, _P]),
    "nq_gemv_fp8row_packed_noalloc": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P]),
    "nq_stream_read_sink_words": (_I64, []),
    "nq_unpack_qbits_to_int8": (_I, [_I, _P, _I64, _I64, _P, _P]),
    "nq_linear_qbits_g64": (_I, [_I, _P, _I64, _P, _P, _I64, _I64, _I, _P, _P, _P, _I, _P, _P, _I64, _P]),
    "nq_gemv_a8_workspace_bytes": (_I64, [_I64, _I64, _I64]),
    "nq_gemv_a8_g64": (_I, [_I, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _I64, _P]),
    "nq_gemv_a8_g64_packed": (_I, [_I, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _I64, _P]),
    "nq_stream_read": (_I, [_P, _I64, _P, _P]),
    "nq_linear_q8g64": (_I, [_P, _I64, _P, _P, _I64, _I64, _I, _P, _P, _I, _P, _P, _I64, _P]),
    "nq_unpack_q4_to_int8": (_I, [_P, _I64, _I64, _P, _P]),
    "nq_linear_q4g64": (_I, [_P, _I64, _P, _P, _I64, _I64, _I, _P, _P, _P, _I, _P, _P, _I64, _P]),
    "nq_quantize_act_fp8_b128": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "nq_rmsnorm": (_I, [_I, _P, _I64, _P, _P, _P, _F, _F, _I64, _I64, _P, _P, _P]),
    "nq_gemm_fp8_b128_workspace_bytes": (_I64, [_I64] * 3),
    "nq_gemm_fp8_b128": (_I, [_P] * 4 + [_I64] * 5 + [_I, _P, _P, _I64, _P]),
    "nq_kv_append_rope": (_I, [_I] + [_P, _I64] * 3 + [_P, _P, _F, _F, _P, _P, _I64, _I, _P, _P, _P, _I64, _P, _P] + [_I64] * 7 +
                          [_P, _I64, _P, _I64, _P, _P, _P]),
    "nq_attn_prompt": (_I, [_P, _I64] * 3 + [_P, _P] + [_I64] * 6 + [_F, _I, _P, _P, _P]),
    "nq_kv_append": (_I, [_I] + [_P, _I64] * 2 + [_P, _P, _P, _I64, _P, _P] + [_I64] * 6 + [_P, _P, _P]),
    "nq_attn_tree_workspace_bytes": (_I64, [_I64] * 6),
    "nq_attn_tree": (_I, [_I, _P, _I64, _P, _P, _P, _P, _P, _I64, _P, _P, _P] + [_I64] * 9 +
                     [_F, _I, _P, _P, _P, _I64, _P]),
    "nq_kv_reserve": (_I, [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _P, _P, _P]),
    "nq_kv_release": (_I, [_P, _I64, _P, _I64, _P, _I64, _I64, _P]),
    "nq_kv_fork": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    "nq_kv_copy_pages": (_I, [_P, _I64, _I64, _I64, _I64, _P, _I64, _P]),
    "nq_kv_compact": (_I, [_P] + [_I64] * 6 + [_P, _I64, _P, _P, _P, _I64, _I64, _P]),
}

_lib = None


class NQError(RuntimeError):
    def __init__(self, status, name):
        self.status = status
        msg = lib().nq_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{name} failed: {msg} (status {status})")


def lib():
    """Load libnq.so (once).  Raises ImportError when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: build it with "
                              "`python -m quantized_weight_linear_amd.build`")
        l = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr() if t.numel() else None


def _size(t, nbytes, what):
    """Raise unless tensor t holds at least nbytes (the C ABI sees raw pointers only)."""
    have = 0 if t is None else t.numel() * t.element_size()
    if nbytes > 0 and have < nbytes:
        raise ValueError(f"{what}: {have} bytes given, {int(nbytes)} needed")


_CODE_BYTES = {NQ_W_Q4G64_F16S: 0.5, NQ_W_Q8G32_F16S: 1, NQ_W_Q8G64_F16S: 1, NQ_W_MXFP8_G32: 1, NQ_W_BF16: 2,
               NQ_W_Q3G64_F16S: 3 / 8, NQ_W_Q5G64_F16S: 5 / 8, NQ_W_Q6G64_F16S: 6 / 8}
_SCALE_BYTES = {NQ_W_Q4G64_F16S: 2 / 64, NQ_W_Q8G32_F16S: 2 / 32, NQ_W_Q8G64_F16S: 2 / 64,
                NQ_W_MXFP8_G32: 1 / 32, NQ_W_BF16: 0, NQ_W_Q3G64_F16S: 2 / 64, NQ_W_Q5G64_F16S: 2 / 64,
                NQ_W_Q6G64_F16S: 2 / 64}


# The current stream's handle by device index: what torch.cuda.current_stream(d).cuda_stream returns, without making
# a Stream object for it (a call's host time is a good part of a small step's).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(*tensors):
    for t in tensors:
        if t is not None and t.is_cuda:
            return _raw_stream(t.get_device()) if _raw_stream else torch.cuda.current_stream(t.device).cuda_stream
    return None


def _check(status, name):
    if status != NQ_OK:
        raise NQError(status, name)


def _out_dt(y):
    return NQ_OUT_BF16 if y.element_size() == 2 else NQ_OUT_F32


def nq_abi_version():
    return lib().nq_abi_version()


def _a8_flags(a8):
    """True / False (prefill A8 allowed or not) or an int of NQ_A8_* flags."""
    if isinstance(a8, bool):
        return NQ_A8_PREFILL if a8 else 0
    return int(a8)


def nq_route(T, a8):
    return lib().nq_route(T, _a8_flags(a8))


def nq_gemv_workspace_bytes(fmt, T, N, K):
    return lib().nq_gemv_workspace_bytes(fmt, T, N, K)


def alloc_gemv_workspace(fmt, T, N, K, device):
    """A zero-filled workspace big enough for nq_gemv_* at (fmt, T, N, K), or None."""
    n = nq_gemv_workspace_bytes(fmt, T, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n > 0 else None


def nq_decode_mxfp8(words, e8m0, N, K, w_out):
    _size(words, N * K, "words"); _size(e8m0, N * K // 32, "e8m0")
    _size(w_out, N * K * w_out.element_size(), "w_out")
    _check(lib().nq_decode_mxfp8(_ptr(words), _ptr(e8m0), N, K, _out_dt(w_out), _ptr(w_out),
                                 _stream(words, w_out)), "nq_decode_mxfp8")


def nq_decode_mlx_affine_int8(codes, scales, biases, N, K, w_out):
    _size(codes, N * K, "codes"); _size(scales, N * (K // 128) * 2, "scales"); _size(biases, N * (K // 128) * 2, "biases")
    _size(w_out, N * K * w_out.element_size(), "w_out")
    _check(lib().nq_decode_mlx_affine_int8(_ptr(codes), _ptr(scales), _ptr(biases), N, K, _out_dt(w_out), _ptr(w_out),
                                           _stream(codes, w_out)), "nq_decode_mlx_affine_int8")


def nq_reencode_block128_to_row(codes, wsi, N, K, row_begin, row_end, out_codes, out_scale):
    gr, gc = wsi.shape
    _size(codes, N * K, "codes"); _size(wsi, 4 * gr * gc, "wsi")
    _size(out_codes, (row_end - row_begin) * K, "out_codes"); _size(out_scale, 2 * (row_end - row_begin), "out_scale")
    _check(lib().nq_reencode_block128_to_row(_ptr(codes), _ptr(wsi), N, K, gr, gc, row_begin, row_end,
                                             _ptr(out_codes), _ptr(out_scale), _stream(codes)),
           "nq_reencode_block128_to_row")


def nq_encode_fp8row_bf16(w, N, K, out_codes, out_scale):
    _size(w, 2 * N * K, "w"); _size(out_codes, N * K, "out_codes"); _size(out_scale, 2 * N, "out_scale")
    _check(lib().nq_encode_fp8row_bf16(_ptr(w), N, K, _ptr(out_codes), _ptr(out_scale), _stream(w)),
           "nq_encode_fp8row_bf16")


def nq_quantize_act_int8_g64(x, T, K, q, scale):
    _size(x, 2 * T * K, "x"); _size(q, T * K, "q"); _size(scale, 4 * T * (K // 64), "scale")
    _check(lib().nq_quantize_act_int8_g64(_ptr(x), T, K, _ptr(q), _ptr(scale), _stream(x)),
           "nq_quantize_act_int8_g64")


def nq_quantize_act_fp8_row(x, M, K, codes, scale):
    _size(x, 2 * M * K, "x"); _size(codes, M * K, "codes"); _size(scale, 4 * M, "scale")
    _check(lib().nq_quantize_act_fp8_row(_ptr(x), M, K, _ptr(codes), _ptr(scale), _stream(x)),
           "nq_quantize_act_fp8_row")


def _ws(workspace):
    return (_ptr(workspace), workspace.numel()) if workspace is not None else (None, 0)


def nq_quantize_act_fp8_b128(x, T, K, codes, scale):
    _size(x, 2 * T * K, "x"); _size(codes, T * K, "codes"); _size(scale, 4 * T * -(-K // 128), "scale")
    _check(lib().nq_quantize_act_fp8_b128(_ptr(x), T, K, _ptr(codes), _ptr(scale), _stream(x)), "nq_quantize_act_fp8_b128")


_ACT_GROUP = {NQ_ACT_INT8_G64: 64, NQ_ACT_E4M3_B128: 128}


def nq_rmsnorm(act_fmt, x, weight, eps, y, y_scale=None, residual=None, residual_out=None, weight_bias=0.0):
    """x [T][K], rows back to back or a slice of longer ones; residual_out may be residual."""
    shape = x.shape
    if len(shape) != 2 or x.dtype not in _TWO_BYTES:
        raise ValueError("x: BF16 rows [T][K] expected")
    t, k = shape
    stride, step = x.stride()
    if step != 1 and k > 1:
        raise ValueError("x: a row's columns must be back to back")
    group = _ACT_GROUP.get(act_fmt)
    if y.shape != shape or y.dtype not in (_ONE_BYTE if group else _TWO_BYTES) or not y.is_contiguous():
        raise ValueError("y: contiguous, the shape of x and the format's type expected")
    rp = op = wp = None
    if residual is not None:
        rp = _like(residual, shape, "residual")
        op = rp if residual_out is residual else None if residual_out is None else _like(residual_out, shape, "residual_out")
    if weight is not None:
        wp = _like(weight, (k,), "weight")
    sp = _floats(y_scale, t * -(-k // group), "y_scale") if group else None
    _check((_lib or lib()).nq_rmsnorm(act_fmt, x.data_ptr(), stride if t > 1 else k, rp, op, wp, weight_bias, eps, t, k,
                                      y.data_ptr(), sp, _stream(x)), "nq_rmsnorm")


def nq_gemv_fp8row(w, w_scale, x, T, N, K, y, workspace=None):
    _size(w, N * K, "w"); _size(w_scale, 2 * N, "w_scale"); _size(x, 2 * T * K, "x")
    _size(y, T * N * y.element_size(), "y")
    wp, wb = _ws(workspace)
    _check(lib().nq_gemv_fp8row(_ptr(w), _ptr(w_scale), _ptr(x), T, N, K, _out_dt(y), _ptr(y), wp, wb,
                                _stream(w, x)), "nq_gemv_fp8row")


def nq_gemv_qgroup(fmt, w_codes, w_scales, x, T, N, K, y, workspace=None):
    if fmt in _CODE_BYTES:
        _size(w_codes, N * K * _CODE_BYTES[fmt], "w_codes")
        _size(w_scales, N * K * _SCALE_BYTES[fmt], "w_scales")
    _size(x, 2 * T * K, "x"); _size(y, T * N * y.element_size(), "y")
    wp, wb = _ws(workspace)
    _check(lib().nq_gemv_qgroup(fmt, _ptr(w_codes), _ptr(w_scales), _ptr(x), T, N, K, _out_dt(y), _ptr(y),
                                wp, wb, _stream(w_codes, x)), "nq_gemv_qgroup")


def nq_gemm_w8a8_g64(a_q, a_scale, w_q, w_scale, M, N, K, y, group_sums=None):
    _size(a_q, M * K, "a_q"); _size(a_scale, 4 * M * (K // 64), "a_scale"); _size(w_q, N * K, "w_q")
    _size(w_scale, 2 * N * (K // 64), "w_scale"); _size(y, M * N * y.element_size(), "y")
    if group_sums is not None:
        _size(group_sums, 4 * M * N * (K // 64), "group_sums")
    _check(lib().nq_gemm_w8a8_g64(_ptr(a_q), _ptr(a_scale), _ptr(w_q), _ptr(w_scale), M, N, K, _out_dt(y),
                                  _ptr(y), _ptr(group_sums), _stream(a_q, w_q)), "nq_gemm_w8a8_g64")


def nq_gemm_fp8row(x, w, w_scale, M, N, K, a_codes, a_scale, y):
    _size(x, 2 * M * K, "x"); _size(w, N * K, "w"); _size(w_scale, 2 * N, "w_scale")
    _size(a_codes, M * K, "a_codes"); _size(a_scale, 4 * M, "a_scale"); _size(y, M * N * y.element_size(), "y")
    _check(lib().nq_gemm_fp8row(_ptr(x), _ptr(w), _ptr(w_scale), M, N, K, _ptr(a_codes), _ptr(a_scale),
                                _out_dt(y), _ptr(y), _stream(x, w)), "nq_gemm_fp8row")


def nq_gemm_fp8_b128_workspace_bytes(M, N, K):
    return lib().nq_gemm_fp8_b128_workspace_bytes(M, N, K)


def alloc_gemm_fp8_b128_workspace(M, N, K, device):
    """A workspace for nq_gemm_fp8_b128 of up to M tokens, or None where none of them needs any."""
    n = nq_gemm_fp8_b128_workspace_bytes(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def nq_gemm_fp8_b128(a_codes, a_scale, w, wsi, M, N, K, y, workspace=None):
    """wsi is [ceil(N/128)][ceil(K/128)]; a_scale [M][ceil(K/128)]."""
    gr, gc = wsi.shape if wsi.dim() == 2 else (-1, -1)
    _size(a_codes, M * K, "a_codes"); _size(w, N * K, "w"); _size(y, M * N * y.element_size(), "y")
    _size(a_scale, 4 * M * -(-K // 128), "a_scale")
    if y.dtype not in _OUT_TYPES:
        raise ValueError("y: float32 or bfloat16 expected")
    wp, wb = _ws(workspace)
    _check((_lib or lib()).nq_gemm_fp8_b128(_ptr(a_codes), _floats(a_scale, 0, "a_scale"), _ptr(w), _floats(wsi, 0, "wsi"), M, N, K,
                                            gr, gc, _OUT_TYPES[y.dtype], _ptr(y), wp, wb, _stream(a_codes, w)), "nq_gemm_fp8_b128")


def nq_linear_q8g64(x, T, w_q, w_scale, N, K, allow_a8, a_q_ws, a_scale_ws, y, workspace=None):
    _size(x, 2 * T * K, "x"); _size(w_q, N * K, "w_q"); _size(w_scale, 2 * N * (K // 64), "w_scale")
    _size(y, T * N * y.element_size(), "y")
    if nq_route(T, allow_a8) != NQ_ROUTE_BF16:
        _size(a_q_ws, T * K, "a_q_ws"); _size(a_scale_ws, 4 * T * (K // 64), "a_scale_ws")
    wp, wb = _ws(workspace)
    _check(lib().nq_linear_q8g64(_ptr(x), T, _ptr(w_q), _ptr(w_scale), N, K, _a8_flags(allow_a8),
                                 _ptr(a_q_ws), _ptr(a_scale_ws), _out_dt(y), _ptr(y), wp, wb,
                                 _stream(x, w_q)), "nq_linear_q8g64")


def nq_unpack_q4_to_int8(codes, N, K, out):
    _size(codes, N * K // 2, "codes"); _size(out, N * K, "out")
    _check(lib().nq_unpack_q4_to_int8(_ptr(codes), N, K, _ptr(out), _stream(codes, out)), "nq_unpack_q4_to_int8")


def nq_linear_q4g64(x, T, w_codes, w_scale, N, K, allow_a8, a_q_ws, a_scale_ws, w_i8_ws, y, workspace=None):
    _size(x, 2 * T * K, "x"); _size(w_codes, N * K // 2, "w_codes"); _size(w_scale, 2 * N * (K // 64), "w_scale")
    _size(y, T * N * y.element_size(), "y")
    route = nq_route(T, allow_a8)
    if route != NQ_ROUTE_BF16:
        _size(a_q_ws, T * K, "a_q_ws"); _size(a_scale_ws, 4 * T * (K // 64), "a_scale_ws")
    if route == NQ_ROUTE_A8:
        _size(w_i8_ws, N * K, "w_i8_ws")
    wp, wb = _ws(workspace)
    _check(lib().nq_linear_q4g64(_ptr(x), T, _ptr(w_codes), _ptr(w_scale), N, K, _a8_flags(allow_a8),
                                 _ptr(a_q_ws), _ptr(a_scale_ws), _ptr(w_i8_ws), _out_dt(y), _ptr(y), wp, wb,
                                 _stream(x, w_codes)), "nq_linear_q4g64")


def nq_gemv_a8_workspace_bytes(T, N, K):
    return lib().nq_gemv_a8_workspace_bytes(T, N, K)


def alloc_gemv_a8_workspace(T, N, K, device):
    """A zero-filled workspace big enough for nq_gemv_a8_* at (T, N, K), or None."""
    n = nq_gemv_a8_workspace_bytes(T, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n > 0 else None


def _gemv_a8(name, fmt, w, w_scale, a_q, a_scale, T, N, K, y, workspace, packed):
    wbytes = nq_packed_weight_bytes(fmt, N, K) if packed else N * K * _CODE_BYTES.get(fmt, 1)
    _size(w, wbytes, "w"); _size(w_scale, 2 * N * (K // 64), "w_scale")
    _size(a_q, T * K, "a_q"); _size(a_scale, 4 * T * (K // 64), "a_scale"); _size(y, T * N * y.element_size(), "y")
    wp, wb = _ws(workspace)
    _check(getattr(lib(), name)(fmt, _ptr(w), _ptr(w_scale), _ptr(a_q), _ptr(a_scale), T, N, K, _out_dt(y), _ptr(y),
                                wp, wb, _stream(w, a_q)), name)


def nq_gemv_a8_g64(fmt, w_codes, w_scale, a_q, a_scale, T, N, K, y, workspace=None):
    _gemv_a8("nq_gemv_a8_g64", fmt, w_codes, w_scale, a_q, a_scale, T, N, K, y, workspace, False)


def nq_gemv_a8_g64_packed(fmt, w_packed, w_scale, a_q, a_scale, T, N, K, y, workspace=None):
    _gemv_a8("nq_gemv_a8_g64_packed", fmt, w_packed, w_scale, a_q, a_scale, T, N, K, y, workspace, True)


def nq_stream_read(src, sink):
    """Read all of src (a device tensor, 16-byte multiple) once; sink is an
    int32 device tensor of at least nq_stream_read_sink_words() elements."""
    nbytes = src.numel() * src.element_size()
    _size(sink, 4 * lib().nq_stream_read_sink_words(), "sink")
    _check(lib().nq_stream_read(_ptr(src), nbytes, _ptr(sink), _stream(src)), "nq_stream_read")


NQ_FMT_FP8ROW = -1     # the format code the packing calls use for row-scaled FP8


def nq_packed_weight_bytes(fmt, N, K):
    return lib().nq_packed_weight_bytes(fmt, N, K)


def nq_pack_weights(fmt, w, N, K, w_packed):
    code_bytes = 1 if fmt == NQ_FMT_FP8ROW else _CODE_BYTES.get(fmt, 1)
    _size(w, N * K * code_bytes, "w")
    _size(w_packed, nq_packed_weight_bytes(fmt, N, K), "w_packed")
    _check(lib().nq_pack_weights(fmt, _ptr(w), N, K, _ptr(w_packed), _stream(w)), "nq_pack_weights")


def nq_gemv_fp8row_packed(w_packed, w_scale, x, T, N, K, y, workspace=None):
    _size(w_packed, nq_packed_weight_bytes(NQ_FMT_FP8ROW, N, K), "w_packed")
    _size(w_scale, 2 * N, "w_scale"); _size(x, 2 * T * K, "x"); _size(y, T * N * y.element_size(), "y")
    wp, wb = _ws(workspace)
    _check(lib().nq_gemv_fp8row_packed(_ptr(w_packed), _ptr(w_scale), _ptr(x), T, N, K, _out_dt(y), _ptr(y),
                                       wp, wb, _stream(w_packed, x)), "nq_gemv_fp8row_packed")


def nq_gemv_qgroup_packed(fmt, w_packed, w_scales, x, T, N, K, y, workspace=None):
    if fmt in _CODE_BYTES:
        _size(w_packed, nq_packed_weight_bytes(fmt, N, K), "w_packed")
        _size(w_scales, N * K * _SCALE_BYTES[fmt], "w_scales")
    _size(x, 2 * T * K, "x"); _size(y, T * N * y.element_size(), "y")
    wp, wb = _ws(workspace)
    _check(lib().nq_gemv_qgroup_packed(fmt, _ptr(w_packed), _ptr(w_scales), _ptr(x), T, N, K, _out_dt(y),
                                       _ptr(y), wp, wb, _stream(w_packed, x)), "nq_gemv_qgroup_packed")


def nq_gemv_fp8row_packed_noalloc(w_packed, w_scale, x, T, N, K, y):
    _size(w_packed, nq_packed_weight_bytes(NQ_FMT_FP8ROW, N, K), "w_packed")
    _size(w_scale, 2 * N, "w_scale"); _size(x, 2 * T * K, "x"); _size(y, T * N * y.element_size(), "y")
    _check(lib().nq_gemv_fp8row_packed_noalloc(_ptr(w_packed), _ptr(w_scale), _ptr(x), T, N, K, _out_dt(y), _ptr(y),
                                               _stream(w_packed, x)), "nq_gemv_fp8row_packed_noalloc")


def nq_unpack_qbits_to_int8(fmt, codes, N, K, out):
    _size(codes, N * K * _CODE_BYTES[fmt], "codes"); _size(out, N * K, "out")
    _check(lib().nq_unpack_qbits_to_int8(fmt, _ptr(codes), N, K, _ptr(out), _stream(codes, out)),
           "nq_unpack_qbits_to_int8")


def nq_linear_qbits_g64(fmt, x, T, w_codes, w_scale, N, K, a8, a_q_ws, a_scale_ws, w_i8_ws, y, workspace=None):
    _size(x, 2 * T * K, "x"); _size(w_codes, N * K * _CODE_BYTES[fmt], "w_codes")
    _size(w_scale, 2 * N * (K // 64), "w_scale"); _size(y, T * N * y.element_size(), "y")
    if nq_route(T, a8) != NQ_ROUTE_BF16:
        _size(a_q_ws, T * K, "a_q_ws"); _size(a_scale_ws, 4 * T * (K // 64), "a_scale_ws")
        _size(w_i8_ws, N * K, "w_i8_ws")
    wp, wb = _ws(workspace)
    _check(lib().nq_linear_qbits_g64(fmt, _ptr(x), T, _ptr(w_codes), _ptr(w_scale), N, K, _a8_flags(a8),
                                     _ptr(a_q_ws), _ptr(a_scale_ws), _ptr(w_i8_ws), _out_dt(y), _ptr(y), wp, wb,
                                     _stream(x, w_codes)), "nq_linear_qbits_g64")


# ---------------------------------------------------------------------------
# Attention and the paged cache.  Sizes come from the tensors' shapes: rows
# [T][heads][D] (a slice of a wider row is fine: heads back to back, any
# distance between tokens), planes [pages][Hkv][page_size][D], pools of planes
# [planes][pages][Hkv][page_size][D], tables [B][width].
# ---------------------------------------------------------------------------

_TWO_BYTES = frozenset((torch.bfloat16, torch.int16, torch.uint16))
_ONE_BYTE = frozenset((torch.uint8, torch.int8, torch.float8_e4m3fn))
_INT32 = frozenset((torch.int32, torch.uint32))
_INT64 = frozenset((torch.int64, torch.uint64))
_OUT_TYPES = {torch.float32: NQ_OUT_F32, torch.bfloat16: NQ_OUT_BF16, torch.int16: NQ_OUT_BF16, torch.uint16: NQ_OUT_BF16}


def _rows(t, shape, what):
    """Address and token stride of rows [T][heads][D]."""
    if t.dtype not in _TWO_BYTES or len(shape) != 3:
        raise ValueError(f"{what}: BF16 rows [T][heads][D] expected")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if n == 0:
        return None, h * d
    if s2 != 1 or (s1 != d and h > 1) or (n > 1 and s0 < h * d):
        raise ValueError(f"{what}: a token's heads must be back to back")
    return t.data_ptr(), s0 if n > 1 else h * d


def _like(t, shape, what):
    """Address of contiguous BF16 values of this shape."""
    if t.shape != shape or t.dtype not in _TWO_BYTES or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous BF16 {list(shape)} expected")
    return t.data_ptr()


def _ints(t, n, what, types=_INT32):
    """Address of at least n integers."""
    if t.dtype not in types or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous integers of {8 if types is _INT64 else 4} bytes expected")
    return t.data_ptr()


def _floats(t, n, what):
    if t is None:
        if n:
            raise ValueError(f"{what}: {n} values expected")
        return None
    if t.dtype is not torch.float32 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous float32 values expected")
    return t.data_ptr()


def _table(t):
    shape = t.shape
    if len(shape) != 2 or t.dtype not in _INT32 or not t.is_contiguous():
        raise ValueError("page table: contiguous 32-bit integers [B][width] expected")
    return t.data_ptr(), shape[0], shape[1]


def _planes(fmt, k_pages, v_pages, hkv, d):
    shape = k_pages.shape
    if len(shape) != 4 or shape != v_pages.shape or shape[1] != hkv or shape[3] != d:
        raise ValueError("pages: [pages][Hkv][page_size][D] expected, the same for keys and values")
    types = _TWO_BYTES if fmt == NQ_KV_BF16 else _ONE_BYTE
    if k_pages.dtype not in types or v_pages.dtype not in types:
        raise ValueError("pages: one byte an element for E4M3, two for BF16")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("pages: tensors must be contiguous")
    return k_pages.data_ptr(), v_pages.data_ptr(), shape[2], shape[0]


def _scales(fmt, k_scale, v_scale, pages):
    """Addresses of the cache's scales: none, one a KV head, or one a row."""
    if fmt == NQ_KV_BF16:
        return None, None
    p, h, ps, _ = pages.shape
    n = h if fmt == NQ_KV_E4M3 else p * h * ps
    return _floats(k_scale, n, "k_scale"), _floats(v_scale, n, "v_scale")


def _out(o, shape):
    """Address and type of the outputs."""
    if o.shape != shape or not o.is_contiguous():
        raise ValueError("o: contiguous, the shape of q expected")
    if o.dtype not in _OUT_TYPES:
        raise ValueError("o: float32 or bfloat16 expected")
    return o.data_ptr(), _OUT_TYPES[o.dtype]


def nq_attn_prompt(q, k, v, cu_q, cu_k, scale, o, lse=None):
    qh, kh = q.shape, k.shape
    qp, qs = _rows(q, qh, "q")
    kp, ks = _rows(k, kh, "k")
    vp, vs = _rows(v, kh, "v")
    b = cu_q.numel() - 1
    if v.shape != kh or kh[2] != qh[2] or cu_k.numel() != b + 1:
        raise ValueError("q, k and v must have the same D, k and v the same shape, cu_q and cu_k the same length")
    op, out = _out(o, qh)
    cq, ck = _ints(cu_q, 0, "cu_q"), _ints(cu_k, 0, "cu_k")
    lp = None if lse is None else _floats(lse, qh[0] * qh[1], "lse")
    _check((_lib or lib()).nq_attn_prompt(qp, qs, kp, ks, vp, vs, cq, ck, b if b > 0 else 0, qh[0], kh[0], qh[1], kh[1], qh[2],
                                          scale, out, op, lp, _stream(q)), "nq_attn_prompt")


def nq_kv_append(fmt, k, v, k_scale, v_scale, page_table, lens, cu, k_pages, v_pages):
    kh = k.shape
    kp, ks = _rows(k, kh, "k")
    vp, vs = _rows(v, kh, "v")
    if v.shape != kh:
        raise ValueError("k and v must have the same shape")
    t, hkv, d = kh
    tp, b, width = _table(page_table)
    kpp, vpp, ps, pages = _planes(fmt, k_pages, v_pages, hkv, d)
    n = hkv if fmt == NQ_KV_E4M3 else 0
    _check((_lib or lib()).nq_kv_append(fmt, kp, ks, vp, vs, _floats(k_scale, n, "k_scale"), _floats(v_scale, n, "v_scale"),
                                        tp, width, _ints(lens, b, "lens"), _ints(cu, b + 1, "cu"), b, t, hkv, d, ps, pages,
                                        kpp, vpp, _stream(k_pages)), "nq_kv_append")


def nq_kv_append_rope(fmt, q, k, v, positions, inv_freq, rope, k_scale, v_scale, page_table, lens, cu, q_out, k_pages, v_pages,
                      q_weight=None, k_weight=None, weight_bias=0.0, eps=1e-6, k_out=None):
    """q (and q_out) None: keys and values only.  inv_freq None: nothing is turned; else its 2 numel first columns are."""
    kh = k.shape
    kp, ks = _rows(k, kh, "k")
    vp, vs = _rows(v, kh, "v")
    if v.shape != kh:
        raise ValueError("k and v must have the same shape")
    t, hkv, d = kh
    qp = qop = kop = qwp = kwp = fp = pp = None
    qs = qos = kos = rot = 0
    hq = hkv
    if q is not None:
        qh = q.shape
        if len(qh) != 3 or qh[0] != t or qh[2] != d or q_out is None or q_out.shape != qh:
            raise ValueError("q and q_out: [T][Hq][D] with k's T and D expected")
        hq = qh[1]
        qp, qs = _rows(q, qh, "q")
        qop, qos = (qp, qs) if q_out is q else _rows(q_out, qh, "q_out")
    if k_out is not None:
        if k_out.shape != kh:
            raise ValueError("k_out: the shape of k expected")
        kop, kos = _rows(k_out, kh, "k_out")
    if q_weight is not None:
        qwp = _like(q_weight, (d,), "q_weight")
    if k_weight is not None:
        kwp = _like(k_weight, (d,), "k_weight")
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        fp, pp = _floats(inv_freq, 0, "inv_freq"), _ints(positions, t, "positions")
    tp, b, width = _table(page_table)
    kpp, vpp, ps, pages = _planes(fmt, k_pages, v_pages, hkv, d)
    ksp, vsp = _scales(fmt, k_scale, v_scale, k_pages)
    _check((_lib or lib()).nq_kv_append_rope(fmt, qp, qs, kp, ks, vp, vs, qwp, kwp, weight_bias, eps, pp, fp, rot, rope, ksp, vsp, tp,
                                             width, _ints(lens, b, "lens"), _ints(cu, b + 1, "cu"), b, t, hq, hkv, d, ps, pages,
                                             qop, qos, kop, kos, kpp, vpp, _stream(k_pages)), "nq_kv_append_rope")


def nq_attn_tree_workspace_bytes(B, max_q, Hq, Hkv, D, max_len):
    return lib().nq_attn_tree_workspace_bytes(B, max_q, Hq, Hkv, D, max_len)


def alloc_attn_tree_workspace(B, max_q, Hq, Hkv, D, max_len, device):
    """A workspace for nq_attn_tree at these sizes, or None where it needs none."""
    n = nq_attn_tree_workspace_bytes(B, max_q, Hq, Hkv, D, max_len)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def nq_attn_tree(fmt, q, k_pages, v_pages, k_scale, v_scale, page_table, lens, cu_q, tree_mask, max_q, max_len, scale, o,
                 lse=None, workspace=None):
    qh = q.shape
    qp, qs = _rows(q, qh, "q")
    t, hq, d = qh
    hkv = k_pages.shape[1] if k_pages.dim() == 4 else 0
    tp, b, width = _table(page_table)
    kpp, vpp, ps, pages = _planes(fmt, k_pages, v_pages, hkv, d)
    kp, vp = _scales(fmt, k_scale, v_scale, k_pages)
    wp, wb = _ws(workspace)
    op, out = _out(o, qh)
    lp = None if lse is None else _floats(lse, t * hq, "lse")
    _check((_lib or lib()).nq_attn_tree(fmt, qp, qs, kpp, vpp, kp, vp, tp, width, _ints(lens, b, "lens"), _ints(cu_q, b + 1, "cu_q"),
                                        _ints(tree_mask, t, "tree_mask", _INT64), b, max_q, t, hq, hkv, d, ps, pages,
                                        max_len, scale, out, op, lp, wp, wb, _stream(q)), "nq_attn_tree")


def nq_kv_reserve(refs, page_table, lens, new_lens, page_size, free_list, shortfall):
    tp, b, width = _table(page_table)
    pages = refs.numel()
    _check((_lib or lib()).nq_kv_reserve(_ints(refs, pages, "refs"), pages, tp, width, _ints(lens, b, "lens"),
                                         _ints(new_lens, b, "new_lens"), b, page_size, _ints(free_list, pages, "free_list"),
                                         _ints(shortfall, 1, "shortfall"), _stream(refs)), "nq_kv_reserve")


def nq_kv_release(refs, page_table, keep_lens, page_size):
    tp, b, width = _table(page_table)
    pages = refs.numel()
    _check((_lib or lib()).nq_kv_release(_ints(refs, pages, "refs"), pages, tp, width, _ints(keep_lens, b, "keep_lens"), b,
                                         page_size, _stream(refs)), "nq_kv_release")


def nq_kv_fork(refs, page_table, lens, parents, page_size, child_table, copies, free_list, shortfall):
    tp, b, width = _table(page_table)
    cp, children, cwidth = _table(child_table)
    pages = refs.numel()
    if cwidth != width or parents.numel() != children:
        raise ValueError("child_table: [children][width] expected")
    _check((_lib or lib()).nq_kv_fork(_ints(refs, pages, "refs"), pages, tp, width, _ints(lens, b, "lens"), b,
                                      _ints(parents, children, "parents"), children, page_size, cp,
                                      _ints(copies, 2 * children, "copies"), _ints(free_list, pages, "free_list"),
                                      _ints(shortfall, 1, "shortfall"), _stream(refs)), "nq_kv_fork")


def _pool(pool):
    """Address, shape, bytes of an element, of a page and of a plane of [planes][pages][Hkv][page_size][D]."""
    shape = pool.shape
    if len(shape) != 5 or not pool.is_contiguous():
        raise ValueError("pool: contiguous [planes][pages][Hkv][page_size][D] expected")
    size = pool.element_size()
    page = shape[2] * shape[3] * shape[4] * size
    return pool.data_ptr(), shape, size, page, shape[1] * page


def nq_kv_copy_pages(pool, copies):
    p, shape, _, page, plane = _pool(pool)
    n = copies.numel() // 2
    _check((_lib or lib()).nq_kv_copy_pages(p, shape[0], plane, page, shape[1], _ints(copies, 2 * n, "copies"), n,
                                            _stream(pool)), "nq_kv_copy_pages")


def nq_kv_compact(pool, page_table, lens, accept, cu_accept):
    p, shape, size, _, plane = _pool(pool)
    tp, b, width = _table(page_table)
    n = accept.numel()
    _check((_lib or lib()).nq_kv_compact(p, shape[0], plane, shape[2], shape[3], shape[4] * size, shape[1], tp, width,
                                         _ints(lens, b, "lens"), _ints(accept, n, "accept"),
                                         _ints(cu_accept, b + 1, "cu_accept"), b, n, _stream(pool)), "nq_kv_compact")
