"""MI355X-native unified-FP8 (W8A8) linear layer: Python binding.

A thin ctypes layer over libfp8w8a8.so (C ABI: include/fp8w8a8.h).  It only
marshals arguments -- torch tensors become device pointers, strides and the
current HIP stream -- and turns status codes into exceptions.  Every step of
the computation runs in the library's gfx950 kernels; there is no fallback:
if the library is missing, importing a function raises.

Entry points (same names as the C ABI):
  fp8_quantize_per_token(x)                -> (q uint8 [M,K], scales fp32 [M])
  fp8_quantize_static(x, scale)            -> (q, scales)   static per-tensor scale (device fp32 [1])
  fp8_quantize_per_token_clipped(x, clip)  -> (q, scales)   per-token scale, absmax clipped at *clip
  fp8_calibrate_percentile(x, num, den)    -> (value fp32 [1], scale fp32 [1])  nearest-rank |x| percentile
  fp8_gemm_scaled(qa, s_tok, qw, s_ch)     -> y bf16 [M,N]
  fp8_quant_gemm_fused(x, qw, s_ch)        -> y bf16 [M,N]  (optionally qa, s_tok)
  fp8_gemm_scaled_fp8out(qa, s_tok, qw, s_ch) -> (q_out uint8 [M,N], s_out fp32 [M])  (optionally y32)
  fp8_gemm_grouped_scaled(qa, s_tok, row_token, expert_offsets, qw, s_ch) -> y bf16 [R,N]
  fp8_kv_append_rope_paged(k, v, positions, cos_sin, scales, slot_mapping, cache, q=q) -> q_out  rotate + FP8 append
  fp8_attn_decode_paged(q, cache, block_table, seq_lens, scales, block_size)  -> out  one new token per sequence
  fp8_attn_prefill_paged(q, cu_q, cache, block_table, seq_lens, scales, block_size) -> out  several new tokens
  fp8_gemm_scaled_act(qa, s_tok, qw, s_ch, bias, act, residual) -> y [M,N]  bias, activation, residual in the epilogue
  fp8_gemm_grouped_scaled_act(qa, s_tok, row_token, expert_offsets, qw, s_ch, bias, act) -> y [R,N]
  fp8_act_quantize(h, act, gated)          -> (q uint8 [M,F], scales fp32 [M])  (gated) activation, quantized per token
  fp8_moe_sort(expert_ids, num_experts)    -> (expert_offsets, row_token, row_of)  choices in the experts' order
  fp8_moe_permute(x, row_of)               -> out [R,H]  tokens moved into that order
  fp8_moe_combine(y, row_of, weights, residual) -> out [T,H]  the experts' rows back to their tokens
  fp8_moe_combine_grad(dout, y, row_of, weights) -> (dy [R,H], dweights fp32 [T,topk])
  fp8_workspace_bytes(M, N, K) (fused call), fp8_gemm_workspace_bytes(M, N, K),
  fp8_fp8out_workspace_bytes(M, N, K), fp8_grouped_workspace_bytes(T, R, E, N, K)
  fp8_status_string(code)
"""
import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8w8a8.so")

FP8_OK = 0
FP8_ERR_INVALID_ARGUMENT = 1
FP8_ERR_UNSUPPORTED = 2
FP8_ERR_WORKSPACE = 3
FP8_ERR_DEVICE = 4

# exported symbols, as declared in include/fp8w8a8.h
EXPORTS = ("fp8_quantize_per_token", "fp8_quantize_static", "fp8_quantize_per_token_clipped",
           "fp8_calibrate_percentile", "fp8_calibrate_workspace_bytes", "fp8_gemm_scaled", "fp8_quant_gemm_fused", "fp8_gemm_scaled_fp8out",
           "fp8_gemm_grouped_scaled", "fp8_workspace_bytes", "fp8_gemm_workspace_bytes", "fp8_fp8out_workspace_bytes",
           "fp8_grouped_workspace_bytes", "fp8_quantize_mx", "fp8_gemm_mx", "fp8_mx_workspace_bytes",
           "fp8_kv_channel_scales", "fp8_kv_scales_workspace_bytes",
           "fp8_kv_quantize_paged", "fp8_kv_dequantize_paged", "fp8_kv_append_rope_paged", "fp8_attn_decode_paged",
           "fp8_attn_prefill_paged", "fp8_attn_decode_workspace_bytes", "fp8_attn_prefill_workspace_bytes",
           "fp8_gemm_scaled_act", "fp8_gemm_act_workspace_bytes", "fp8_gemm_grouped_scaled_act", "fp8_act_quantize",
           "fp8_moe_sort", "fp8_moe_sort_workspace_bytes", "fp8_moe_permute", "fp8_moe_combine", "fp8_moe_combine_grad",
           "fp8_stream_read", "fp8_quant_gemm_fused_noalloc",
           "fp8_status_string")

_lib = None
_torch_module = None


class Fp8Error(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__(f"{fn} failed: {status_name(code)}")


def lib():
    """Load libfp8w8a8.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run python fp8_w8a8_quantized_quantize_amd/_build.py")
        L = ctypes.CDLL(LIB_PATH)
        i64, vp, sz, st = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.fp8_quantize_per_token.restype = st
        L.fp8_quantize_per_token.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp]
        L.fp8_quantize_static.restype = st
        L.fp8_quantize_static.argtypes = [vp, i64, i64, i64, vp, vp, i64, vp, vp]
        L.fp8_quantize_per_token_clipped.restype = st
        L.fp8_quantize_per_token_clipped.argtypes = [vp, i64, i64, i64, vp, vp, i64, vp, vp]
        L.fp8_calibrate_percentile.restype = st
        L.fp8_calibrate_percentile.argtypes = [vp, i64, i64, i64, vp, vp, vp, sz, vp]
        L.fp8_calibrate_workspace_bytes.restype = sz
        L.fp8_calibrate_workspace_bytes.argtypes = []
        L.fp8_gemm_scaled.restype = st
        L.fp8_gemm_scaled.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, i64, vp, sz, vp]
        L.fp8_quant_gemm_fused.restype = st
        L.fp8_quant_gemm_fused.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, vp, vp, vp, sz, vp]
        L.fp8_gemm_scaled_fp8out.restype = st
        L.fp8_gemm_scaled_fp8out.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, vp, sz, vp]
        L.fp8_fp8out_workspace_bytes.restype = sz
        L.fp8_fp8out_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8_gemm_grouped_scaled.restype = st
        L.fp8_gemm_grouped_scaled.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, sz, vp]
        L.fp8_workspace_bytes.restype = sz
        L.fp8_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8_gemm_workspace_bytes.restype = sz
        L.fp8_gemm_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8_grouped_workspace_bytes.restype = sz
        L.fp8_grouped_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
        L.fp8_quantize_mx.restype = st
        L.fp8_quantize_mx.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp]
        L.fp8_gemm_mx.restype = st
        L.fp8_gemm_mx.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, i64, i64, i64, vp, sz, vp]
        L.fp8_mx_workspace_bytes.restype = sz
        L.fp8_mx_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8_kv_channel_scales.restype = st
        L.fp8_kv_channel_scales.argtypes = [vp, st, i64, i64, i64, st, vp, vp, sz, vp]
        L.fp8_kv_scales_workspace_bytes.restype = sz
        L.fp8_kv_scales_workspace_bytes.argtypes = [i64, i64]
        L.fp8_kv_quantize_paged.restype = st
        L.fp8_kv_quantize_paged.argtypes = [vp, st, i64, i64, i64, vp, st, vp, vp, i64, vp]
        L.fp8_kv_dequantize_paged.restype = st
        L.fp8_kv_dequantize_paged.argtypes = [vp, i64, vp, i64, i64, vp, st, vp, st, i64, vp]
        f32, i32 = ctypes.c_float, ctypes.c_int32
        L.fp8_kv_append_rope_paged.restype = st
        L.fp8_kv_append_rope_paged.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, st, i64, i64, i64, i64, vp, vp, i64,
                                               i64, i32, vp, st, vp, vp, i64, vp]
        L.fp8_attn_decode_workspace_bytes.restype = sz
        L.fp8_attn_decode_workspace_bytes.argtypes = [i64] * 7
        L.fp8_attn_decode_paged.restype = st
        L.fp8_attn_decode_paged.argtypes = [vp, i64, st, vp, i64, i64, vp, st, vp, i64, i64, vp, i64, i64, i64, i64,
                                            i64, f32, f32, vp, i64, vp, i64, vp, vp, sz, vp]
        L.fp8_attn_prefill_workspace_bytes.restype = sz
        L.fp8_attn_prefill_workspace_bytes.argtypes = [i64] * 9
        L.fp8_attn_prefill_paged.restype = st
        L.fp8_attn_prefill_paged.argtypes = [vp, i64, st, vp, i64, vp, i64, i64, vp, st, vp, i64, i64, vp, i64, i64,
                                             i64, i64, i64, i64, i32, vp, f32, f32, vp, i64, vp, i64, vp, vp, sz, vp]
        L.fp8_quant_gemm_fused_noalloc.restype = st
        L.fp8_quant_gemm_fused_noalloc.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, i64, vp, vp, vp]
        L.fp8_gemm_act_workspace_bytes.restype = sz
        L.fp8_gemm_act_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8_gemm_scaled_act.restype = st
        L.fp8_gemm_scaled_act.argtypes = [vp, i64, vp, vp, i64, vp, vp, st, vp, i64, vp, st, i64, i64, i64, i64, vp, sz,
                                          vp]
        L.fp8_gemm_grouped_scaled_act.restype = st
        L.fp8_gemm_grouped_scaled_act.argtypes = [vp, vp, vp, vp, vp, vp, vp, st, vp, st, i64, i64, i64, i64, i64, i64,
                                                  vp, sz, vp]
        L.fp8_act_quantize.restype = st
        L.fp8_act_quantize.argtypes = [vp, i64, st, i64, i64, st, i32, vp, i64, vp, vp, vp]
        L.fp8_moe_sort_workspace_bytes.restype = sz
        L.fp8_moe_sort_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8_moe_sort.restype = st
        L.fp8_moe_sort.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, vp, sz, vp]
        L.fp8_moe_permute.restype = st
        L.fp8_moe_permute.argtypes = [vp, i64, vp, vp, i64, i64, i64, i64, i64, vp, i64, vp, vp]
        L.fp8_moe_combine.restype = st
        L.fp8_moe_combine.argtypes = [vp, i64, st, vp, vp, vp, i64, vp, st, i64, i64, i64, i64, i64, vp]
        L.fp8_moe_combine_grad.restype = st
        L.fp8_moe_combine_grad.argtypes = [vp, i64, st, vp, i64, st, vp, vp, vp, i64, vp, i64, i64, i64, i64, vp]
        L.fp8_stream_read.restype = st
        L.fp8_stream_read.argtypes = [vp, sz, ctypes.c_int32, ctypes.c_int32, vp, vp]
        L.fp8_status_string.restype = ctypes.c_char_p
        L.fp8_status_string.argtypes = [st]
        _lib = L
    return _lib


def status_name(code):
    return lib().fp8_status_string(int(code)).decode()


def _check(fn, code):
    if code != FP8_OK:
        raise Fp8Error(fn, code)


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_tensor_class = None


def _tensor():
    """torch.Tensor."""
    global _tensor_class
    if _tensor_class is None:
        _tensor_class = _torch().Tensor
    return _tensor_class


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


SIZE_MAX = (1 << 64) - 1


def _on_device(t, dtype, name, device=None):
    """t must be a torch tensor of `dtype` in GPU memory (on `device` when
    given): the library takes raw pointers and cannot tell a host address from
    a device one, so a host tensor is rejected here, before any call."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name}: expected a {dtype} CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _rows(t, dtype, name, device=None):
    _on_device(t, dtype, name, device)
    if t.dim() != 2 or (t.shape[0] > 0 and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a 2-D row-major tensor (unit stride along the last dim)")
    return t.shape[0], t.shape[1], (t.stride(0) if t.shape[0] > 1 else t.shape[1])


def _vec(t, dtype, name, n, device=None):
    _on_device(t, dtype, name, device)
    if not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous {dtype} CUDA tensor")
    if t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")


def _dense(t, dtype, name, shape, device=None):
    """A contiguous device tensor of exactly `shape` (optional outputs)."""
    _on_device(t, dtype, name, device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}")


def _workspace(ws, need, fn, device):
    """The caller's workspace (checked: a uint8 device tensor on `device` of at
    least `need` bytes), or a new one when ws is None; None when nothing is
    needed.  need == SIZE_MAX (the library's answer for invalid sizes) raises
    the library's FP8_ERR_INVALID_ARGUMENT."""
    torch = _torch()
    if need == SIZE_MAX:
        raise Fp8Error(fn, FP8_ERR_INVALID_ARGUMENT)
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
    _on_device(ws, torch.uint8, "ws", device)
    if not ws.is_contiguous():
        raise ValueError("ws: expected a contiguous uint8 tensor")
    return ws


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def fp8_workspace_bytes(M, N, K):
    """Workspace bytes of fp8_quant_gemm_fused (codes staged + the GEMM's)."""
    return int(lib().fp8_workspace_bytes(M, N, K))


def fp8_gemm_workspace_bytes(M, N, K):
    """Workspace bytes of fp8_gemm_scaled alone."""
    return int(lib().fp8_gemm_workspace_bytes(M, N, K))


def fp8_fp8out_workspace_bytes(M, N, K):
    return int(lib().fp8_fp8out_workspace_bytes(M, N, K))


def fp8_grouped_workspace_bytes(T, R, E, N, K):
    return int(lib().fp8_grouped_workspace_bytes(T, R, E, N, K))


def fp8_status_string(code):
    return status_name(code)


def fp8_quantize_per_token(x, q=None, scales=None, stream=None):
    """Per-row absmax E4M3 quantization of fp32 x [M, K] -> (q uint8 [M, K], scales fp32 [M])."""
    torch = _torch()
    M, K, ldx = _rows(x, torch.float32, "x")
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=x.device)
    Mq, Kq, ldq = _rows(q, torch.uint8, "q", x.device)
    if (Mq, Kq) != (M, K):
        raise ValueError("q: expected shape [M, K]")
    _vec(scales, torch.float32, "scales", M, x.device)
    _check("fp8_quantize_per_token",
           lib().fp8_quantize_per_token(_ptr(x), M, K, ldx, _ptr(q), ldq, _ptr(scales), _stream(stream)))
    return q, scales


def _scalar(t, name, device):
    torch = _torch()
    _on_device(t, torch.float32, name, device)
    if t.numel() < 1:
        raise TypeError(f"{name}: expected a float32 CUDA tensor holding one value")


def fp8_quantize_static(x, scale, q=None, scales_out=None, stream=None):
    """Static per-tensor quantization of fp32 x [M, K] with the device scalar
    `scale` -> (q uint8 [M, K], scales_out fp32 [M] filled with the scale)."""
    torch = _torch()
    M, K, ldx = _rows(x, torch.float32, "x")
    _scalar(scale, "scale", x.device)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if scales_out is None:
        scales_out = torch.empty(M, dtype=torch.float32, device=x.device)
    Mq, Kq, ldq = _rows(q, torch.uint8, "q", x.device)
    if (Mq, Kq) != (M, K):
        raise ValueError("q: expected shape [M, K]")
    _vec(scales_out, torch.float32, "scales_out", M, x.device)
    _check("fp8_quantize_static", lib().fp8_quantize_static(_ptr(x), M, K, ldx, _ptr(scale), _ptr(q), ldq,
                                                            _ptr(scales_out), _stream(stream)))
    return q, scales_out


def fp8_quantize_per_token_clipped(x, clip, q=None, scales=None, stream=None):
    """Per-token quantization with the row absmax clipped at the device scalar `clip`."""
    torch = _torch()
    M, K, ldx = _rows(x, torch.float32, "x")
    _scalar(clip, "clip", x.device)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=x.device)
    Mq, Kq, ldq = _rows(q, torch.uint8, "q", x.device)
    if (Mq, Kq) != (M, K):
        raise ValueError("q: expected shape [M, K]")
    _vec(scales, torch.float32, "scales", M, x.device)
    _check("fp8_quantize_per_token_clipped",
           lib().fp8_quantize_per_token_clipped(_ptr(x), M, K, ldx, _ptr(clip), _ptr(q), ldq, _ptr(scales),
                                                _stream(stream)))
    return q, scales


def fp8_calibrate_percentile(x, num, den, value=None, scale=None, ws=None, stream=None):
    """Nearest-rank percentile num/den of |x| over all of x (fp32, contiguous)
    -> (value fp32 [1], static scale fp32 [1]) on the device."""
    torch = _torch()
    _on_device(x, torch.float32, "x")
    if not x.is_contiguous():
        raise TypeError("x: expected a contiguous float32 CUDA tensor")
    if value is None:
        value = torch.empty(1, dtype=torch.float32, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _vec(value, torch.float32, "value", 1, x.device)
    _vec(scale, torch.float32, "scale", 1, x.device)
    ws = _workspace(ws, int(lib().fp8_calibrate_workspace_bytes()), "fp8_calibrate_percentile", x.device)
    _check("fp8_calibrate_percentile",
           lib().fp8_calibrate_percentile(_ptr(x), x.numel(), int(num), int(den), _ptr(value), _ptr(scale), _ptr(ws),
                                          _nbytes(ws), _stream(stream)))
    return value, scale


def fp8_mx_workspace_bytes(M, N, K):
    return int(lib().fp8_mx_workspace_bytes(M, N, K))


def _mx_scales(t, name, rows, K, device):
    _dense(t, _torch().uint8, name, (K // 128, rows, 4), device)


def fp8_quantize_mx(x, q=None, scales=None, stream=None):
    """Block-scaled E4M3 quantization of fp32 x [M, K] (K % 128 == 0) ->
    (q uint8 [M, K], scales uint8 [K/128, M, 4] chunk-major exponent bytes)."""
    torch = _torch()
    M, K, ldx = _rows(x, torch.float32, "x")
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((K // 128, M, 4), dtype=torch.uint8, device=x.device)
    Mq, Kq, ldq = _rows(q, torch.uint8, "q", x.device)
    if (Mq, Kq) != (M, K):
        raise ValueError("q: expected shape [M, K]")
    _mx_scales(scales, "scales", M, K, x.device)
    _check("fp8_quantize_mx", lib().fp8_quantize_mx(_ptr(x), M, K, ldx, _ptr(q), ldq, _ptr(scales), _stream(stream)))
    return q, scales


def fp8_gemm_mx(qa, sa, qw, sw, y=None, ws=None, stream=None):
    """y = bf16(sum over 32-blocks of 2^(ea + ew - 254) * block dot) for block-scaled
    E4M3 operands qa [M, K], qw [N, K] with chunk-major exponent bytes sa [K/128, M, 4],
    sw [K/128, N, 4]."""
    torch = _torch()
    M, K, lda = _rows(qa, torch.uint8, "qa")
    dev = qa.device
    N, K2, ldw = _rows(qw, torch.uint8, "qw", dev)
    if K2 != K:
        raise ValueError("qa and qw disagree on K")
    _mx_scales(sa, "sa", M, K, dev)
    _mx_scales(sw, "sw", N, K, dev)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    My, Ny, ldy = _rows(y, torch.bfloat16, "y", dev)
    if (My, Ny) != (M, N):
        raise ValueError("y: expected shape [M, N]")
    ws = _workspace(ws, fp8_mx_workspace_bytes(M, N, K), "fp8_gemm_mx", dev)
    _check("fp8_gemm_mx", lib().fp8_gemm_mx(_ptr(qa), lda, _ptr(sa), _ptr(qw), ldw, _ptr(sw), _ptr(y), ldy, M, N, K,
                                            _ptr(ws), _nbytes(ws), _stream(stream)))
    return y


FP8_KV_E4M3 = 0
FP8_KV_E5M2 = 1
FP8_KV_F32 = 0
FP8_KV_BF16 = 1
FP8_KV_F16 = 2
_KV_FORMATS = {"e4m3": FP8_KV_E4M3, "e5m2": FP8_KV_E5M2, FP8_KV_E4M3: FP8_KV_E4M3, FP8_KV_E5M2: FP8_KV_E5M2}


def _kv_fmt(fmt):
    if fmt not in _KV_FORMATS:
        raise ValueError(f"fmt: expected 'e4m3' or 'e5m2', got {fmt!r}")
    return _KV_FORMATS[fmt]


def fp8_kv_scales_workspace_bytes(T, C):
    return int(lib().fp8_kv_scales_workspace_bytes(T, C))


def _kv_dtype(t, name, device=None):
    torch = _torch()
    codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    if not isinstance(t, torch.Tensor) or t.dtype not in codes or not t.is_cuda:
        raise TypeError(f"{name}: expected a float32, bfloat16 or float16 CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    return codes[t.dtype]


def _kv_rows(t, name, device=None):
    dt = _kv_dtype(t, name, device)
    if t.dim() != 2 or (t.shape[0] > 0 and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a 2-D row-major tensor (unit stride along the last dim)")
    return t.shape[0], t.shape[1], (t.stride(0) if t.shape[0] > 1 else t.shape[1]), dt


def _kv_cache(cache, C=None, device=None):
    torch = _torch()
    _on_device(cache, torch.uint8, "cache", device)
    if not cache.is_contiguous() or cache.dim() != 2 or (C is not None and cache.shape[1] != C):
        raise TypeError("cache: expected a contiguous uint8 CUDA tensor [num_slots, C]")


def fp8_kv_channel_scales(kv, fmt="e5m2", scales=None, ws=None, stream=None):
    """Per-channel scales max(fl32(max_t |kv[t,c]| / fmt_max), 1e-12f) of kv [T, C]
    (float32, bfloat16 or float16) -> scales fp32 [C]."""
    torch = _torch()
    T, C, ldkv, dt = _kv_rows(kv, "kv")
    if scales is None:
        scales = torch.empty(C, dtype=torch.float32, device=kv.device)
    _vec(scales, torch.float32, "scales", C, kv.device)
    ws = _workspace(ws, fp8_kv_scales_workspace_bytes(T, C), "fp8_kv_channel_scales", kv.device)
    _check("fp8_kv_channel_scales",
           lib().fp8_kv_channel_scales(_ptr(kv), dt, T, C, ldkv, _kv_fmt(fmt), _ptr(scales), _ptr(ws),
                                       _nbytes(ws), _stream(stream)))
    return scales


def fp8_kv_quantize_paged(kv, scales, slot_mapping, cache, fmt="e5m2", stream=None):
    """Write kv [T, C] (float32, bfloat16 or float16) into the rows slot_mapping[t]
    of the uint8 cache [num_slots, C] (contiguous) as FP8 codes of kv / scales;
    returns cache."""
    torch = _torch()
    T, C, ldkv, dt = _kv_rows(kv, "kv")
    _vec(scales, torch.float32, "scales", C, kv.device)
    _vec(slot_mapping, torch.int32, "slot_mapping", T, kv.device)
    _kv_cache(cache, C, kv.device)
    _check("fp8_kv_quantize_paged",
           lib().fp8_kv_quantize_paged(_ptr(kv), dt, T, C, ldkv, _ptr(scales), _kv_fmt(fmt), _ptr(slot_mapping),
                                       _ptr(cache), cache.shape[0], _stream(stream)))
    return cache


def fp8_kv_dequantize_paged(cache, slot_mapping, scales, fmt="e5m2", out=None, out_dtype=None, stream=None):
    """Read cache rows slot_mapping[t] back -> out [T, C] (float32 by default, or
    bfloat16 / float16: out's dtype, else out_dtype)."""
    torch = _torch()
    _kv_cache(cache)
    dev = cache.device
    num_slots, C = cache.shape
    T = slot_mapping.numel() if isinstance(slot_mapping, torch.Tensor) else -1
    _vec(slot_mapping, torch.int32, "slot_mapping", T, dev)
    _vec(scales, torch.float32, "scales", C, dev)
    if out is None:
        out = torch.empty((T, C), dtype=out_dtype or torch.float32, device=dev)
    T2, C2, ldo, odt = _kv_rows(out, "out", dev)
    if (T2, C2) != (T, C):
        raise ValueError("out: expected shape [T, C]")
    _check("fp8_kv_dequantize_paged",
           lib().fp8_kv_dequantize_paged(_ptr(cache), num_slots, _ptr(slot_mapping), T, C, _ptr(scales),
                                         _kv_fmt(fmt), _ptr(out), odt, ldo, _stream(stream)))
    return out


# The attention calls are a few microseconds of GPU work at small sizes, so
# their argument checks take a tensor's facts once and only spell out what is
# wrong (through the checks above) when something is.

def _on_stream(fn):
    """Runs fn with the first argument's device current and, when a stream is
    given, with that stream current: what fn allocates (outputs, workspace)
    then belongs to the stream that uses it, so the allocator cannot hand it to
    other work while the call still runs."""

    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        t = args[0] if args else kwargs.get(first)
        try:
            di = t.get_device()
        except AttributeError:
            di = -1
        if di < 0:
            raise TypeError(f"{fn.__name__}: expected CUDA tensors")
        if stream is None and di == _current_device():
            return fn(*args, **kwargs)
        torch = _torch()
        if stream is not None:
            if stream.device != t.device:
                raise ValueError(f"stream: on {stream.device}, expected {t.device}")
            with torch.cuda.stream(stream):
                return fn(*args, **kwargs)
        with torch.cuda.device(t.device):
            return fn(*args, **kwargs)

    return call


_device_of = None


def _current_device():
    """The number of the current device (some tensor is on one: the runtime is up)."""
    global _device_of
    if _device_of is None:
        _device_of = getattr(_torch()._C, "_cuda_getDevice", None) or _torch().cuda.current_device
    return _device_of()


_raw_stream_of = None


def _raw_stream(di):
    """The current stream of device number di, as a pointer."""
    global _raw_stream_of
    if _raw_stream_of is None:
        _raw_stream_of = getattr(_torch()._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: _torch().cuda.current_stream(d).cuda_stream)
    return _raw_stream_of(di)


def _heads(t, name, di=None, dtype=None):
    """[T, H, D] with the heads of a row adjacent, on device number di and of
    dtype when given -> (T, H, D, row stride, address)."""
    if dtype is None or not isinstance(t, _torch().Tensor) or t.dtype is not dtype or t.get_device() != di:
        _kv_dtype(t, name)
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
        if di is not None and t.get_device() != di:
            raise ValueError(f"{name}: on {t.device}, expected device {di}")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected a 3-D tensor [tokens, heads, head_dim]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1 or s1 != d and h > 1) and n and h and d:
        raise ValueError(f"{name}: expected the heads of a token adjacent (strides [*, head_dim, 1])")
    return n, h, d, (s0 if n > 1 else h * d), t.data_ptr()


def _flat(t, dtype, name, n, di):
    """Address of a contiguous tensor of n elements on device number di."""
    if isinstance(t, _tensor()) and t.dtype is dtype and t.get_device() == di and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    _vec(t, dtype, name, n)
    raise ValueError(f"{name}: on {t.device}, expected device {di}")


def _paged_cache(cache, di):
    """(slots, channels, address) of a uint8 cache [num_slots, channels]."""
    torch = _torch()
    if not (isinstance(cache, torch.Tensor) and cache.dtype is torch.uint8 and cache.get_device() == di and cache.dim() == 2
            and cache.is_contiguous()):
        _kv_cache(cache)
        raise ValueError(f"cache: on {cache.device}, expected device {di}")
    slots, C = cache.shape
    return slots, C, cache.data_ptr()


@_on_stream
def fp8_kv_append_rope_paged(k, v, positions, cos_sin, scales, slot_mapping, cache, fmt="e5m2", q=None, q_out=None,
                             interleaved=False):
    """Rotate k [T, Hkv, D] (and q [T, Hq, D]) by positions int32 [T] with the table
    cos_sin fp32 [P, rot_dim] (cosines, then sines) and write k and v as FP8 codes
    of value / scales [2 * Hkv * D] into the rows slot_mapping int32 [T] of the
    uint8 cache [num_slots, 2 * Hkv * D]; returns the rotated q (q_out, which may
    be q itself), or None without q.  stream: the stream to run on."""
    torch = _torch()
    dt = _kv_dtype(k, "k")
    dtype, di = k.dtype, k.get_device()
    T, Hkv, D, ldk, kp = _heads(k, "k", di, dtype)
    Tv, Hv, Dv, ldv, vp = _heads(v, "v", di, dtype)
    if (Tv, Hv, Dv) != (T, Hkv, D):
        raise ValueError("v: expected k's shape")
    Hq = ldq = ldqo = qp = qop = 0
    if q is not None:
        Tq, Hq, Dq, ldq, qp = _heads(q, "q", di, dtype)
        if (Tq, Dq) != (T, D):
            raise ValueError("q: expected shape [T, Hq, D] with k's T and D")
        if q_out is None:
            q_out = q.new_empty((T, Hq, D))
        To, Ho, Do, ldqo, qop = _heads(q_out, "q_out", di, dtype)
        if (To, Ho, Do) != (T, Hq, D):
            raise ValueError("q_out: expected q's shape")
    elif q_out is not None:
        raise ValueError("q_out: given without q")
    C = 2 * Hkv * D
    if not isinstance(cos_sin, torch.Tensor) or cos_sin.dim() != 2:
        raise TypeError("cos_sin: expected a contiguous float32 CUDA tensor [P, rot_dim]")
    P, rot = cos_sin.shape
    slots, cols, cp = _paged_cache(cache, di)
    if cols != C:
        raise TypeError("cache: expected a contiguous uint8 CUDA tensor [num_slots, 2 * Hkv * D]")
    i32, f32 = torch.int32, torch.float32
    _check("fp8_kv_append_rope_paged",
           lib().fp8_kv_append_rope_paged(qp, ldq, qop, ldqo, kp, ldk, vp, ldv, dt, T, Hq, Hkv, D,
                                          _flat(positions, i32, "positions", T, di),
                                          _flat(cos_sin, f32, "cos_sin", P * rot, di), P, rot,
                                          1 if interleaved else 0, _flat(scales, f32, "scales", C, di), _kv_fmt(fmt),
                                          _flat(slot_mapping, i32, "slot_mapping", T, di), cp, slots, _raw_stream(di)))
    return q_out


def _attn_args(q, cache, block_table, seq_lens, scales, block_size, alibi_slopes, out, lse):
    """What both attention calls check -> (rows, B, table width, Hq, Hkv, D, blocks, ldq, ldo, ld_table, out, and the
    addresses of q, cache, scales, block_table, seq_lens, alibi_slopes, out, lse)."""
    torch = _torch()
    dtype, di = q.dtype, q.get_device()
    rows, Hq, D, ldq, qp = _heads(q, "q", di, dtype)
    slots, C, cp = _paged_cache(cache, di)
    if block_size < 1 or slots % block_size:
        raise ValueError("cache: expected [num_blocks * block_size, 2 * Hkv * D]")
    if D == 0 or C == 0 or C % (2 * D):
        raise ValueError("cache: rows are not 2 * Hkv * D codes of q's D")
    if not isinstance(block_table, torch.Tensor) or block_table.dtype is not torch.int32 or block_table.get_device() != di:
        _on_device(block_table, torch.int32, "block_table", q.device)
    if block_table.dim() != 2:
        raise ValueError("block_table: expected a 2-D row-major int32 tensor [B, max_blocks]")
    B, width = block_table.shape
    ld_table, one = block_table.stride()
    if one != 1 and width > 1:
        raise ValueError("block_table: expected a 2-D row-major int32 tensor [B, max_blocks]")
    f32 = torch.float32
    sp, lp = _flat(scales, f32, "scales", C, di), _flat(seq_lens, torch.int32, "seq_lens", B, di)
    ap = 0 if alibi_slopes is None else _flat(alibi_slopes, f32, "alibi_slopes", Hq, di)
    if out is None:
        out = q.new_empty((rows, Hq, D))
    ro, ho, do, ldo, op = _heads(out, "out", di, dtype)
    if (ro, ho, do) != (rows, Hq, D):
        raise ValueError("out: expected q's shape")
    ep = 0
    if lse is not None:
        _dense(lse, f32, "lse", (rows, Hq), q.device)
        ep = lse.data_ptr()
    return (rows, B, width, Hq, C // (2 * D), D, slots // block_size, ldq, ldo, ld_table if B > 1 else width, out,
            qp, cp, sp, block_table.data_ptr(), lp, ap, op, ep)


def _attn_ws(ws, need, device):
    """(workspace kept alive over the call, its address, its bytes)."""
    torch = _torch()
    if ws is None:
        if need == 0 or need == SIZE_MAX:   # sizes the library refuses: the call says so
            return None, 0, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _on_device(ws, torch.uint8, "ws", device)
        if not ws.is_contiguous():
            raise ValueError("ws: expected a contiguous uint8 tensor")
    return ws, ws.data_ptr(), ws.numel()


@_on_stream
def fp8_attn_decode_paged(q, cache, block_table, seq_lens, scales, block_size, fmt="e5m2", max_len=None, sm_scale=None,
                          softcap=0.0, alibi_slopes=None, window=0, out=None, lse=None, ws=None):
    """Attention of one new token per sequence, q [B, Hq, D], over its seq_lens int32
    [B] cached tokens (the new one's among them) in the pages block_table int32
    [B, max_blocks] of the uint8 cache [num_blocks * block_size, 2 * Hkv * D] with
    channel scales fp32 [2 * Hkv * D] -> out [B, Hq, D] in q's type.

    max_len: the longest sequence's length when the host knows it (plans the
    launch; by default the block table's width).  sm_scale: D ** -0.5 by default.
    softcap, alibi_slopes fp32 [Hq], window: 0 / None for off.  lse: fp32 [B, Hq]
    that receives the log-sum-exp; with it a bfloat16 out is computed from operands
    of 2^-22, as other types are, without it of 2^-11.  ws: uint8 workspace of at least
    fp8_attn_decode_workspace_bytes(...) bytes, allocated when not given.
    stream: the stream to run on."""
    dt = _kv_dtype(q, "q")
    (rows, B, width, Hq, Hkv, D, blocks, ldq, ldo, ld_table, out, qp, cp, sp, tp, lp, ap, op, ep) = _attn_args(
        q, cache, block_table, seq_lens, scales, block_size, alibi_slopes, out, lse)
    if rows != B:
        raise ValueError("q: expected one row per sequence of block_table")
    max_len = max_len or 0
    ws, wp, wn = _attn_ws(ws, fp8_attn_decode_workspace_bytes(B, Hq, Hkv, D, block_size, width, max_len), q.device)
    _check("fp8_attn_decode_paged",
           lib().fp8_attn_decode_paged(qp, ldq, dt, cp, blocks, block_size, sp, _kv_fmt(fmt), tp, ld_table, width, lp, B,
                                       Hq, Hkv, D, max_len, D ** -0.5 if sm_scale is None else sm_scale,
                                       softcap or 0.0, ap, window or 0, op, ldo, ep, wp, wn, _raw_stream(q.get_device())))
    return out


@_on_stream
def fp8_attn_prefill_paged(q, cu_q, cache, block_table, seq_lens, scales, block_size, fmt="e5m2", max_q=None,
                           max_len=None, causal=True, prefix_lens=None, sm_scale=None, softcap=0.0, alibi_slopes=None,
                           window=0, out=None, lse=None, ws=None):
    """Attention of several new tokens per sequence -- a prompt, a chunk of one, drafted
    tokens -- over the cache: rows cu_q[b] .. cu_q[b + 1] (int32 [B + 1]) of q
    [T, Hq, D] are sequence b's newest tokens, the last of seq_lens[b] cached ones
    -> out [T, Hq, D] in q's type.  Causal (each token sees its own and earlier
    keys, and the first prefix_lens[b] int32 [B] of them in any case), or every key
    of the sequence when causal is false.  Rows no sequence owns are left as they
    were (uninitialised when out is allocated here).  max_q: the most new tokens of
    one sequence when the host knows it; by default the launch goes by their mean.
    The other arguments as for fp8_attn_decode_paged."""
    dt = _kv_dtype(q, "q")
    (T, B, width, Hq, Hkv, D, blocks, ldq, ldo, ld_table, out, qp, cp, sp, tp, lp, ap, op, ep) = _attn_args(
        q, cache, block_table, seq_lens, scales, block_size, alibi_slopes, out, lse)
    i32, di = _torch().int32, q.get_device()
    cup = _flat(cu_q, i32, "cu_q", B + 1, di)
    pp = 0 if prefix_lens is None else _flat(prefix_lens, i32, "prefix_lens", B, di)
    max_q, max_len = max_q or 0, max_len or 0
    ws, wp, wn = _attn_ws(ws, fp8_attn_prefill_workspace_bytes(T, B, Hq, Hkv, D, block_size, width, max_q, max_len),
                          q.device)
    _check("fp8_attn_prefill_paged",
           lib().fp8_attn_prefill_paged(qp, ldq, dt, cup, T, cp, blocks, block_size, sp, _kv_fmt(fmt), tp, ld_table,
                                        width, lp, B, Hq, Hkv, D, max_q, max_len, 1 if causal else 0, pp,
                                        D ** -0.5 if sm_scale is None else sm_scale, softcap or 0.0, ap, window or 0, op,
                                        ldo, ep, wp, wn, _raw_stream(di)))
    return out


@functools.lru_cache(maxsize=1024)
def fp8_attn_decode_workspace_bytes(B, Hq, Hkv, D, block_size, max_blocks, max_len=0):
    """Workspace bytes of fp8_attn_decode_paged."""
    return int(lib().fp8_attn_decode_workspace_bytes(B, Hq, Hkv, D, block_size, max_blocks, max_len))


@functools.lru_cache(maxsize=1024)
def fp8_attn_prefill_workspace_bytes(T, B, Hq, Hkv, D, block_size, max_blocks, max_q=0, max_len=0):
    """Workspace bytes of fp8_attn_prefill_paged."""
    return int(lib().fp8_attn_prefill_workspace_bytes(T, B, Hq, Hkv, D, block_size, max_blocks, max_q, max_len))


def fp8_gemm_scaled(qa, s_tok, qw, s_ch, y=None, ws=None, stream=None):
    """y[m,n] = bf16(sum_k e4m3(qa[m,k]) e4m3(qw[n,k]) * s_tok[m] * s_ch[n]).

    ws: optional uint8 device workspace of at least fp8_gemm_workspace_bytes(M, N, K)
    bytes (scratch: its contents on entry do not matter); allocated per call
    when not given and the shape needs one."""
    torch = _torch()
    M, K, lda = _rows(qa, torch.uint8, "qa")
    dev = qa.device
    N, K2, ldw = _rows(qw, torch.uint8, "qw", dev)
    if K2 != K:
        raise ValueError("qa and qw disagree on K")
    _vec(s_tok, torch.float32, "s_tok", M, dev)
    _vec(s_ch, torch.float32, "s_ch", N, dev)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    My, Ny, ldy = _rows(y, torch.bfloat16, "y", dev)
    if (My, Ny) != (M, N):
        raise ValueError("y: expected shape [M, N]")
    ws = _workspace(ws, fp8_gemm_workspace_bytes(M, N, K), "fp8_gemm_scaled", dev)
    _check("fp8_gemm_scaled",
           lib().fp8_gemm_scaled(_ptr(qa), lda, _ptr(s_tok), _ptr(qw), ldw, _ptr(s_ch), _ptr(y), ldy, M, N, K,
                                 _ptr(ws), _nbytes(ws), _stream(stream)))
    return y


def fp8_quant_gemm_fused(x, qw, s_ch, y=None, qa_out=None, s_tok_out=None, ws=None, stream=None):
    """Quantize x per token, then the scaled FP8 GEMM, in one call -> y bf16 [M, N]."""
    torch = _torch()
    M, K, ldx = _rows(x, torch.float32, "x")
    dev = x.device
    N, K2, ldw = _rows(qw, torch.uint8, "qw", dev)
    if K2 != K:
        raise ValueError("x and qw disagree on K")
    _vec(s_ch, torch.float32, "s_ch", N, dev)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    My, Ny, ldy = _rows(y, torch.bfloat16, "y", dev)
    if (My, Ny) != (M, N):
        raise ValueError("y: expected shape [M, N]")
    if qa_out is not None:
        _dense(qa_out, torch.uint8, "qa_out", (M, K), dev)
    if s_tok_out is not None:
        _vec(s_tok_out, torch.float32, "s_tok_out", M, dev)
    ws = _workspace(ws, fp8_workspace_bytes(M, N, K), "fp8_quant_gemm_fused", dev)
    _check("fp8_quant_gemm_fused",
           lib().fp8_quant_gemm_fused(_ptr(x), ldx, _ptr(qw), ldw, _ptr(s_ch), _ptr(y), ldy, M, N, K,
                                      _ptr(qa_out), _ptr(s_tok_out), _ptr(ws), _nbytes(ws), _stream(stream)))
    return y


# size of the static device scratch array of fp8_quant_gemm_fused_noalloc
FP8_NOALLOC_SCRATCH_BYTES = 72 << 20


def fp8_quant_gemm_fused_noalloc(x, qw, s_ch, y, qa_out=None, s_tok_out=None, stream=None):
    """fp8_quant_gemm_fused without a workspace: the library's static device
    scratch array holds the staged codes and split-K partial sums, so the call
    allocates nothing (y, and qa_out / s_tok_out when wanted, are the caller's)."""
    torch = _torch()
    M, K, ldx = _rows(x, torch.float32, "x")
    dev = x.device
    N, K2, ldw = _rows(qw, torch.uint8, "qw", dev)
    if K2 != K:
        raise ValueError("x and qw disagree on K")
    _vec(s_ch, torch.float32, "s_ch", N, dev)
    My, Ny, ldy = _rows(y, torch.bfloat16, "y", dev)
    if (My, Ny) != (M, N):
        raise ValueError("y: expected shape [M, N]")
    if qa_out is not None:
        _dense(qa_out, torch.uint8, "qa_out", (M, K), dev)
    if s_tok_out is not None:
        _vec(s_tok_out, torch.float32, "s_tok_out", M, dev)
    _check("fp8_quant_gemm_fused_noalloc",
           lib().fp8_quant_gemm_fused_noalloc(_ptr(x), ldx, _ptr(qw), ldw, _ptr(s_ch), _ptr(y), ldy, M, N, K,
                                              _ptr(qa_out), _ptr(s_tok_out), _stream(stream)))
    return y


def fp8_gemm_scaled_fp8out(qa, s_tok, qw, s_ch, q_out=None, s_out=None, y32_out=None, ws=None, stream=None):
    """FP8-output GEMM: y32 = acc * s_tok * s_ch in fp32, re-quantized per token
    -> (q_out uint8 [M, N], s_out fp32 [M]); y32_out (fp32 [M, N]) optional."""
    torch = _torch()
    M, K, lda = _rows(qa, torch.uint8, "qa")
    dev = qa.device
    N, K2, ldw = _rows(qw, torch.uint8, "qw", dev)
    if K2 != K:
        raise ValueError("qa and qw disagree on K")
    _vec(s_tok, torch.float32, "s_tok", M, dev)
    _vec(s_ch, torch.float32, "s_ch", N, dev)
    if q_out is None:
        q_out = torch.empty((M, N), dtype=torch.uint8, device=dev)
    Mq, Nq, ldq = _rows(q_out, torch.uint8, "q_out", dev)
    if (Mq, Nq) != (M, N):
        raise ValueError("q_out: expected shape [M, N]")
    if s_out is None:
        s_out = torch.empty(M, dtype=torch.float32, device=dev)
    _vec(s_out, torch.float32, "s_out", M, dev)
    if y32_out is not None:
        _dense(y32_out, torch.float32, "y32_out", (M, N), dev)
    need = fp8_fp8out_workspace_bytes(M, N, K)
    if need != SIZE_MAX and y32_out is not None:
        need = int(lib().fp8_gemm_workspace_bytes(M, N, K))   # y32 lives in y32_out, not in ws
    ws = _workspace(ws, need, "fp8_gemm_scaled_fp8out", dev)
    _check("fp8_gemm_scaled_fp8out",
           lib().fp8_gemm_scaled_fp8out(_ptr(qa), lda, _ptr(s_tok), _ptr(qw), ldw, _ptr(s_ch), _ptr(q_out), ldq,
                                        _ptr(s_out), _ptr(y32_out), M, N, K, _ptr(ws), _nbytes(ws), _stream(stream)))
    return q_out, s_out


def fp8_gemm_grouped_scaled(qa, s_tok, row_token, expert_offsets, qw, s_ch, y=None, ws=None, stream=None):
    """Grouped MoE GEMM over expert-sorted routed rows -> y bf16 [R, N]."""
    torch = _torch()
    T, K, _ = _rows(qa, torch.uint8, "qa")
    dev = qa.device
    if not qa.is_contiguous():
        raise ValueError("qa: expected contiguous [T, K]")
    _on_device(qw, torch.uint8, "qw", dev)
    if qw.dim() != 3 or not qw.is_contiguous():
        raise ValueError("qw: expected a contiguous uint8 CUDA tensor [E, N, K]")
    E, N, K2 = qw.shape
    if K2 != K:
        raise ValueError("qa and qw disagree on K")
    _on_device(row_token, torch.int32, "row_token", dev)
    R = row_token.numel()
    _vec(s_tok, torch.float32, "s_tok", T, dev)
    _vec(row_token, torch.int32, "row_token", R, dev)
    _vec(expert_offsets, torch.int32, "expert_offsets", E + 1, dev)
    _dense(s_ch, torch.float32, "s_ch", (E, N), dev)
    if y is None:
        y = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
    _dense(y, torch.bfloat16, "y", (R, N), dev)
    ws = _workspace(ws, fp8_grouped_workspace_bytes(T, R, E, N, K), "fp8_gemm_grouped_scaled", dev)
    _check("fp8_gemm_grouped_scaled",
           lib().fp8_gemm_grouped_scaled(_ptr(qa), _ptr(s_tok), _ptr(row_token), _ptr(expert_offsets), _ptr(qw),
                                         _ptr(s_ch), _ptr(y), T, R, E, N, K, _ptr(ws), _nbytes(ws), _stream(stream)))
    return y


FP8_ACT_NONE = 0
FP8_ACT_RELU = 1
FP8_ACT_SILU = 2
FP8_ACT_GELU = 3
FP8_ACT_GELU_TANH = 4
_ACTS = {None: FP8_ACT_NONE, "none": FP8_ACT_NONE, "relu": FP8_ACT_RELU, "silu": FP8_ACT_SILU, "gelu": FP8_ACT_GELU,
         "gelu_tanh": FP8_ACT_GELU_TANH}
_ACTS.update({v: v for v in list(_ACTS.values())})


def _act(act):
    if act not in _ACTS:
        raise ValueError(f"act: expected 'none', 'relu', 'silu', 'gelu' or 'gelu_tanh', got {act!r}")
    return _ACTS[act]


# Like the attention calls, the calls below run on the device and stream of their
# first argument and check a tensor's facts once.

def _mat(t, name, di, dtype=None, cols=None, rows=None):
    """A 2-D row-major tensor on device number di, of dtype, rows and cols when given -> (rows, cols, row stride, address)."""
    if not isinstance(t, _tensor()) or (dtype is not None and t.dtype is not dtype) or t.get_device() != di or t.dim() != 2:
        if dtype is not None:
            _on_device(t, dtype, name)
        elif not isinstance(t, _tensor()) or not t.is_cuda:
            raise TypeError(f"{name}: expected a CUDA tensor")
        if t.get_device() != di:
            raise ValueError(f"{name}: on {t.device}, expected device {di}")
        raise ValueError(f"{name}: expected a 2-D row-major tensor (unit stride along the last dim)")
    n, c = t.shape
    s0, s1 = t.stride()
    if s1 != 1 and c > 1 and n > 0:
        raise ValueError(f"{name}: expected a 2-D row-major tensor (unit stride along the last dim)")
    if rows is not None and n != rows or cols is not None and c != cols:
        raise ValueError(f"{name}: expected shape [{'*' if rows is None else rows}, {'*' if cols is None else cols}]")
    return n, c, (s0 if n > 1 else c), t.data_ptr()


_DTYPE_CODES = {}


def _dtype_code(dtype, name):
    """fp8_kv_dtype_t of a row element type."""
    if not _DTYPE_CODES:
        torch = _torch()
        _DTYPE_CODES.update({torch.float32: FP8_KV_F32, torch.bfloat16: FP8_KV_BF16, torch.float16: FP8_KV_F16})
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name}: expected float32, bfloat16 or float16")
    return code


@functools.lru_cache(maxsize=1024)
def fp8_gemm_act_workspace_bytes(M, N, K):
    """Workspace bytes of fp8_gemm_scaled_act."""
    return int(lib().fp8_gemm_act_workspace_bytes(M, N, K))


def _out_type(out, dtype, like, name):
    """The type of an output: its own, which a dtype given beside it has to be, else dtype, else that of the tensor
    `like`, else bfloat16."""
    for t, n in ((out, name), (like, "residual")):
        if t is not None and not isinstance(t, _tensor()):
            raise TypeError(f"{n}: expected a CUDA tensor")
    if out is None:
        return dtype or (like.dtype if like is not None else _torch().bfloat16)
    if dtype is not None and dtype is not out.dtype:
        raise TypeError(f"{name}: of {out.dtype}, expected {name}_dtype {dtype}")
    return out.dtype


@_on_stream
def fp8_gemm_scaled_act(qa, s_tok, qw, s_ch, bias=None, act="none", residual=None, y=None, y_dtype=None, ws=None):
    """y[m,n] = round(act(sum_k e4m3(qa[m,k]) e4m3(qw[n,k]) * s_tok[m] * s_ch[n] + bias[n]) + residual[m,n]).

    bias: fp32 [N] or None.  act: 'none', 'relu', 'silu', 'gelu' (erf) or 'gelu_tanh'.
    residual: [M, N] in y's type or None; it may be y itself.  y: [M, N] float32,
    bfloat16 or float16 with any row stride; allocated when not given, in y_dtype
    (by default the residual's type, else bfloat16; of a y given, its own type).  ws: uint8 workspace of at least
    fp8_gemm_act_workspace_bytes(M, N, K) bytes, allocated when not given.
    stream: the stream to run on."""
    torch = _torch()
    di, u8, f32 = qa.get_device(), torch.uint8, torch.float32
    M, K, lda, qp = _mat(qa, "qa", di, u8)
    N, _, ldw, wp = _mat(qw, "qw", di, u8, cols=K)
    tp, cp = _flat(s_tok, f32, "s_tok", M, di), _flat(s_ch, f32, "s_ch", N, di)
    bp = 0 if bias is None else _flat(bias, f32, "bias", N, di)
    dtype = _out_type(y, y_dtype, residual, "y")
    code = _dtype_code(dtype, "y")
    if y is None:
        y = qa.new_empty((M, N), dtype=dtype)
        ldy, yp = N, y.data_ptr()
    else:
        _, _, ldy, yp = _mat(y, "y", di, dtype, N, M)
    ldr = rp = 0
    if residual is not None:
        _, _, ldr, rp = _mat(residual, "residual", di, dtype, N, M)
    ws, wsp, wsn = _attn_ws(ws, fp8_gemm_act_workspace_bytes(M, N, K), qa.device)
    _check("fp8_gemm_scaled_act",
           lib().fp8_gemm_scaled_act(qp, lda, tp, wp, ldw, cp, bp, _act(act), rp, ldr, yp, code, ldy, M, N, K, wsp, wsn,
                                     _raw_stream(di)))
    return y


@_on_stream
def fp8_gemm_grouped_scaled_act(qa, s_tok, row_token, expert_offsets, qw, s_ch, bias=None, act="none", y=None,
                                y_dtype=None, ws=None):
    """The expert product over rows sorted by expert, with an epilogue: row r of expert e is
    y[r,n] = round(act(sum_k e4m3(qa[t,k]) e4m3(qw[e,n,k]) * s_tok[t] * s_ch[e,n] + bias[e,n])), t = row_token[r].

    qa uint8 [T, K], qw uint8 [E, N, K], s_ch and bias fp32 [E, N] (bias may be
    None), row_token int32 [R], expert_offsets int32 [E + 1] as fp8_moe_sort gives
    them; rows from expert_offsets[E] on are left as they were (uninitialised when y
    is allocated here).  y and y_dtype as for fp8_gemm_scaled_act."""
    torch = _torch()
    di, u8, f32, i32 = qa.get_device(), torch.uint8, torch.float32, torch.int32
    T, K, _, qp = _mat(qa, "qa", di, u8)
    if not qa.is_contiguous():
        raise ValueError("qa: expected contiguous [T, K]")
    _on_device(qw, u8, "qw", qa.device)
    if qw.dim() != 3 or not qw.is_contiguous() or qw.shape[2] != K:
        raise ValueError("qw: expected a contiguous uint8 CUDA tensor [E, N, K] with qa's K")
    E, N, _ = qw.shape
    _on_device(row_token, i32, "row_token", qa.device)
    R = row_token.numel()
    tp, rp = _flat(s_tok, f32, "s_tok", T, di), _flat(row_token, i32, "row_token", R, di)
    op = _flat(expert_offsets, i32, "expert_offsets", E + 1, di)
    cp = _flat(s_ch, f32, "s_ch", E * N, di)
    bp = 0 if bias is None else _flat(bias, f32, "bias", E * N, di)
    dtype = _out_type(y, y_dtype, None, "y")
    code = _dtype_code(dtype, "y")
    if y is None:
        y = qa.new_empty((R, N), dtype=dtype)
        ldy, yp = N, y.data_ptr()
    else:
        _, _, ldy, yp = _mat(y, "y", di, dtype, N, R)
    ws, wsp, wsn = _attn_ws(ws, fp8_grouped_workspace_bytes(T, R, E, N, K), qa.device)
    _check("fp8_gemm_grouped_scaled_act",
           lib().fp8_gemm_grouped_scaled_act(qp, tp, rp, op, qw.data_ptr(), cp, bp, _act(act), yp, code, ldy, T, R, E, N,
                                             K, wsp, wsn, _raw_stream(di)))
    return y


@_on_stream
def fp8_act_quantize(h, act="silu", gated=True, q=None, scales=None, live_rows=None):
    """v = act(h[:, :F]) * h[:, F:] (gated) or act(h), quantized per token to E4M3 ->
    (q uint8 [M, F], scales fp32 [M]).

    h: [M, 2 F] (gated) or [M, F], float32, bfloat16 or float16.  live_rows: int32
    tensor of one element on the device (e.g. expert_offsets[-1:]): rows from it on
    are left as they were (uninitialised when q is allocated here)."""
    torch = _torch()
    di = h.get_device()
    code = _dtype_code(h.dtype, "h")
    M, C, ldh, hp = _mat(h, "h", di)
    if gated and C % 2:
        raise ValueError("h: expected [M, 2 F] (gated)")
    F = C // 2 if gated else C
    if q is None:
        q = h.new_empty((M, F), dtype=torch.uint8)
    if scales is None:
        scales = h.new_empty(M, dtype=torch.float32)
    _, _, ldq, qp = _mat(q, "q", di, torch.uint8, F, M)
    lp = 0 if live_rows is None else _flat(live_rows, torch.int32, "live_rows", 1, di)
    _check("fp8_act_quantize",
           lib().fp8_act_quantize(hp, ldh, code, M, F, _act(act), 1 if gated else 0, qp, ldq,
                                  _flat(scales, torch.float32, "scales", M, di), lp, _raw_stream(di)))
    return q, scales


@functools.lru_cache(maxsize=1024)
def fp8_moe_sort_workspace_bytes(T, topk, E):
    """Workspace bytes of fp8_moe_sort."""
    return int(lib().fp8_moe_sort_workspace_bytes(T, topk, E))


@_on_stream
def fp8_moe_sort(expert_ids, num_experts, expert_offsets=None, row_token=None, row_of=None, ws=None):
    """The choices expert_ids [T, topk] (int32 or int64, contiguous) in the stable order of
    their experts -> (expert_offsets int32 [num_experts + 1], row_token int32 [T * topk],
    row_of int32 [T, topk]): choice (t, j) is row row_of[t, j] of token
    row_token[row] == t.  An id outside [0, num_experts) has row_of -1; row_token is -1
    from row expert_offsets[num_experts] on."""
    torch = _torch()
    di, i32 = expert_ids.get_device(), torch.int32
    if expert_ids.dtype is not i32 and expert_ids.dtype is not torch.int64:
        raise TypeError("expert_ids: expected an int32 or int64 CUDA tensor")
    if expert_ids.dim() != 2 or not expert_ids.is_contiguous():
        raise ValueError("expert_ids: expected a contiguous tensor [T, topk]")
    T, topk = expert_ids.shape
    R = T * topk
    if expert_offsets is None:
        expert_offsets = expert_ids.new_empty(max(num_experts, 0) + 1, dtype=i32)
        op = expert_offsets.data_ptr()
    else:
        op = _flat(expert_offsets, i32, "expert_offsets", max(num_experts, 0) + 1, di)
    if row_token is None:
        row_token = expert_ids.new_empty(R, dtype=i32)
        tp = row_token.data_ptr()
    else:
        tp = _flat(row_token, i32, "row_token", R, di)
    if row_of is None:
        row_of = expert_ids.new_empty((T, topk), dtype=i32)
        rp = row_of.data_ptr()
    else:
        rp = _flat(row_of, i32, "row_of", R, di)
    ws, wsp, wsn = _attn_ws(ws, fp8_moe_sort_workspace_bytes(T, topk, num_experts), expert_ids.device)
    _check("fp8_moe_sort",
           lib().fp8_moe_sort(expert_ids.data_ptr(), 0 if expert_ids.dtype is i32 else 1, T, topk, num_experts, op, tp, rp,
                              wsp, wsn, _raw_stream(di)))
    return expert_offsets, row_token, row_of


def _choices(row_of, di):
    """(T, topk, address) of row_of int32 [T, topk]."""
    torch = _torch()
    if not isinstance(row_of, torch.Tensor) or row_of.dtype is not torch.int32 or row_of.get_device() != di:
        _on_device(row_of, torch.int32, "row_of", torch.device("cuda", di))
    if row_of.dim() != 2 or not row_of.is_contiguous():
        raise ValueError("row_of: expected a contiguous int32 tensor [T, topk]")
    return row_of.shape[0], row_of.shape[1], row_of.data_ptr()


@_on_stream
def fp8_moe_permute(x, row_of, num_rows=None, s_tok=None, out=None, s_out=None):
    """Tokens x [T, H] (uint8 codes, float32, bfloat16 or float16) moved to the rows
    row_of int32 [T, topk] -> out [num_rows, H], or (out, s_out) with the tokens' scales
    s_tok fp32 [T].  num_rows: T * topk by default (out's rows when out is given).
    Entries outside [0, num_rows) are skipped and rows no entry names left as they
    were (uninitialised when out is allocated here).  The gradient with respect to x
    is fp8_moe_combine(dout, row_of)."""
    torch = _torch()
    di = x.get_device()
    if x.dtype not in (torch.uint8, torch.bfloat16, torch.float16, torch.float32):
        raise TypeError("x: expected uint8, float32, bfloat16 or float16")
    T, topk, rp = _choices(row_of, di)
    _, H, ldx, xp = _mat(x, "x", di, rows=T)
    if out is None:
        out = x.new_empty((T * topk if num_rows is None else num_rows, H))
    R, _, ldo, op = _mat(out, "out", di, x.dtype, H, num_rows)
    tp = sp = 0
    if s_tok is not None:
        tp = _flat(s_tok, torch.float32, "s_tok", T, di)
        if s_out is None:
            s_out = x.new_empty(R, dtype=torch.float32)
        sp = _flat(s_out, torch.float32, "s_out", R, di)
    elif s_out is not None:
        raise ValueError("s_out: given without s_tok")
    _check("fp8_moe_permute",
           lib().fp8_moe_permute(xp, ldx, tp, rp, T, topk, R, H, x.element_size(), op, ldo, sp, _raw_stream(di)))
    return out if s_tok is None else (out, s_out)


@_on_stream
def fp8_moe_combine(y, row_of, weights=None, residual=None, out=None, out_dtype=None):
    """out[t] = round(residual[t] + sum_j weights[t, j] * y[row_of[t, j]]): the experts' rows
    y [R, H] back to the tokens, weights fp32 [T, topk] (None: ones), residual [T, H] in
    out's type (None: nothing; it may be out itself) -> out [T, H].  Entries of row_of
    int32 [T, topk] outside [0, R) add nothing.  out_dtype: of an out given, its own;
    else by default the residual's type, else y's."""
    torch = _torch()
    di = y.get_device()
    code = _dtype_code(y.dtype, "y")
    T, topk, rp = _choices(row_of, di)
    R, H, ldy, yp = _mat(y, "y", di)
    wp = 0 if weights is None else _flat(weights, torch.float32, "weights", T * topk, di)
    dtype = _out_type(out, out_dtype, y if residual is None else residual, "out")
    out_code = _dtype_code(dtype, "out")
    if out is None:
        out = y.new_empty((T, H), dtype=dtype)
        ldo, op = H, out.data_ptr()
    else:
        _, _, ldo, op = _mat(out, "out", di, dtype, H, T)
    ldr = sp = 0
    if residual is not None:
        _, _, ldr, sp = _mat(residual, "residual", di, dtype, H, T)
    _check("fp8_moe_combine",
           lib().fp8_moe_combine(yp, ldy, code, rp, wp, sp, ldr, op, out_code, ldo, T, topk, R, H, _raw_stream(di)))
    return out


@_on_stream
def fp8_moe_combine_grad(dout, y, row_of, weights=None, dy=None, dweights=None, need_dy=True, need_dweights=True):
    """The gradient of fp8_moe_combine for dout [T, H]: dy[row_of[t, j]] = round(weights[t, j] *
    dout[t]) in y's type and dweights[t, j] = <dout[t], y[row_of[t, j]]> -> (dy [R, H],
    dweights fp32 [T, topk]), None for the one not needed.  The residual's gradient is
    dout.  Entries outside [0, R) write no row and a dweights of 0; rows no entry names
    are left as they were (uninitialised when dy is allocated here).  dy may be y itself."""
    torch = _torch()
    di = dout.get_device()
    code = _dtype_code(dout.dtype, "dout")
    T, topk, rp = _choices(row_of, di)
    _, H, ldd, dp = _mat(dout, "dout", di, rows=T)
    R, _, ldy, yp = _mat(y, "y", di, cols=H)
    y_code = _dtype_code(y.dtype, "y")
    wp = 0 if weights is None else _flat(weights, torch.float32, "weights", T * topk, di)
    lddy = yg = wg = 0
    if dy is not None or need_dy:
        if dy is None:
            dy = y.new_empty((R, H))
        _, _, lddy, yg = _mat(dy, "dy", di, y.dtype, H, R)
    if dweights is not None or need_dweights:
        if dweights is None:
            dweights = y.new_empty((T, topk), dtype=torch.float32)
        wg = _flat(dweights, torch.float32, "dweights", T * topk, di)
    _check("fp8_moe_combine_grad",
           lib().fp8_moe_combine_grad(dp, ldd, code, yp, ldy, y_code, rp, wp, yg, lddy, wg, T, topk, R, H,
                                      _raw_stream(di)))
    return dy, dweights


def fp8_stream_read(buf, workgroups=256, nontemporal=False, sink=None, stream=None):
    """Read every byte of the contiguous device tensor `buf` once (the HBM read
    ceiling the decode kernels are measured against); returns the sink tensor."""
    torch = _torch()
    if not isinstance(buf, torch.Tensor) or not buf.is_cuda or not buf.is_contiguous():
        raise TypeError("buf: expected a contiguous CUDA tensor")
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device=buf.device)
    _vec(sink, torch.int32, "sink", 1, buf.device)
    _check("fp8_stream_read", lib().fp8_stream_read(_ptr(buf), _nbytes(buf), int(workgroups), int(bool(nontemporal)),
                                                    _ptr(sink), _stream(stream)))
    return sink
