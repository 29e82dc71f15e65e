"""ctypes binding of libw4.so: one Python function per C entry point, same
names, argument marshalling only (torch tensors -> device pointers, dtype
codes, the current HIP stream). Every step runs in the HIP library; there
is no fallback. A missing library or a failed call raises."""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libw4.so")

W4_BF16, W4_F16, W4_F32, W4_I8, W4_FP8_E4M3 = 1, 2, 3, 4, 5
W4_LAYOUT_GPTQ_KN, W4_LAYOUT_CT_NK, W4_LAYOUT_S4_NK, W4_LAYOUT_I8_NK = 1, 2, 3, 4
W4_LINEAR_MIN_TOKENS_INT8 = 33          # include/w4.h: the library's default dispatch threshold
ERRORS = {0: "OK", -1: "INVALID", -2: "ALIGN", -3: "GROUP", -4: "DTYPE", -5: "UNSUPPORTED", -6: "HIP"}

_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int

_SIGS = {
    "w4a8_quantize_act": [_P, _I, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _P],
    "w4a8_quantize_act_static": [_P, _I, _I64, _I64, _I64, _P, _P, _I, _P, _P, _I64, _P],
    "w4_repack_bytes": [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4_repack": [_P, _I, _I64, _I64, _I64, _P, _P],
    "w4a8_gemm": [_P, _P, _P, _P, _I, _I64, _P, _P, _I, _I64, _I64, _I64, _P],
    "w4a8_gemm_partials": [_P, _P, _I64, _P, _I64, _I64, _I64, _P],
    "w4a16_repack_bytes": [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)],
    "w4a16_repack": [_P, _P, _P, _I, _I64, _I64, _I64, _P, _P, _P],
    "w4a16_gemm": [_P, _P, _P, _I64, _P, _I64, _I64, _I64, _P],
    "w4a8_grouped_gemm": [_P, _I, _P, _P, _P, _P, _I64, _P, _P, _I, _I64, _P, _I, _I64, _I64, _I64, _I64, _P],
    "w4a16_tiled_gemm": [_P, _I, _P, _P, _I, _I64, _P, _P, _I64, _I64, _I64, _P],
    "w4_linear_workspace_bytes": [_I64, _I64, _I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4_linear": [_P, _I, _P, _P, _I, _I64, _P, _P, _I64, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
    "w4_linear_noalloc": [_P, _I, _P, _P, _I, _I64, _P, _P, _I64, _I64, _I64, _I64, _P],
    "w4a16_dequantize": [_P, _P, _P, _I, _I64, _I64, _I64, _P, _P],
    "w4a16_prefill_gemm": [_P, _P, _P, _I64, _I64, _I64, _P],
    "w4a16_prefill_workspace_bytes": [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4a16_prefill": [_P, _P, _P, _P, _I, _I64, _P, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
    "w4_quantize_groupwise": [_P, _I, _I64, _I64, _I64, _P, _P, _P, _I, _P],
    "w4a16_embedding": [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P],
    "w4a8_quantize_act_asym": [_P, _I, _I64, _I64, _I64, _P, _P, _P, _P],
    "w4a8_weight_offsets": [_P, _P, _I, _I64, _I64, _I64, _P, _P],
    "w4a8_gemm_asym": [_P, _P, _P, _P, _P, _I, _I64, _P, _P, _P, _I, _I64, _I64, _I64, _P],
    "w4_fp8_encode_range": [ctypes.c_uint32, _I64, _P, _P],
    "w4_probe_mfma": [_I, _I64, _P, _I64, ctypes.POINTER(ctypes.c_double), _P],
    "w4_pack_nibbles": [_P, _I64, _I64, _P, _P],
    "w4_unpack_nibbles": [_P, _I64, _I64, _P, _P],
    "w4_route_workspace_bytes": [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4_route": [_P, _I, _I64, _I64, _I64, _I, _P, _I64, _I64, _I64, _I64, _I, ctypes.c_double, _P, _P, _P, _P, _P,
                 _P, ctypes.c_size_t, _P],
    "w4_fp8_block_quantize": [_P, _I, _I64, _I64, _I64, _I, _P, _P, _P],
    "w4_fp8_block_gemm_workspace_bytes": [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4_fp8_block_gemm": [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
    "w4_fp8_block_grouped_gemm": [_P, _P, _P, _P, _I64, _P, _P, _P, _I, _I64, _I64, _I64, _I64, _P],
    "w4_combine": [_P, _I, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P],
    "w4_mxfp4_quantize": [_P, _I, _I64, _I64, _I64, _I, _P, _P, _P],
    "w4_mxfp4_dequantize": [_P, _P, _I64, _I64, _P, _I, _P],
    "w4_mxfp4_gemm_workspace_bytes": [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4_mxfp4_gemm": [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
    "w4_mxfp4_linear_workspace_bytes": [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4_mxfp4_linear": [_P, _I, _P, _P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
    "w4_mxfp4_grouped_gemm": [_P, _P, _P, _P, _I64, _P, _P, _P, _I, _I64, _I64, _I64, _I64, _P],
    "w4_moe_decode_workspace_bytes": [_I64, _I64, _I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "w4_moe_decode": [_P, _I, _P, _I, _I64, _I, _P, _I64, _I64, _I64, _I64, _I, ctypes.c_double, _I, _P, _P, _P, _P, _I64,
                      _P, _P, _I64, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
    "w4_last_error": [],
    "w4_version": [],
}


class W4Error(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {ERRORS.get(code, code)} ({code}): {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libw4.so (built in-tree by build.py). Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with int4_weight_quantized_amd/build.py "
                               "(or __graft_entry__.build()); there is no fallback")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_char_p if name == "w4_last_error" else ctypes.c_int
        _lib = L
    return _lib


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise W4Error(fn, rc, lib().w4_last_error().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr() or None


def _stream(stream=None) -> int | None:
    if stream is None:      # the handle alone: building a Stream object costs a microsecond
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) or None
    return stream.cuda_stream or None


def _half_code(dt) -> int:
    if dt == torch.bfloat16:
        return W4_BF16
    if dt == torch.float16:
        return W4_F16
    raise TypeError(f"unsupported half dtype {dt}")


# ----------------------------------------------------------------- entry points

def w4a8_quantize_act(x: torch.Tensor, code_dtype: str = "i8", group_sums_group: int | None = None,
                      stream=None):
    """x [M, K] bf16/fp16 -> (codes [M, K] int8 or uint8 E4M3 bits, scales fp32 [M],
    group_sums fp32 [M, K/group] or None)."""
    M, K = x.shape
    fp8 = code_dtype == "fp8"
    codes = torch.empty((M, K), dtype=torch.uint8 if fp8 else torch.int8, device=x.device)
    scales = torch.empty((M,), dtype=torch.float32, device=x.device)
    gs = None
    if group_sums_group is not None:
        gs = torch.empty((M, K // group_sums_group), dtype=torch.float32, device=x.device)
    quantize_act_into(x, codes, scales, gs, group_sums_group or 0, fp8, stream)
    return codes, scales, gs


def quantize_act_into(x, codes, scales, group_sums=None, group=0, fp8=False, stream=None):
    M, K = x.shape
    _check("w4a8_quantize_act", lib().w4a8_quantize_act(
        _ptr(x), _half_code(x.dtype), M, K, K, _ptr(codes), W4_FP8_E4M3 if fp8 else W4_I8,
        _ptr(scales), _ptr(group_sums), group, _stream(stream)))


def w4a8_quantize_act_static(x: torch.Tensor, static_scale: torch.Tensor, code_dtype: str = "i8",
                             group_sums_group: int | None = None, stream=None):
    """As w4a8_quantize_act with a calibrated per-tensor scale (device fp32 tensor of one element)."""
    M, K = x.shape
    fp8 = code_dtype == "fp8"
    codes = torch.empty((M, K), dtype=torch.uint8 if fp8 else torch.int8, device=x.device)
    scales = torch.empty((M,), dtype=torch.float32, device=x.device)
    gs = None
    if group_sums_group is not None:
        gs = torch.empty((M, K // group_sums_group), dtype=torch.float32, device=x.device)
    _check("w4a8_quantize_act_static", lib().w4a8_quantize_act_static(
        _ptr(x), _half_code(x.dtype), M, K, K, _ptr(static_scale), _ptr(codes), W4_FP8_E4M3 if fp8 else W4_I8,
        _ptr(scales), _ptr(gs), group_sums_group or 0, _stream(stream)))
    return codes, scales, gs


def w4a8_quantize_act_asym(x: torch.Tensor, stream=None):
    """x [M, K] bf16/fp16 -> (codes int8 [M, K], scales fp32 [M], offsets fp32 [M]),
    x ~ code * scale + offset per row."""
    M, K = x.shape
    codes = torch.empty((M, K), dtype=torch.int8, device=x.device)
    scales = torch.empty((M,), dtype=torch.float32, device=x.device)
    offsets = torch.empty((M,), dtype=torch.float32, device=x.device)
    w4a8_quantize_act_asym_into(x, codes, scales, offsets, stream)
    return codes, scales, offsets


def w4a8_quantize_act_asym_into(x, codes, scales, offsets, stream=None):
    M, K = x.shape
    _check("w4a8_quantize_act_asym", lib().w4a8_quantize_act_asym(
        _ptr(x), _half_code(x.dtype), M, K, K, _ptr(codes), _ptr(scales), _ptr(offsets), _stream(stream)))


def w4a8_weight_offsets(w_tiled, w_scale, group: int, K: int, N: int, stream=None) -> torch.Tensor:
    """fp32 [N]: sum_g w_scale[g, n] * sum_{k in g} (q[k, n] - 8), from the tiled weights."""
    out = torch.empty((N,), dtype=torch.float32, device=w_tiled.device)
    sdt = W4_F16 if w_scale.dtype == torch.float16 else (W4_BF16 if w_scale.dtype == torch.bfloat16 else W4_F32)
    _check("w4a8_weight_offsets", lib().w4a8_weight_offsets(
        _ptr(w_tiled), _ptr(w_scale), sdt, group, K, N, _ptr(out), _stream(stream)))
    return out


def w4a8_gemm_asym(a, a_scale, a_offset, w_tiled, w_scale, group: int, w_offsets, N: int,
                   out_dtype=torch.bfloat16, bias=None, out=None, stream=None):
    M, K = a.shape
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    sdt = W4_F16 if w_scale.dtype == torch.float16 else (W4_BF16 if w_scale.dtype == torch.bfloat16 else W4_F32)
    _check("w4a8_gemm_asym", lib().w4a8_gemm_asym(
        _ptr(a), _ptr(a_scale), _ptr(a_offset), _ptr(w_tiled), _ptr(w_scale), sdt, group, _ptr(w_offsets),
        _ptr(bias), _ptr(out), _half_code(out.dtype), M, N, K, _stream(stream)))
    return out


def w4_repack_bytes(K: int, N: int) -> int:
    n = ctypes.c_size_t(0)
    _check("w4_repack_bytes", lib().w4_repack_bytes(K, N, ctypes.byref(n)))
    return n.value


def w4_repack(src: torch.Tensor, layout: int, K: int, N: int, batch: int = 1, stream=None) -> torch.Tensor:
    """Repack `batch` int4 matrices into the kernel-tiled layout (uint8 buffer)."""
    nbytes = w4_repack_bytes(K, N)
    dst = torch.empty((batch, nbytes), dtype=torch.uint8, device=src.device)
    _check("w4_repack", lib().w4_repack(_ptr(src), layout, K, N, batch, _ptr(dst), _stream(stream)))
    return dst


def w4_fp8_encode_range(first_bits: int, n: int, out=None, device="cuda", stream=None) -> torch.Tensor:
    """E4M3 codes (uint8 [n]) of the fp32 values with bit patterns
    first_bits .. first_bits + n - 1, by the quantizer's own conversion."""
    if out is None:
        out = torch.empty((n,), dtype=torch.uint8, device=device)
    _check("w4_fp8_encode_range", lib().w4_fp8_encode_range(first_bits, n, _ptr(out), _stream(stream)))
    return out


def w4_probe_mfma(kind: int, iters: int, sink: torch.Tensor, stream=None) -> float:
    """Launch the pure-MFMA loop (0 int8, 1 fp8, 2 bf16); returns its op count."""
    ops_ = ctypes.c_double(0.0)
    _check("w4_probe_mfma", lib().w4_probe_mfma(kind, iters, _ptr(sink), sink.numel(), ctypes.byref(ops_),
                                                _stream(stream)))
    return ops_.value


def w4_pack_nibbles(codes: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """codes uint8 [N, K] (0..15) -> uint8 [N, K/2], low nibble first."""
    N, K = codes.shape
    if out is None:
        out = torch.empty((N, K // 2), dtype=torch.uint8, device=codes.device)
    _check("w4_pack_nibbles", lib().w4_pack_nibbles(_ptr(codes), N, K, _ptr(out), _stream(stream)))
    return out


def w4_unpack_nibbles(packed: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """uint8 [N, K/2] -> codes uint8 [N, K]."""
    N, K = packed.shape[0], packed.shape[1] * 2
    if out is None:
        out = torch.empty((N, K), dtype=torch.uint8, device=packed.device)
    _check("w4_unpack_nibbles", lib().w4_unpack_nibbles(_ptr(packed), N, K, _ptr(out), _stream(stream)))
    return out


def w4a8_gemm(a, a_scale, w_tiled, w_scale, group: int, N: int, out_dtype=torch.bfloat16, bias=None,
              out=None, stream=None):
    M, K = a.shape
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    sdt = W4_F16 if w_scale.dtype == torch.float16 else (W4_BF16 if w_scale.dtype == torch.bfloat16 else W4_F32)
    _check("w4a8_gemm", lib().w4a8_gemm(
        _ptr(a), _ptr(a_scale), _ptr(w_tiled), _ptr(w_scale), sdt, group, _ptr(bias), _ptr(out),
        _half_code(out.dtype), M, N, K, _stream(stream)))
    return out


def w4a8_gemm_partials(a, w_tiled, group: int, N: int, stream=None):
    M, K = a.shape
    G = 1 if group == -1 else K // group
    P = torch.empty((M, G, N), dtype=torch.int32, device=a.device)
    _check("w4a8_gemm_partials", lib().w4a8_gemm_partials(
        _ptr(a), _ptr(w_tiled), group, _ptr(P), M, N, K, _stream(stream)))
    return P


def w4a16_repack_bytes(K: int, N: int, group: int):
    wb, sb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("w4a16_repack_bytes", lib().w4a16_repack_bytes(K, N, group, ctypes.byref(wb), ctypes.byref(sb)))
    return wb.value, sb.value


def w4a16_repack(w, scale, zero, group: int, stream=None):
    """Load-time repack of byte-layout weights [N, K/2] with bf16 scale/zero [N, K/group]
    into (w_tiled, sz_tiled) uint8 buffers."""
    N, K = w.shape[0], w.shape[1] * 2
    wb, sb = w4a16_repack_bytes(K, N, group)
    wt = torch.empty((wb,), dtype=torch.uint8, device=w.device)
    st = torch.empty((sb,), dtype=torch.uint8, device=w.device)
    _check("w4a16_repack", lib().w4a16_repack(
        _ptr(w), _ptr(scale), _ptr(zero), _half_code(scale.dtype), group, K, N, _ptr(wt), _ptr(st),
        _stream(stream)))
    return wt, st


def w4a16_gemm(x, w_tiled, sz_tiled, group: int, N: int, out=None, stream=None):
    M, K = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check("w4a16_gemm", lib().w4a16_gemm(
        _ptr(x), _ptr(w_tiled), _ptr(sz_tiled), group, _ptr(out), M, N, K, _stream(stream)))
    return out


def w4a8_grouped_gemm(a8, a_scale, a_group_sums, row_token, expert_offsets, w_tiled, w_scale,
                      group: int, N: int, out=None, stream=None):
    T, K = a8.shape
    R = row_token.shape[0]
    E = expert_offsets.shape[0] - 1
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=a8.device)
    _check("w4a8_grouped_gemm", lib().w4a8_grouped_gemm(
        _ptr(a8), W4_FP8_E4M3, _ptr(a_scale), _ptr(a_group_sums), _ptr(row_token), _ptr(expert_offsets),
        E, _ptr(w_tiled), _ptr(w_scale), W4_F16, group, _ptr(out), W4_BF16, T, R, N, K, _stream(stream)))
    return out


def w4a16_tiled_gemm(x, w_tiled, w_scale, group: int, N: int, bias=None, out=None, stream=None):
    """Weight-only path on the w4_repack tiles: x [M <= 16, K] bf16/fp16 -> out [M, N] (x dtype)."""
    M, K = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    _check("w4a16_tiled_gemm", lib().w4a16_tiled_gemm(
        _ptr(x), _half_code(x.dtype), _ptr(w_tiled), _ptr(w_scale), W4_F16 if w_scale.dtype == torch.float16 else W4_BF16,
        group, _ptr(bias), _ptr(out), M, N, K, _stream(stream)))
    return out


def w4_linear_workspace_bytes(M: int, N: int, K: int, group: int, min_tokens_int8: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check("w4_linear_workspace_bytes", lib().w4_linear_workspace_bytes(M, N, K, group, min_tokens_int8,
                                                                        ctypes.byref(n)))
    return n.value


def w4_linear(x, w_tiled, w_scale, group: int, N: int, bias=None, min_tokens_int8: int = 0, out=None,
              workspace=None, stream=None):
    """The layer with its per-call dispatch: int8 path from min_tokens_int8 rows up (<= 0: the library's
    default), weight-only path below. The workspace (uint8, device) is allocated here if not given."""
    M, K = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    need = w4_linear_workspace_bytes(M, N, K, group, min_tokens_int8)
    if workspace is None and need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    _check("w4_linear", lib().w4_linear(
        _ptr(x), _half_code(x.dtype), _ptr(w_tiled), _ptr(w_scale), W4_F16 if w_scale.dtype == torch.float16 else W4_BF16,
        group, _ptr(bias), _ptr(out), M, N, K, min_tokens_int8, _ptr(workspace) if need else None,
        workspace.numel() if workspace is not None else 0, _stream(stream)))
    return out


W4_LINEAR_NOALLOC_SCRATCH_BYTES = 64 << 20     # include/w4.h


def w4_linear_noalloc(x, w_tiled, w_scale, group: int, N: int, bias=None, min_tokens_int8: int = 0, out=None,
                      stream=None):
    """w4_linear with the library's own device scratch (no workspace argument)."""
    M, K = x.shape
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    _check("w4_linear_noalloc", lib().w4_linear_noalloc(
        _ptr(x), _half_code(x.dtype), _ptr(w_tiled), _ptr(w_scale), W4_F16, group, _ptr(bias), _ptr(out), M, N, K,
        min_tokens_int8, _stream(stream)))
    return out


def w4a16_dequantize(w, scale, zero, group: int, out=None, stream=None):
    """Row-major int4 bytes [N, K/2] with bf16 scale/zero [N, K/group] -> bf16 weights [N, K]."""
    N, K = w.shape[0], w.shape[1] * 2
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=w.device)
    _check("w4a16_dequantize", lib().w4a16_dequantize(
        _ptr(w), _ptr(scale), _ptr(zero), _half_code(scale.dtype), group, K, N, _ptr(out), _stream(stream)))
    return out


def w4_quantize_groupwise(w, group: int, sz_dtype=torch.float32, stream=None):
    """w [N, K] bf16/fp16/fp32 -> (packed uint8 [N, K/2], scale [N, K/group], zero [N, K/group])."""
    N, K = w.shape
    wdt = {torch.bfloat16: W4_BF16, torch.float16: W4_F16, torch.float32: W4_F32}[w.dtype]
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    scale = torch.empty((N, K // group), dtype=sz_dtype, device=w.device)
    zero = torch.empty_like(scale)
    _check("w4_quantize_groupwise", lib().w4_quantize_groupwise(
        _ptr(w), wdt, N, K, group, _ptr(packed), _ptr(scale), _ptr(zero),
        W4_F32 if sz_dtype == torch.float32 else W4_BF16, _stream(stream)))
    return packed, scale, zero


def w4a16_embedding(ids, w_tiled, sz_tiled, group: int, V: int, K: int, out=None, stream=None):
    """ids int32 [T] -> bf16 [T, K]: rows of the tiled [V, K] table, dequantized."""
    T = ids.numel()
    if out is None:
        out = torch.empty((T, K), dtype=torch.bfloat16, device=ids.device)
    _check("w4a16_embedding", lib().w4a16_embedding(
        _ptr(ids), T, _ptr(w_tiled), _ptr(sz_tiled), group, V, K, _ptr(out), _stream(stream)))
    return out


def w4_version() -> int:
    return lib().w4_version()


def w4a16_prefill_gemm(x, w, out=None, stream=None):
    """bf16 x [M, K] times bf16 w [N, K] transposed -> bf16 [M, N]."""
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check("w4a16_prefill_gemm", lib().w4a16_prefill_gemm(_ptr(x), _ptr(w), _ptr(out), M, N, K, _stream(stream)))
    return out


def w4a16_prefill_workspace_bytes(N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    _check("w4a16_prefill_workspace_bytes", lib().w4a16_prefill_workspace_bytes(N, K, ctypes.byref(n)))
    return n.value


def w4a16_prefill(x, w, scale, zero, group: int, out=None, workspace=None, stream=None):
    """The W4A16 prefill path: dequantize the byte-layout weights [N, K/2] to bf16 (in the workspace) and
    run the bf16 GEMM. The workspace (uint8, device) is allocated here if not given."""
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    need = w4a16_prefill_workspace_bytes(N, K)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    _check("w4a16_prefill", lib().w4a16_prefill(
        _ptr(x), _ptr(w), _ptr(scale), _ptr(zero), _half_code(scale.dtype), group, _ptr(out), M, N, K,
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


# ----------------------------------------------------------------- the FP8 expert path

W4_SCORES = {"softmax": 0, "sigmoid": 1}
W4_ACTS = {"none": 0, "swiglu": 1}
_FLOAT_CODES = {torch.bfloat16: W4_BF16, torch.float16: W4_F16, torch.float32: W4_F32}


def _float_code(dt) -> int:
    if dt not in _FLOAT_CODES:
        raise TypeError(f"unsupported dtype {dt}: bf16, fp16 or fp32")
    return _FLOAT_CODES[dt]


def _arg(t, dtype, shape: tuple, what: str):
    """Pointer of a contiguous GPU tensor, its type and shape checked (None passes). One pass over the common case:
    these checks are most of a small call's host time. A tensor that is not on the GPU, or not contiguous, is returned
    itself, for _call to refuse once every type and shape has been looked at."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")
    return t.data_ptr() if t.is_cuda and t.is_contiguous() else t


def _new(shape, dtype, device, stream):
    """A tensor of the stream that will write it: memory of another stream could still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(fn: str, *args) -> None:
    try:
        rc = getattr(lib(), fn)(*args)
    except ctypes.ArgumentError:
        for v in args:
            if isinstance(v, torch.Tensor):
                _ptr(v)                                  # names what is wrong with it
        raise
    _check(fn, rc)


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _on_current_device(stream, first, *others) -> None:
    """A launch goes to the current device, whatever memory it is given: refuses tensors or a stream of another one. (One
    that is not on a GPU is refused for that.)"""
    here = first.get_device()
    if here < 0:
        return
    if here != _current_device():
        raise ValueError(f"a tensor is on cuda:{here}, the current device is cuda:{_current_device()}")
    if stream is not None and stream.device_index != here:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, the current device is cuda:{here}")
    for t in others:
        if t is not None and t.get_device() != here and t.is_cuda:
            raise ValueError(f"a tensor is on cuda:{t.get_device()}, the current device is cuda:{here}")


def _e4m3_codes(t, what: str):
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"{what} must hold E4M3 codes (torch.float8_e4m3fn or uint8), got {t.dtype}")
    return t


def _rows_ptr(t, what: str):
    """Pointer and row stride of a matrix whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if t.dim() != 2 or (t.numel() and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a matrix with contiguous rows")
    return t.data_ptr() or None, (t.stride(0) if t.numel() and t.shape[0] > 1 else t.shape[1])


def w4_route_workspace(T: int, E: int, topk: int, device="cuda", stream=None) -> torch.Tensor:
    """Device scratch for w4_route at these sizes (uint8, possibly empty), for use on `stream`."""
    n = ctypes.c_size_t(0)
    _check("w4_route_workspace_bytes", lib().w4_route_workspace_bytes(T, E, topk, ctypes.byref(n)))
    return _new((n.value,), torch.uint8, device, stream)


def w4_route(logits, topk: int, score: str = "softmax", bias=None, n_groups: int = 1, topk_groups: int = 1,
             group_top: int = 1, renorm: bool = True, scale: float = 1.0, out=None, workspace=None, stream=None):
    """logits [T, E] bf16/fp16/fp32 (rows may be strided) -> (ids int32 [T, topk], weights fp32 [T, topk],
    row_token int32 [T * topk], expert_offsets int32 [E + 1], row_of int32 [T, topk]); include/w4.h has the
    definition. `out` is such a tuple to write into; the workspace (w4_route_workspace) is allocated if not given."""
    T, E = logits.shape
    ptr, ld = _rows_ptr(logits, "logits")
    dev = logits.device
    if score not in W4_SCORES:
        raise ValueError(f"score must be one of {sorted(W4_SCORES)}, got {score!r}")
    if out is None:
        out = (_new((T, topk), torch.int32, dev, stream), _new((T, topk), torch.float32, dev, stream),
               _new((T * topk,), torch.int32, dev, stream), _new((E + 1,), torch.int32, dev, stream),
               _new((T, topk), torch.int32, dev, stream))
    ids, weights, row_token, offsets, row_of = out
    p_bias = _arg(bias, torch.float32, (E,), "bias")
    p_ids = _arg(ids, torch.int32, (T, topk), "ids")
    p_weights = _arg(weights, torch.float32, (T, topk), "weights")
    p_token = _arg(row_token, torch.int32, (T * topk,), "row_token")
    p_off = _arg(offsets, torch.int32, (E + 1,), "expert_offsets")
    p_row = _arg(row_of, torch.int32, (T, topk), "row_of")
    if workspace is None:
        workspace = w4_route_workspace(T, E, topk, dev, stream)
    _call("w4_route",
        ptr, _float_code(logits.dtype), T, E, ld, W4_SCORES[score], p_bias, n_groups, topk_groups, group_top, topk,
        int(renorm), scale, p_ids, p_weights, p_token, p_off, p_row, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    return out


def w4_fp8_block_quantize(x, act: str = "none", out=None, stream=None):
    """x [M, K] ([M, 2K] = gate | up with act="swiglu") bf16/fp16, rows may be strided -> (codes uint8 [M, K] of E4M3
    bits, scales fp32 [M, ceil(K / 128)])."""
    if act not in W4_ACTS:
        raise ValueError(f"act must be one of {sorted(W4_ACTS)}, got {act!r}")
    M, wide = x.shape
    if act == "swiglu" and wide % 2:
        raise ValueError(f"swiglu takes gate and up side by side: {wide} columns cannot be halved")
    K = wide // 2 if act == "swiglu" else wide
    ptr, ldx = _rows_ptr(x, "x")
    KB = (K + 127) // 128
    if out is None:
        out = (_new((M, K), torch.uint8, x.device, stream), _new((M, KB), torch.float32, x.device, stream))
    codes, scales = out
    p_codes = _arg(_e4m3_codes(codes, "codes"), codes.dtype, (M, K), "codes")
    _call("w4_fp8_block_quantize",
        ptr, _half_code(x.dtype), M, K, ldx, W4_ACTS[act], p_codes, _arg(scales, torch.float32, (M, KB), "scales"),
        _stream(stream))
    return out


def w4_fp8_block_gemm_workspace(M: int, N: int, K: int, device="cuda", stream=None) -> torch.Tensor:
    """Device scratch for w4_fp8_block_gemm at these sizes (uint8, possibly empty), for use on `stream`."""
    n = ctypes.c_size_t(0)
    _check("w4_fp8_block_gemm_workspace_bytes", lib().w4_fp8_block_gemm_workspace_bytes(M, N, K, ctypes.byref(n)))
    return _new((n.value,), torch.uint8, device, stream)


def w4_fp8_block_gemm(a, a_scale, w, w_scale, bias=None, out=None, out_dtype=torch.bfloat16, workspace=None,
                      stream=None):
    """a [M, K] and w [N, K] E4M3 codes with fp32 scales [M, ceil(K/128)] and [ceil(N/128), ceil(K/128)]
    -> out [M, N] bf16/fp16/fp32 (+ bias [N] of the same type)."""
    (M, K), (N, Kw) = _e4m3_codes(a, "a").shape, _e4m3_codes(w, "w").shape
    if K != Kw:
        raise ValueError(f"a has {K} columns, w {Kw}")
    KB, NB = (K + 127) // 128, (N + 127) // 128
    if out is None:
        out = _new((M, N), out_dtype, a.device, stream)
    p_as = _arg(a_scale, torch.float32, (M, KB), "a_scale")
    p_ws = _arg(w_scale, torch.float32, (NB, KB), "w_scale")
    p_bias = _arg(bias, out.dtype, (N,), "bias")
    p_out = _arg(out, out.dtype, (M, N), "out")
    if workspace is None:
        workspace = w4_fp8_block_gemm_workspace(M, N, K, a.device, stream)
    _call("w4_fp8_block_gemm",
        _ptr(a), p_as, _ptr(w), p_ws, p_bias, p_out, _float_code(out.dtype), M, N, K, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    return out


def w4_fp8_block_grouped_gemm(a, a_scale, row_token, expert_offsets, w, w_scale, out=None, out_dtype=torch.bfloat16,
                              stream=None):
    """The block-scaled product over expert segments: w [E, N, K], w_scale [E, ceil(N/128), ceil(K/128)]; output row r
    of expert e (expert_offsets) takes activation row row_token[r], or row r itself with row_token None. -> out [R, N]
    bf16/fp16; rows past expert_offsets[E] are not written."""
    (T, K), (E, N, Kw) = _e4m3_codes(a, "a").shape, _e4m3_codes(w, "w").shape
    if K != Kw:
        raise ValueError(f"a has {K} columns, w {Kw}")
    KB, NB = (K + 127) // 128, (N + 127) // 128
    R = T if row_token is None else row_token.shape[0]
    if out is None:
        out = _new((R, N), out_dtype, a.device, stream)
    p_as = _arg(a_scale, torch.float32, (T, KB), "a_scale")
    p_token = _arg(row_token, torch.int32, (R,), "row_token")
    p_off = _arg(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    p_ws = _arg(w_scale, torch.float32, (E, NB, KB), "w_scale")
    p_out = _arg(out, out.dtype, (R, N), "out")
    _call("w4_fp8_block_grouped_gemm",
        _ptr(a), p_as, p_token, p_off, E, _ptr(w), p_ws, p_out, _half_code(out.dtype), T, R, N, K, _stream(stream))
    return out


def w4_combine(y, row_of, weights, add=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * y[row_of[t, j]] (+ add[t]): y [R, N] bf16/fp16/fp32, row_of int32 and weights fp32
    [T, topk] from w4_route."""
    R, N = y.shape
    T, topk = row_of.shape
    if out is None:
        out = _new((T, N), y.dtype, y.device, stream)
    _call("w4_combine",
        _ptr(y), _float_code(y.dtype), _arg(row_of, torch.int32, (T, topk), "row_of"),
        _arg(weights, torch.float32, (T, topk), "weights"), _arg(add, y.dtype, (T, N), "add"),
        _arg(out, y.dtype, (T, N), "out"), T, R, topk, N, _stream(stream))
    return out


# ----------------------------------------------------------------- MXFP4

def _mx_row(K: int) -> int:
    """Scale bytes of a row: one per 32 columns, padded to whole blocks of 128."""
    return 4 * ((K + 127) // 128)


def w4_mxfp4_quantize(x, act: str = "none", out=None, stream=None):
    """x [M, K] ([M, 2K] = gate | up with act="swiglu") bf16/fp16/fp32, rows may be strided -> (codes uint8 [M, K / 2] of
    E2M1 pairs, scales uint8 [M, 4 * ceil(K / 128)] of E8M0 bits, one per 32 columns, then padding)."""
    if act not in W4_ACTS:
        raise ValueError(f"act must be one of {sorted(W4_ACTS)}, got {act!r}")
    M, wide = x.shape
    if act == "swiglu" and wide % 2:
        raise ValueError(f"swiglu takes gate and up side by side: {wide} columns cannot be halved")
    K = wide // 2 if act == "swiglu" else wide
    ptr, ldx = _rows_ptr(x, "x")
    if out is None:
        out = (_new((M, K // 2), torch.uint8, x.device, stream), _new((M, _mx_row(K)), torch.uint8, x.device, stream))
    codes, scales = out
    _on_current_device(stream, x, codes, scales)
    _call("w4_mxfp4_quantize",
        ptr, _float_code(x.dtype), M, K, ldx, W4_ACTS[act], _arg(codes, torch.uint8, (M, K // 2), "codes"),
        _arg(scales, torch.uint8, (M, _mx_row(K)), "scales"), _stream(stream))
    return out


def w4_mxfp4_dequantize(codes, scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """codes uint8 [M, K / 2] and scales uint8 [M, 4 * ceil(K / 128)] -> the values they stand for, [M, K]
    bf16/fp16/fp32."""
    M, K = codes.shape[0], 2 * codes.shape[1]
    if out is None:
        out = _new((M, K), out_dtype, codes.device, stream)
    _on_current_device(stream, codes, scales, out)
    _call("w4_mxfp4_dequantize",
        _arg(codes, torch.uint8, (M, K // 2), "codes"), _arg(scales, torch.uint8, (M, _mx_row(K)), "scales"), M, K,
        _arg(out, out.dtype, (M, K), "out"), _float_code(out.dtype), _stream(stream))
    return out


def w4_mxfp4_gemm_workspace(M: int, N: int, K: int, device="cuda", stream=None) -> torch.Tensor:
    """Device scratch for w4_mxfp4_gemm at these sizes (uint8, possibly empty), for use on `stream`."""
    n = ctypes.c_size_t(0)
    _check("w4_mxfp4_gemm_workspace_bytes", lib().w4_mxfp4_gemm_workspace_bytes(M, N, K, ctypes.byref(n)))
    return _new((n.value,), torch.uint8, device, stream)


def w4_mxfp4_gemm(a, a_scale, w, w_scale, bias=None, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """a [M, K] and w [N, K] as MXFP4 codes (uint8 [., K / 2]) and scales (uint8 [., 4 * ceil(K / 128)]) -> out [M, N]
    bf16/fp16/fp32 (+ bias [N] of the same type)."""
    (M, KH), (N, Kw) = a.shape, w.shape
    if KH != Kw:
        raise ValueError(f"a has {2 * KH} columns, w {2 * Kw}")
    K, KS = 2 * KH, _mx_row(2 * KH)
    if out is None:
        out = _new((M, N), out_dtype, a.device, stream)
    p_a, p_as = _arg(a, torch.uint8, (M, KH), "a"), _arg(a_scale, torch.uint8, (M, KS), "a_scale")
    p_w, p_ws = _arg(w, torch.uint8, (N, KH), "w"), _arg(w_scale, torch.uint8, (N, KS), "w_scale")
    p_bias = _arg(bias, out.dtype, (N,), "bias")
    p_out = _arg(out, out.dtype, (M, N), "out")
    if workspace is None:
        workspace = w4_mxfp4_gemm_workspace(M, N, K, a.device, stream)
    _on_current_device(stream, a, a_scale, w, w_scale, bias, out, workspace)
    _call("w4_mxfp4_gemm",
        p_a, p_as, p_w, p_ws, p_bias, p_out, _float_code(out.dtype), M, N, K, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    return out


def w4_mxfp4_linear_workspace(M: int, N: int, K: int, device="cuda", stream=None) -> torch.Tensor:
    """Device scratch for w4_mxfp4_linear at these sizes (uint8, possibly empty), for use on `stream`."""
    n = ctypes.c_size_t(0)
    _check("w4_mxfp4_linear_workspace_bytes", lib().w4_mxfp4_linear_workspace_bytes(M, N, K, ctypes.byref(n)))
    return _new((n.value,), torch.uint8, device, stream)


def w4_mxfp4_linear(x, w, w_scale, bias=None, out=None, workspace=None, stream=None):
    """x [M, K] bf16/fp16, quantized to MXFP4 on the way, times w [N, K] in MXFP4 (codes uint8 [N, K / 2], scales uint8
    [N, 4 * ceil(K / 128)]) -> out [M, N] in x's type (+ bias [N])."""
    (M, K), (N, KH) = x.shape, w.shape
    if K != 2 * KH:
        raise ValueError(f"x has {K} columns, w {2 * KH}")
    if out is None:
        out = _new((M, N), x.dtype, x.device, stream)
    p_x = _arg(x, x.dtype, (M, K), "x")
    p_w, p_ws = _arg(w, torch.uint8, (N, KH), "w"), _arg(w_scale, torch.uint8, (N, _mx_row(K)), "w_scale")
    p_bias = _arg(bias, x.dtype, (N,), "bias")
    p_out = _arg(out, x.dtype, (M, N), "out")
    if workspace is None:
        workspace = w4_mxfp4_linear_workspace(M, N, K, x.device, stream)
    _on_current_device(stream, x, w, w_scale, bias, out, workspace)
    _call("w4_mxfp4_linear",
        p_x, _half_code(x.dtype), p_w, p_ws, p_bias, p_out, M, N, K, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    return out


def w4_mxfp4_grouped_gemm(a, a_scale, row_token, expert_offsets, w, w_scale, out=None, out_dtype=torch.bfloat16,
                          stream=None):
    """The MXFP4 product over expert segments: w [E, N, K / 2], w_scale [E, N, 4 * ceil(K / 128)]; output row r of expert
    e (expert_offsets) takes activation row row_token[r], or row r itself with row_token None. -> out [R, N] bf16/fp16;
    rows past expert_offsets[E] are not written."""
    (T, KH), (E, N, Kw) = a.shape, w.shape
    if KH != Kw:
        raise ValueError(f"a has {2 * KH} columns, w {2 * Kw}")
    K, KS = 2 * KH, _mx_row(2 * KH)
    R = T if row_token is None else row_token.shape[0]
    if out is None:
        out = _new((R, N), out_dtype, a.device, stream)
    p_a, p_as = _arg(a, torch.uint8, (T, KH), "a"), _arg(a_scale, torch.uint8, (T, KS), "a_scale")
    p_token = _arg(row_token, torch.int32, (R,), "row_token")
    p_off = _arg(expert_offsets, torch.int32, (E + 1,), "expert_offsets")
    p_w, p_ws = _arg(w, torch.uint8, (E, N, KH), "w"), _arg(w_scale, torch.uint8, (E, N, KS), "w_scale")
    p_out = _arg(out, out.dtype, (R, N), "out")
    _on_current_device(stream, a, a_scale, row_token, expert_offsets, w, w_scale, out)
    _call("w4_mxfp4_grouped_gemm",
        p_a, p_as, p_token, p_off, E, p_w, p_ws, p_out, _half_code(out.dtype), T, R, N, K, _stream(stream))
    return out


# ----------------------------------------------------------------- the whole layer for a few tokens

W4_MOE_DECODE_MAX_TOKENS = 32            # include/w4.h
W4_MOE_FORMATS = {"fp8_block": 1, "mxfp4": 2, "int4": 3}


def w4_moe_decode_workspace(T: int, E: int, topk: int, H: int, I: int, device="cuda", stream=None) -> torch.Tensor:
    """Device scratch for w4_moe_decode at these sizes (uint8, possibly empty), for use on `stream`."""
    n = ctypes.c_size_t(0)
    _check("w4_moe_decode_workspace_bytes", lib().w4_moe_decode_workspace_bytes(T, E, topk, H, I, ctypes.byref(n)))
    return _new((n.value,), torch.uint8, device, stream)


def w4_moe_decode(x, logits, topk: int, w13, w13_scale, w2, w2_scale, fmt: str = "fp8_block", score: str = "softmax",
                  bias=None, n_groups: int = 1, topk_groups: int = 1, group_top: int = 1, renorm: bool = True,
                  scale: float = 1.0, add=None, out=None, workspace=None, stream=None):
    """The expert layer of at most W4_MOE_DECODE_MAX_TOKENS tokens: x [T, H] bf16/fp16 and logits [T, E] -> [T, H]
    (+ add [T, H]); include/w4.h has the definition, w4_route the routing arguments. Weights by `fmt`:
    "fp8_block": w13 [E, 2I, H] and w2 [E, H, I] E4M3 codes, scales fp32 [E, ceil(2I/128), ceil(H/128)] and
    [E, ceil(H/128), ceil(I/128)];
    "mxfp4": w13 uint8 [E, 2I, H/2], w2 uint8 [E, H, I/2], scales uint8 [E, 2I, 4 ceil(H/128)], [E, H, 4 ceil(I/128)];
    "int4": w13 and w2 from w4_repack (batch = E), scales fp16 [E, G, 2I] and [E, G, H] with G = H / group and I / group
    (one group of 128 m for both), or 1 and 1 per channel."""
    if fmt not in W4_MOE_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(W4_MOE_FORMATS)}, got {fmt!r}")
    if score not in W4_SCORES:
        raise ValueError(f"score must be one of {sorted(W4_SCORES)}, got {score!r}")
    (T, H), E = x.shape, logits.shape[1]
    ptr, ld = _rows_ptr(logits, "logits")
    group = -1
    if fmt == "int4":
        I = w13_scale.shape[2] // 2
        G13, G2 = w13_scale.shape[1], w2_scale.shape[1]
        if (G13, G2) != (1, 1):
            group = H // G13 if G13 else 0
            if group <= 0 or G13 * group != H or G2 * group != I:
                raise ValueError(f"w13_scale and w2_scale must share a group along H={H} and I={I}: got {G13} and {G2} groups")
        p_w13 = _arg(w13, torch.uint8, (E, w4_repack_bytes(H, 2 * I)), "w13")
        p_w2 = _arg(w2, torch.uint8, (E, w4_repack_bytes(I, H)), "w2")
        p_s13 = _arg(w13_scale, torch.float16, (E, G13, 2 * I), "w13_scale")
        p_s2 = _arg(w2_scale, torch.float16, (E, G2, H), "w2_scale")
    elif fmt == "mxfp4":
        I = 2 * w2.shape[2]
        p_w13 = _arg(w13, torch.uint8, (E, 2 * I, H // 2), "w13")
        p_w2 = _arg(w2, torch.uint8, (E, H, I // 2), "w2")
        p_s13 = _arg(w13_scale, torch.uint8, (E, 2 * I, _mx_row(H)), "w13_scale")
        p_s2 = _arg(w2_scale, torch.uint8, (E, H, _mx_row(I)), "w2_scale")
    else:
        I = w2.shape[2]
        HB, IB = (H + 127) // 128, (I + 127) // 128
        p_w13 = _arg(_e4m3_codes(w13, "w13"), w13.dtype, (E, 2 * I, H), "w13")
        p_w2 = _arg(_e4m3_codes(w2, "w2"), w2.dtype, (E, H, I), "w2")
        p_s13 = _arg(w13_scale, torch.float32, (E, (2 * I + 127) // 128, HB), "w13_scale")
        p_s2 = _arg(w2_scale, torch.float32, (E, HB, IB), "w2_scale")
    if logits.shape[0] != T:
        raise ValueError(f"logits have {logits.shape[0]} rows, x {T}")
    if out is None:
        out = _new((T, H), x.dtype, x.device, stream)
    p_bias = _arg(bias, torch.float32, (E,), "bias")
    p_add, p_out = _arg(add, x.dtype, (T, H), "add"), _arg(out, x.dtype, (T, H), "out")
    if workspace is None:
        workspace = w4_moe_decode_workspace(T, E, topk, H, I, x.device, stream)
    _on_current_device(stream, x, logits, w13, w13_scale, w2, w2_scale, bias, add, out, workspace)
    _call("w4_moe_decode",
        _arg(x, x.dtype, (T, H), "x"), _half_code(x.dtype), ptr, _float_code(logits.dtype), ld, W4_SCORES[score], p_bias,
        n_groups, topk_groups, group_top, topk, int(renorm), scale, W4_MOE_FORMATS[fmt], p_w13, p_s13, p_w2, p_s2, group,
        p_add, p_out, T, E, H, I, _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    return out
