// MXFP4 quantization and its inverse.
//
// Per block of 32 columns: scale = 2^(floor(log2 max |v|) - 2), at least
// 2^-127; code = E2M1(v / scale), nearest even, saturating at 6. The quotient
// is exact (a power of two), so the one rounding is the conversion's own.
// v = x, or silu(gate) * up in fp32. A block that holds a NaN or an infinity
// has the scale NaN and codes 0.
//
// Both are bound by memory: n (size + 17/32) bytes and as many back (8192 x
// 14336 from fp16: 64 us, 4.7 TB/s, where a copy reaches 4.8). 16 lanes
// take one row's 128 columns, 8 columns each (16-byte loads of 16-bit values,
// side by side); 4 lanes share a block's maximum (DPP), and the first of the 16
// writes the four scale bytes as one word, the padding of a row's end among them.
#include "mxfp4.h"

namespace w4 {

constexpr int kMxThreads = 256;
constexpr int kMxUnits = kMxThreads / 16;            // 128-column units per block

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}

// 8 values at p as fp32. DT: 0 bf16, 1 fp16, 2 fp32.
template <int DT>
__device__ __forceinline__ void load8(const void* x, int64_t at, float (&v)[8]) {
  if constexpr (DT == 2) {
    const v4f a = *reinterpret_cast<const v4f*>(static_cast<const float*>(x) + at);
    const v4f b = *reinterpret_cast<const v4f*>(static_cast<const float*>(x) + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const v4i r = *reinterpret_cast<const v4i*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t h = (uint16_t)((uint32_t)r[i / 2] >> (16 * (i % 2)));
      v[i] = DT == 0 ? bf16_to_f32(h) : f16_to_f32(h);
    }
  }
}

template <int DT, bool SWIGLU>
__global__ __launch_bounds__(kMxThreads) void mx_quant_kernel(const void* __restrict__ x, int64_t ldx, int K,
                                                              uint32_t KB, uint32_t units,
                                                              uint8_t* __restrict__ codes,
                                                              uint32_t* __restrict__ scales) {
  const uint32_t u = blockIdx.x * kMxUnits + (threadIdx.x >> 4);
  if (u >= units) return;                            // whole groups of 16 lanes leave
  const int64_t m = u / KB;
  const int k = (int)(u % KB) * 128 + (threadIdx.x & 15) * 8;
  const bool in = k < K;                             // K is a multiple of 32: whole blocks of 4 lanes
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (in) {
    load8<DT>(x, m * ldx + k, v);
    if constexpr (SWIGLU) {
      float g[8];
      load8<DT>(x, m * ldx + K + k, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * g[i];
    }
  }
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  amax = max(amax, dpp_u<0xB1>(amax));               // lane ^ 1
  amax = max(amax, dpp_u<0x4E>(amax));               // lane ^ 2
  const uint32_t sc = mx_scale_code(amax);
  uint32_t c = 0;
  if (sc != kMxNan) {
    const float s = mx_scale_value(sc);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  }
  // the four blocks' scale bytes in the first lane: from lanes 4, 8 and 12
  uint32_t w = sc | dpp_u<0x104>(sc) << 8;           // row_shl 4
  w |= dpp_u<0x108>(w) << 16;                        // row_shl 8
  if (in) *reinterpret_cast<uint32_t*>(codes + m * (K >> 1) + (k >> 1)) = c;
  if ((threadIdx.x & 15) == 0) scales[u] = w;
}

// 8 columns per thread, side by side, so that a wave's stores are whole lines (8192 x 14336 to bf16: 59 us, 5.1 TB/s; 32
// columns per thread took 78, and several turns of 8 per thread gain nothing). DT as above, of the output.
template <int DT>
__global__ __launch_bounds__(kMxThreads) void mx_dequant_kernel(const uint32_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, uint32_t K8, int KS,
                                                                uint32_t units, void* __restrict__ out) {
  const uint32_t u = blockIdx.x * kMxThreads + threadIdx.x;
  if (u >= units) return;
  const uint32_t m = u / K8, c = codes[u], sc = scales[(int64_t)m * KS + (u - m * K8) / 4];
  typedef float v2f __attribute__((ext_vector_type(2)));
  const float s = mx_scale_value(sc);
  const v2f p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3)};
  float f[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] = sc == kMxNan ? __uint_as_float(0x7FC00000u) : p[q / 2][q % 2];
  if constexpr (DT == 2) {
    float* o = static_cast<float*>(out) + (int64_t)u * 8;
    *reinterpret_cast<v4f*>(o) = v4f{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<v4f*>(o + 4) = v4f{f[4], f[5], f[6], f[7]};
  } else {
    v4i r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t lo = DT == 0 ? f32_to_bf16_rne(f[2 * q]) : f32_to_f16_rne(f[2 * q]);
      const uint32_t hi = DT == 0 ? f32_to_bf16_rne(f[2 * q + 1]) : f32_to_f16_rne(f[2 * q + 1]);
      r[q] = (int)(lo | hi << 16);
    }
    *reinterpret_cast<v4i*>(static_cast<uint16_t*>(out) + (int64_t)u * 8) = r;
  }
}

hipError_t launch_mx_quant(const void* x, int dt, bool swiglu, int64_t M, int64_t K, int64_t ldx, void* codes,
                           void* scales, hipStream_t stream) {
  if (M == 0 || K == 0) return hipSuccess;
  // a launch takes fewer than 2^32 threads: row ranges in turn past 2^28 units of 16 lanes
  const int64_t KB = (K + 127) / 128, per = (((int64_t)1 << 28) - kMxUnits) / KB;
  const int64_t size = dt == 2 ? 4 : 2;
  for (int64_t m0 = 0; m0 < M; m0 += per) {
    const int64_t units = (M - m0 < per ? M - m0 : per) * KB;
    const dim3 grid((unsigned)((units + kMxUnits - 1) / kMxUnits)), block(kMxThreads);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, stream, static_cast<const uint8_t*>(x) + m0 * ldx * size, ldx, (int)K,
                         (uint32_t)KB, (uint32_t)units, static_cast<uint8_t*>(codes) + m0 * (K / 2),
                         static_cast<uint32_t*>(scales) + m0 * KB);
    };
    if (dt == 0) swiglu ? go(mx_quant_kernel<0, true>) : go(mx_quant_kernel<0, false>);
    else if (dt == 1) swiglu ? go(mx_quant_kernel<1, true>) : go(mx_quant_kernel<1, false>);
    else swiglu ? go(mx_quant_kernel<2, true>) : go(mx_quant_kernel<2, false>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_dequant(const void* codes, const void* scales, int64_t M, int64_t K, void* out, int dt,
                             hipStream_t stream) {
  if (M == 0 || K == 0) return hipSuccess;
  const int64_t K8 = K / 8, per = (((int64_t)1 << 32) - 2 * kMxThreads) / K8, KS = mx_scale_bytes(K);
  const int64_t size = dt == 2 ? 4 : 2;
  for (int64_t m0 = 0; m0 < M; m0 += per) {
    const int64_t units = (M - m0 < per ? M - m0 : per) * K8;
    const dim3 grid((unsigned)((units + kMxThreads - 1) / kMxThreads)), block(kMxThreads);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, stream, static_cast<const uint32_t*>(codes) + m0 * K8,
                         static_cast<const uint8_t*>(scales) + m0 * KS, (uint32_t)K8, (int)KS, (uint32_t)units,
                         static_cast<void*>(static_cast<uint8_t*>(out) + m0 * K * size));
    };
    if (dt == 0) go(mx_dequant_kernel<0>);
    else if (dt == 1) go(mx_dequant_kernel<1>);
    else go(mx_dequant_kernel<2>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace w4
