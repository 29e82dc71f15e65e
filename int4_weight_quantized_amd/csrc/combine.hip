// Combine: the experts' rows of each token, weighted and summed.
//
//   out[t, n] = sum_j weights[t, j] * y[row_of[t, j], n]  (+ add[t, n])
//
// in fp32, j ascending, rounded once to the output type; slots whose row is
// outside [0, R) (a token without that expert) add nothing. The sum gathers
// by the router's inverse map (row_of), so no atomics are needed and its
// order is fixed.
//
// HBM-bound: every routed row is read once (topk * N elements a token) and
// the token's row written once. Nothing is read twice, so loads and stores
// pass the caches by: 8192 tokens x 8 rows x 7168 bf16 in 196 us (5.4 TB/s; 214
// with ordinary ones).
#include "w4_device.h"

namespace w4 {

constexpr int kCThreads = 256;

template <int DT>   // 0 bf16, 1 fp16, 2 fp32
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&f)[8]) {
  if constexpr (DT == 2) {
    const v4f a = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i));
    const v4f b = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i + 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  } else {
    const v4i raw = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(static_cast<const uint16_t*>(p) + i));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = (uint32_t)raw[e];
      f[2 * e] = DT == 0 ? __uint_as_float(w << 16) : f16_to_f32((uint16_t)w);
      f[2 * e + 1] = DT == 0 ? __uint_as_float(w & 0xFFFF0000u) : f16_to_f32((uint16_t)(w >> 16));
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  if constexpr (DT == 2) {
    float* o = static_cast<float*>(p) + i;
    __builtin_nontemporal_store(v4f{f[0], f[1], f[2], f[3]}, reinterpret_cast<v4f*>(o));
    __builtin_nontemporal_store(v4f{f[4], f[5], f[6], f[7]}, reinterpret_cast<v4f*>(o + 4));
  } else {
    v4i w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = DT == 0 ? f32_to_bf16_rne(f[2 * e]) : f32_to_f16_rne(f[2 * e]);
      const uint32_t hi = DT == 0 ? f32_to_bf16_rne(f[2 * e + 1]) : f32_to_f16_rne(f[2 * e + 1]);
      w[e] = (int)(lo | (hi << 16));
    }
    __builtin_nontemporal_store(w, reinterpret_cast<v4i*>(static_cast<uint16_t*>(p) + i));
  }
}

// One thread per 8 columns of a token; chunk c of the T * N/8 belongs to
// token c / (N/8), a 32-bit division. (Loading the rows of 4 slots ahead of
// their use was 12% slower.)
template <int DT>
__global__ __launch_bounds__(kCThreads) void combine_kernel(const void* __restrict__ y,
                                                            const int32_t* __restrict__ row_of,
                                                            const float* __restrict__ weights,
                                                            const void* add, void* out,
                                                            uint32_t T, int R, int topk, int N) {
  const uint32_t nc = (uint32_t)N >> 3;
  const uint32_t c = blockIdx.x * kCThreads + threadIdx.x;
  const uint32_t t = c / nc;
  if (t >= T) return;
  const int64_t n = (int64_t)(c - t * nc) * 8;
  const int32_t* rows = row_of + (int64_t)t * topk;
  const float* ws = weights + (int64_t)t * topk;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < topk; ++j) {
    const int r = rows[j];
    if ((unsigned)r >= (unsigned)R) continue;
    const float w = ws[j];
    float f[8];
    load8<DT>(y, (int64_t)r * N + n, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = fmaf(w, f[e], s[e]);
  }
  if (add) {
    float f[8];
    load8<DT>(add, (int64_t)t * N + n, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += f[e];
  }
  store8<DT>(out, (int64_t)t * N + n, s);
}

hipError_t launch_combine(const void* y, int dt, const int32_t* row_of, const float* weights, const void* add,
                          void* out, int64_t T, int64_t R, int64_t topk, int64_t N, hipStream_t stream) {
  if (T == 0 || N == 0) return hipSuccess;
  // a launch takes fewer than 2^32 threads: past 2^31 chunks, token ranges in turn
  const int64_t per = (((int64_t)1 << 31) - 1) / (N / 8), size = dt == 2 ? 4 : 2;
  for (int64_t t0 = 0; t0 < T; t0 += per) {
    const int64_t n = T - t0 < per ? T - t0 : per;
    const dim3 grid((unsigned)((n * (N / 8) + kCThreads - 1) / kCThreads)), block(kCThreads);
    const int64_t at = t0 * N * size;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, stream, y, row_of + t0 * topk, weights + t0 * topk,
                         add ? static_cast<const char*>(add) + at : nullptr, static_cast<char*>(out) + at, (uint32_t)n,
                         (int)R, (int)topk, (int)N);
    };
    if (dt == 0) go(combine_kernel<0>);
    else if (dt == 1) go(combine_kernel<1>);
    else go(combine_kernel<2>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace w4
