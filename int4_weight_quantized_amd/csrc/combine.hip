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
// the token's row written once.
#include "w4_device.h"

namespace w4 {

constexpr int kCThreads = 256;

template <int DT>   // 0 bf16, 1 fp16, 2 fp32
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&f)[8]) {
  if constexpr (DT == 2) {
    const v4f a = *reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i);
    const v4f b = *reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  } else {
    const v4i raw = *reinterpret_cast<const v4i*>(static_cast<const uint16_t*>(p) + i);
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
    *reinterpret_cast<v4f*>(o) = v4f{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<v4f*>(o + 4) = v4f{f[4], f[5], f[6], f[7]};
  } else {
    v4i w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = DT == 0 ? f32_to_bf16_rne(f[2 * e]) : f32_to_f16_rne(f[2 * e]);
      const uint32_t hi = DT == 0 ? f32_to_bf16_rne(f[2 * e + 1]) : f32_to_f16_rne(f[2 * e + 1]);
      w[e] = (int)(lo | (hi << 16));
    }
    *reinterpret_cast<v4i*>(static_cast<uint16_t*>(p) + i) = w;
  }
}

// One thread per 8 columns of a token; chunk c of the T * N/8 belongs to
// token c / (N/8).
template <int DT>
__global__ __launch_bounds__(kCThreads) void combine_kernel(const void* __restrict__ y,
                                                            const int32_t* __restrict__ row_of,
                                                            const float* __restrict__ weights,
                                                            const void* add, void* out,
                                                            int64_t T, int R, int topk, int N) {
  const int nc = N >> 3;
  const int64_t c = (int64_t)blockIdx.x * kCThreads + threadIdx.x;
  const int64_t t = c / nc;
  if (t >= T) return;
  const int64_t n = (c - t * nc) * 8;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < topk; ++j) {
    const int r = row_of[t * topk + j];
    if ((unsigned)r >= (unsigned)R) continue;
    const float w = weights[t * topk + j];
    float f[8];
    load8<DT>(y, (int64_t)r * N + n, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = fmaf(w, f[e], s[e]);
  }
  if (add) {
    float f[8];
    load8<DT>(add, t * N + n, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] += f[e];
  }
  store8<DT>(out, t * N + n, s);
}

hipError_t launch_combine(const void* y, int dt, const int32_t* row_of, const float* weights, const void* add,
                          void* out, int64_t T, int64_t R, int64_t topk, int64_t N, hipStream_t stream) {
  if (T == 0 || N == 0) return hipSuccess;
  const int64_t chunks = T * (N / 8);
  const dim3 grid((unsigned)((chunks + kCThreads - 1) / kCThreads)), block(kCThreads);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, y, row_of, weights, add, out, T, (int)R, (int)topk, (int)N);
  };
  if (dt == 0) go(combine_kernel<0>);
  else if (dt == 1) go(combine_kernel<1>);
  else go(combine_kernel<2>);
  return hipGetLastError();
}

}  // namespace w4
