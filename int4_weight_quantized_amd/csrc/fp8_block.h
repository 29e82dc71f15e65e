// Shared by the block-scaled FP8 products (fp8_block_gemm.hip: tiles through
// LDS; fp8_block_stream.hip: few rows, weights streamed into registers) and,
// where P is a type parameter, by the MXFP4 products.
#pragma once

#include "w4_device.h"

namespace w4 {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kFK = 128;                             // K step: one scale block
constexpr uint32_t kPast = 0x80000000u;              // buffer offset past any buffer: reads as zero

struct Fp8Args {
  const uint8_t* a;
  const float* a_scale;
  const int32_t* row_token;                          // grouped: null = rows in segment order
  const int32_t* offsets;                            // grouped: [E + 1]
  const uint8_t* w;
  const float* w_scale;
  const void* bias;                                  // dense
  void* out;                                         // splits > 1: fp32 [splits][M][N]
  int64_t M;                                         // dense rows, or activation rows (T) of the grouped form
  int64_t R;                                         // output rows
  int E, N, K, KB, NT, NBLK, splits;                 // KB, NBLK: 128-blocks of K and N
  int64_t tiles;                                     // dense: row tiles * NT
};

// 8 E4M3 bytes (words w, w + 1 of a fragment) as fp16
__device__ __forceinline__ v8h e4m3_to_f16(const v8i& f, int w) {
  v8h h;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const v2h lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[w + q], 1.0f, false);
    const v2h hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[w + q], 1.0f, true);
    h[4 * q] = lo[0];
    h[4 * q + 1] = lo[1];
    h[4 * q + 2] = hi[0];
    h[4 * q + 3] = hi[1];
  }
  return h;
}

// One scale block: 16 weight rows x 16 activation rows x 128, the weights as
// the A operand: lane l holds activation row l % 16, weight rows 4 (l / 16) ..
// + 3. F16: the operands as fp16 (exact), whose sums the matrix unit keeps in
// fp32; else as E4M3, twice as fast, each 8 products added on a grid of 2^-13
// of the largest one's power of two.
template <bool F16>
__device__ __forceinline__ v4f block_product(const v8i& w, const v8i& a) {
  const v4f z = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (F16) {
    v4f d = z;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      d = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3_to_f16(w, 2 * c), e4m3_to_f16(a, 2 * c), d, 0, 0, 0);
    return d;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, 0, 0, 0);
  }
}

// Work item of a grouped block: expert, row tile inside its segment, column
// tile; the segment's first row and its length. e < 0: an idle block (the
// grid is an upper bound). Block ids go to the 8 XCDs in turn: XCD x takes
// the x-th eighth of the items, column tile fastest, so that its blocks share
// gathered rows and an expert's weights.
struct Segment {
  int e, mt, tn, left;                               // left: items behind it in the XCD's eighth
  int64_t row0, rows;
};

template <int BM, typename P>
__device__ __forceinline__ Segment find_segment(const P& p) {
  const int lane = threadIdx.x & 63;
  Segment s;
  s.e = -1;
  int total = 0;
  for (int c = 0; c < p.E; c += 64) {
    int mt = 0;
    if (c + lane < p.E) mt = (p.offsets[c + lane + 1] - p.offsets[c + lane] + BM - 1) / BM;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) mt += __shfl_xor(mt, off, kWave);
    total += mt;
  }
  total = __builtin_amdgcn_readfirstlane(total) * p.NT;
  const int per = (total + 7) / 8, xi = (int)(blockIdx.x / 8);
  const int t = (int)(blockIdx.x % 8) * per + xi;
  if (xi >= per || t >= total) return s;
  const int want = t / p.NT;                         // row tile, over all experts
  s.tn = t - want * p.NT;
  s.left = min(per - xi, total - t) - 1;
  int cum = 0;
  for (int c = 0; c < p.E && s.e < 0; c += 64) {     // 64 experts per round, one per lane
    int o0 = 0, o1 = 0;
    if (c + lane < p.E) {
      o0 = p.offsets[c + lane];
      o1 = p.offsets[c + lane + 1];
    }
    const int n = (o1 - o0 + BM - 1) / BM;
    int inc = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(inc, off, kWave);
      if (lane >= off) inc += o;
    }
    const unsigned long long hit = __ballot(want < cum + inc);
    if (hit) {
      const int src = __ffsll(hit) - 1;
      s.e = __builtin_amdgcn_readfirstlane(c + src);
      s.mt = __builtin_amdgcn_readfirstlane(want - cum - (__shfl(inc, src, kWave) - __shfl(n, src, kWave)));
      s.row0 = __builtin_amdgcn_readfirstlane(__shfl(o0, src, kWave));
      s.rows = __builtin_amdgcn_readfirstlane(__shfl(o1, src, kWave)) - s.row0;
      if (s.row0 + s.rows > p.R) s.rows = p.R - s.row0;   // offsets past the output rows
    }
    cum += __shfl(inc, 63, kWave);
  }
  return s;
}

// Store C (4 or 8) consecutive columns of a row, with the bias added first.
template <int OUT, int C, typename P>
__device__ __forceinline__ void store_columns(const P& p, float (&f)[C], int64_t orow, int n, bool bias) {
  if (bias) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      f[c] += OUT == 2 ? static_cast<const float*>(p.bias)[n + c]
                       : (OUT == 0 ? bf16_to_f32(static_cast<const uint16_t*>(p.bias)[n + c])
                                   : f16_to_f32(static_cast<const uint16_t*>(p.bias)[n + c]));
  }
  if constexpr (OUT == 2) {
    float* o = static_cast<float*>(p.out) + orow + n;
#pragma unroll
    for (int c = 0; c < C; c += 4) *reinterpret_cast<v4f*>(o + c) = v4f{f[c], f[c + 1], f[c + 2], f[c + 3]};
  } else {
    uint32_t w[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c) {
      const uint32_t lo = OUT == 0 ? f32_to_bf16_rne(f[2 * c]) : f32_to_f16_rne(f[2 * c]);
      const uint32_t hi = OUT == 0 ? f32_to_bf16_rne(f[2 * c + 1]) : f32_to_f16_rne(f[2 * c + 1]);
      w[c] = lo | (hi << 16);
    }
    uint16_t* o = static_cast<uint16_t*>(p.out) + orow + n;
    if constexpr (C == 8)
      *reinterpret_cast<v4i*>(o) = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    else
      *reinterpret_cast<v2i*>(o) = v2i{(int)w[0], (int)w[1]};
  }
}

// Split K: the partial sums [splits][rows][N], in order, to the output.
template <int OUT, typename P>
__global__ __launch_bounds__(256) void split_reduce_kernel(P p, const float* __restrict__ part) {
  const int nc = p.N >> 3;
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.M * nc) return;
  const int64_t span = p.M * p.N;
  const float* q = part + c * 8;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, q += span) {
    const v4f x = *reinterpret_cast<const v4f*>(q), y = *reinterpret_cast<const v4f*>(q + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] += x[e];
      f[4 + e] += y[e];
    }
  }
  store_columns<OUT, 8>(p, f, c / nc * p.N, (int)(c % nc) * 8, p.bias != nullptr);
}

// Blocks of a grouped launch with BM x BN tiles.
int64_t grouped_blocks(int64_t E, int64_t R, int64_t N, int64_t BM, int64_t BN);

hipError_t launch_fp8_stream(const Fp8Args& p, int out_dt, hipStream_t stream);
// Threads that it takes: dense (E = 0) or grouped.
int64_t fp8_stream_threads(int64_t M, int64_t N, int64_t E, int64_t R);

}  // namespace w4
