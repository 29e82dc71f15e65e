// Block-scaled FP8 products of few rows (a decode step: up to 16 dense rows,
// or experts that hold a handful each): the weights are streamed once.
//
// The arithmetic is that of fp8_block_gemm.hip; with so few rows the time is
// the weights' bytes. A block of WS waves owns 16 NJ weight rows (output
// columns) and 16 activation rows; its waves take the K blocks in turn,
// each loading weights and activations straight into the registers the matrix
// instruction reads (a weight byte is used by one wave only, so LDS would add
// a copy), and their sums meet in LDS at the end. Without a barrier in the
// loop, every resident wave keeps U K blocks of loads in flight.
#include "fp8_block.h"

namespace w4 {

template <int NJ, int WS, int U, bool GROUPED, bool F16, int OUT>
__global__ __launch_bounds__(64 * WS) void fp8_stream_kernel(Fp8Args p) {
  constexpr int BM = 16, BN = 16 * NJ, NQ = NJ * 64;   // NQ: quads of results
  __shared__ __attribute__((aligned(16))) v4f red[WS][NQ];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  int e = 0, tn;
  int64_t r0, rows, out0 = 0;                        // first row of the tile, end of the rows (segment-local if grouped)
  if constexpr (GROUPED) {
    const Segment s = find_segment<BM>(p);
    if (s.e < 0) return;
    e = s.e;
    tn = s.tn;
    r0 = (int64_t)s.mt * BM;
    out0 = s.row0;
    rows = s.rows;
  } else {
    tn = (int)(blockIdx.x % (unsigned)p.NT);
    r0 = (int64_t)(blockIdx.x / (unsigned)p.NT) * BM;
    rows = p.M;
  }
  const int n0 = tn * BN;

  const bool gather = GROUPED && p.row_token;
  const int64_t base = gather ? 0 : out0 + r0, left = gather ? p.M : min((int64_t)BM, p.M - base);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(p.a + base * p.K, (uint32_t)max(left * p.K, (int64_t)0));
  const __amdgpu_buffer_rsrc_t asr = make_rsrc(p.a_scale + base * p.KB, (uint32_t)max(left * p.KB * 4, (int64_t)0));
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.w + ((int64_t)e * p.N + n0) * p.K, (uint32_t)(min(BN, p.N - n0) * (int64_t)p.K));
  const float* __restrict__ ws = p.w_scale + ((int64_t)e * p.NBLK + n0 / 128) * p.KB;   // BN divides 128: one row of scales
  uint32_t w_off[NJ];
  const int64_t r = r0 + l16;                        // this lane's row
  int64_t t = r < rows ? (gather ? (int64_t)p.row_token[out0 + r] : l16) : -1;
  if (t >= left) t = -1;
  const uint32_t a_off = t >= 0 ? (uint32_t)(t * p.K + 16 * g) : kPast;
  const uint32_t s_off = t >= 0 ? (uint32_t)(t * p.KB * 4) : kPast;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    w_off[j] = n0 + 16 * j + l16 < p.N ? (uint32_t)((16 * j + l16) * (int64_t)p.K + 16 * g) : kPast;

  // the 16-byte chunks g and g + 4 of a K block; past K's end they read as zero
  auto load = [&](const __amdgpu_buffer_rsrc_t rs, uint32_t off, int kb) -> v8i {
    const uint32_t ks = (uint32_t)kb * kFK, end = (uint32_t)p.K - ks;
    const v4i x = __builtin_amdgcn_raw_buffer_load_b128(rs, 16u * g < end ? off : kPast, ks, 0);
    const v4i y = __builtin_amdgcn_raw_buffer_load_b128(rs, 16u * g + 64u < end ? (off == kPast ? kPast : off + 64u) : kPast, ks, 0);
    return v8i{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  v4f acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < p.KB; kb += WS * U) {
    v8i wf[U][NJ], af[U];
    float s[U], sw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(kb + WS * u, p.KB - 1);      // past the end: loaded again, not used
#pragma unroll
      for (int j = 0; j < NJ; ++j) wf[u][j] = load(wr, w_off[j], k);
      af[u] = load(ar, a_off, k);
      s[u] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(asr, s_off, 4u * (uint32_t)k, 0));
      sw[u] = ws[k];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + WS * u >= p.KB) break;
      const float sc = s[u] * sw[u];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const v4f d = block_product<F16>(wf[u][j], af[u]);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = fmaf(d[q], sc, acc[j][q]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) red[wave][j * 64 + lane] = acc[j];
  __syncthreads();
  for (int q = tid; q < NQ; q += 64 * WS) {          // 64 WS is a multiple of 64: q keeps the lane's row
    const int n = n0 + 16 * (q / 64) + 4 * g;
    if (r >= rows || n >= p.N) continue;
    v4f v = red[0][q];
#pragma unroll
    for (int w = 1; w < WS; ++w) v += red[w][q];
    float f[4] = {v[0], v[1], v[2], v[3]};
    store_columns<OUT, 4>(p, f, (out0 + r) * p.N, n, !GROUPED && p.bias);
  }
}

template <int NJ, int TH, typename F>
static hipError_t stream_go(Fp8Args p, F kernel, hipStream_t stream) {
  constexpr int BN = 16 * NJ;
  p.NT = (p.N + BN - 1) / BN;
  const dim3 grid((unsigned)(p.offsets ? grouped_blocks(p.E, p.R, p.N, 16, BN) : (p.M + 15) / 16 * p.NT)), block(TH);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, p);
  return hipGetLastError();
}

template <int NJ, int WS, int U>
static hipError_t dense_go(const Fp8Args& p, int out_dt, hipStream_t stream) {
  auto go = [&](auto kernel) { return stream_go<NJ, 64 * WS>(p, kernel, stream); };
  if (out_dt == 0) return go(fp8_stream_kernel<NJ, WS, U, false, false, 0>);
  if (out_dt == 1) return go(fp8_stream_kernel<NJ, WS, U, false, false, 1>);
  return go(fp8_stream_kernel<NJ, WS, U, false, true, 2>);
}

// Dense: 32 columns a block; 16, with 16 waves along K, where the former would leave
// CUs without a block (1 x 4096 x 14336: 11.4 us, 22.6 with 32 columns and 4
// waves; 1 x 14336 x 4096: 11.8 us with the latter, 14.7 with the former).
static bool narrow(int64_t N) { return N < 32 * 256; }

hipError_t launch_fp8_stream(const Fp8Args& p, int out_dt, hipStream_t stream) {
  if (p.offsets)
    return out_dt == 0 ? stream_go<2, 256>(p, fp8_stream_kernel<2, 4, 2, true, false, 0>, stream)
                       : stream_go<2, 256>(p, fp8_stream_kernel<2, 4, 2, true, false, 1>, stream);
  return narrow(p.N) ? dense_go<1, 16, 2>(p, out_dt, stream) : dense_go<2, 4, 2>(p, out_dt, stream);
}

int64_t fp8_stream_threads(int64_t M, int64_t N, int64_t E, int64_t R) {
  if (E > 0) return grouped_blocks(E, R, N, 16, 32) * 256;
  return (M + 15) / 16 * (narrow(N) ? (N + 15) / 16 * 1024 : (N + 31) / 32 * 256);
}

}  // namespace w4
