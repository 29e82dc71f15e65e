// MXFP4 products of few rows (a decode step: up to 16 dense rows, or experts
// that hold a handful each): the weights are streamed once, and their bytes
// are the time.
//
// A block of WS waves owns 16 NJ weight rows (output columns) and 16
// activation rows; its waves take the K steps of 256 in turn, each loading
// weights and activations straight into the registers that
// v_mfma_scale_f32_16x16x128_f8f6f4 reads (a weight byte is used by one wave
// only, so LDS would add a copy), and their sums meet in LDS at the end. Lane
// (row l16, group g) holds the blocks g and 4 + g of a step: 64 consecutive
// bytes of each of 16 rows per load. Its two scales are bytes g of the step's
// two scale words.
//
// XQ: the activations come as bf16 or fp16 and are quantized on the way. A
// lane's 32 values of an MFMA are exactly one block of the format, so its scale
// and codes need no exchange; a single token's linear layer is one launch.
#include "mxfp4.h"

namespace w4 {

// XQ: 0 codes, 1 bf16 activations, 2 fp16 ones.
template <int NJ, int WS, int U, bool GROUPED, int XQ, int OUT>
__global__ __launch_bounds__(64 * WS) void mx_stream_kernel(MxArgs p) {
  constexpr int BM = 16, BN = 16 * NJ, NQ = NJ * 64;   // NQ: quads of results
  constexpr int kStep = 256;
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

  const int64_t KH = p.K >> 1, arow = XQ ? 2 * (int64_t)p.K : KH;   // bytes of a row of weights, of activations
  const bool gather = GROUPED && p.row_token;
  const int64_t base = gather ? 0 : out0 + r0, left = gather ? p.M : min((int64_t)BM, p.M - base);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(p.a + base * arow, (uint32_t)max(left * arow, (int64_t)0));
  const __amdgpu_buffer_rsrc_t asr = make_rsrc(p.a_scale + (XQ ? 0 : base * p.KS), XQ ? 0u : (uint32_t)max(left * p.KS, (int64_t)0));
  const int64_t wrow0 = (int64_t)e * p.N + n0;
  const int wrows = min(BN, p.N - n0);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(p.w + wrow0 * KH, (uint32_t)(wrows * KH));
  const __amdgpu_buffer_rsrc_t wsr = make_rsrc(p.w_scale + wrow0 * p.KS, (uint32_t)((int64_t)wrows * p.KS));
  const int64_t r = r0 + l16;                        // this lane's row
  int64_t t = r < rows ? (gather ? (int64_t)p.row_token[out0 + r] : l16) : -1;
  if (t >= left) t = -1;
  const uint32_t a_off = t >= 0 ? (uint32_t)(t * arow + (XQ ? 64 : 16) * g) : kPast;
  const uint32_t as_off = t >= 0 ? (uint32_t)(t * p.KS) : kPast;
  uint32_t w_off[NJ], ws_off[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const bool in = 16 * j + l16 < wrows;
    w_off[j] = in ? (uint32_t)((16 * j + l16) * KH + 16 * g) : kPast;
    ws_off[j] = in ? (uint32_t)((16 * j + l16) * (int64_t)p.KS) : kPast;
  }

  v4f acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kt = wave; kt < p.KT; kt += WS * U) {
    v4i wf[U][NJ][2];
    v4i af[U][XQ ? 8 : 2];
    v2i sw[U][NJ], sa[U];
    uint32_t live[U];                                // bit q: block 4 q + g of the step lies inside K
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = min(kt + WS * u, p.KT - 1);      // past the end: loaded again, not used
      const int left_k = p.K - k * kStep;
      live[u] = (32 * g < left_k ? 1u : 0u) | (128 + 32 * g < left_k ? 2u : 0u);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          wf[u][j][q] = __builtin_amdgcn_raw_buffer_load_b128(
              wr, (live[u] >> q & 1) && w_off[j] != kPast ? w_off[j] + 64u * q : kPast, (uint32_t)k * (kStep / 2), 0);
        sw[u][j] = __builtin_amdgcn_raw_buffer_load_b64(wsr, ws_off[j], (uint32_t)k * 8u, 0);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool in = (live[u] >> q & 1) && a_off != kPast;
        if constexpr (XQ) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            af[u][4 * q + i] = __builtin_amdgcn_raw_buffer_load_b128(ar, in ? a_off + 256u * q + 16u * i : kPast,
                                                                     (uint32_t)k * (2 * kStep), 0);
        } else {
          af[u][q] = __builtin_amdgcn_raw_buffer_load_b128(ar, in ? a_off + 64u * q : kPast, (uint32_t)k * (kStep / 2), 0);
        }
      }
      if constexpr (!XQ) sa[u] = __builtin_amdgcn_raw_buffer_load_b64(asr, as_off, (uint32_t)k * 8u, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kt + WS * u >= p.KT) break;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool in = live[u] >> q & 1;
        v4i a;
        int s;
        if constexpr (XQ) {
          int raw[16], codes[4];
#pragma unroll
          for (int i = 0; i < 16; ++i) raw[i] = af[u][4 * q + i / 4][i % 4];
          const uint32_t sc = mx_scale_code(mx_amax16<XQ == 1>(raw));
          mx_encode16<XQ == 1>(raw, mx_scale_value(sc), codes);
          a = v4i{codes[0], codes[1], codes[2], codes[3]};   // with a NaN scale whatever they are, as with zeros
          s = (int)sc;
        } else {
          a = af[u][q];
          s = in ? (int)((uint32_t)sa[u][q] >> (8 * g) & 0xFF) : 0;   // past K: the padding, or the next row's
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const v4i w = wf[u][j][q];
          const int sq = in ? (int)((uint32_t)sw[u][j][q] >> (8 * g) & 0xFF) : 0;
          acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v8i{w[0], w[1], w[2], w[3], 0, 0, 0, 0},
                                                                    v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, acc[j], 4, 4,
                                                                    0, sq, 0, s);
        }
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
static hipError_t stream_go(MxArgs p, F kernel, hipStream_t stream) {
  constexpr int BN = 16 * NJ;
  p.NT = (p.N + BN - 1) / BN;
  const dim3 grid((unsigned)(p.offsets ? grouped_blocks(p.E, p.R, p.N, 16, BN) : (p.M + 15) / 16 * p.NT)), block(TH);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, p);
  return hipGetLastError();
}

template <int NJ, int WS, int U>
static hipError_t dense_go(const MxArgs& p, int xq, int out_dt, hipStream_t stream) {
  auto go = [&](auto kernel) { return stream_go<NJ, 64 * WS>(p, kernel, stream); };
  if (xq == 1) return go(mx_stream_kernel<NJ, WS, U, false, 1, 0>);
  if (xq == 2) return go(mx_stream_kernel<NJ, WS, U, false, 2, 1>);
  if (out_dt == 0) return go(mx_stream_kernel<NJ, WS, U, false, 0, 0>);
  if (out_dt == 1) return go(mx_stream_kernel<NJ, WS, U, false, 0, 1>);
  return go(mx_stream_kernel<NJ, WS, U, false, 0, 2>);
}

static bool narrow(int64_t N) { return N < 32 * 256; }

hipError_t launch_mx_stream(const MxArgs& p, int xq, int out_dt, hipStream_t stream) {
  if (p.offsets)
    return out_dt == 0 ? stream_go<2, 256>(p, mx_stream_kernel<2, 4, 2, true, 0, 0>, stream)
                       : stream_go<2, 256>(p, mx_stream_kernel<2, 4, 2, true, 0, 1>, stream);
  return narrow(p.N) ? dense_go<1, 16, 2>(p, xq, out_dt, stream) : dense_go<2, 4, 2>(p, xq, out_dt, stream);
}

int64_t mx_stream_threads(int64_t M, int64_t N, int64_t E, int64_t R) {
  if (E > 0) return grouped_blocks(E, R, N, 16, 32) * 256;
  return (M + 15) / 16 * (narrow(N) ? (N + 15) / 16 * 1024 : (N + 31) / 32 * 256);
}

}  // namespace w4
