// MXFP4 products of few rows (a decode step: up to 64 dense rows, or experts
// that hold a handful each): the weights are streamed once per 16 rows, and their
// bytes are the time (1 x 14336 x 4096: 7.3 us, 4.3 TB/s, of which about 2.5 are the
// launch; 64 rows of 64 experts, 2048 x 7168: 62 us, 5.3 TB/s).
//
// A block owns 16 NJ weight rows (output columns) and 16 activation rows; its
// waves each take a run of the K steps of 256, weights, scales and activations'
// codes through LDS of their own (lds_weights.h), into
// v_mfma_scale_f32_16x16x128_f8f6f4, and their sums meet in LDS at the end.
// Lane (row l16, group g) holds the blocks g and 4 + g of a step; its two scales
// are bytes g of the step's two scale words.
//
// XQ: the activations come as bf16 or fp16, few enough that every block can
// quantize them all into LDS first, a block of the format per thread, while its first
// weights are on their way: a single token's linear layer is one launch.
#include "lds_weights.h"

namespace w4 {

// XQ: 0 codes, 1 bf16 activations, 2 fp16 ones.
template <int NJ, int WS, bool GROUPED, int XQ, int OUT>
__global__ __launch_bounds__(64 * WS) void mx_stream_kernel(MxArgs p) {
  constexpr int BM = 16, BN = 16 * NJ, NQ = NJ * 64;   // NQ: quads of results
  constexpr int kStep = 256;
  using S = Scales<kMx, NJ>;
  // a step in LDS: weights, activations; and the scales of both (the latter as one more set of 16 rows) in places of their own
  constexpr int kA = 2048 * NJ, kSlot = kA + (XQ ? 0 : 2048), kScales = 1024 * (NJ + (XQ ? 0 : 1));
  __shared__ __attribute__((aligned(16))) union {
    struct {
      uint8_t step[WS][kSlot], scales[WS][kScales];
    } r;
    v4f red[WS][NQ];
  } s;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];   // XQ: codes [M][KT][128], scales [M][KT][8]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  int e = 0, tn;
  int64_t r0, rows, out0 = 0;                        // first row of the tile, end of the rows (segment-local if grouped)
  if constexpr (GROUPED) {
    const Segment seg = find_segment<BM>(p);
    if (seg.e < 0) return;
    e = __builtin_amdgcn_readfirstlane(seg.e);
    tn = __builtin_amdgcn_readfirstlane(seg.tn);
    r0 = (int64_t)__builtin_amdgcn_readfirstlane(seg.mt) * BM;
    out0 = __builtin_amdgcn_readfirstlane((int)seg.row0);
    rows = __builtin_amdgcn_readfirstlane((int)seg.rows);
  } else {
    tn = (int)(blockIdx.x % (unsigned)p.NT);
    r0 = (int64_t)(blockIdx.x / (unsigned)p.NT) * BM;
    rows = p.M;
  }
  const int n0 = tn * BN;
  const int64_t KH = p.K >> 1;
  const bool gather = GROUPED && p.row_token;
  const int64_t base = gather ? 0 : out0 + r0, left = gather ? p.M : min((int64_t)BM, p.M - base);
  if (left <= 0) return;
  Rows<kMx> wt[NJ], at;
  S sc;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int n = n0 + 16 * j < p.N ? n0 + 16 * j : n0;   // a set past N: the first again, not stored
    wt[j].lane(0, p.K, lane);
    wt[j].open(p.w, e, p.N, n, p.K, min(16, p.N - n));
  }
  sc.lane(p.N, n0, 16, p.K, 0, lane);
  sc.open(p.w_scale, e, p.N, n0, 16, p.K, 0, min(BN, p.N - n0) - 16 * (NJ - 1));
  uint32_t as_off = kPast;
  __amdgpu_buffer_rsrc_t asr;
  if constexpr (!XQ) {
    at.lane(0, p.K, lane);
    at.w = make_rsrc(p.a + base * KH, (uint32_t)(left * KH));
    asr = make_rsrc(p.a_scale + base * p.KS, (uint32_t)(left * p.KS));
    auto token = [&](int i) {                        // of the tile's row i; -1: none
      if (r0 + i >= rows) return (int64_t)-1;
      const int64_t t = gather ? (int64_t)p.row_token[out0 + r0 + i] : i;
      return t < left ? t : -1;
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * i + (lane >> 3);
      const int64_t t = token(r);
      at.off[i] = t >= 0 ? (uint32_t)(t * KH + 16 * ((lane & 7) ^ (r & 7))) : kPast;
    }
    const int r = lane >> 2;
    const int64_t t = token(r);
    if (t >= 0) as_off = (uint32_t)(t * p.KS + 16 * ((lane & 3) ^ (r >> 2 & 3)));
  }

  const uint8_t *step = &s.r.step[wave][0], *scales = &s.r.scales[wave][0];
  const uint32_t to = lds_address(step), to_scales = lds_address(scales);
  const int k0 = p.KT * wave / WS, k1 = p.KT * (wave + 1) / WS;
  auto fetch = [&](int k) {
    const bool last = k == p.KT - 1;
#pragma unroll
    for (int j = 0; j < NJ; ++j) wt[j].fetch(k, last, to + 2048 * j);
    if constexpr (!XQ) at.fetch(k, last, to + kA);
    if (k == k0 || S::begins(k)) {
      sc.fetch(k, to_scales, lane);
      if constexpr (!XQ) dma16(asr, to_scales + 1024 * NJ, as_off, (uint32_t)(k & ~7) * 8);
    }
  };
  if (k0 < k1) fetch(k0);
  const int M = (int)p.M, row = min(l16, M - 1);     // XQ: M <= 16; rows past the last: the last again, not stored
  const uint8_t* xs = smem + M * p.KT * 128;
  if constexpr (XQ) {
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.a, (uint32_t)(2 * M * p.K));
    for (int b = tid; b < M * p.KT * 8; b += 64 * WS) {
      const int r = b / (p.KT * 8), i = b - r * p.KT * 8;
      int raw[16], codes[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4i v = __builtin_amdgcn_raw_buffer_load_b128(xr, 32 * i < p.K ? (uint32_t)(2 * (r * p.K + 32 * i) + 16 * q) : kPast, 0, 0);
#pragma unroll
        for (int d = 0; d < 4; ++d) raw[4 * q + d] = v[d];
      }
      const uint32_t c = mx_scale_code(mx_amax16<XQ == 1>(raw));
      mx_encode16<XQ == 1>(raw, mx_scale_value(c), codes);   // with a NaN scale whatever they are, as with zeros
      *reinterpret_cast<v4i*>(smem + (r * p.KT + i / 8) * 128 + 16 * ((i & 7) ^ (r & 7))) = v4i{codes[0], codes[1], codes[2], codes[3]};
      smem[M * p.KT * 128 + b] = (uint8_t)c;
    }
    __syncthreads();
  }

  v4f acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int k = k0; k < k1; ++k) {
    const int left_k = p.K - k * kStep;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    v4i wf[NJ][2], af[2];
    int sw[NJ][2], sa[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        wf[j][q] = weight_piece<kMx>(step + 2048 * j, q, l16, g);
        sw[j][q] = (int)S::code(scales, k, j, q, left_k, l16, g);
      }
      if constexpr (XQ) {
        af[q] = *reinterpret_cast<const v4i*>(smem + (row * p.KT + k) * 128 + 16 * ((4 * q + g) ^ (row & 7)));
        sa[q] = xs[(row * p.KT + k) * 8 + 4 * q + g];
      } else {
        af[q] = weight_piece<kMx>(step + kA, q, l16, g);
        sa[q] = (int)S::code(scales, k, NJ, q, left_k, l16, g);
      }
    }
    // the step is in registers: its place takes the next
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (k + 1 < k1) fetch(k + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const v4i w = wf[j][q], a = af[q];
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v8i{w[0], w[1], w[2], w[3], 0, 0, 0, 0},
                                                                  v8i{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, acc[j], 4, 4,
                                                                  0, sw[j][q], 0, sa[q]);
      }
    }
  }
  __syncthreads();                                   // nothing is on its way into what takes the sums
#pragma unroll
  for (int j = 0; j < NJ; ++j) s.red[wave][j * 64 + lane] = acc[j];
  __syncthreads();
  const int64_t r = r0 + l16;                        // this lane's row
  for (int q = tid; q < NQ; q += 64 * WS) {          // 64 WS is a multiple of 64: q keeps the lane's row
    const int n = n0 + 16 * (q / 64) + 4 * g;
    if (r >= rows || n >= p.N) continue;
    v4f v = s.red[0][q];
#pragma unroll
    for (int w = 1; w < WS; ++w) v += s.red[w][q];
    float f[4] = {v[0], v[1], v[2], v[3]};
    store_columns<OUT, 4>(p, f, (out0 + r) * p.N, n, !GROUPED && p.bias);
  }
}

// 32 columns per block, 4 waves: 64 rows of 64 experts, 2048 x 7168, take 64 us; 16 columns 77, 64 columns 67; 2 waves 63, 8
// waves 70. A single row of 14336 x 4096 takes 7.4 to 7.6 us in each of these.
constexpr int kSets = 2, kWaves = 4;

template <typename F>
static hipError_t stream_go(MxArgs p, F kernel, hipStream_t stream, size_t lds = 0) {
  p.NT = (p.N + 16 * kSets - 1) / (16 * kSets);
  const dim3 grid((unsigned)(p.offsets ? grouped_blocks(p.E, p.R, p.N, 16, 16 * kSets) : (p.M + 15) / 16 * p.NT));
  hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), lds, stream, p);
  return hipGetLastError();
}

hipError_t launch_mx_stream(const MxArgs& p, int xq, int out_dt, hipStream_t stream) {
  if (p.offsets)
    return out_dt == 0 ? stream_go(p, mx_stream_kernel<kSets, kWaves, true, 0, 0>, stream)
                       : stream_go(p, mx_stream_kernel<kSets, kWaves, true, 0, 1>, stream);
  const size_t lds = (size_t)(p.M * p.KT * 136);     // codes and scales of activations that the kernel quantizes
  if (xq == 1) return stream_go(p, mx_stream_kernel<kSets, kWaves, false, 1, 0>, stream, lds);
  if (xq == 2) return stream_go(p, mx_stream_kernel<kSets, kWaves, false, 2, 1>, stream, lds);
  if (out_dt == 0) return stream_go(p, mx_stream_kernel<kSets, kWaves, false, 0, 0>, stream);
  if (out_dt == 1) return stream_go(p, mx_stream_kernel<kSets, kWaves, false, 0, 1>, stream);
  return stream_go(p, mx_stream_kernel<kSets, kWaves, false, 0, 2>, stream);
}

int64_t mx_stream_threads(int64_t M, int64_t N, int64_t E, int64_t R) {
  if (E > 0) return grouped_blocks(E, R, N, 16, 16 * kSets) * 64 * kWaves;
  return (M + 15) / 16 * ((N + 16 * kSets - 1) / (16 * kSets)) * 64 * kWaves;
}

}  // namespace w4
