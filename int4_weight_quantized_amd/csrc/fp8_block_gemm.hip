// FP8 (E4M3) matrix products with a scale for each block of 128: dense, and
// grouped over the row segments of routed experts.
//
//   out[r, n] = sum_b sa[t, b] * sw[n / 128, b] * sum_{k in block b} a[t, k] * w[n, k]  (+ bias[n])
//
// with t = r, or the row's token in the grouped form.
//
// v_mfma_f32_16x16x128_f8f6f4 spans one scale block: it starts from zero,
// and its 4 results per lane are scaled into fp32 accumulators (4 FMAs per
// MFMA of 32 cycles). Inside, the FP8 matrix unit sums each 8 products on a
// grid of 2^-13 of the largest one's power of two (measured; the 8-products'
// sums themselves add in fp32): below 1.4e-5 of the result on normal data,
// far under half a step of bf16 and fp16 (2^-9, 2^-12 on average), but above
// fp32's. So fp32 outputs convert both operands to fp16, which holds every
// E4M3 value, and take v_mfma_f32_16x16x32_f16, whose sums are fp32 (1e-8
// measured), at half the rate. The weights are the A operand and the activations the
// B operand, so a lane's 4 results lie in one activation row and share one
// scale sa * sw, and a lane holds consecutive output columns.
//
// Tile kernel: WM x WN waves, each with a tile of 16 MI rows x 16 NJ columns.
// - Both operands pass through LDS (two stages, one K block each) by LDS DMA.
//   The DMA is an asm statement: with the builtin the compiler waits for all
//   of it before the next LDS read, which cost 40% (1149 to 1834 TFLOP/s, with
//   the order of work below).
// - A step's last row of MFMAs runs behind the barrier that ends the step:
//   every fragment of the step is in registers by then, so its stage is free
//   for the DMA two steps ahead (a whole step in flight) and the next step's
//   first fragments are read under those MFMAs.
// - The FMAs of an MFMA follow it by kLag MFMAs, pinned there (left alone the
//   compiler sinks them past the barrier and keeps every result alive: 60
//   registers more, and spills in the 256 x 256 tile).
// - The scales of 4 steps come by one DMA of 16 bytes per row (one of 4 bytes
//   per step cost the experts 6%); a lane reads its rows' at the step's start.
// - 256 x 256 with 8 waves is the largest tile whose accumulators (128
//   registers a lane: vector FMAs cannot reach the other 256) leave room; it
//   reads 3/4 of the LDS bytes per MFMA of a 64 x 64 wave tile.
// 4096 x 14336 x 4096, bf16 out: 240 to 252 us, 1.9 to 2.0 PFLOP/s, the matrix
// units 45% busy at the 2.0 GHz the power limit leaves; 65536 rows of 64
// experts, 2048 x 7168: 1.00 to 1.05 ms, 1.8 to 1.9 PFLOP/s. From K = 1024 to
// 8192 the time grows by 6.8 us per K step, of which the matrix units need 4.1
// (four rounds of tiles), over 31 us for the tiles' first loads and stores.
// Without FMAs 5% less time, without DMA 16%. With fp32 output (128 x 128
// tiles, fp16 operands) 464 us, 1.04 PFLOP/s.
#include "fp8_block.h"

namespace w4 {

constexpr int kLag = 3;                              // 2: 273 us where 3 takes 262, 4 and 5 no faster

// OUT: 0 bf16, 1 fp16, 2 fp32.
template <int MI, int NJ, int WM, int WN, bool GROUPED, bool F16, int OUT>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_tile_kernel(Fp8Args p) {
  constexpr int TH = 64 * WM * WN, BM = 16 * MI * WM, BN = 16 * NJ * WN;
  constexpr int RA = BM * 8 / TH, RB = BN * 8 / TH;  // LDS DMAs per thread and K step
  constexpr int NB = BN > 128 ? BN / 128 : 1;        // weight scale rows per tile
  static_assert(MI % 2 == 0 && NJ % 2 == 0, "pairs of rows and of column blocks");
  static_assert(RA * TH == BM * 8 && RB * TH == BN * 8, "whole DMAs");
  constexpr int STAGE = (BM + BN) * kFK, CHUNK = TH * 16;
  static_assert(BM + NB <= TH, "a row of scales per thread");
  // two stages (activation rows, then weight rows), two chunks of the scales of 4 K steps (sa of each row, then sw)
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE + 2 * CHUNK];

  // ---- work item
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, l16 = lane & 15;
  int e = 0, tn, split = 0;
  int64_t r0, row_end, out0 = 0;                     // first row and end of this tile's rows (segment-local if grouped)
  if constexpr (GROUPED) {
    const Segment s = find_segment<BM>(p);
    if (s.e < 0) return;
    e = s.e;
    tn = s.tn;
    r0 = (int64_t)s.mt * BM;
    out0 = s.row0;
    row_end = s.rows;
  } else {
    const int64_t t = xcd_remap((int)blockIdx.x, (int)gridDim.x);
    split = (int)(t / p.tiles);
    const int64_t tile = t - (int64_t)split * p.tiles;
    r0 = tile / p.NT * BM;
    tn = (int)(tile % p.NT);
    row_end = p.M;
  }
  const int n0 = tn * BN;
  const int k0 = (int)((int64_t)p.KB * split / p.splits), k1 = (int)((int64_t)p.KB * (split + 1) / p.splits);

  // ---- LDS DMA: wave w's load i fills 8 rows (one KiB), lane L at row L/8,
  // physical 16-byte chunk L%8. Row r holds logical chunk c at physical chunk
  // c ^ f(r), with f(r) = r & 7 for the activations and (r & 3) + 4 of the
  // fragment's row-group parity for the weights, so that the 8 rows that a
  // fragment read touches at a time lie in 8 different chunks. Rows and
  // columns past the end get an offset past the buffer, which reads as zero.
  const int lrow = lane >> 3, lchunk = lane & 7;
  const int64_t abase = (GROUPED && p.row_token) ? 0 : (out0 + r0) * p.K;
  const int64_t aspan = (GROUPED && p.row_token) ? p.M * p.K : min((int64_t)BM, p.M - out0 - r0) * p.K;
  const __amdgpu_buffer_rsrc_t arsrc = make_rsrc(p.a + abase, (uint32_t)max(aspan, (int64_t)0));
  const int64_t wrow0 = (int64_t)e * p.N + n0;
  const __amdgpu_buffer_rsrc_t wrsrc = make_rsrc(p.w + wrow0 * p.K, (uint32_t)((int64_t)min(BN, p.N - n0) * p.K));
  auto token = [&](int r) -> int64_t {               // activation row of tile row r, relative to abase; -1: none
    if (r0 + r >= row_end) return -1;
    if (GROUPED && p.row_token) {
      const int t = p.row_token[out0 + r0 + r];
      return (unsigned)t < (uint64_t)p.M ? t : -1;
    }
    return (!GROUPED || out0 + r0 + r < p.M) ? r : -1;
  };
  uint32_t a_off[RA], b_off[RB];
  uint32_t a_dead = 0, b_dead = 0;                   // bit i: load i's chunk lies past K in the last step
  const int klast = p.K - (p.KB - 1) * kFK;          // columns of the last K step
#pragma unroll
  for (int i = 0; i < RA; ++i) {
    const int r = (TH / 8) * i + 8 * wave + lrow;
    const int c = lchunk ^ (r & 7);
    const int64_t t = token(r);
    a_off[i] = t >= 0 ? (uint32_t)(t * p.K + 16 * c) : kPast;
    if (16 * c >= klast) a_dead |= 1u << i;
  }
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int r = (TH / 8) * i + 8 * wave + lrow;
    const int c = lchunk ^ ((r & 3) + 4 * ((r >> 3) & 1));
    b_off[i] = n0 + r < p.N ? (uint32_t)((int64_t)r * p.K + 16 * c) : kPast;
    if (16 * c >= klast) b_dead |= 1u << i;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t ldsw = __builtin_amdgcn_readfirstlane(lds0 + 8 * wave * kFK);
  // m0 holds the LDS address. The compiler keeps nothing in it here, and a clobber of a reserved register is not honoured.
  auto dma = [&](const __amdgpu_buffer_rsrc_t rs, uint32_t dst, uint32_t off, uint32_t ks) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(dst), "v"(off), "s"(rs), "s"(ks) : "memory");
  };
  // the row of scales that this thread fetches
  const int64_t sspan = (GROUPED && p.row_token) ? p.M * p.KB : min((int64_t)BM, p.M - out0 - r0) * p.KB;
  const __amdgpu_buffer_rsrc_t asr = make_rsrc(p.a_scale + ((GROUPED && p.row_token) ? 0 : (out0 + r0) * p.KB),
                                               (uint32_t)max(sspan * 4, (int64_t)0));
  const __amdgpu_buffer_rsrc_t wsr = make_rsrc(p.w_scale + ((int64_t)e * p.NBLK + n0 / 128) * p.KB,
                                               (uint32_t)((int64_t)min(NB, p.NBLK - n0 / 128) * p.KB * 4));
  const bool rows_wave = 64 * wave < BM;             // BM is a multiple of 64: a wave fetches sa or sw
  uint32_t s_off;
  if (rows_wave) {
    const int64_t t = token(tid);
    s_off = t >= 0 ? (uint32_t)(t * p.KB * 4) : kPast;
  } else {
    s_off = tid - BM < NB ? (uint32_t)((tid - BM) * p.KB * 4) : kPast;
  }
  // DMA q of a K step: the activations' RA, the weights' RB, then every 4
  // steps the scales (of steps past K: whatever follows, not used)
  constexpr int ND = RA + RB + 1;
  auto gload1 = [&](int tk, uint32_t stage, int q) {
    const uint32_t ks = (uint32_t)tk * kFK;
    if (q == RA + RB) {
      const int rel = tk - k0;
      if (rel & 3) return;
      const uint32_t dst = lds0 + 2 * STAGE + ((rel >> 2) & 1) * CHUNK + 1024 * wave;
      if (rows_wave) dma(asr, dst, s_off, (uint32_t)tk * 4);
      else dma(wsr, dst, s_off, (uint32_t)tk * 4);
      return;
    }
    const bool act = q < RA;
    const int i = act ? q : q - RA;
    uint32_t off = act ? a_off[i] : b_off[i];
    if (tk == p.KB - 1 && (((act ? a_dead : b_dead) >> i) & 1)) off = kPast;
    dma(act ? arsrc : wrsrc, ldsw + stage + ((act ? 0 : BM) + (TH / 8) * i) * kFK, off, ks);
  };
  auto gload = [&](int tk, uint32_t stage) {
#pragma unroll
    for (int q = 0; q < ND; ++q) gload1(tk, stage, q);
  };

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // ---- fragments: lane group g takes logical chunks g and g + 4 of its row.
  // Row rho of weight block j is column 32 (j / 2) + 8 (rho / 4) + 4 (j % 2) +
  // rho % 4 of the wave's 16 NJ, so that two blocks give a lane 8 consecutive
  // columns and four lanes a run of 32 (stores of 16 bytes in runs of 64; with
  // 8-byte stores the 4096 x 14336 x 4096 product took 24 us longer).
  const int ar = 16 * MI * wm + l16;                 // + 16 i; 16 i leaves f unchanged
  const int a_ro = ar * kFK + 16 * (g ^ (ar & 7)), a_rx = ar * kFK + 16 * ((g + 4) ^ (ar & 7));
  const int br = 16 * NJ * wn + 8 * (l16 >> 2) + (l16 & 3);   // + 32 (j / 2) + 4 (j % 2): those leave f unchanged
  const int bfx = (l16 & 3) + 4 * ((l16 >> 2) & 1);
  const int b_ro = (BM + br) * kFK + 16 * (g ^ bfx), b_rx = (BM + br) * kFK + 16 * ((g + 4) ^ bfx);
  const int snb = (16 * NJ * wn) / 128 % NB;
  auto frag = [&](const uint8_t* q0, const uint8_t* q1) -> v8i {
    const v4i x0 = *reinterpret_cast<const v4i*>(q0);
    const v4i x1 = *reinterpret_cast<const v4i*>(q1);
    return v8i{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
  };

  constexpr int NM = MI * NJ;
  if (k0 < k1) {
    gload(k0, 0);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    if (k0 + 1 < k1) gload(k0 + 1, STAGE);
    if (GROUPED && r0 + 16 * MI * wm >= row_end) {   // a wave whose rows all lie past the segment only fetches
      for (int tk = k0; tk < k1; ++tk) {
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        if (tk + 2 < k1) gload(tk + 2, ((tk - k0) & 1) * STAGE);
      }
      return;
    }
    v8i bf[NJ], af[2];
    af[0] = frag(lds + a_ro, lds + a_rx);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      bf[j] = frag(lds + b_ro + (32 * (j / 2) + 4 * (j % 2)) * kFK, lds + b_rx + (32 * (j / 2) + 4 * (j % 2)) * kFK);
    for (int tk = k0; tk < k1; ++tk) {
      const int rel = tk - k0;
      const uint32_t st = (rel & 1) * STAGE;         // this step's stage
      const uint8_t* cur = lds + st;
      const uint8_t* nxt = lds + (STAGE - st);
      const float* sp = reinterpret_cast<const float*>(lds + 2 * STAGE + ((rel >> 2) & 1) * CHUNK) + (rel & 3);
      const float sw = sp[4 * (BM + snb)];
      float s[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) s[i] = sp[4 * (16 * (MI * wm + i) + l16)];
      v4f d[kLag + 1];
#pragma unroll
      for (int n = 0; n < NM + kLag; ++n) {
        const int i = n / NJ, j = n % NJ;
        if (n < NM) {
          if (j == 0) {
            if (i + 1 < MI) {
              af[(i + 1) & 1] = frag(cur + a_ro + 16 * (i + 1) * kFK, cur + a_rx + 16 * (i + 1) * kFK);
            } else {
              // every fragment of this step is in registers; once the next step's tiles have landed: swap
              asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          d[n % (kLag + 1)] = block_product<F16>(bf[j], af[i & 1]);
          if (i == MI - 1) {
            // the next step's fragments (at the end: of a stage whose contents are not used)
            bf[j] = frag(nxt + b_ro + (32 * (j / 2) + 4 * (j % 2)) * kFK, nxt + b_rx + (32 * (j / 2) + 4 * (j % 2)) * kFK);
            if (j == 0) af[0] = frag(nxt + a_ro, nxt + a_rx);
            constexpr int Q = (ND + NJ - 1) / NJ;
            if (tk + 2 < k1) {
#pragma unroll
              for (int q = j * Q; q < (j + 1) * Q && q < ND; ++q) gload1(tk + 2, st, q);
            }
          }
        }
        if (n == kLag) {
#pragma unroll
          for (int i2 = 0; i2 < MI; ++i2) s[i2] *= sw;
        }
        if (n >= kLag) {
          const int m = n - kLag;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[m / NJ][m % NJ][r] = fmaf(d[m % (kLag + 1)][r], s[m / NJ], acc[m / NJ][m % NJ][r]);
          asm volatile("" : "+v"(acc[m / NJ][m % NJ]));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // ---- output: lane's row per i, runs of 8 consecutive columns
  const int nw = n0 + 16 * NJ * wn + 8 * g;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t r = r0 + 16 * MI * wm + 16 * i + l16;
    if (r >= row_end) continue;
    const int64_t orow = (out0 + r + (int64_t)split * p.M) * p.N;
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      const int n = nw + 16 * j;
      if (n >= p.N) continue;
      float f[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] = acc[i][j + c / 4][c % 4];
      store_columns<OUT, 8>(p, f, orow, n, !GROUPED && p.bias && p.splits == 1);
    }
  }
}

// The 256 x 256 tile does a third more work per time than four of 128 x 128, as
// long as its padding takes no more than that.
static bool wide_pays(int64_t t256, int64_t t128) { return 3 * t256 <= t128; }

// What the dense product runs as: rows streamed (tile 0), or a tile and its
// K splits.
struct DensePlan {
  int tile, splits;
};

// The smaller tiles run one step in about 0.9 us while at most two of their
// blocks share a CU (the next step's tiles arrive from memory), so K is split
// while the steps saved outweigh the partial sums' way to memory and back
// (4.5 TB/s) and the second kernel (2 us, 0.1 us per split). 200 x 4096 x
// 14336: 8 splits 29 us, 4 36; 256 x 4096 x 4096: 4 splits 18 us, 8 24; 1024 x
// 4096 x 4096: none 27 us, 2 34. The 256 x 256 tile takes over where it fills
// most CUs (1024 x 14336 x 4096: 62 us; 128 x 128 2 us slower), and streaming
// up to 16 rows (12 x 4096 x 4096: 7 us; 64 x 128 tiles 11).
static DensePlan plan_dense(int64_t M, int64_t N, int64_t K) {
  if (M <= 16) return {0, 1};
  const int64_t KB = (K + 127) / 128;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  if (tiles(256, 256) >= 192 && wide_pays(tiles(256, 256), tiles(128, 128))) return {256, 1};
  const int tile = M <= 64 ? 64 : 128;
  const int64_t t = tiles(tile, 128);
  int64_t best = 1, cost = 4000 + 900 * KB;   // ns
  for (int64_t s = 2; s * t <= 512 && 2 * s <= KB; ++s) {
    const int64_t c = 6000 + 900 * ((KB + s - 1) / s) + 100 * s + s * M * N * 8 / 4500;
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return {tile, (int)best};
}

size_t fp8_block_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const DensePlan pl = plan_dense(M, N, K);
  return pl.splits > 1 ? (size_t)pl.splits * (size_t)M * (size_t)N * 4 : 0;
}

// Threads of the largest launch of a product, for the host's check against a
// launch's limit. (A dense product planned for 256 x 256 tiles takes 128 x 128
// ones for fp32 outputs: more threads.)
int64_t fp8_block_gemm_threads(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const DensePlan pl = plan_dense(M, N, K);
  if (pl.tile == 0) return fp8_stream_threads(M, N, 0, 0);
  const int64_t bm = pl.tile == 64 ? 64 : 128;
  return (M + bm - 1) / bm * ((N + 127) / 128) * pl.splits * 256;
}

template <int BM, int BN, int TH, typename F>
static hipError_t grouped_go(Fp8Args p, F kernel, hipStream_t stream) {
  p.NT = (p.N + BN - 1) / BN;
  const dim3 grid((unsigned)grouped_blocks(p.E, p.R, p.N, BM, BN)), block(TH);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, p);
  return hipGetLastError();
}

template <int BM, int BN, int TH, typename F>
static hipError_t dense_go(Fp8Args p, F kernel, hipStream_t stream) {
  p.NT = (p.N + BN - 1) / BN;
  p.tiles = (p.M + BM - 1) / BM * p.NT;
  const dim3 grid((unsigned)(p.tiles * p.splits)), block(TH);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, p);
  return hipGetLastError();
}

// The tiles with K splits: fp32 outputs and partial sums among them.
// f16: the fp32-exact products (fp32 results).
template <int MI, int NJ>
static hipError_t split_tile_go(const Fp8Args& p, bool f16, int out_dt, hipStream_t stream) {
  constexpr int BM = 32 * MI, BN = 32 * NJ;
  auto go = [&](auto kernel) { return dense_go<BM, BN, 256>(p, kernel, stream); };
  if (f16) return go(fp8_tile_kernel<MI, NJ, 2, 2, false, true, 2>);
  if (out_dt == 0) return go(fp8_tile_kernel<MI, NJ, 2, 2, false, false, 0>);
  if (out_dt == 1) return go(fp8_tile_kernel<MI, NJ, 2, 2, false, false, 1>);
  return go(fp8_tile_kernel<MI, NJ, 2, 2, false, false, 2>);   // partial sums
}

hipError_t launch_fp8_block_gemm(const void* a, const float* a_scale, const void* w, const float* w_scale,
                                 const void* bias, void* out, int out_dt, int64_t M, int64_t N, int64_t K, void* ws,
                                 hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  Fp8Args p{};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scale = a_scale;
  p.w = static_cast<const uint8_t*>(w);
  p.w_scale = w_scale;
  p.bias = bias;
  p.out = out;
  p.M = p.R = M;
  p.E = 1;
  p.N = (int)N;
  p.K = (int)K;
  p.KB = (int)((K + 127) / 128);
  p.NBLK = (int)((N + 127) / 128);
  const DensePlan pl = plan_dense(M, N, K);
  p.splits = pl.splits;
  if (pl.tile == 0) return launch_fp8_stream(p, out_dt, stream);
  Fp8Args part = p;
  if (p.splits > 1) part.out = ws;
  const int dt = p.splits > 1 ? 2 : out_dt;
  // (converting to fp16 in the 256 x 256 tile spills registers)
  hipError_t e;
  if (pl.tile == 64) e = split_tile_go<2, 4>(part, out_dt == 2, dt, stream);
  else if (pl.tile == 128 || out_dt == 2) e = split_tile_go<4, 4>(part, out_dt == 2, dt, stream);
  else if (dt == 0) e = dense_go<256, 256, 512>(part, fp8_tile_kernel<8, 4, 2, 4, false, false, 0>, stream);
  else e = dense_go<256, 256, 512>(part, fp8_tile_kernel<8, 4, 2, 4, false, false, 1>, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 grid((unsigned)((M * (N / 8) + 255) / 256)), block(256);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, p, static_cast<const float*>(ws)); };
  if (out_dt == 0) go(split_reduce_kernel<0, Fp8Args>);
  else if (out_dt == 1) go(split_reduce_kernel<1, Fp8Args>);
  else go(split_reduce_kernel<2, Fp8Args>);
  return hipGetLastError();
}

// What the grouped product runs as: rows streamed (0), or the tile.
static int plan_grouped(int64_t E, int64_t R, int64_t N) {
  // by the average rows of an expert (64 experts of 2048 x 7168): 4 rows 157 us streamed, 159 in 128-row tiles; 8 rows
  // 184 and 163; 96 rows 203 in 128-row tiles, 202 in 256-row ones; 128 rows 280 and 237
  if (R <= 4 * E) return 0;
  // few tiles: the smaller ones reach more CUs (4 experts, 2000 rows, 512 x 4096: 26 us, 52 in 256-row tiles; about 144
  // tiles 38 and 56, about 160 109 and 98); 128 columns: 16384 rows 28 us, 52 in 256-wide tiles
  const int64_t c256 = (N + 255) / 256, c128 = (N + 127) / 128;
  if (R <= 96 * E || (R / 256 + E / 2) * c256 < 160 || !wide_pays(2 * c256, 4 * c128)) return 128;
  return 256;
}

// Blocks of a grouped launch with BM x BN tiles: no segment's last tile is
// shared, so at most one more than the full ones for each expert with rows;
// a multiple of 8.
int64_t grouped_blocks(int64_t E, int64_t R, int64_t N, int64_t BM, int64_t BN) {
  return ((R / BM + (E < R ? E : R)) * ((N + BN - 1) / BN) + 7) / 8 * 8;
}

int64_t fp8_block_grouped_threads(int64_t E, int64_t R, int64_t N) {
  if (R == 0 || N == 0 || E == 0) return 0;
  const int tile = plan_grouped(E, R, N);
  if (tile == 0) return fp8_stream_threads(0, N, E, R);
  return grouped_blocks(E, R, N, tile, tile) * (tile == 128 ? 256 : 512);
}

hipError_t launch_fp8_block_grouped(const void* a, const float* a_scale, const int32_t* row_token,
                                    const int32_t* offsets, int64_t E, const void* w, const float* w_scale, void* out,
                                    int out_dt, int64_t T, int64_t R, int64_t N, int64_t K, hipStream_t stream) {
  if (R == 0 || N == 0 || E == 0) return hipSuccess;
  Fp8Args p{};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scale = a_scale;
  p.row_token = row_token;
  p.offsets = offsets;
  p.w = static_cast<const uint8_t*>(w);
  p.w_scale = w_scale;
  p.out = out;
  p.M = T;
  p.R = R;
  p.E = (int)E;
  p.N = (int)N;
  p.K = (int)K;
  p.KB = (int)((K + 127) / 128);
  p.NBLK = (int)((N + 127) / 128);
  p.splits = 1;
  const int tile = plan_grouped(E, R, N);
  if (tile == 0) return launch_fp8_stream(p, out_dt, stream);
  if (tile == 128)
    return out_dt == 0 ? grouped_go<128, 128, 256>(p, fp8_tile_kernel<4, 4, 2, 2, true, false, 0>, stream)
                       : grouped_go<128, 128, 256>(p, fp8_tile_kernel<4, 4, 2, 2, true, false, 1>, stream);
  return out_dt == 0 ? grouped_go<256, 256, 512>(p, fp8_tile_kernel<8, 4, 2, 4, true, false, 0>, stream)
                     : grouped_go<256, 256, 512>(p, fp8_tile_kernel<8, 4, 2, 4, true, false, 1>, stream);
}

}  // namespace w4
