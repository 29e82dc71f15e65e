// MXFP4 matrix products: dense, and grouped over the row segments of routed
// experts.
//
//   out[r, n] = sum_b 2^(ea[t, b] + ew[n, b]) * sum_{k in block b} a[t, k] * w[n, k]  (+ bias[n])
//
// over the blocks b of 32 columns, with t = r, or the row's token in the
// grouped form. v_mfma_scale_f32_32x32x64_f8f6f4 takes both blocks' powers of
// two with its operands, so its fp32 accumulators need no other arithmetic
// (measured: 4e-8 of the absolute sum off over 128 columns, as fp32's own sums;
// the 16x16x128 form runs at half its rate).
//
// Tile kernel: WM x WN waves, each with a tile of 32 MI rows x 32 NJ columns,
// K in steps of 256 (128 bytes of a row).
// - Both operands pass through LDS in two stages, by LDS DMA (an asm statement:
//   with the builtin the compiler waits for all of it before the next LDS read).
// - The matrix unit reads, from lane (row, half h), 16 bytes = one block of 32
//   columns. MFMA c of a step takes the blocks c (h = 0) and 4 + c (h = 1), so
//   a lane's four scales of a step are one word of LDS, byte c of it MFMA c's.
// - A step is four groups of MFMAs, one per c. Under group 0 the fragments of the
//   other three are read; a barrier, and the stage is free: the DMA two steps
//   ahead goes out under group 1. A second barrier before group 3, by which the
//   next step's tiles have landed; its first fragments are read under group 3.
//   (With the last group behind the barrier that ends the step, in the compiler's
//   order, the 256 x 256 tile took 192 us for 4096 x 14336 x 4096; so 154.)
// - The weights are the A operand and the activations the B operand: a lane's
//   results lie in one activation row. Row q of a weight fragment is its column
//   16 (q / 4 % 2) + 4 (q / 8) + q % 4, which gives a lane 16 consecutive ones.
// - Results leave through LDS as whole rows: straight from the registers a store
//   would be half a cache line of each of 32 rows (154 us, 151 so).
// What bounds it: 4096 x 14336 x 4096 takes 146 us, 3.3 PFLOP/s, K = 16384 reaches
// 4.1, where the fp4 matrix rate alone is 8.4. At K = 4096 the clock is 2.0 GHz, as in a
// loop of the matrix instruction alone, and 39% of the SIMDs' cycles are MFMA: what is
// lost are stores, rounds and the loop's waits. Each round of tiles ends in a
// burst of stores that memory takes 7 us for and nothing overlaps (about 30 of the
// 146 us, from the times of K = 512 to 16384), and 896 tiles are 3.5 rounds of 256 CUs.
// Within the loop a step of 256 columns takes 1.8 us; without its DMA 1.4, with a quarter
// of its MFMAs 1.1. Only at K = 16384 the power limit holds the clock near 1.6 GHz and
// the step takes 2.1 us.
#include <cmath>
#include <type_traits>

#include "mxfp4.h"

namespace w4 {

constexpr int kMK = 256;                             // columns per step
constexpr int kMB = kMK / 2;                         // bytes of a row per step

__device__ __forceinline__ v8i mx_operand(v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <int C>
__device__ __forceinline__ v16f mx_mfma(v4i w, v4i a, v16f d, int sw, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(w), mx_operand(a), d, 4, 4, C, sw, C, sa);
}

// Two results as bf16 (OUT 0) or fp16, nearest even.
template <int OUT>
__device__ __forceinline__ int pack16(float x, float y) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  if constexpr (OUT == 0) return __builtin_bit_cast(int, __builtin_convertvector(v2f{x, y}, v2bf));
  else return __builtin_bit_cast(int, __builtin_convertvector(v2f{x, y}, v2h));
}

// Two words at a uniform address, through the scalar cache: the vector memory counter stays the DMAs' own.
__device__ __forceinline__ v2i scalar_load2(const int32_t* at) {
  v2i r;
  asm volatile("s_load_dwordx2 %0, %1, 0x0\n\ts_waitcnt lgkmcnt(0)" : "=&s"(r) : "s"(at) : "memory");
  return r;
}

// OUT: 0 bf16, 1 fp16, 2 fp32.
template <int WM, int WN, int MI, int NJ, bool GROUPED, int OUT>
__global__ __launch_bounds__(64 * WM * WN, MI * NJ > 4 ? 1 : 2) void mx_tile_kernel(MxArgs p) {
  constexpr int NW = WM * WN, TH = 64 * NW, BM = 32 * MI * WM, BN = 32 * NJ * WN;
  // Grouped tiles of 192 and 256 rows: one block per CU takes its XCD's items in turn, and fetches an item's first step while the last
  // one's results leave (1024 tokens x 8 of 64 experts, 7168 x 2048: 174 us with a block per item, 160 so; 8192 tokens, 2048 x
  // 7168: 593 and 592). The dense tile has no registers left for that.
  constexpr bool STAY = GROUPED && MI * NJ > 4;
  constexpr int RA = BM * 8 / TH, RB = BN * 8 / TH;  // LDS DMAs of codes per thread and step
  constexpr int RS = ((BM + BN) / 64 + NW - 1) / NW; // of scales, every second step
  static_assert(BM % 64 == 0 && BN % 64 == 0, "a wave fetches scales of activations or of weights");
  static_assert(RA * TH == BM * 8 && RB * TH == BN * 8, "whole DMAs");
  constexpr int STAGE = (BM + BN) * kMB, SCALES = (BM + BN) * 16;
  // two stages (activation rows, then weight rows), two chunks of the scales of 2 steps (16 bytes per row)
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * STAGE + 2 * SCALES];

  // ---- work item
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int h = lane >> 5, l32 = lane & 31;
  int e = 0, tn, mt = 0, split = 0;                  // mt: grouped: within the expert's rows
  int length = 0, more = 0;                          // of the expert's segment; work items after this one
  int64_t r0, row_end, out0 = 0;                     // first row and end of this tile's rows (segment-local if grouped)
  if constexpr (GROUPED) {
    const Segment s = find_segment<BM>(p);
    if (s.e < 0) return;
    e = __builtin_amdgcn_readfirstlane(s.e);
    tn = __builtin_amdgcn_readfirstlane(s.tn);
    mt = __builtin_amdgcn_readfirstlane(s.mt);
    out0 = __builtin_amdgcn_readfirstlane((int)s.row0);
    row_end = __builtin_amdgcn_readfirstlane((int)s.rows);
    if constexpr (STAY) {
      const v2i o = scalar_load2(p.offsets + e);
      length = o[1] - o[0];
      more = __builtin_amdgcn_readfirstlane(s.left) / (int)(gridDim.x / 8);
    }
  } else {
    const int t = xcd_remap((int)blockIdx.x, (int)gridDim.x), tiles = (int)p.tiles;   // below 2^24
    split = t / tiles;
    const int tile = t - split * tiles;
    // four row tiles at a time, column by column: the tiles that an XCD holds at once share rows and columns
    const int MT = tiles / p.NT, grp = tile / (4 * p.NT);
    const int rows = min(4, MT - 4 * grp), in = tile - grp * 4 * p.NT;
    mt = 4 * grp + in % rows;
    tn = in / rows;
    row_end = p.M;
  }
  r0 = (int64_t)mt * BM;
  const int k0 = p.KT * split / p.splits, k1 = p.KT * (split + 1) / p.splits;   // KT at most 2^14, splits 2^9
  const int64_t KH = p.K >> 1;                       // code bytes of a row

  // ---- LDS DMA: a wave's load fills 8 rows (one KiB), lane L at row L / 8, physical 16-byte chunk L % 8. Row r holds logical
  // chunk c at physical chunk c ^ f(r), so that the 16 rows that a read touches at a time fill two rows' width of banks.
  // f repeats every TH / 8 rows. Rows past the end lie past the buffer, which reads as zero; so do gathered rows without a
  // token, and chunks past K, by an offset of their own. (The scalar part of an address never passes the buffer's size.)
  const int lrow = lane >> 3, lchunk = lane & 7;
  const bool gather = GROUPED && p.row_token;
  __amdgpu_buffer_rsrc_t arsrc, asr, wrsrc, wsr;
  const int drow = 8 * wave + lrow;                  // + TH / 8 per load
  const int ca = lchunk ^ ((drow >> 1) & 7), cb = lchunk ^ (((drow >> 1) & 3) + 4 * ((drow >> 4) & 1));
  static_assert(TH / 8 % 32 == 0, "f repeats");
  const uint32_t KHu = (uint32_t)KH;
  const int klast = p.K - (p.KT - 1) * kMK;          // columns of the last step
  const bool a_dead = 32 * ca >= klast, b_dead = 32 * cb >= klast;   // the lane's chunk lies past K there
  uint32_t a_off[RA], b_off[RB], s_off[RS];
#pragma unroll
  for (int i = 0; i < RB; ++i) b_off[i] = (uint32_t)((TH / 8) * i + drow) * KHu + 16 * cb;
  auto open = [&]() __attribute__((always_inline)) {   // the item's buffers and rows
    const int64_t abase = gather ? 0 : out0 + r0;
    const int64_t mine = GROUPED ? min((int64_t)BM, row_end - r0) : (int64_t)BM;
    const int64_t arows = gather ? p.M : min(mine, p.M - abase);
    const int64_t wrow0 = (int64_t)e * p.N + tn * BN;
    const int wrows = min(BN, p.N - tn * BN);
    arsrc = make_rsrc(p.a + abase * KH, (uint32_t)max(arows * KH, (int64_t)0));
    asr = make_rsrc(p.a_scale + abase * p.KS, (uint32_t)max(arows * p.KS, (int64_t)0));
    wrsrc = make_rsrc(p.w + wrow0 * KH, (uint32_t)(wrows * KH));
    wsr = make_rsrc(p.w_scale + wrow0 * p.KS, (uint32_t)((int64_t)wrows * p.KS));
    // gathered: activation row of tile row r; -1: none (no branch: all rows' loads are on their way together)
    const int trows = (int)min((int64_t)BM, row_end - r0);
    const __amdgpu_buffer_rsrc_t trs = make_rsrc(p.row_token + out0 + r0, (uint32_t)max(trows, 0) * 4);
    auto token = [&](int r) -> int {
      const int t = __builtin_amdgcn_raw_buffer_load_b32(trs, 4 * r, 0, 0);
      return r < trows && (unsigned)t < (uint64_t)p.M ? t : -1;
    };
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const int t = gather ? token((TH / 8) * i + drow) : (TH / 8) * i + drow;
      a_off[i] = t >= 0 ? (uint32_t)t * KHu + 16 * ca : kPast;
    }
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      const int r = 64 * (NW * i + wave) + lane;     // activation rows, then weight rows
      const int t = 64 * (NW * i + wave) >= BM ? r - BM : (gather ? token(r) : r);
      s_off[i] = t >= 0 ? (uint32_t)t * (uint32_t)p.KS : kPast;
    }
  };
  open();
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t ldsw = __builtin_amdgcn_readfirstlane(lds0 + 8 * wave * kMB);
  // m0 holds the LDS address. The compiler keeps nothing in it here, and a clobber of a reserved register is not honoured.
  auto dma = [&](const __amdgpu_buffer_rsrc_t rs, uint32_t dst, uint32_t off, uint32_t ks) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(dst), "v"(off), "s"(rs), "s"(ks) : "memory");
  };
  // DMA q of a step: the activations' RA, the weights' RB, then with every second step the scales' RS (of steps past K:
  // whatever follows, not used). Steps past the split's end read no memory.
  constexpr int ND = RA + RB + RS;
  auto gload1 = [&](int tk, uint32_t stage, int q) __attribute__((always_inline)) {
    if (q >= RA + RB) {
      const int i = q - RA - RB;
      const int grp = NW * i + wave;                 // 64 rows
      if (64 * grp >= BM + BN) return;
      const uint32_t dst = lds0 + 2 * STAGE + (((tk - k0) >> 1) & 1) * SCALES + 1024 * grp;
      const uint32_t off = tk < k1 ? s_off[i] : kPast, ks = tk < k1 ? (uint32_t)tk * 8 : 0u;
      if (64 * grp < BM) dma(asr, dst, off, ks);
      else dma(wsr, dst, off, ks);
      return;
    }
    const uint32_t ks = tk < k1 ? (uint32_t)tk * kMB : 0u;
    const bool last = tk == p.KT - 1;
    if (q < RA) dma(arsrc, ldsw + stage + (TH / 8) * q * kMB, tk >= k1 || (last && a_dead) ? kPast : a_off[q], ks);
    else dma(wrsrc, ldsw + stage + (BM + (TH / 8) * (q - RA)) * kMB, tk >= k1 || (last && b_dead) ? kPast : b_off[q - RA], ks);
  };

  // the accumulators start from the bias, of 16 consecutive columns each (without one an empty buffer, which reads as zero).
  // One of 16-bit values may begin in the middle of a word: whole words are loaded, from there on, and shifted.
  constexpr int SZ = OUT == 2 ? 4 : 2;               // bytes of a result
  v4i bias[NJ][SZ];
  if constexpr (!GROUPED) {
    const uint32_t odd = (uint32_t)(uintptr_t)p.bias & 2;
    const __amdgpu_buffer_rsrc_t brs = make_rsrc(static_cast<const uint8_t*>(p.bias) - odd,
                                                 p.bias && p.splits == 1 ? (uint32_t)p.N * SZ + 2 * odd : 0u);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint32_t at = (uint32_t)(tn * BN + 32 * (NJ * wn + j) + 16 * h) * SZ;
#pragma unroll
      for (int q = 0; q < SZ; ++q) bias[j][q] = buffer_load16(brs, at + 16 * q);
      if constexpr (OUT != 2) {
        const int next = __builtin_amdgcn_raw_buffer_load_b32(brs, at + 32, 0, 0);
#pragma unroll
        for (int d = 0; d < 8; ++d)
          bias[j][d / 4][d % 4] = (int)__builtin_amdgcn_alignbyte((uint32_t)(d < 7 ? bias[j][(d + 1) / 4][(d + 1) % 4] : next),
                                                                  (uint32_t)bias[j][d / 4][d % 4], odd);
      }
    }
  }

  // ---- fragments
  const int ar = 32 * MI * wm + l32;                 // + 32 i, which leaves f unchanged
  const int br = 32 * NJ * wn + 16 * ((l32 >> 2) & 1) + 4 * (l32 >> 3) + (l32 & 3);   // + 32 j, likewise
  const int af7 = (l32 >> 1) & 7, bf7 = ((br >> 1) & 3) + 4 * ((br >> 4) & 1);
  auto afrag = [&](uint32_t stage, int i, int c) -> v4i {
    return *reinterpret_cast<const v4i*>(lds + stage + (ar + 32 * i) * kMB + 16 * ((4 * h + c) ^ af7));
  };
  auto bfrag = [&](uint32_t stage, int j, int c) -> v4i {
    return *reinterpret_cast<const v4i*>(lds + stage + (BM + br + 32 * j) * kMB + 16 * ((4 * h + c) ^ bf7));
  };
  // the four scales of a step; blocks past K (of the row's padding, or of the next row) are none
  int smask = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (32 * (4 * h + c) < klast) smask |= 0xFF << (8 * c);
  auto scale = [&](int tk, int row) -> int {
    const int rel = tk - k0;
    const uint8_t* q = lds + 2 * STAGE + ((rel >> 1) & 1) * SCALES + row * 16 + 8 * (rel & 1) + 4 * h;
    return *reinterpret_cast<const int*>(q) & (tk < k1 ? (tk == p.KT - 1 ? smask : -1) : 0);
  };

  constexpr int NM = MI * NJ;
  if (k0 < k1) {
#pragma unroll
    for (int q = 0; q < ND; ++q) gload1(k0, 0, q);
  }
  for (;;) {                                         // a work item; its first step is on its way
    v16f acc[MI][NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v16f f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if constexpr (GROUPED) f[c] = 0.f;
        else if constexpr (OUT == 2) f[c] = __int_as_float(bias[j][c / 4][c % 4]);
        else {
          const uint16_t b = (uint16_t)((uint32_t)bias[j][c / 8][c % 8 / 2] >> (16 * (c % 2)));
          f[c] = OUT == 0 ? bf16_to_f32(b) : f16_to_f32(b);
        }
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i][j] = f;
    }
    const bool idle = GROUPED && r0 + 32 * MI * wm >= row_end;   // a wave whose rows all lie past the segment only fetches
    if (k0 < k1) {
      asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
      for (int q = 0; q < RA + RB; ++q) gload1(k0 + 1, STAGE, q);
      if (idle) {
        for (int tk = k0; tk < k1 + ((k1 - k0) & 1); ++tk) {   // as many barriers as the others
          asm volatile("s_barrier" ::: "memory");
          const bool odd = (tk - k0) & 1;
#pragma unroll
          for (int q = 0; q < ND; ++q)
            if (q < RA + RB || !odd) gload1(tk + 2, odd * STAGE, q);
          asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"(RA + RB) : "memory");
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      } else {
        v4i af[4][MI], bf[4][NJ];
        int sa[2][MI], sb[2][NJ];                        // by the step's parity
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          af[0][i] = afrag(0, i, 0);
          sa[0][i] = scale(k0, ar + 32 * i);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          bf[0][j] = bfrag(0, j, 0);
          sb[0][j] = scale(k0, BM + br + 32 * j);
        }
        // One step; P: its parity, and so its stage. No branch inside, and every MFMA is pinned where it stands (the empty
        // statement names its result): left alone the compiler sinks all 64 behind the barrier and reads every fragment first.
        auto step = [&](auto parity, int tk) __attribute__((always_inline)) {
          constexpr int P = decltype(parity)::value;
          constexpr uint32_t st = P * STAGE;
          constexpr int NF = MI + NJ;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c == 1) {
              // every fragment of this step is in every wave's registers: its stage is free
              asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
              __builtin_amdgcn_sched_barrier(0);
            }
            if (c == 3) {
              // the next step's tiles have landed (what was issued since is the step after's)
              asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier"
                           :: "n"(RA + RB + (P == 0 && NW * 64 * RS == BM + BN ? RS : 0)) : "memory");
              __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int n = 0; n < NM; ++n) {
              const int i = n / NJ, j = n % NJ;
              if (c == 0) {                              // groups 1 to 3's fragments
#pragma unroll
                for (int q = n * 3 * NF / NM; q < (n + 1) * 3 * NF / NM; ++q) {
                  if (q % NF < NJ) bf[1 + q / NF][q % NF] = bfrag(st, q % NF, 1 + q / NF);
                  else af[1 + q / NF][q % NF - NJ] = afrag(st, q % NF - NJ, 1 + q / NF);
                }
              }
              if (c == 3) {                          // the next step's group 0 (at the end: of a stage that is not used)
#pragma unroll
                for (int q = n * NF / NM; q < (n + 1) * NF / NM; ++q) {
                  if (q < NJ) {
                    bf[0][q] = bfrag(STAGE - st, q, 0);
                    sb[1 - P][q] = scale(tk + 1, BM + br + 32 * q);
                  } else {
                    af[0][q - NJ] = afrag(STAGE - st, q - NJ, 0);
                    sa[1 - P][q - NJ] = scale(tk + 1, ar + 32 * (q - NJ));
                  }
                }
              }
              if (c == 0) acc[i][j] = mx_mfma<0>(bf[0][j], af[0][i], acc[i][j], sb[P][j], sa[P][i]);
              if (c == 1) acc[i][j] = mx_mfma<1>(bf[1][j], af[1][i], acc[i][j], sb[P][j], sa[P][i]);
              if (c == 2) acc[i][j] = mx_mfma<2>(bf[2][j], af[2][i], acc[i][j], sb[P][j], sa[P][i]);
              if (c == 3) acc[i][j] = mx_mfma<3>(bf[3][j], af[3][i], acc[i][j], sb[P][j], sa[P][i]);
              asm volatile("" : "+a"(acc[i][j]));
              if (c == 1) {
                constexpr int NDP = P == 0 ? ND : RA + RB;
#pragma unroll
                for (int q = n * NDP / NM; q < (n + 1) * NDP / NM; ++q) gload1(tk + 2, st, q);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        };
        for (int tk = k0; tk < k1; tk += 2) {            // an odd number's last step adds zeros
          step(std::integral_constant<int, 0>{}, tk);
          step(std::integral_constant<int, 1>{}, tk + 1);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
    }

    // ---- output. A lane's results are 16 columns of one row, which as stores would be half a cache line from each of 32
    // rows; 32 rows at a time go through the wave's own LDS and leave as whole rows. Chunk c (16 bytes) of row r lies at c ^
    // f(r), so that 16 lanes that write one chunk of 16 rows, or read 16 of a row, fill the banks.
    constexpr int CH = 32 * NJ * SZ / 16, PER = 16 / SZ;   // chunks of a row, columns of a chunk
    constexpr uint32_t ROWS = STAY ? STAGE : 0;        // where: the first stage takes the next item's first step
    static_assert(CH >= 8 && ROWS + NW * 32 * CH * 16 <= 2 * STAGE, "the waves' rows fit the stages");
    auto swizzle = [](int r) { return CH == 8 ? (r >> 1) & 7 : r & 15; };
    __syncthreads();                                   // no wave's tiles are on their way any more
    uint8_t* mine = lds + ROWS + wave * (32 * CH * 16);
    const int nw = tn * BN + 32 * NJ * wn;
    const int col = nw + PER * (lane % CH), row = lane / CH;
    constexpr int RPI = 64 / CH;                       // rows of a store
    const int left = col < p.N ? (int)min((int64_t)BM, row_end - r0) : 0;
    const int64_t row0 = out0 + r0 + (int64_t)split * p.M;
    const bool last = !STAY || more == 0;
    if constexpr (STAY) {
      if (!last) {                                   // the next item; its first step comes while this one's results leave
        --more;
        tn += (int)(gridDim.x / 8);
        while (tn >= p.NT) {
          tn -= p.NT;
          ++mt;
          while (mt * BM >= length && e + 1 < p.E) {
            ++e;
            mt = 0;
            const v2i o = scalar_load2(p.offsets + e);
            out0 = o[0];
            length = o[1] - o[0];
            row_end = min((int64_t)length, p.R - out0);
          }
        }
        r0 = (int64_t)mt * BM;
        open();
#pragma unroll
        for (int q = 0; q < ND; ++q) gload1(k0, 0, q);
      }
    }
    if (!idle) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
          for (int q = 0; q < SZ; ++q) {                 // SZ chunks of the lane's 16 columns
            v4i w;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if constexpr (OUT == 2) w[c] = __float_as_int(acc[i][j][4 * q + c]);
              else w[c] = pack16<OUT>(acc[i][j][8 * q + 2 * c], acc[i][j][8 * q + 2 * c + 1]);
            }
            *reinterpret_cast<v4i*>(mine + (l32 * CH + ((2 * j + h) * SZ + q ^ swizzle(l32))) * 16) = w;
          }
        }
        const int first = 32 * (MI * wm + i) + row;      // of the tile's rows
        uint8_t* o = static_cast<uint8_t*>(p.out) + ((row0 + first) * p.N + col) * SZ;
#pragma unroll
        for (int k = 0; k < 32 / RPI; ++k) {
          const int rr = row + RPI * k;
          const v4i w = *reinterpret_cast<const v4i*>(mine + (rr * CH + (lane % CH ^ swizzle(rr))) * 16);
          if (first + RPI * k < left) *reinterpret_cast<v4i*>(o) = w;
          o += (int64_t)RPI * p.N * SZ;
        }
      }
    }
    if (last) break;
  }
}

// What the dense product runs as: rows streamed (tile 0), or a tile and its K splits.
struct MxPlan {
  int tile, splits;
};

// Streaming reads the weights once per 16 rows, mostly from L2, and needs no second launch: 64 rows of 4096 x 4096 7.1 us
// (tiles 10.2), of 4096 x 14336 12.7 (13.4), of 14336 x 4096 11.8 (10.6). Above that the cheapest by a model of what was
// measured: a launch, steps of 256 columns (slower where two blocks share a CU), and for splits a second launch that adds
// the parts. It comes within 20% of the measured times from 65 to 1024 rows of the sizes above, of 1024 x 4096 and of
// 7168 x 2048, and takes the fastest plan or one within 5% of it. For instance 128 rows of 14336 x 4096: 11.8 us in tiles of
// 64 x 128, 13.7 of 128 x 128, 28 of 256 x 256; 200 rows of 4096 x 14336: 20.3 in 4 splits of 128 x 128, 22.2 in 4 of 64 x
// 128, 76 in tiles of 256 x 256; 1024 rows of 14336 x 4096: 37.9 in tiles of 256 x 256, 45.2 of 128 x 128.
static MxPlan plan_dense(int64_t M, int64_t N, int64_t K) {
  if (M <= 64) return {0, 1};
  struct Form {
    int64_t bm, bn, launch, step, shared;            // ns; shared: a step where two blocks share a CU (0: they cannot)
  };
  constexpr Form forms[] = {{64, 128, 4000, 450, 800}, {128, 128, 4000, 650, 1300}, {256, 256, 6000, 1500, 0}};
  const int64_t KT = (K + kMK - 1) / kMK;
  MxPlan best{0, 1};
  int64_t least = INT64_MAX;
  for (const Form& f : forms) {
    const int64_t t = ((M + f.bm - 1) / f.bm) * ((N + f.bn - 1) / f.bn), slots = f.shared ? 512 : 256;
    for (int64_t s = 1; s == 1 || (f.shared && s * t <= slots && 2 * s <= KT); ++s) {
      const int64_t step = s * t <= 256 || !f.shared ? f.step : f.shared;
      const int64_t cost = f.launch + step * ((KT + s - 1) / s) * ((s * t + slots - 1) / slots) +
                           (s > 1 ? 4500 + s * M * N / 1000 : 0);
      if (cost < least) {
        least = cost;
        best = {(int)f.bm, (int)s};
      }
    }
  }
  return best;
}

size_t mx_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const MxPlan pl = plan_dense(M, N, K);
  return pl.splits > 1 ? (size_t)pl.splits * (size_t)M * (size_t)N * 4 : 0;
}

// Threads of the largest launch of a product, for the host's check against a launch's limit.
int64_t mx_gemm_threads(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const MxPlan pl = plan_dense(M, N, K);
  if (pl.tile == 0) return mx_stream_threads(M, N, 0, 0);
  const int64_t bm = pl.tile, bn = pl.tile == 256 ? 256 : 128;
  const int64_t reduce = pl.splits > 1 ? M * (N / 8) : 0, product = (M + bm - 1) / bm * ((N + bn - 1) / bn) * pl.splits * 256;
  return product > reduce ? product : reduce;
}

// Whether the linear layer's product quantizes the rows itself, every block all of them, instead of a launch before it: the
// more the blocks, the fewer. With weights from memory, us (two launches): 16 x 256 x 4096 7.2 (7.1); 12 x 4096 x 4096 8.6
// (9.1), 14 rows 9.0 (9.2), 16 rows 9.3 (9.1); 8 x 4096 x 7168 11.7 (12.1); 4 x 4096 x 14336 19.1 (19.2); 8 x 8192 x 4096
// 9.2 (10.0), 12 rows 10.3 (10.0); 8 x 14336 x 4096 10.8 (11.1); 4 x 28672 x 4096 16.4 (18.0), 8 rows 20.5 (18.0).
bool mx_inline(int64_t M, int64_t N, int64_t K) {
  return M <= 16 && M * K <= (N <= 512 ? 65536 : N <= 4096 ? 57344 : N <= 8192 ? 40960 : N <= 16384 ? 32768 : 16384);
}

template <int BM, int BN, typename F>
static hipError_t tile_go(MxArgs p, F kernel, hipStream_t stream) {
  p.NT = (p.N + BN - 1) / BN;
  p.tiles = (p.M + BM - 1) / BM * p.NT;
  int64_t blocks = p.offsets ? grouped_blocks(p.E, p.R, p.N, BM, BN) : p.tiles * p.splits;
  if (p.offsets && BM > 128) blocks = blocks < 256 ? blocks : 256;   // they stay
  const dim3 grid((unsigned)blocks), block(256);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, p);
  return hipGetLastError();
}

template <int WM, int WN, int MI, int NJ>
static hipError_t dense_go(const MxArgs& p, int out_dt, hipStream_t stream) {
  auto go = [&](auto kernel) { return tile_go<32 * MI * WM, 32 * NJ * WN>(p, kernel, stream); };
  if (out_dt == 0) return go(mx_tile_kernel<WM, WN, MI, NJ, false, 0>);
  if (out_dt == 1) return go(mx_tile_kernel<WM, WN, MI, NJ, false, 1>);
  return go(mx_tile_kernel<WM, WN, MI, NJ, false, 2>);
}

static MxArgs mx_args(const void* a, const void* a_scale, const void* w, const void* w_scale, void* out, int64_t M,
                      int64_t N, int64_t K) {
  MxArgs p{};
  p.a = static_cast<const uint8_t*>(a);
  p.a_scale = static_cast<const uint8_t*>(a_scale);
  p.w = static_cast<const uint8_t*>(w);
  p.w_scale = static_cast<const uint8_t*>(w_scale);
  p.out = out;
  p.M = p.R = M;
  p.E = 1;
  p.N = (int)N;
  p.K = (int)K;
  p.KS = (int)mx_scale_bytes(K);
  p.KT = (int)((K + kMK - 1) / kMK);
  p.splits = 1;
  return p;
}

// Few rows of 16-bit activations, quantized on the way (a: bf16 or fp16 [M, K]).
hipError_t launch_mx_linear_few(const void* x, bool bf16, const void* w, const void* w_scale, const void* bias, void* out,
                                int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  MxArgs p = mx_args(x, nullptr, w, w_scale, out, M, N, K);
  p.bias = bias;
  return launch_mx_stream(p, bf16 ? 1 : 2, bf16 ? 0 : 1, stream);
}

hipError_t launch_mx_gemm(const void* a, const void* a_scale, const void* w, const void* w_scale, const void* bias,
                          void* out, int out_dt, int64_t M, int64_t N, int64_t K, void* ws, hipStream_t stream) {
  if (M == 0 || N == 0) return hipSuccess;
  MxArgs p = mx_args(a, a_scale, w, w_scale, out, M, N, K);
  p.bias = bias;
  const MxPlan pl = plan_dense(M, N, K);
  p.splits = pl.splits;
  if (pl.tile == 0) return launch_mx_stream(p, 0, out_dt, stream);
  MxArgs part = p;
  if (p.splits > 1) part.out = ws;
  const int dt = p.splits > 1 ? 2 : out_dt;
  hipError_t e;
  if (pl.tile == 64) e = dense_go<2, 2, 1, 2>(part, dt, stream);
  else if (pl.tile == 128) e = dense_go<2, 2, 2, 2>(part, dt, stream);
  else e = dense_go<2, 2, 4, 4>(part, dt, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 grid((unsigned)((M * (N / 8) + 255) / 256)), block(256);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, p, static_cast<const float*>(ws)); };
  if (out_dt == 0) go(split_reduce_kernel<0, MxArgs>);
  else if (out_dt == 1) go(split_reduce_kernel<1, MxArgs>);
  else go(split_reduce_kernel<2, MxArgs>);
  return hipGetLastError();
}

// Row tiles of bm that an expert takes, if its rows spread about their mean as by chance.
static double tiles_of(double mean, int bm) {
  double t = 1.0;
  for (int j = 1; j * bm < mean + 4.0 * std::sqrt(mean); ++j) t += 0.5 * std::erfc((j * bm - mean) / std::sqrt(2.0 * mean));
  return t;
}

// What the grouped product runs as: rows streamed (0), or the tile's rows. By rows per expert; measured with 64 experts of
// 4096 x 7168 (us): 4 rows 162 streamed, 168 in tiles of 64 x 128, 176 of 128 x 128; 16 rows 224, 182 and 187; 48 rows 211 and
// 202, 199 of 192 x 256; 96 rows (-), 229, 222, and 235 of 256 x 256; 128 rows (-), 289, 240 and 263; 256 rows (-), 456, 433
// and 394; 320 rows (-), 545, 455 and 513. Of 7168 x 2048, whose K leaves a streaming wave two steps, tiles win from the
// start (4 rows 104, 96 and 100) and those of 128 up to 112 rows (138, of 192 147). A tile of 192 rows costs about 0.87 of one
// of 256. Few of the larger tiles would leave CUs idle, or their last column tile be mostly empty.
static int plan_grouped(int64_t E, int64_t R, int64_t N, int64_t K) {
  if (R <= 8 * E && K >= 4096) return 0;
  if (R <= 32 * E) return 64;
  const int64_t c256 = (N + 255) / 256, c128 = (N + 127) / 128;
  if (R <= (K < 6144 ? 104 : 48) * E || (R / 256 + E / 2) * c256 < 160 || 3 * 2 * c256 > 4 * c128) return 128;
  const double mean = (double)R / (double)E;
  return mean <= 2048 && 0.87 * tiles_of(mean, 192) < tiles_of(mean, 256) ? 192 : 256;
}

int64_t mx_grouped_threads(int64_t E, int64_t R, int64_t N, int64_t K) {
  if (R == 0 || N == 0 || E == 0) return 0;
  const int tile = plan_grouped(E, R, N, K);
  if (tile == 0) return mx_stream_threads(0, N, E, R);
  return grouped_blocks(E, R, N, tile, tile > 128 ? 256 : 128) * 256;
}

hipError_t launch_mx_grouped(const void* a, const void* a_scale, const int32_t* row_token, const int32_t* offsets,
                             int64_t E, const void* w, const void* w_scale, void* out, int out_dt, int64_t T, int64_t R,
                             int64_t N, int64_t K, hipStream_t stream) {
  if (R == 0 || N == 0 || E == 0) return hipSuccess;
  MxArgs p = mx_args(a, a_scale, w, w_scale, out, T, N, K);
  p.row_token = row_token;
  p.offsets = offsets;
  p.R = R;
  p.E = (int)E;
  const int tile = plan_grouped(E, R, N, K);
  if (tile == 0) return launch_mx_stream(p, 0, out_dt, stream);
  if (tile == 64)
    return out_dt == 0 ? tile_go<64, 128>(p, mx_tile_kernel<2, 2, 1, 2, true, 0>, stream)
                       : tile_go<64, 128>(p, mx_tile_kernel<2, 2, 1, 2, true, 1>, stream);
  if (tile == 128)
    return out_dt == 0 ? tile_go<128, 128>(p, mx_tile_kernel<2, 2, 2, 2, true, 0>, stream)
                       : tile_go<128, 128>(p, mx_tile_kernel<2, 2, 2, 2, true, 1>, stream);
  if (tile == 192)
    return out_dt == 0 ? tile_go<192, 256>(p, mx_tile_kernel<2, 2, 3, 4, true, 0>, stream)
                       : tile_go<192, 256>(p, mx_tile_kernel<2, 2, 3, 4, true, 1>, stream);
  return out_dt == 0 ? tile_go<256, 256>(p, mx_tile_kernel<2, 2, 4, 4, true, 0>, stream)
                     : tile_go<256, 256>(p, mx_tile_kernel<2, 2, 4, 4, true, 1>, stream);
}

}  // namespace w4
