// The whole routed-expert layer for a few tokens (T <= 32), weights only
// quantized: router logits and hidden rows in, the experts' weighted sum out.
//
//   out[t] = sum_j w[t, j] * W2[e] (silu(W1[e] x[t]) * (W3[e] x[t]))  (+ add[t]),  e = ids[t, j]
//
// With so few rows the time is the chosen experts' weights, each read once. Two
// kernels: gate and up products with the activation, then the down products with
// the sum over a token's experts. Up to kInline tokens the first one routes too,
// every block for itself (a wave per token): one token 47 us, where a launch that
// routes takes 7 and the first kernel 42 then; two tokens 50 and 7 + 45. More
// tokens are routed by a block before it.
//
// The plan: pairs (token, expert) are rows, ordered by expert, then token. Tiles
// of at most 8 (gate and up) or 4 or 5 (down) rows of an expert name it, their
// first row and their tokens as bits.
//
// Both kernels stream weights through the matrix unit, 16 weight rows as its A
// operand, a tile's rows as its B operand. Weights become bf16 (exactly, with
// MXFP4's scale applied; v_mfma_f32_16x16x32_bf16), or fp16 for fp16 activations of
// FP8 and int4 weights; FP8's and int4's scales multiply the sums of 128 columns.
//
// What a wave reads passes through LDS of its own (lds_weights.h): rows lie there with their 16-byte chunks permuted by the
// row, so that the reads of 8 rows touch 8 different chunks.
//
// What lies between the two stays fp32: it is held as the sum of three bf16 numbers,
// 8 bits of mantissa each, exactly. The matrix unit takes them in one go: of its 16
// columns the first are a tile's rows' first numbers, the next ones their second and
// third ones, added at the end; hence tiles of at most 5 rows. MXFP4 with fp16
// activations takes x apart in two such numbers, exactly (11 bits).
//
// 64 experts, 8 chosen, 7168 x 2048, kernels only (medians): one token FP8 47 + 23 us
// (5.1 TB/s of weights); two tokens int4 50 + 28; 8 tokens MXFP4 9 + 113 + 62, int4 8 +
// 123 + 68; 32 tokens FP8 15 + 320 + 194, MXFP4 21 + 189 + 143, int4 14 + 199 + 135. What
// bounds them is memory and, with many rows, the activations and the middle, which every
// block reads from L2: with a middle of two bf16 numbers (16 bits) and so tiles of 8 rows
// the down products took 59 us for the 8 tokens of MXFP4, 160 for the 32 of FP8. Tiles of
// 10 rows in two turns on the same weights instead of two tiles of 5 gain 2% there and
// cost as much in smaller layers.
#include <type_traits>

#include "lds_weights.h"
#include "route_token.h"

namespace w4 {

constexpr int kInline = 2;                           // tokens that the first kernel routes itself
constexpr int kInlineE = 256;
constexpr int kInlineRows = kInline * 64;
constexpr int kUpRows = 8, kFewRows = 4, kDownRows = 5;   // most rows of a tile: up, down, down where experts hold many
constexpr int kParts = 3;                            // bf16 numbers of a value of the middle
constexpr int kMaxT = 32, kMaxTopk = 64;             // the host lets no more through
constexpr size_t kLds = 160 * 1024;                  // of a CU

struct MoeTile {
  uint16_t e, row0;
  uint32_t tokens;
};

struct MoeArgs {
  const uint16_t* x;
  const uint8_t *w13, *w2;
  const void *s13, *s2;
  const uint16_t* add;
  uint16_t* out;
  int T, E, topk, H, I;
  int G13, G2;                                       // int4: scale groups along K
  int kg13, kg2;                                     // and steps per group
  int NT;                                            // column tiles of the first kernel
  int inl;                                           // the first kernel routes
  int down_rows;                                     // most rows of a tile of the second
  // workspace
  int32_t* counts;                                   // tiles of the first kernel, of the second
  MoeTile *up, *down;
  float* weights;                                    // of the rows
  uint16_t* mid;                                     // [kParts][R][I]: the middle
  RouteArgs route;
};

// 8 codes of a lane's word w as the matrix unit's operand.
template <bool F16>
struct Operand {
  using V = typename std::conditional<F16, v8h, v8bf>::type;
};

template <bool F16>
__device__ __forceinline__ v4f mfma16(typename Operand<F16>::V a, typename Operand<F16>::V b, v4f c) {
  if constexpr (F16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ int cvt_fp8(int w, float scale, bool high) {
  if constexpr (F16)
    return high ? __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true))
                : __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false));
  else
    return high ? __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))
                : __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false));
}

// Rows of 16-bit activations: a DMA takes kCols columns of 4 (FP8) or 2 rows; row r, chunk c at 2 kCols r + 16 (c ^ (by & 7)),
// by: the row, or the column of the product that it becomes.
template <int FMT>
constexpr int kRowsPerDma = 512 / kCols<FMT>;
template <int FMT>
__device__ __forceinline__ int act_row(int j, int lane) { return j * kRowsPerDma<FMT> + lane / (kCols<FMT> / 8); }
template <int FMT>
__device__ __forceinline__ int act_column(int by, int lane) { return 8 * ((lane & (kCols<FMT> / 8 - 1)) ^ (by & 7)); }
// MFMA c's 8 activations of a lane (of the step's half q: MXFP4 and int4 have 4 MFMAs in each): FP8: columns 64 (c / 2) +
// 16 g + 8 (c % 2) ..; MXFP4: 128 q + 32 g + 8 c ..; int4: 128 q + 32 g + 4 c .. + 3 and 16 after them.
template <int FMT>
__device__ __forceinline__ v4i act_chunk(const uint8_t* at, int row, int by, int chunk) {
  return *reinterpret_cast<const v4i*>(at + 2 * kCols<FMT> * row + 16 * (chunk ^ (by & 7)));
}
template <int FMT>
__device__ __forceinline__ v4i act_piece(const v4i (&X)[4], int c) {
  if constexpr (FMT == kInt4) {
    const v4i a = X[c / 2], b = X[2 + c / 2];
    return c % 2 ? v4i{a[2], a[3], b[2], b[3]} : v4i{a[0], a[1], b[0], b[1]};
  } else {
    return X[c];
  }
}

// 8 weights for MFMA c from a lane's pieces. int4 codes come as the code itself, 0..15 (E4M3's codes 0..15 are 0..15 times
// 2^-9); the sums start from -8 sum x. So a term counts up to 23 steps of the scale in fp32's rounding where a signed code
// counts 8: of two tokens' output the error before its own rounding is 2.1e-7, of FP8's 1.9e-7. (Codes in sign and
// magnitude would take 11 instructions more per word of 8.)
template <int FMT, bool F16>
__device__ __forceinline__ typename Operand<F16>::V decode(const v4i (&w)[2], int q, int c, float scale) {
  v4i r;
  if constexpr (FMT == kFp8) {
    const int lo = w[c / 2][2 * (c % 2)], hi = w[c / 2][2 * (c % 2) + 1];
    r = v4i{cvt_fp8<F16>(lo, 1.0f, false), cvt_fp8<F16>(lo, 1.0f, true), cvt_fp8<F16>(hi, 1.0f, false),
            cvt_fp8<F16>(hi, 1.0f, true)};
  } else if constexpr (FMT == kMx) {
    static_assert(!F16, "its scales need bf16's range");
    const uint32_t v = (uint32_t)w[q][c];
    r = v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0)),
            __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1)),
            __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2)),
            __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3))};
  } else {
    const uint32_t v = (uint32_t)w[q][c] ^ 0x88888888u;
    const int lo = (int)(v & 0x0F0F0F0Fu), hi = (int)((v >> 4) & 0x0F0F0F0Fu);
    r = v4i{cvt_fp8<F16>(lo, 512.0f, false), cvt_fp8<F16>(lo, 512.0f, true), cvt_fp8<F16>(hi, 512.0f, false),
            cvt_fp8<F16>(hi, 512.0f, true)};
  }
  return __builtin_bit_cast(typename Operand<F16>::V, r);
}

__device__ __forceinline__ v8bf bf(v4i v) { return __builtin_bit_cast(v8bf, v); }

// fp16 pairs as the sum of two bf16 numbers each (exact: the upper 8 of 11 bits, and the
// rest; bf16's range is wider): the first of them, or the second. An infinity's
// remainder, a NaN, becomes a finite number, which changes nothing.
__device__ __forceinline__ v4i part_of_f16(v4i x, uint32_t taken) {   // taken: 0, or the upper half's bits
  v4i r;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const float a = f16_to_f32((uint16_t)x[d]), b = f16_to_f32((uint16_t)((uint32_t)x[d] >> 16));
    const float ra = a - __uint_as_float(__float_as_uint(a) & taken), rb = b - __uint_as_float(__float_as_uint(b) & taken);
    r[d] = (int)__builtin_amdgcn_perm(__float_as_uint(taken ? fmaxf(rb, -64.f * 1024.f) : rb),
                                      __float_as_uint(taken ? fmaxf(ra, -64.f * 1024.f) : ra), 0x07060302u);
  }
  return r;
}

// The token of a tile's i-th row (the i-th bit of its tokens), -1 past the last.
__device__ __forceinline__ int tile_token(uint32_t tokens, int i) {
  for (int q = 0; q < i; ++q) tokens &= tokens - 1;
  return tokens ? __builtin_ctz(tokens) : -1;
}

// Tile i of an expert's tokens, at most `most` of them each.
__device__ __forceinline__ MoeTile tile_of(int e, int row0, uint32_t tokens, int i, int most) {
  for (int q = 0; q < i * most; ++q) tokens &= tokens - 1;
  uint32_t rest = tokens;
  for (int q = 0; q < most; ++q) rest &= rest - 1;
  return MoeTile{(uint16_t)e, (uint16_t)(row0 + i * most), tokens ^ rest};
}

// The plan of up to kInline tokens in LDS, by every block for itself; block 0 leaves the second kernel's in the workspace.
// (Two tokens of an expert fit one tile.)
struct InlinePlan {
  float w[kInlineRows];
  MoeTile tile[kInlineRows];
  int tiles;
};
struct InlineScratch {
  int raw_e[kInlineRows];
  float raw_w[kInlineRows];
  double keys[kInline][kInlineE];
};

__device__ __forceinline__ void route_one(const RouteArgs& a, int t, int lane, double* keys, int& id, double& w) {
  if (a.E <= 64) {
    if (a.bias || a.G > 1) route_token<3, 1, true>(a, t, lane, LaneExperts<1, true>(a, lane), keys, id, w);
    else route_token<3, 1, false>(a, t, lane, LaneExperts<1, false>(a, lane), keys, id, w);
  } else {
    constexpr int V = kInlineE / 64;
    if (a.bias || a.G > 1) route_token<3, V, true>(a, t, lane, LaneExperts<V, true>(a, lane), keys, id, w);
    else route_token<3, V, false>(a, t, lane, LaneExperts<V, false>(a, lane), keys, id, w);
  }
}

__device__ __forceinline__ void plan_inline(const MoeArgs& p, InlinePlan& s, InlineScratch& x) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RouteArgs& a = p.route;
  if (wave < p.T) {
    int id;
    double w;
    route_one(a, wave, lane, x.keys[wave], id, w);
    if (lane < p.topk) {
      x.raw_e[wave * p.topk + lane] = id;
      x.raw_w[wave * p.topk + lane] = (float)(w * a.scale);
    }
  }
  __syncthreads();
  // One wave: lane i holds both tokens' choice i. A pair's row counts the pairs before it, its tile the experts.
  if (wave == 0) {
    const bool two = p.T == 2;
    const int e0 = lane < p.topk ? x.raw_e[lane] : -1, e1 = two && lane < p.topk ? x.raw_e[p.topk + lane] : -1;
    bool dup0 = false, dup1 = false;                 // the other token chose it too
    for (int q = 0; q < p.topk; ++q) {
      dup1 = dup1 || (e1 >= 0 && x.raw_e[q] == e1);
      dup0 = dup0 || (two && e0 >= 0 && x.raw_e[p.topk + q] == e0);
    }
    const unsigned long long dups = __ballot(dup1);
    int r0 = 0, r1 = dup1 ? 1 : 0, s0 = 0, s1 = 0;
    for (int q = 0; q < p.topk; ++q) {
      const int a = x.raw_e[q], b = two ? x.raw_e[p.topk + q] : -1;
      const int a0 = a >= 0 && a < e0, a1 = a >= 0 && a < e1, b0 = b >= 0 && b < e0, b1 = b >= 0 && b < e1;
      const int once = (dups >> q & 1) ? 0 : 1;
      r0 += a0 + b0;
      r1 += a1 + b1;
      s0 += a0 + b0 * once;
      s1 += a1 + b1 * once;
    }
    if (e0 >= 0) {
      s.w[r0] = x.raw_w[lane];
      s.tile[s0] = MoeTile{(uint16_t)e0, (uint16_t)r0, dup0 ? 3u : 1u};
    }
    if (e1 >= 0) {
      s.w[r1] = x.raw_w[p.topk + lane];
      if (!dup1) s.tile[s1] = MoeTile{(uint16_t)e1, (uint16_t)r1, 2u};
    }
    const int n = __popcll(__ballot(e0 >= 0)) + __popcll(__ballot(e1 >= 0 && !dup1));
    if (lane == 0) s.tiles = n;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = tid; i < s.tiles; i += blockDim.x) p.down[i] = s.tile[i];
    if (tid == 0) p.counts[1] = s.tiles;
  }
}

// The plan of more tokens, by one block of its own: a wave per token; a token is one bit of a mask per expert, so that
// rows need no sort and no order of atomics.
constexpr int kPThreads = 1024;
template <int V, bool GENERAL>
__global__ __launch_bounds__(kPThreads) void moe_plan_kernel(MoeArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ uint32_t mask[kMaxE];
  __shared__ int row0[kMaxE], part[3][kPThreads / kWave];
  double* keys = reinterpret_cast<double*>(smem);    // (groups) the waves' choice values
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RouteArgs& a = p.route;
  mask[tid] = 0;
  __syncthreads();
  int id[2] = {-1, -1};
  float w[2] = {0.f, 0.f};
  const LaneExperts<V, GENERAL> own(a, lane);
#pragma unroll
  for (int q = 0; q < 2; ++q) {                      // T <= 32 = 2 x 16 waves
    const int t = wave + 16 * q;
    if (t < p.T) {
      double v;
      route_token<3, V, GENERAL>(a, t, lane, own, keys + wave * a.E, id[q], v);
      w[q] = (float)(v * a.scale);
      if (id[q] >= 0) atomicOr(&mask[id[q]], 1u << t);
    }
  }
  __syncthreads();
  // thread e: the expert's rows and tiles, and the sums of those before it (the waves that hold experts)
  const int waves = (a.E + kWave - 1) / kWave;
  const uint32_t m = mask[tid];
  const int n = __popc(m), up = (n + kUpRows - 1) / kUpRows, dn = (n + p.down_rows - 1) / p.down_rows;
  int s[3] = {n, up, dn};
  if (wave < waves) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(s[k], off, kWave);
        if (lane >= off) s[k] += o;
      }
      if (lane == 63) part[k][wave] = s[k];
    }
  }
  if (waves > 1) __syncthreads();
  if (wave < waves) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      for (int v = 0; v < wave; ++v) s[k] += part[k][v];
    row0[tid] = s[0] - n;
    for (int i = 0; i < up; ++i) p.up[s[1] - up + i] = tile_of(tid, s[0] - n, m, i, kUpRows);
    for (int i = 0; i < dn; ++i) p.down[s[2] - dn + i] = tile_of(tid, s[0] - n, m, i, p.down_rows);
    if (tid == waves * kWave - 1) {
      p.counts[0] = s[1];
      p.counts[1] = s[2];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (id[q] >= 0) p.weights[row0[id[q]] + __popc(mask[id[q]] & ((1u << (wave + 16 * q)) - 1))] = w[q];
}

// Gate and up: WS waves of a block share the steps of 16 gate rows and the 16 up rows beside them. NX: DMAs of a step's
// activations.
template <int FMT, bool XF16, int NX, int WS>
__global__ __launch_bounds__(64 * WS) void moe_up_kernel(MoeArgs p) {
  constexpr bool OPF16 = XF16 && FMT != kMx;         // the operands' type
  constexpr bool PARTS = XF16 && FMT == kMx;         // x as two numbers
  constexpr bool FEW = kRowsPerDma<FMT> * NX < kUpRows;   // up to kInline tokens
  constexpr int COLS = kCols<FMT>, HALVES = FMT == kFp8 ? 1 : 2;
  using Op = typename Operand<OPF16>::V;
  using S = Scales<FMT, 2>;
  constexpr int kX = 4096, kSlot = kX + 1024 * NX;   // a step in LDS: gate, up, activations
  __shared__ __attribute__((aligned(16))) union {
    InlineScratch route;
    struct {
      uint8_t step[WS][kSlot], scales[WS][S::kBytes];
    } r;
    v4f red[WS][2][64];
  } s;
  __shared__ InlinePlan plan;                        // (takes no place where FEW is false)
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int row = l16 & 7;                           // this lane's row of a tile (columns 8 and on: again, or second parts)
  const bool inl = FEW && p.inl;
  if (inl) plan_inline(p, plan, s.route);
  const int items = __builtin_amdgcn_readfirstlane(inl ? plan.tiles : p.counts[0]) * p.NT;
  for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
    const int ti = item / p.NT, tn = item - ti * p.NT;
    const MoeTile tile = inl ? plan.tile[ti] : p.up[ti];
    const int rows = __popc(__builtin_amdgcn_readfirstlane(tile.tokens));
    const bool mine = row < rows;
    const float weight = mine ? (inl ? plan.w[tile.row0 + row] : p.weights[tile.row0 + row]) : 0.f;
    __syncthreads();                                   // the last item's sums were read (or the plan's scratch)
    const int e = __builtin_amdgcn_readfirstlane(tile.e);
    const int KT = (p.H + COLS - 1) / COLS, n0 = 16 * tn;
    Rows<FMT> wg, wu;
    wg.lane(n0, p.H, lane);
    wu.lane(p.I + n0, p.H, lane);
    wg.open(p.w13, e, 2 * (int64_t)p.I, n0, p.H);
    wu.open(p.w13, e, 2 * (int64_t)p.I, p.I + n0, p.H);
    S sc;
    sc.lane(2 * (int64_t)p.I, n0, p.I, p.H, p.kg13, lane);
    sc.open(p.s13, e, 2 * (int64_t)p.I, n0, p.I, p.H, p.G13);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x, (uint32_t)(p.T * (int64_t)p.H * 2));
    uint32_t xo[NX];
    bool xdead[NX];                                    // past H in the last step
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const int r = act_row<FMT>(j, lane), col = act_column<FMT>(r, lane), token = tile_token(tile.tokens, r);
      xo[j] = token >= 0 ? (uint32_t)(((int64_t)token * p.H + col) * 2) : kPast;
      xdead[j] = col >= p.H - (KT - 1) * COLS;
    }
    const uint8_t *step = &s.r.step[wave][0], *scales = &s.r.scales[wave][0];
    const uint32_t to = lds_address(step), to_scales = lds_address(scales);
    const int k0 = KT * wave / WS, k1 = KT * (wave + 1) / WS;
    auto fetch = [&](int k) {
      const bool last = k == KT - 1;
      wg.fetch(k, last, to);
      wu.fetch(k, last, to + 2048);
#pragma unroll
      for (int j = 0; j < NX; ++j)                   // (rows that the tile does not have: whatever lies there, not stored)
        if (kRowsPerDma<FMT> * j < rows)
          dma16(xr, to + kX + 1024 * j, last && xdead[j] ? kPast : xo[j], (uint32_t)k * (2 * COLS));
      if (k == k0 || S::begins(k)) sc.fetch(k, to_scales, lane);
    };
    const uint32_t taken = l16 >= 8 ? 0xFFFF0000u : 0u;
    v4f ag = v4f{0.f, 0.f, 0.f, 0.f}, au = ag;
    if (k0 < k1) {
      fetch(k0);
      for (int k = k0; k < k1; ++k) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        v4i qg[2], qu[2], X[HALVES][4];
        float lg[HALVES], lu[HALVES];
        v4f mg[HALVES], mu[HALVES];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          qg[q] = weight_piece<FMT>(step, q, l16, g);
          qu[q] = weight_piece<FMT>(step + 2048, q, l16, g);
        }
#pragma unroll
        for (int q = 0; q < HALVES; ++q) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            X[q][c] = act_chunk<FMT>(step + kX, row & (kRowsPerDma<FMT> * NX - 1), row & (kRowsPerDma<FMT> * NX - 1),
                                     FMT == kFp8 ? 8 * (c / 2) + 2 * g + c % 2 : 16 * q + 4 * g + c);
          if constexpr (FMT == kMx) {
            lg[q] = S::block(scales, k, 0, q, p.H - k * COLS, l16, g);
            lu[q] = S::block(scales, k, 1, q, p.H - k * COLS, l16, g);
          } else {
            mg[q] = S::sums(scales, k, 0, q, g);
            mu[q] = S::sums(scales, k, 1, q, g);
          }
        }
        // the step is in registers: its place takes the next
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        if (k + 1 < k1) fetch(k + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < HALVES; ++q) {
          v4f dg = FMT == kMx ? ag : v4f{0.f, 0.f, 0.f, 0.f}, du = FMT == kMx ? au : dg;
          if constexpr (FMT == kInt4) {                // -8 sum x
            const int m8 = OPF16 ? (int)0xC800C800 : (int)0xC100C100;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              dg = mfma16<OPF16>(__builtin_bit_cast(Op, v4i{m8, m8, m8, m8}), __builtin_bit_cast(Op, act_piece<FMT>(X[q], c)), dg);
            du = dg;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            v4i xp = act_piece<FMT>(X[q], c);
            if constexpr (PARTS) xp = part_of_f16(xp, taken);
            dg = mfma16<OPF16>(decode<FMT, OPF16>(qg, q, c, lg[q]), __builtin_bit_cast(Op, xp), dg);
            du = mfma16<OPF16>(decode<FMT, OPF16>(qu, q, c, lu[q]), __builtin_bit_cast(Op, xp), du);
          }
          if constexpr (FMT == kMx) {
            ag = dg;
            au = du;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ag[i] = fmaf(dg[i], mg[q][i], ag[i]);
              au[i] = fmaf(du[i], mu[q][i], au[i]);
            }
          }
        }
      }
    }
    __syncthreads();                                   // nothing is on its way into what takes the sums
    s.red[wave][0][lane] = ag;
    s.red[wave][1][lane] = au;
    __syncthreads();
    if (wave != 0) continue;
    v4f vg = s.red[0][0][lane], vu = s.red[0][1][lane];
#pragma unroll
    for (int w = 1; w < WS; ++w) {
      vg += s.red[w][0][lane];
      vu += s.red[w][1][lane];
    }
    if constexpr (PARTS) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        vg[q] += __shfl_xor(vg[q], 8, kWave);
        vu[q] += __shfl_xor(vu[q], 8, kWave);
      }
    }
    if (l16 >= 8 || !mine) continue;
    uint32_t part[kParts][4];                        // the upper 8 bits of mantissa, of what is left the next 8, the last 8
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float m = vg[q] / (1.0f + expf(-vg[q])) * vu[q] * weight;
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        part[k][q] = __float_as_uint(m) & 0xFFFF0000u;
        // (an infinity or a NaN, whose quiet bit the upper half holds, leaves no remainder)
        m = (part[k][q] & 0x7F800000u) != 0x7F800000u ? m - __uint_as_float(part[k][q]) : 0.f;
      }
    }
    uint16_t* o = p.mid + (int64_t)(tile.row0 + row) * p.I + n0 + 4 * g;
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      *reinterpret_cast<v2i*>(o + k * ((int64_t)p.T * p.topk * p.I)) =
          v2i{(int)(part[k][0] >> 16 | part[k][1]), (int)(part[k][2] >> 16 | part[k][3])};
  }
}

// DMAs of a step's middle.
template <int FMT, int ROWS>
constexpr int kMidDmas = (kParts * ROWS + kRowsPerDma<FMT> - 1) / kRowsPerDma<FMT>;

// Down: a block owns 16 NJ output columns of all tokens; its waves share the (tile, step) pairs, each a run of them. At a
// tile's end a wave adds its sums to its own place in LDS by token: no token takes anything of an expert that it did not
// choose, and the order is fixed. ROWS: most rows of a tile; number k of row r is row 3 r + k of a step's middle in LDS, and
// column ROWS k + r of the products.
template <int FMT, bool F16OUT, int ROWS, int WS, int NJ>
__global__ __launch_bounds__(64 * WS) void moe_down_kernel(MoeArgs p) {
  constexpr int COLS = kCols<FMT>, HALVES = FMT == kFp8 ? 1 : 2;
  using S = Scales<FMT, NJ>;
  constexpr int NM = kMidDmas<FMT, ROWS>, kX = 2048 * NJ, kSlot = kX + 1024 * NM;
  static_assert(kParts * ROWS <= 16, "the parts of a tile's rows are columns of one product");
  __shared__ __attribute__((aligned(16))) uint8_t room[WS][kSlot], room_scales[WS][S::kBytes];
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  v4f* sum = reinterpret_cast<v4f*>(smem);           // [WS][T][4 NJ]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int n0 = 16 * NJ * (int)blockIdx.x;
  const int KT = (p.I + COLS - 1) / COLS, tiles = p.counts[1], steps = tiles * KT;
  MoeTile* list = reinterpret_cast<MoeTile*>(sum + WS * p.T * 4 * NJ);
  for (int i = tid; i < tiles; i += 64 * WS) list[i] = p.down[i];
  for (int i = tid; i < WS * p.T * 4 * NJ; i += 64 * WS) sum[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const int64_t plane = (int64_t)p.T * p.topk * p.I * 2;
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(p.mid, (uint32_t)(kParts * plane));
  __syncthreads();
  v4f* mine = sum + wave * p.T * 4 * NJ;
  const int i0 = (int)((int64_t)steps * wave / WS), i1 = (int)((int64_t)steps * (wave + 1) / WS);
  const uint8_t *step = &room[wave][0], *scales = &room_scales[wave][0];
  const uint32_t to = lds_address(step), to_scales = lds_address(scales);
  uint32_t mo[NM];
  bool mdead[NM];
#pragma unroll
  for (int j = 0; j < NM; ++j) {
    const int r = act_row<FMT>(j, lane), col = act_column<FMT>(ROWS * (r % kParts) + r / kParts, lane);
    mo[j] = (uint32_t)((int64_t)(r / kParts) * p.I * 2 + 2 * col + r % kParts * plane);
    mdead[j] = col >= p.I - (KT - 1) * COLS;
  }
  // the tile and step that are fetched next, and those that are computed
  int ft = i0 / KT, fk = i0 - ft * KT, ct = ft, ck = fk;
  Rows<FMT> w[NJ];
  S sc;
  int rows = 0;
  uint32_t row0 = 0;
  auto open_tile = [&]() {                           // past the last: the last again, not used
    const MoeTile tile = list[min(ft, tiles - 1)];
    const int e = __builtin_amdgcn_readfirstlane(tile.e);
    rows = __popc(__builtin_amdgcn_readfirstlane(tile.tokens));
    row0 = (uint32_t)__builtin_amdgcn_readfirstlane(tile.row0) * (uint32_t)p.I * 2u;
#pragma unroll
    for (int j = 0; j < NJ; ++j) w[j].open(p.w2, e, p.H, n0 + 16 * j, p.I);
    sc.open(p.s2, e, p.H, n0, 16, p.I, p.G2);
  };
  auto fetch = [&](bool first) {
    const bool last = fk == KT - 1;
#pragma unroll
    for (int j = 0; j < NJ; ++j) w[j].fetch(fk, last, to + 2048 * j);
#pragma unroll
    for (int j = 0; j < NM; ++j)                     // (rows that the tile does not have: whatever lies there, not stored)
      if (kRowsPerDma<FMT> * j < kParts * rows)
        dma16(mr, to + kX + 1024 * j, act_row<FMT>(j, lane) / kParts >= rows || (last && mdead[j]) ? kPast : mo[j] + row0,
              (uint32_t)fk * (2 * COLS));
    if (first || S::begins(fk)) sc.fetch(fk, to_scales, lane);
    if (++fk == KT) {
      fk = 0;
      ++ft;
      open_tile();
    }
  };
  if (i0 < i1) {
    v4f acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
      w[j].lane(n0 + 16 * j, p.I, lane);
    }
    sc.lane(p.H, n0, 16, p.I, p.kg2, lane);
    open_tile();
    fetch(true);
    const int mrow = l16 < kParts * ROWS ? l16 % ROWS * kParts + l16 / ROWS : 0;   // (columns past the parts: not used)
    for (int i = i0; i < i1; ++i) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      v4i qw[NJ][2], M[HALVES][4];
      float ls[NJ][HALVES];
      v4f ms[NJ][HALVES];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) qw[j][q] = weight_piece<FMT>(step + 2048 * j, q, l16, g);
#pragma unroll
      for (int q = 0; q < HALVES; ++q) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          M[q][c] = act_chunk<FMT>(step + kX, mrow, l16, FMT == kFp8 ? 8 * (c / 2) + 2 * g + c % 2 : 16 * q + 4 * g + c);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if constexpr (FMT == kMx) ls[j][q] = S::block(scales, ck, j, q, p.I - ck * COLS, l16, g);
          else ms[j][q] = S::sums(scales, ck, j, q, g);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if (i + 1 < i1) fetch(false);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < HALVES; ++q) {
        v4f v[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) v[j] = FMT == kMx ? acc[j] : v4f{0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT == kInt4) {
          const int m8 = (int)0xC100C100;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[0] = mfma16<false>(bf(v4i{m8, m8, m8, m8}), bf(act_piece<FMT>(M[q], c)), v[0]);
#pragma unroll
          for (int j = 1; j < NJ; ++j) v[j] = v[0];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            v[j] = mfma16<false>(decode<FMT, false>(qw[j], q, c, ls[j][q]), bf(act_piece<FMT>(M[q], c)), v[j]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          if constexpr (FMT == kMx) {
            acc[j] = v[j];
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[j][c] = fmaf(v[j][c], ms[j][q][c], acc[j][c]);
          }
        }
      }
      if (++ck == KT || i == i1 - 1) {               // the tile's last step here
        const MoeTile tile = list[ct];
        const int token = tile_token(tile.tokens, min(l16, ROWS - 1));
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          v4f t = acc[j];                            // the smallest parts first
#pragma unroll
          for (int c = 0; c < 4; ++c)
            t[c] += __shfl(t[c], lane + ROWS, kWave) + __shfl(t[c], lane + 2 * ROWS, kWave);
          if (l16 < ROWS && token >= 0) mine[(token * NJ + j) * 4 + g] += t;
          acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        ck = 0;
        ++ct;
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < p.T * 4 * NJ; i += 64 * WS) {
    v4f v = sum[i];
#pragma unroll
    for (int w = 1; w < WS; ++w) v += sum[w * p.T * 4 * NJ + i];
    const int64_t at = (int64_t)(i / (4 * NJ)) * p.H + n0 + 4 * (i % (4 * NJ));
    if (p.add) {
      const v2i a = *reinterpret_cast<const v2i*>(p.add + at);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint16_t b = (uint16_t)((uint32_t)a[q / 2] >> (16 * (q % 2)));
        v[q] += F16OUT ? f16_to_f32(b) : bf16_to_f32(b);
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      o[q] = F16OUT ? f32_to_f16_rne(v[q]) : f32_to_bf16_rne(v[q]);
    }
    *reinterpret_cast<v2i*>(p.out + at) = v2i{(int)(o[0] | o[1] << 16), (int)(o[2] | o[3] << 16)};
  }
}

// ---- workspace: the tiles, the rows' weights, the middle
static size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Most tiles of `most` rows: one partial one for each expert with rows.
static constexpr int64_t most_tiles(int64_t E, int64_t R, int64_t most) { return R / most + (E < R ? E : R); }

struct MoeSpace {
  size_t up, down, weights, mid, end;
};
static MoeSpace moe_space(int64_t T, int64_t E, int64_t topk, int64_t I) {
  const int64_t R = T * topk;
  MoeSpace s;
  s.up = 16;
  s.down = s.up + up16(sizeof(MoeTile) * (size_t)most_tiles(E, R, kUpRows));
  s.weights = s.down + up16(sizeof(MoeTile) * (size_t)most_tiles(E, R, kFewRows));
  s.mid = s.weights + up16((size_t)R * 4);
  s.end = s.mid + up16((size_t)(kParts * R * I) * 2);
  return s;
}

size_t moe_workspace(int64_t T, int64_t E, int64_t topk, int64_t I) {
  return T == 0 ? 0 : moe_space(T, E, topk, I).end;
}

template <int FMT, bool F16, int NX, int ROWS, int WD, int NJ>
static hipError_t moe_stream(const MoeArgs& p, int64_t tiles, hipStream_t stream) {
  constexpr int WU = 4;                              // (2, 3 and 8 waves: within 5%)
  // Blocks of the first kernel that route for themselves do so once, for several column tiles each: at most 4 blocks per CU,
  // equally many tiles for each (2 tokens of 64 experts, int4: 55 us with a tile per block, 50 so). Where a kernel before
  // it routes, a tile per block is as fast or faster (32 tokens FP8: 314 us; 1024 blocks, 326).
  const int64_t items = tiles * p.NT, turns = p.inl ? (items + 1023) / 1024 : 1;
  // LDS of the second kernel: its waves' steps, their sums by token, the tiles; with the most of everything (32 tokens of 1024
  // experts, 64 chosen) at most 156 KiB
  const size_t lds = (size_t)WD * p.T * 64 * NJ + sizeof(MoeTile) * (size_t)most_tiles(p.E, (int64_t)p.T * p.topk, ROWS);
  constexpr size_t steps = (size_t)WD * (2048 * NJ + 1024 * kMidDmas<FMT, ROWS> + Scales<FMT, NJ>::kBytes);
  constexpr int64_t maxT = ROWS == kInline ? kInline : kMaxT;
  static_assert(steps + (size_t)WD * maxT * 64 * NJ + sizeof(MoeTile) * (size_t)most_tiles(kMaxE, maxT * kMaxTopk, ROWS) <= kLds,
                "every accepted size fits a CU's LDS");
  hipLaunchKernelGGL((moe_up_kernel<FMT, F16, NX, WU>), dim3((unsigned)((items + turns - 1) / turns)), dim3(64 * WU), 0,
                     stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<FMT, F16, ROWS, WD, NJ>), dim3((unsigned)(p.H / (16 * NJ))), dim3(64 * WD), lds, stream, p);
  return hipGetLastError();
}

template <int FMT, bool F16>
static hipError_t moe_go(MoeArgs& p, hipStream_t stream) {
  const int64_t R = (int64_t)p.T * p.topk;
  p.NT = p.I / 16;
  // Longer tiles of the second kernel read an expert's weights once for more rows and hold more LDS (32 tokens of 64
  // experts, 7168 x 2048: FP8 222 us with 4 rows, 205 with 5, MXFP4 157 and 152; 16 tokens: the same).
  p.down_rows = p.T <= kInline ? kInline : R >= 2 * p.E ? kDownRows : kFewRows;
  if (!p.inl) {
    const bool general = p.route.bias || p.route.G > 1;
    const size_t keys = p.route.G > 1 ? (size_t)8 * p.E * (kPThreads / kWave) : 0;
    static_assert(8 * kMaxE * (kPThreads / kWave) + 8 * kMaxE + 3 * 4 * (kPThreads / kWave) <= kLds, "as does the plan");
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(1), dim3(kPThreads), keys, stream, p); };
    if (p.E <= 64) general ? go(moe_plan_kernel<1, true>) : go(moe_plan_kernel<1, false>);
    else if (p.E <= 256) general ? go(moe_plan_kernel<4, true>) : go(moe_plan_kernel<4, false>);
    else general ? go(moe_plan_kernel<16, true>) : go(moe_plan_kernel<16, false>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // up to 2 tokens tiles have at most 2 rows
  constexpr int C = kCols<FMT> / 128;
  if (p.T <= kInline)
    return moe_stream<FMT, F16, 1, kInline, 8, 1>(p, p.inl ? (R < p.E ? R : p.E) : most_tiles(p.E, R, kUpRows), stream);
  const int64_t tiles = most_tiles(p.E, R, kUpRows);
  // The second kernel reads the middle, from L2, once per block: with 32 columns per block half as often (measured with a
  // middle of two numbers and tiles of 8 rows: 32 tokens, 7168 x 2048, FP8: 199 us with 16 columns, 160 with 32; 8 tokens
  // of MXFP4: 66 and 58), if that leaves enough blocks; else more
  // waves share the steps (32 tokens, 2048 x 1024, FP8: 32 columns 70 us, 16 columns 58, with 12 waves 51; 8 tokens of
  // 4096 x 2048, MXFP4: 54, 46 and 39). LDS bounds the waves of long tiles.
  if (p.H >= 6144)
    return p.down_rows == kFewRows ? moe_stream<FMT, F16, 2 * C, kFewRows, 8, 2>(p, tiles, stream)
                                   : moe_stream<FMT, F16, 2 * C, kDownRows, 8, 2>(p, tiles, stream);
  return p.down_rows == kFewRows ? moe_stream<FMT, F16, 2 * C, kFewRows, 12, 1>(p, tiles, stream)
                                 : moe_stream<FMT, F16, 2 * C, kDownRows, 10, 1>(p, tiles, stream);
}

// fmt: 0 FP8 with block scales, 1 MXFP4, 2 int4 tiles (group: 128 m, or -1).
hipError_t launch_moe_decode(const void* x, bool f16, const void* logits, int dt, int64_t ld, int score, const float* bias,
                             int64_t G, int64_t topk_groups, int64_t group_top, int64_t topk, bool renorm, double scale,
                             int fmt, const void* w13, const void* s13, const void* w2, const void* s2, int64_t group,
                             const void* add, void* out, int64_t T, int64_t E, int64_t H, int64_t I, void* ws,
                             hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const MoeSpace sp = moe_space(T, E, topk, I);
  uint8_t* base = static_cast<uint8_t*>(ws);
  MoeArgs p{};
  p.x = static_cast<const uint16_t*>(x);
  p.w13 = static_cast<const uint8_t*>(w13);
  p.w2 = static_cast<const uint8_t*>(w2);
  p.s13 = s13;
  p.s2 = s2;
  p.add = static_cast<const uint16_t*>(add);
  p.out = static_cast<uint16_t*>(out);
  p.T = (int)T; p.E = (int)E; p.topk = (int)topk; p.H = (int)H; p.I = (int)I;
  p.G13 = group == -1 ? 1 : (int)(H / group);
  p.G2 = group == -1 ? 1 : (int)(I / group);
  p.kg13 = (int)((group == -1 ? H : group) / 128);
  p.kg2 = (int)((group == -1 ? I : group) / 128);
  p.counts = reinterpret_cast<int32_t*>(base);
  p.up = reinterpret_cast<MoeTile*>(base + sp.up);
  p.down = reinterpret_cast<MoeTile*>(base + sp.down);
  p.weights = reinterpret_cast<float*>(base + sp.weights);
  p.mid = reinterpret_cast<uint16_t*>(base + sp.mid);
  RouteArgs& a = p.route;
  a.x = logits; a.bias = bias; a.T = T; a.ld = ld; a.dt = dt;
  a.E = (int)E; a.topk = (int)topk; a.G = (int)G; a.per_group = (int)(E / G);
  a.topk_groups = (int)topk_groups; a.group_top = (int)group_top; a.score = score; a.renorm = renorm ? 1 : 0;
  a.scale = scale;
  p.inl = T <= kInline && E <= kInlineE;
  if (fmt == kFp8) return f16 ? moe_go<kFp8, true>(p, stream) : moe_go<kFp8, false>(p, stream);
  if (fmt == kMx) return f16 ? moe_go<kMx, true>(p, stream) : moe_go<kMx, false>(p, stream);
  return f16 ? moe_go<kInt4, true>(p, stream) : moe_go<kInt4, false>(p, stream);
}

}  // namespace w4
