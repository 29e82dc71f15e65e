// The whole routed-expert layer for a few tokens (T <= 32), weights only
// quantized: router logits and hidden rows in, the experts' weighted sum out.
//
//   out[t] = sum_j w[t, j] * W2[e] (silu(W1[e] x[t]) * (W3[e] x[t]))  (+ add[t]),  e = ids[t, j]
//
// With so few rows the time is the chosen experts' weights, each read once. Two
// kernels: gate and up products with the activation, then the down products with
// the sum over a token's experts. Up to kInline tokens the first one routes too,
// every block for itself (a wave per token); more tokens are routed by a block
// before it, once instead of once per block.
//
// The plan: pairs (token, expert) are rows, ordered by expert, then token. Tiles
// of at most 8 (gate and up) or 4 (down) rows of an expert name it, their first
// row and their tokens as bits.
//
// Both kernels stream weights through the matrix unit, 16 weight rows as its A
// operand, a tile's rows as its B operand. Weights become bf16 (exactly, with
// MXFP4's scale applied; v_mfma_f32_16x16x32_bf16), or fp16 for fp16 activations of
// FP8 and int4 weights; FP8's and int4's scales multiply the sums of 128 columns.
//
// What a wave reads passes through a ring of its own in LDS, by LDS DMA: no wave
// waits for another, and D steps are in flight without a register. Loading straight
// into the matrix unit's layout (lane = row + 16 * column group) would touch 64
// cache lines per load and cost the address unit 60 clocks where a DMA of 8 rows'
// full lines costs 16 (measured); it bound such a kernel at 2 to 4 TB/s. Rows
// lie in LDS with their 16-byte chunks permuted by the row, so that the reads of 8
// rows touch 8 different chunks.
//
// What lies between the two is held to 16 bits of mantissa as the sum of two bf16
// numbers (2^-17 relative, below what the output's own rounding leaves visible).
// The matrix unit takes them in one go: columns 0..7 are 8 rows' first numbers,
// columns 8..15 their second ones, added at the end. MXFP4 with fp16 activations
// takes x apart in the same way, exactly (11 bits).
#include <type_traits>

#include "mxfp4.h"
#include "route_token.h"

namespace w4 {

constexpr int kInline = 2;                           // tokens that the first kernel routes itself
constexpr int kInlineE = 256;
constexpr int kInlineRows = kInline * 64;
constexpr int kUpRows = 8, kDownRows = 4;            // most rows of a tile
enum { kFp8 = 0, kMx = 1, kInt4 = 2 };

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
  int NT;                                            // column tiles of the launch
  int inl;                                           // the first kernel routes
  // workspace
  int32_t* counts;                                   // tiles of the first kernel, of the second
  MoeTile *up, *down;
  float* weights;                                    // of the rows
  uint16_t* mid;                                     // [2][R][I]: the middle, as two bf16
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

// Columns of a step: 128 bytes of a weight row (int4: two tiles).
template <int FMT>
constexpr int kCols = FMT == kFp8 ? 128 : 256;

// LDS DMA of 16 or 4 bytes per lane to dst + lane * 16 (4). Memory past the buffer
// reads as zero. m0 holds the LDS address: the compiler keeps nothing in it here, and
// a clobber of a reserved register is not honoured.
__device__ __forceinline__ void dma16(const __amdgpu_buffer_rsrc_t rs, uint32_t dst, uint32_t off, uint32_t ks) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(dst), "v"(off), "s"(rs), "s"(ks) : "memory");
}
__device__ __forceinline__ void dma4(const __amdgpu_buffer_rsrc_t rs, uint32_t dst, uint32_t off, uint32_t ks) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(dst), "v"(off), "s"(rs), "s"(ks) : "memory");
}

// 16 rows n .. n + 15 of weight matrix e, [N, K]: 2 KiB of LDS per step, by two DMAs.
// FP8, MXFP4: row r, chunk c at 128 r + 16 (c ^ (r & 7)); int4: tile q, unit (r, g) at
// 1024 q + 64 r + 16 (g ^ (r / 4 & 3)).
template <int FMT>
struct Rows {
  __amdgpu_buffer_rsrc_t w;
  uint32_t off[2];
  bool dead[2];                                      // the chunk lies past K in the last step
  int kt;                                            // int4: tiles along K
  // what depends on the lane alone, and on the matrix
  __device__ __forceinline__ void lane(int64_t n, int64_t K, int lane) {
    if constexpr (FMT == kInt4) {
      kt = (int)(K / kTileK);
      const int r = lane >> 2, g = (lane & 3) ^ (r >> 2 & 3);
      off[0] = off[1] = (uint32_t)((n % kTileN + r) * 64 + 16 * g);
    } else {
      const int64_t bytes = FMT == kFp8 ? K : K / 2;
      const int left = (int)(K - (K - 1) / kCols<FMT> * kCols<FMT>);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * i + (lane >> 3), c = (lane & 7) ^ (r & 7);
        off[i] = (uint32_t)(r * bytes + 16 * c);
        dead[i] = kCols<FMT> / 8 * c >= left;
      }
    }
  }
  __device__ __forceinline__ void open(const uint8_t* base, int64_t e, int64_t N, int64_t n, int64_t K) {
    if constexpr (FMT == kInt4) {
      const int64_t tk = K / kTileK, tiles = (N + kTileN - 1) / kTileN * tk;
      w = make_rsrc(base + (e * tiles + n / kTileN * tk) * kTileBytes, (uint32_t)(tk * kTileBytes));
    } else {
      const int64_t bytes = FMT == kFp8 ? K : K / 2;
      w = make_rsrc(base + (e * N + n) * bytes, (uint32_t)(16 * bytes));
    }
  }
  __device__ __forceinline__ void fetch(int k, bool last, uint32_t dst) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (FMT == kInt4) dma16(w, dst + 1024 * i, 2 * k + i < kt ? off[i] : kPast, (uint32_t)(2 * k + i) * kTileBytes);
      else dma16(w, dst + 1024 * i, last && dead[i] ? kPast : off[i], (uint32_t)k * 128u);
    }
  }
};
// A lane's two 16-byte pieces: FP8: columns 16 g .. and 64 + 16 g ..; MXFP4: blocks g and 4 + g; int4: units (row, g).
template <int FMT>
__device__ __forceinline__ v4i weight_piece(const uint8_t* at, int q, int l16, int g) {
  return *reinterpret_cast<const v4i*>(FMT == kInt4 ? at + 1024 * q + 64 * l16 + 16 * (g ^ (l16 >> 2 & 3))
                                                    : at + 128 * l16 + 16 * ((4 * q + g) ^ (l16 & 7)));
}

// Rows of 16-bit activations: a DMA takes kCols columns of 4 (FP8) or 2 rows; row r, chunk c at 2 kCols r + 16 (c ^ (r & 7)).
template <int FMT>
constexpr int kRowsPerDma = 512 / kCols<FMT>;
template <int FMT>
__device__ __forceinline__ int act_row(int j, int lane) { return j * kRowsPerDma<FMT> + lane / (kCols<FMT> / 8); }
template <int FMT>
__device__ __forceinline__ int act_column(int row, int lane) { return 8 * ((lane & (kCols<FMT> / 8 - 1)) ^ (row & 7)); }
// MFMA c's 8 activations of a lane (of the step's half q: MXFP4 and int4 have 4 MFMAs in each): FP8: columns 64 (c / 2) +
// 16 g + 8 (c % 2) ..; MXFP4: 128 q + 32 g + 8 c ..; int4: 128 q + 32 g + 4 c .. + 3 and 16 after them.
template <int FMT>
__device__ __forceinline__ v4i act_chunk(const uint8_t* at, int row, int chunk) {
  return *reinterpret_cast<const v4i*>(at + 2 * kCols<FMT> * row + 16 * (chunk ^ (row & 7)));
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
// 2^-9); the sums start from -8 sum x.
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

// The scales of MATS sets of 16 rows (the second `gap` rows after the first). FP8 and MXFP4: of 8 steps at a time, with the
// first of them (steps one by one would ask for a cache line that is still on its way, which holds up the whole cache: 46 us
// of one token's gate and up products where 8 at a time take $UP): FP8 8 floats of each set; MXFP4 64 bytes of each row,
// piece c of row r at 64 r + 16 (c ^ (r / 4 & 3)). int4: of each step: half q, set m: 16 fp16.
template <int FMT, int MATS>
struct Scales {
  static constexpr int kSteps = FMT == kInt4 ? 1 : 8;
  static constexpr int kDmas = FMT == kMx ? MATS : 1;
  static constexpr int kLanes = FMT == kMx ? 64 : (FMT == kFp8 ? 8 : 16) * MATS;
  static constexpr int kBytes = FMT == kMx ? 1024 * MATS : 64 * MATS;
  __amdgpu_buffer_rsrc_t s;
  uint32_t off, next;                                // next: from set to set
  int per, N, halves;
  __device__ __forceinline__ void lane(int64_t N_, int64_t n, int64_t gap, int64_t K, int per_, int lane) {
    per = per_;
    N = (int)N_;
    if constexpr (FMT == kFp8) {
      off = (uint32_t)((n + (lane >> 3) * gap) / 128 * ((K + 127) / 128) * 4 + 4 * (lane & 7));
    } else if constexpr (FMT == kMx) {
      const int r = lane >> 2;
      off = (uint32_t)(r * mx_scale_bytes(K) + 16 * ((lane & 3) ^ (r >> 2 & 3)));
      next = (uint32_t)(gap * mx_scale_bytes(K));
    } else {
      halves = (int)(K / 128);
      off = (uint32_t)((n + (lane >> 3) % MATS * gap) * 2 + 4 * (lane & 7));
    }
  }
  __device__ __forceinline__ void open(const void* base, int64_t e, int64_t N_, int64_t n, int64_t gap, int64_t K, int G) {
    const uint8_t* b = static_cast<const uint8_t*>(base);
    if constexpr (FMT == kFp8) {
      const int64_t size = (K + 127) / 128 * ((N_ + 127) / 128) * 4;
      s = make_rsrc(b + e * size, (uint32_t)size);
    } else if constexpr (FMT == kMx) {
      const int64_t ks = mx_scale_bytes(K);
      s = make_rsrc(b + (e * N_ + n) * ks, (uint32_t)(((MATS - 1) * gap + 16) * ks));
    } else {
      s = make_rsrc(b + e * G * N_ * 2, (uint32_t)(G * N_ * 2));
    }
  }
  // begins: whether a step's scales come with it (a run's first step, and every kSteps)
  static __device__ __forceinline__ bool begins(int k) { return k % kSteps == 0; }
  __device__ __forceinline__ void fetch(int k, uint32_t dst, int lane) const {
    dst = __builtin_amdgcn_readfirstlane(dst);       // (the compiler does not see that it is uniform)
    if (lane >= kLanes) return;
    if constexpr (FMT == kFp8) {
      dma4(s, dst, off, (uint32_t)(k & ~7) * 4);
    } else if constexpr (FMT == kMx) {
#pragma unroll
      for (int m = 0; m < MATS; ++m) dma16(s, dst + 1024 * m, off + m * next, (uint32_t)(k & ~7) * 8);
    } else {
      // (the second half of an odd number's last step: the first's)
      const int a = 2 * k / per * N * 2, b = min(2 * k + 1, halves - 1) / per * N * 2;
      dma4(s, dst, off + (lane < 8 * MATS ? (uint32_t)a : (uint32_t)b), 0u);
    }
  }
  // what multiplies the sums of rows 4 g .. 4 g + 3 of set m over half q of step k
  static __device__ __forceinline__ v4f sums(const uint8_t* at, int k, int m, int q, int g) {
    if constexpr (FMT == kFp8) {
      const float v = reinterpret_cast<const float*>(at)[8 * m + (k & 7)];
      return v4f{v, v, v, v};
    } else {
      const v2i v = *reinterpret_cast<const v2i*>(at + 32 * (MATS * q + m) + 8 * g);
      return v4f{f16_to_f32((uint16_t)v[0]), f16_to_f32((uint16_t)((uint32_t)v[0] >> 16)), f16_to_f32((uint16_t)v[1]),
                 f16_to_f32((uint16_t)((uint32_t)v[1] >> 16))};
    }
  }
  // MXFP4: a lane's scale of half q of step k; left: the columns from the step's first to the end
  static __device__ __forceinline__ float block(const uint8_t* at, int k, int m, int q, int left, int l16, int g) {
    const int piece = (k & 7) >> 1 ^ (l16 >> 2 & 3);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(at + 1024 * m + 64 * l16 + 16 * piece + 8 * (k & 1) + 4 * q);
    const uint32_t c = 128 * q + 32 * g < left ? w >> (8 * g) & 0xFF : 0u;   // past K: the padding, or the next row's
    return c == kMxNan ? __uint_as_float(0x7FC00000u) : mx_scale_value(c);
  }
};

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
  int raw_e[kInlineRows];
  float raw_w[kInlineRows];
  MoeTile tile[kInlineRows];
  int tiles;
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

__device__ __forceinline__ void plan_inline(const MoeArgs& p, InlinePlan& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RouteArgs& a = p.route;
  if (wave < p.T) {
    int id;
    double w;
    route_one(a, wave, lane, s.keys[wave], id, w);
    if (lane < p.topk) {
      s.raw_e[wave * p.topk + lane] = id;
      s.raw_w[wave * p.topk + lane] = (float)(w * a.scale);
    }
  }
  __syncthreads();
  // One wave: lane i holds both tokens' choice i. A pair's row counts the pairs before it, its tile the experts.
  if (wave == 0) {
    const bool two = p.T == 2;
    const int e0 = lane < p.topk ? s.raw_e[lane] : -1, e1 = two && lane < p.topk ? s.raw_e[p.topk + lane] : -1;
    bool dup0 = false, dup1 = false;                 // the other token chose it too
    for (int q = 0; q < p.topk; ++q) {
      dup1 = dup1 || (e1 >= 0 && s.raw_e[q] == e1);
      dup0 = dup0 || (two && e0 >= 0 && s.raw_e[p.topk + q] == e0);
    }
    const unsigned long long dups = __ballot(dup1);
    int r0 = 0, r1 = dup1 ? 1 : 0, s0 = 0, s1 = 0;
    for (int q = 0; q < p.topk; ++q) {
      const int a = s.raw_e[q], b = two ? s.raw_e[p.topk + q] : -1;
      const int a0 = a >= 0 && a < e0, a1 = a >= 0 && a < e1, b0 = b >= 0 && b < e0, b1 = b >= 0 && b < e1;
      const int once = (dups >> q & 1) ? 0 : 1;
      r0 += a0 + b0;
      r1 += a1 + b1;
      s0 += a0 + b0 * once;
      s1 += a1 + b1 * once;
    }
    if (e0 >= 0) {
      s.w[r0] = s.raw_w[lane];
      s.tile[s0] = MoeTile{(uint16_t)e0, (uint16_t)r0, dup0 ? 3u : 1u};
    }
    if (e1 >= 0) {
      s.w[r1] = s.raw_w[p.topk + lane];
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
  // thread e: the expert's rows and tiles, and the sums of those before it
  const uint32_t m = mask[tid];
  const int n = __popc(m), up = (n + kUpRows - 1) / kUpRows, dn = (n + kDownRows - 1) / kDownRows;
  int s[3] = {n, up, dn};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int o = __shfl_up(s[k], off, kWave);
      if (lane >= off) s[k] += o;
    }
    if (lane == 63) part[k][wave] = s[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k)
    for (int v = 0; v < wave; ++v) s[k] += part[k][v];
  row0[tid] = s[0] - n;
  for (int i = 0; i < up; ++i) p.up[s[1] - up + i] = tile_of(tid, s[0] - n, m, i, kUpRows);
  for (int i = 0; i < dn; ++i) p.down[s[2] - dn + i] = tile_of(tid, s[0] - n, m, i, kDownRows);
  if (tid == kPThreads - 1) {
    p.counts[0] = s[1];
    p.counts[1] = s[2];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (id[q] >= 0) p.weights[row0[id[q]] + __popc(mask[id[q]] & ((1u << (wave + 16 * q)) - 1))] = w[q];
}

// Gate and up: WS waves of a block share the steps of 16 gate rows and the 16 up rows beside them. NX: DMAs of a step's
// activations.
template <int FMT, bool XF16, int NX, int WS, int D>
__global__ __launch_bounds__(64 * WS) void moe_up_kernel(MoeArgs p) {
  constexpr bool OPF16 = XF16 && FMT != kMx;         // the operands' type
  constexpr bool PARTS = XF16 && FMT == kMx;         // x as two numbers
  constexpr int COLS = kCols<FMT>, HALVES = FMT == kFp8 ? 1 : 2;
  using Op = typename Operand<OPF16>::V;
  using S = Scales<FMT, 2>;
  // a step in LDS: gate, up, activations; and the scales in places of their own. kDmas: the fewest of a step
  constexpr int kX = 4096, kSlot = kX + 1024 * NX, kDmas = 4 + NX + (S::kSteps == 1 ? S::kDmas : 0);
  __shared__ __attribute__((aligned(16))) union {
    InlinePlan plan;
    struct {
      uint8_t ring[WS][D][kSlot], scales[WS][D][S::kBytes];
    } r;
    v4f red[WS][2][64];
  } s;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int ti = (int)blockIdx.x / p.NT, tn = (int)blockIdx.x % p.NT;
  MoeTile tile;
  const int row = l16 & 7;                           // this lane's row of the tile (columns 8 and on: again, or second parts)
  float weight = 0.f;
  if (p.inl) {
    plan_inline(p, s.plan);
    if (ti >= s.plan.tiles) return;
    tile = s.plan.tile[ti];
    if (row < __popc(tile.tokens)) weight = s.plan.w[tile.row0 + row];
    __syncthreads();                                 // the plan's place becomes the ring
  } else {
    if (ti >= p.counts[0]) return;
    tile = p.up[ti];
    if (row < __popc(tile.tokens)) weight = p.weights[tile.row0 + row];
  }
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
  const uint32_t ring0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&s.r.ring[wave][0][0]);
  const uint32_t scales0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&s.r.scales[wave][0][0]);
  const int k0 = KT * wave / WS, k1 = KT * (wave + 1) / WS;
  int fs = -1, cs = -1;                              // the scales' places that were fetched and are used last
  auto fetch = [&](int k, int d) {                   // past the run's end: the last step again, not used
    const bool begins = k == k0 || (k < k1 && S::begins(k));
    k = min(k, k1 - 1);
    const uint32_t at = ring0 + d * kSlot;
    const bool last = k == KT - 1;
    wg.fetch(k, last, at);
    wu.fetch(k, last, at + 2048);
#pragma unroll
    for (int j = 0; j < NX; ++j) dma16(xr, at + kX + 1024 * j, last && xdead[j] ? kPast : xo[j], (uint32_t)k * (2 * COLS));
    if (begins || S::kSteps == 1) {
      fs = fs + 1 == D ? 0 : fs + 1;
      sc.fetch(k, scales0 + fs * S::kBytes, lane);
    }
  };
  const uint32_t taken = l16 >= 8 ? 0xFFFF0000u : 0u;
  v4f ag = v4f{0.f, 0.f, 0.f, 0.f}, au = ag;
  if (k0 < k1) {
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(k0 + d, d);
    int d = 0;
    for (int k = k0; k < k1; ++k) {
      const uint8_t* at = &s.r.ring[wave][d][0];
      if (k == k0 || S::begins(k)) cs = cs + 1 == D ? 0 : cs + 1;
      const uint8_t* as = &s.r.scales[wave][cs][0];
      asm volatile("s_waitcnt vmcnt(%0)" :: "n"((D - 1) * kDmas) : "memory");
      v4i qg[2], qu[2], X[HALVES][4];
      float lg[HALVES], lu[HALVES];
      v4f mg[HALVES], mu[HALVES];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        qg[q] = weight_piece<FMT>(at, q, l16, g);
        qu[q] = weight_piece<FMT>(at + 2048, q, l16, g);
      }
#pragma unroll
      for (int q = 0; q < HALVES; ++q) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          X[q][c] = act_chunk<FMT>(at + kX, row & (kRowsPerDma<FMT> * NX - 1),
                                   FMT == kFp8 ? 8 * (c / 2) + 2 * g + c % 2 : 16 * q + 4 * g + c);
        if constexpr (FMT == kMx) {
          lg[q] = S::block(as, k, 0, q, p.H - k * COLS, l16, g);
          lu[q] = S::block(as, k, 1, q, p.H - k * COLS, l16, g);
        } else {
          mg[q] = S::sums(as, k, 0, q, g);
          mu[q] = S::sums(as, k, 1, q, g);
        }
      }
      // the step is in registers: its place takes the one D on
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      fetch(k + D, d);
      __builtin_amdgcn_sched_barrier(0);
      d = d + 1 == D ? 0 : d + 1;
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
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // nothing may land in what the ring becomes
  }
  __syncthreads();
  s.red[wave][0][lane] = ag;
  s.red[wave][1][lane] = au;
  __syncthreads();
  if (wave != 0) return;
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
  if (l16 >= 8 || row >= __popc(tile.tokens)) return;
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float m = vg[q] / (1.0f + expf(-vg[q])) * vu[q] * weight;
    hi[q] = f32_to_bf16_rne(m);
    const float rest = m - __uint_as_float(hi[q] << 16);
    lo[q] = (hi[q] & 0x7F80u) != 0x7F80u ? f32_to_bf16_rne(rest) : 0u;   // (an infinity has no remainder)
  }
  uint16_t* o = p.mid + (int64_t)(tile.row0 + row) * p.I + n0 + 4 * g;
  *reinterpret_cast<v2i*>(o) = v2i{(int)(hi[0] | hi[1] << 16), (int)(hi[2] | hi[3] << 16)};
  *reinterpret_cast<v2i*>(o + (int64_t)p.T * p.topk * p.I) = v2i{(int)(lo[0] | lo[1] << 16), (int)(lo[2] | lo[3] << 16)};
}

// Down: a block owns 16 output columns of all tokens; its waves share the (tile, step) pairs, each a run of them. At a
// tile's end a wave adds its sums to its own place in LDS by token: no token takes anything of an expert that it did not
// choose, and the order is fixed. NM: DMAs of a step's middle (row r's first numbers as row 2 r, its second as 2 r + 1).
template <int FMT, bool F16OUT, int NM, int WS, int D>
__global__ __launch_bounds__(64 * WS) void moe_down_kernel(MoeArgs p) {
  constexpr int COLS = kCols<FMT>, HALVES = FMT == kFp8 ? 1 : 2;
  using S = Scales<FMT, 1>;
  constexpr int kX = 2048, kSlot = kX + 1024 * NM, kDmas = 2 + NM + (S::kSteps == 1 ? S::kDmas : 0);
  constexpr int kMost = kRowsPerDma<FMT> * NM / 2;   // rows that fit
  __shared__ __attribute__((aligned(16))) uint8_t ring[WS][D][kSlot], scales[WS][D][S::kBytes];
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  v4f* sum = reinterpret_cast<v4f*>(smem);           // [WS][T][4]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int n0 = 16 * (int)blockIdx.x;
  const int KT = (p.I + COLS - 1) / COLS, tiles = p.counts[1], steps = tiles * KT;
  MoeTile* list = reinterpret_cast<MoeTile*>(sum + WS * p.T * 4);
  for (int i = tid; i < tiles; i += 64 * WS) list[i] = p.down[i];
  for (int i = tid; i < WS * p.T * 4; i += 64 * WS) sum[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const int64_t plane = (int64_t)p.T * p.topk * p.I * 2;
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(p.mid, (uint32_t)(2 * plane));
  __syncthreads();
  v4f* mine = sum + wave * p.T * 4;
  const int i0 = (int)((int64_t)steps * wave / WS), i1 = (int)((int64_t)steps * (wave + 1) / WS);
  const uint32_t ring0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&ring[wave][0][0]);
  const uint32_t scales0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&scales[wave][0][0]);
  uint32_t mo[NM];
  bool mdead[NM];
#pragma unroll
  for (int j = 0; j < NM; ++j) {
    const int r = act_row<FMT>(j, lane), col = act_column<FMT>(r, lane);
    mo[j] = (uint32_t)((int64_t)(r >> 1) * p.I * 2 + 2 * col + (r & 1) * plane);
    mdead[j] = col >= p.I - (KT - 1) * COLS;
  }
  // the tile and step that are fetched next, and those that are computed
  int ft = i0 / KT, fk = i0 - ft * KT, ct = ft, ck = fk;
  int fs = -1, cs = -1;                              // the scales' places that were fetched and are used last
  Rows<FMT> w;
  S sc;
  int rows = 0;
  uint32_t row0 = 0;
  auto open_tile = [&]() {                           // past the last: the last again, not used
    const MoeTile tile = list[min(ft, tiles - 1)];
    const int e = __builtin_amdgcn_readfirstlane(tile.e);
    rows = __popc(__builtin_amdgcn_readfirstlane(tile.tokens));
    row0 = (uint32_t)__builtin_amdgcn_readfirstlane(tile.row0) * (uint32_t)p.I * 2u;
    w.open(p.w2, e, p.H, n0, p.I);
    sc.open(p.s2, e, p.H, n0, 0, p.I, p.G2);
  };
  auto fetch = [&](int d, bool first) {
    const uint32_t at = ring0 + d * kSlot;
    const bool last = fk == KT - 1;
    w.fetch(fk, last, at);
#pragma unroll
    for (int j = 0; j < NM; ++j)
      dma16(mr, at + kX + 1024 * j, (act_row<FMT>(j, lane) >> 1) >= rows || (last && mdead[j]) ? kPast : mo[j] + row0,
            (uint32_t)fk * (2 * COLS));
    if (first || S::begins(fk)) {
      fs = fs + 1 == D ? 0 : fs + 1;
      sc.fetch(fk, scales0 + fs * S::kBytes, lane);
    }
    if (++fk == KT) {
      fk = 0;
      ++ft;
      open_tile();
    }
  };
  if (i0 < i1) {
    v4f acc = v4f{0.f, 0.f, 0.f, 0.f};
    w.lane(n0, p.I, lane);
    sc.lane(p.H, n0, 0, p.I, p.kg2, lane);
    open_tile();
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, d == 0);
    const int mrow = (2 * (l16 & 7) + (l16 >> 3)) & (2 * kMost - 1);
    int d = 0;
    for (int i = i0; i < i1; ++i) {
      const uint8_t* at = &ring[wave][d][0];
      if (i == i0 || S::begins(ck)) cs = cs + 1 == D ? 0 : cs + 1;
      const uint8_t* as = &scales[wave][cs][0];
      asm volatile("s_waitcnt vmcnt(%0)" :: "n"((D - 1) * kDmas) : "memory");
      v4i qw[2], M[HALVES][4];
      float ls[HALVES];
      v4f ms[HALVES];
#pragma unroll
      for (int q = 0; q < 2; ++q) qw[q] = weight_piece<FMT>(at, q, l16, g);
#pragma unroll
      for (int q = 0; q < HALVES; ++q) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          M[q][c] = act_chunk<FMT>(at + kX, mrow, FMT == kFp8 ? 8 * (c / 2) + 2 * g + c % 2 : 16 * q + 4 * g + c);
        if constexpr (FMT == kMx) ls[q] = S::block(as, ck, 0, q, p.I - ck * COLS, l16, g);
        else ms[q] = S::sums(as, ck, 0, q, g);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      fetch(d, false);
      __builtin_amdgcn_sched_barrier(0);
      d = d + 1 == D ? 0 : d + 1;
#pragma unroll
      for (int q = 0; q < HALVES; ++q) {
        v4f v = FMT == kMx ? acc : v4f{0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT == kInt4) {
          const int m8 = (int)0xC100C100;
#pragma unroll
          for (int c = 0; c < 4; ++c) v = mfma16<false>(bf(v4i{m8, m8, m8, m8}), bf(act_piece<FMT>(M[q], c)), v);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) v = mfma16<false>(decode<FMT, false>(qw, q, c, ls[q]), bf(act_piece<FMT>(M[q], c)), v);
        if constexpr (FMT == kMx) {
          acc = v;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[c] = fmaf(v[c], ms[q][c], acc[c]);
        }
      }
      if (++ck == KT || i == i1 - 1) {               // the tile's last step here
        const MoeTile tile = list[ct];
        const int token = tile_token(tile.tokens, l16 & 7);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] += __shfl_xor(acc[c], 8, kWave);
        if (l16 < 8 && token >= 0) mine[token * 4 + g] += acc;
        acc = v4f{0.f, 0.f, 0.f, 0.f};
        ck = 0;
        ++ct;
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // what was fetched past the end has landed
  }
  __syncthreads();
  for (int i = tid; i < p.T * 4; i += 64 * WS) {
    v4f v = sum[i];
#pragma unroll
    for (int w = 1; w < WS; ++w) v += sum[w * p.T * 4 + i];
    const int64_t at = (int64_t)(i / 4) * p.H + n0 + 4 * (i % 4);
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
static int64_t most_tiles(int64_t E, int64_t R, int64_t most) { return R / most + (E < R ? E : R); }

struct MoeSpace {
  size_t up, down, weights, mid, end;
};
static MoeSpace moe_space(int64_t T, int64_t E, int64_t topk, int64_t I) {
  const int64_t R = T * topk;
  MoeSpace s;
  s.up = 16;
  s.down = s.up + up16(sizeof(MoeTile) * (size_t)most_tiles(E, R, kUpRows));
  s.weights = s.down + up16(sizeof(MoeTile) * (size_t)most_tiles(E, R, kDownRows));
  s.mid = s.weights + up16((size_t)R * 4);
  s.end = s.mid + up16((size_t)(2 * R * I) * 2);
  return s;
}

size_t moe_workspace(int64_t T, int64_t E, int64_t topk, int64_t I) {
  return T == 0 ? 0 : moe_space(T, E, topk, I).end;
}

template <int FMT, bool F16, int NX, int NM>
static hipError_t moe_stream(const MoeArgs& p, int64_t tiles, hipStream_t stream) {
  constexpr int WU = 4, DU = 2, WD = 8, DD = 2;
  hipLaunchKernelGGL((moe_up_kernel<FMT, F16, NX, WU, DU>), dim3((unsigned)(tiles * p.NT)), dim3(64 * WU), 0, stream, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<FMT, F16, NM, WD, DD>), dim3((unsigned)(p.H / 16)), dim3(64 * WD),
                     (size_t)WD * p.T * 64 + sizeof(MoeTile) * (size_t)most_tiles(p.E, (int64_t)p.T * p.topk, kDownRows), stream, p);
  return hipGetLastError();
}

template <int FMT, bool F16>
static hipError_t moe_go(MoeArgs& p, hipStream_t stream) {
  const int64_t R = (int64_t)p.T * p.topk;
  p.NT = p.I / 16;
  if (!p.inl) {
    const bool general = p.route.bias || p.route.G > 1;
    const size_t keys = p.route.G > 1 ? (size_t)8 * p.E * (kPThreads / kWave) : 0;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(1), dim3(kPThreads), keys, stream, p); };
    if (p.E <= 64) general ? go(moe_plan_kernel<1, true>) : go(moe_plan_kernel<1, false>);
    else if (p.E <= 256) general ? go(moe_plan_kernel<4, true>) : go(moe_plan_kernel<4, false>);
    else general ? go(moe_plan_kernel<16, true>) : go(moe_plan_kernel<16, false>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // up to 2 tokens tiles have at most 2 rows
  constexpr int C = kCols<FMT> / 128;
  return p.T <= 2 ? moe_stream<FMT, F16, 1, C>(p, p.inl ? (R < p.E ? R : p.E) : most_tiles(p.E, R, kUpRows), stream)
                  : moe_stream<FMT, F16, 2 * C, 2 * C>(p, most_tiles(p.E, R, kUpRows), stream);
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
