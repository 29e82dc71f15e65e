// The whole routed-expert layer for a few tokens (T <= 32), weights only
// quantized: router logits and hidden rows in, the experts' weighted sum out.
//
//   out[t] = sum_j w[t, j] * W2[e] (silu(W1[e] x[t]) * (W3[e] x[t]))  (+ add[t]),  e = ids[t, j]
//
// With so few rows the time is the chosen experts' weights, each read once. Two
// kernels: gate and up products with the activation, then the down products with
// the sum over a token's experts. Up to kInline tokens the first one routes too,
// every block for itself (a wave per token, a microsecond); more tokens are
// routed by w4_route's kernel before it, once instead of once per block.
//
// Both are streams of weights through the matrix unit, 16 weight rows as its A
// operand, up to 16 tokens (RT times) as its B operand, nothing staged in LDS: a
// weight byte is used by one wave only. Weights become bf16 (exactly, with MXFP4's
// scale applied; a product with v_mfma_f32_16x16x32_bf16), or fp16 for fp16
// activations of FP8 and int4 weights. A wave's K step is 128 columns, lane (row
// l16, group g) holding 32 of them. FP8's and int4's scales multiply the sums of a
// step or group.
//
// What lies between the two is rounded to 16 bits of mantissa: the sum of two bf16
// numbers, each of which goes through the matrix unit (2^-17 relative, below what
// the output's own rounding leaves visible). MXFP4 with fp16 activations takes x
// apart in the same way, exactly (11 bits).
#include <type_traits>

#include "mxfp4.h"
#include "route_token.h"

namespace w4 {

constexpr int kInline = 2;                           // tokens that the first kernel routes itself
constexpr int kInlineE = 256;
constexpr int kInlineRows = kInline * 64;
enum { kFp8 = 0, kMx = 1, kInt4 = 2 };

// The experts with rows: e, their first row in the plan, the mask of their tokens.
struct MoeSlot {
  int e, row0;
  uint32_t tokens;
  int pad;
};

struct MoeArgs {
  const uint16_t* x;
  const uint8_t *w13, *w2;
  const void *s13, *s2;
  const uint16_t* add;
  uint16_t* out;
  int T, E, topk, H, I;
  int G13, G2;                                       // int4: scale groups along K
  int kg13, kg2;                                     // and K steps per group
  int NT;                                            // column tiles of the launch
  int inl;                                           // the first kernel routes
  // workspace
  int32_t* nslots;
  MoeSlot* slots;
  uint16_t *hi, *lo;                                 // [R][I]: the middle, as two bf16
  RouteArgs route;                                   // ids .. row_of in the workspace too (not inl)
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

// The weights of a lane for one K step (16 rows x 128 columns of a wave).
// FP8: the 16-byte chunks g and g + 4 of the row's 128 bytes; MXFP4: the row's
// block g and the step's scale word; int4: the unit (row, g) of its tile.
template <int FMT>
struct Weights {
  v4i q[FMT == kFp8 ? 2 : 1];
  uint32_t s;
};

// The lane's columns of MFMA c (0..3), as 16-byte pieces of 8 activations: FP8:
// columns 64 (c / 2) + 16 g + 8 (c % 2) ..; MXFP4: 32 g + 8 c ..; int4: 32 g + 4 c
// .. + 3 and 16 after them. A lane loads four pieces X[0..3]; this is MFMA c's.
template <int FMT>
__device__ __forceinline__ int piece_column(int g, int c) {
  return FMT == kFp8 ? 64 * (c / 2) + 16 * g + 8 * (c % 2) : 32 * g + 8 * c;
}
template <int FMT>
__device__ __forceinline__ v4i piece(const v4i (&X)[4], int c) {
  if constexpr (FMT == kInt4) {
    const v4i a = X[c / 2], b = X[2 + c / 2];
    return c % 2 ? v4i{a[2], a[3], b[2], b[3]} : v4i{a[0], a[1], b[0], b[1]};
  } else {
    return X[c];
  }
}

// MFMA c's 8 weights. int4 codes come as the code itself, 0..15 (E4M3's codes 0..15
// are 0..15 times 2^-9); the caller starts the sum from -8 sum x.
template <int FMT, bool F16>
__device__ __forceinline__ typename Operand<F16>::V decode(const Weights<FMT>& w, int c, float scale) {
  v4i r;
  if constexpr (FMT == kFp8) {
    const int lo = w.q[c / 2][2 * (c % 2)], hi = w.q[c / 2][2 * (c % 2) + 1];
    r = v4i{cvt_fp8<F16>(lo, 1.0f, false), cvt_fp8<F16>(lo, 1.0f, true), cvt_fp8<F16>(hi, 1.0f, false),
            cvt_fp8<F16>(hi, 1.0f, true)};
  } else if constexpr (FMT == kMx) {
    static_assert(!F16, "its scales need bf16's range");
    const uint32_t v = (uint32_t)w.q[0][c];
    r = v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0)),
            __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1)),
            __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2)),
            __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3))};
  } else {
    const uint32_t v = (uint32_t)w.q[0][c] ^ 0x88888888u;
    const int lo = (int)(v & 0x0F0F0F0Fu), hi = (int)((v >> 4) & 0x0F0F0F0Fu);
    r = v4i{cvt_fp8<F16>(lo, 512.0f, false), cvt_fp8<F16>(lo, 512.0f, true), cvt_fp8<F16>(hi, 512.0f, false),
            cvt_fp8<F16>(hi, 512.0f, true)};
  }
  return __builtin_bit_cast(typename Operand<F16>::V, r);
}

// 16 rows of a weight matrix: rows n .. n + 15 of [N, K] of expert e. Reads past the
// matrix's end (its last, partial K step) give zeros.
template <int FMT>
struct Rows {
  __amdgpu_buffer_rsrc_t w, s;
  const void* scales;                                // FP8: the tile's row of block scales; int4: [G, N] at column n
  uint32_t off, soff;
  int N;
  __device__ __forceinline__ Rows(const uint8_t* base, const void* sc, int64_t e, int64_t N_, int64_t n, int64_t K, int G,
                                  int l16, int g) {
    N = (int)N_;
    if constexpr (FMT == kFp8) {
      w = make_rsrc(base + (e * N_ + n) * K, (uint32_t)(16 * K));
      off = (uint32_t)(l16 * K + 16 * g);
      scales = static_cast<const float*>(sc) + (e * ((N_ + 127) / 128) + n / 128) * ((K + 127) / 128);
    } else if constexpr (FMT == kMx) {
      w = make_rsrc(base + (e * N_ + n) * (K / 2), (uint32_t)(8 * K));
      off = (uint32_t)(l16 * (K / 2) + 16 * g);
      const int64_t ks = mx_scale_bytes(K);
      s = make_rsrc(static_cast<const uint8_t*>(sc) + (e * N_ + n) * ks, (uint32_t)(16 * ks));
      soff = (uint32_t)(l16 * ks);
    } else {
      // tiles [n / 128][k / 128] of 8 KiB, unit (n % 128) * 4 + g: the 16 rows are 1 KiB of each
      const int64_t kt = K / kTileK, tiles = (N_ + kTileN - 1) / kTileN * kt;
      w = make_rsrc(base + (e * tiles + n / kTileN * kt) * kTileBytes, (uint32_t)(kt * kTileBytes));
      off = (uint32_t)((n % kTileN + l16) * 64 + 16 * g);
      scales = static_cast<const uint16_t*>(sc) + e * (int64_t)G * N_ + n + 4 * g;
    }
  }
  __device__ __forceinline__ Weights<FMT> load(int kb, int left, int g) const {   // left: columns from the step's first
    Weights<FMT> r;
    if constexpr (FMT == kFp8) {
      r.q[0] = __builtin_amdgcn_raw_buffer_load_b128(w, 16 * g < left ? off : kPast, (uint32_t)kb * 128u, 0);
      r.q[1] = __builtin_amdgcn_raw_buffer_load_b128(w, 64 + 16 * g < left ? off + 64u : kPast, (uint32_t)kb * 128u, 0);
    } else if constexpr (FMT == kMx) {
      r.q[0] = __builtin_amdgcn_raw_buffer_load_b128(w, 32 * g < left ? off : kPast, (uint32_t)kb * 64u, 0);
      r.s = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(s, 32 * g < left ? soff : kPast, (uint32_t)kb * 4u, 0);
    } else {
      r.q[0] = __builtin_amdgcn_raw_buffer_load_b128(w, off, (uint32_t)kb * kTileBytes, 0);
    }
    return r;
  }
  // MXFP4: this lane's scale of the step
  __device__ __forceinline__ float lane_scale(const Weights<FMT>& r, int g) const {
    if constexpr (FMT != kMx) return 1.0f;
    const uint32_t c = r.s >> (8 * g) & 0xFF;
    return c == kMxNan ? __uint_as_float(0x7FC00000u) : mx_scale_value(c);
  }
  // what multiplies the step's sums of weight rows 4 g .. 4 g + 3
  __device__ __forceinline__ v4f sum_scale(int kb, int per_group) const {
    if constexpr (FMT == kFp8) {
      const float v = static_cast<const float*>(scales)[kb];
      return v4f{v, v, v, v};
    } else if constexpr (FMT == kInt4) {
      const v2i v = *reinterpret_cast<const v2i*>(static_cast<const uint16_t*>(scales) + (int64_t)(kb / per_group) * N);
      return v4f{f16_to_f32((uint16_t)v[0]), f16_to_f32((uint16_t)((uint32_t)v[0] >> 16)), f16_to_f32((uint16_t)v[1]),
                 f16_to_f32((uint16_t)((uint32_t)v[1] >> 16))};
    } else {
      return v4f{1.f, 1.f, 1.f, 1.f};
    }
  }
};

// fp16 pairs as the sum of two bf16 numbers each (exact: 11 bits, and bf16's range is wider). An infinity's remainder,
// a NaN, becomes a finite number, which changes nothing.
__device__ __forceinline__ void split_f16(v4i x, v4i& hi, v4i& lo) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const float a = f16_to_f32((uint16_t)x[d]), b = f16_to_f32((uint16_t)((uint32_t)x[d] >> 16));
    const uint32_t ha = f32_to_bf16_rne(a), hb = f32_to_bf16_rne(b);
    const float ra = fmaxf(a - __uint_as_float(ha << 16), -64.f), rb = fmaxf(b - __uint_as_float(hb << 16), -64.f);
    hi[d] = (int)(ha | hb << 16);
    lo[d] = (int)((uint32_t)f32_to_bf16_rne(ra) | (uint32_t)f32_to_bf16_rne(rb) << 16);
  }
}

__device__ __forceinline__ v8bf bf(v4i v) { return __builtin_bit_cast(v8bf, v); }

// Everything a block of the first kernel has to know: its expert and the rows.
struct MoeWork {
  int e, row0, rows;
};

// The plan of up to kInline tokens in LDS, by one block: routes, orders the pairs
// by expert and token, and lists the experts. Block 0 leaves the list in the workspace.
struct InlinePlan {
  int t[kInlineRows];
  float w[kInlineRows];
  int raw_e[kInlineRows];
  float raw_w[kInlineRows];
  MoeSlot slot[kInlineRows];
  int nslots;
  double keys[kInline][kInlineE];
};

__device__ __forceinline__ void plan_inline(const MoeArgs& p, InlinePlan& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const RouteArgs& a = p.route;
  if (wave < p.T) {
    int id;
    double w;
    if (a.bias || a.G > 1) {
      const LaneExperts<kInlineE / 64, true> own(a, lane);
      route_token<3, kInlineE / 64, true>(a, wave, lane, own, s.keys[wave], id, w);
    } else {
      const LaneExperts<kInlineE / 64, false> own(a, lane);
      route_token<3, kInlineE / 64, false>(a, wave, lane, own, s.keys[wave], id, w);
    }
    if (lane < p.topk) {
      s.raw_e[wave * p.topk + lane] = id;
      s.raw_w[wave * p.topk + lane] = (float)(w * a.scale);
    }
  }
  __syncthreads();
  // One wave: lane i holds both tokens' choice i. A pair's row counts the pairs before it, its slot the experts.
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
      s.t[r0] = 0;
      s.w[r0] = s.raw_w[lane];
      s.slot[s0] = MoeSlot{e0, r0, dup0 ? 3u : 1u, 0};
    }
    if (e1 >= 0) {
      s.t[r1] = 1;
      s.w[r1] = s.raw_w[p.topk + lane];
      if (!dup1) s.slot[s1] = MoeSlot{e1, r1, 2u, 0};
    }
    const int n = __popcll(__ballot(e0 >= 0)) + __popcll(__ballot(e1 >= 0 && !dup1));
    if (lane == 0) s.nslots = n;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = tid; i < s.nslots; i += blockDim.x) p.slots[i] = s.slot[i];
    if (tid == 0) *p.nslots = s.nslots;
  }
}

// The list of experts from the plan's offsets, by the first block's first wave.
__device__ __forceinline__ void list_slots(const MoeArgs& p) {
  const int lane = threadIdx.x;
  const RouteArgs& a = p.route;
  int n = 0;
  for (int c = 0; c < p.E; c += 64) {
    const int e = c + lane;
    const int r0 = e < p.E ? a.offsets[e] : 0, r1 = e < p.E ? a.offsets[e + 1] : 0;
    const unsigned long long have = __ballot(r1 > r0);
    if (r1 > r0) {
      uint32_t tokens = 0;
      for (int r = r0; r < r1; ++r) tokens |= 1u << a.row_token[r];
      p.slots[n + __popcll(have & ((1ull << lane) - 1))] = MoeSlot{e, r0, tokens, 0};
    }
    n += __popcll(have);
  }
  if (lane == 0) *p.nslots = n;
}

// Gate and up: WS waves of a block take the K steps of 16 gate rows and the 16 up
// rows beside them in turn.
template <int FMT, bool XF16, int RT, int WS, int U>
__global__ __launch_bounds__(64 * WS) void moe_up_kernel(MoeArgs p) {
  constexpr bool OPF16 = XF16 && FMT != kMx;         // the operands' type
  constexpr int PARTS = XF16 && FMT == kMx ? 2 : 1;
  __shared__ union {
    InlinePlan plan;
    v4f red[WS][2 * RT][64];
  } s;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  MoeWork k;
  int tn = (int)blockIdx.x % p.NT;
  int token[RT], mine[RT];                           // this lane's activation row, and that of the results it keeps
  float weight[RT];
  if (p.inl) {
    plan_inline(p, s.plan);
    const int sl = (int)blockIdx.x / p.NT;
    if (sl >= s.plan.nslots) return;
    k.e = __builtin_amdgcn_readfirstlane(s.plan.slot[sl].e);
    k.row0 = __builtin_amdgcn_readfirstlane(s.plan.slot[sl].row0);
    k.rows = __builtin_amdgcn_readfirstlane(__popc(s.plan.slot[sl].tokens));
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int i = 16 * r + l16;
      token[r] = i < k.rows ? s.plan.t[k.row0 + i] : -1;
      weight[r] = i < k.rows ? s.plan.w[k.row0 + i] : 0.f;
      mine[r] = k.row0 + i;
    }
    __syncthreads();                                 // the plan's place becomes the sums'
  } else {
    if (blockIdx.x == gridDim.x - 1 && wave == 0) list_slots(p);
    struct { const int32_t* offsets; int E, NT; int64_t R; } f{p.route.offsets, p.E, p.NT, (int64_t)p.T * p.topk};
    const Segment seg = find_segment<16 * RT>(f);
    if (seg.e < 0) return;
    k.e = seg.e;
    k.row0 = (int)seg.row0;
    k.rows = (int)seg.rows;
    tn = seg.tn;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int i = 16 * r + l16;
      token[r] = i < k.rows ? p.route.row_token[k.row0 + i] : -1;
      mine[r] = k.row0 + i;
      weight[r] = 0.f;
      if (i < k.rows)
        for (int j = 0; j < p.topk; ++j)
          if (p.route.row_of[token[r] * p.topk + j] == mine[r]) weight[r] = p.route.weights[token[r] * p.topk + j];
    }
  }
  const int KB = (p.H + 127) / 128, n0 = 16 * tn;
  const Rows<FMT> wg(p.w13, p.s13, k.e, 2 * (int64_t)p.I, n0, p.H, p.G13, l16, g);
  const Rows<FMT> wu(p.w13, p.s13, k.e, 2 * (int64_t)p.I, p.I + n0, p.H, p.G13, l16, g);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(p.x, (uint32_t)(p.T * (int64_t)p.H * 2));
  uint32_t xo[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) xo[r] = token[r] >= 0 ? (uint32_t)((int64_t)token[r] * p.H * 2) : kPast;

  v4f ag[RT], au[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) ag[r] = au[r] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < KB; kb += WS * U) {
    Weights<FMT> qg[U], qu[U];
    v4i X[U][RT][4];
    v4f sg[U], su[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kk = min(kb + WS * u, KB - 1);       // past the end: loaded again, not used
      const int left = p.H - 128 * kk;
      qg[u] = wg.load(kk, left, g);
      qu[u] = wu.load(kk, left, g);
      sg[u] = wg.sum_scale(kk, p.kg13);
      su[u] = wu.sum_scale(kk, p.kg13);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = piece_column<FMT>(g, c);
          X[u][r][c] = __builtin_amdgcn_raw_buffer_load_b128(xr, col < left && xo[r] != kPast ? xo[r] + 2 * col : kPast,
                                                             256u * (uint32_t)kk, 0);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + WS * u >= KB) break;
      const float lg = wg.lane_scale(qg[u], g), lu = wu.lane_scale(qu[u], g);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (16 * r >= k.rows) break;
        v4f dg = v4f{0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT == kInt4) {                // -8 sum x
          const int m8 = OPF16 ? (int)0xC800C800 : (int)0xC100C100;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            dg = mfma16<OPF16>(__builtin_bit_cast(typename Operand<OPF16>::V, v4i{m8, m8, m8, m8}),
                               __builtin_bit_cast(typename Operand<OPF16>::V, piece<FMT>(X[u][r], c)), dg);
        }
        v4f du = dg;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const v4i xp = piece<FMT>(X[u][r], c);
          const auto a = decode<FMT, OPF16>(qg[u], c, lg), b = decode<FMT, OPF16>(qu[u], c, lu);
          if constexpr (PARTS == 2) {
            v4i hi, lo;
            split_f16(xp, hi, lo);
            dg = mfma16<false>(a, bf(lo), dg);
            du = mfma16<false>(b, bf(lo), du);
            dg = mfma16<false>(a, bf(hi), dg);
            du = mfma16<false>(b, bf(hi), du);
          } else {
            const auto x = __builtin_bit_cast(typename Operand<OPF16>::V, xp);
            dg = mfma16<OPF16>(a, x, dg);
            du = mfma16<OPF16>(b, x, du);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          ag[r][q] = FMT == kMx ? ag[r][q] + dg[q] : fmaf(dg[q], sg[u][q], ag[r][q]);
          au[r][q] = FMT == kMx ? au[r][q] + du[q] : fmaf(du[q], su[u][q], au[r][q]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    s.red[wave][2 * r][lane] = ag[r];
    s.red[wave][2 * r + 1][lane] = au[r];
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (16 * r + l16 >= k.rows) break;
    v4f vg = s.red[0][2 * r][lane], vu = s.red[0][2 * r + 1][lane];
#pragma unroll
    for (int w = 1; w < WS; ++w) {
      vg += s.red[w][2 * r][lane];
      vu += s.red[w][2 * r + 1][lane];
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float m = vg[q] / (1.0f + expf(-vg[q])) * vu[q] * weight[r];
      hi[q] = f32_to_bf16_rne(m);
      // (an infinity has no remainder)
      const float rest = m - __uint_as_float(hi[q] << 16);
      lo[q] = (hi[q] & 0x7F80u) != 0x7F80u ? f32_to_bf16_rne(rest) : 0u;
    }
    const int64_t at = (int64_t)mine[r] * p.I + n0 + 4 * g;
    *reinterpret_cast<v2i*>(p.hi + at) = v2i{(int)(hi[0] | hi[1] << 16), (int)(hi[2] | hi[3] << 16)};
    *reinterpret_cast<v2i*>(p.lo + at) = v2i{(int)(lo[0] | lo[1] << 16), (int)(lo[2] | lo[3] << 16)};
  }
}

// Down: a block owns 16 output columns of all tokens; its waves take the (expert, K
// step) pairs in turn. The matrix unit's columns are the tokens themselves, so the
// sum over a token's experts is the accumulator's own.
template <int FMT, bool F16OUT, int RT, int WS, int U>
__global__ __launch_bounds__(64 * WS) void moe_down_kernel(MoeArgs p) {
  __shared__ v4f red[WS][RT][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int n0 = 16 * (int)blockIdx.x;
  const int KB = (p.I + 127) / 128, items = *p.nslots * KB;
  const __amdgpu_buffer_rsrc_t hr = make_rsrc(p.hi, (uint32_t)((int64_t)p.T * p.topk * p.I * 2));
  const __amdgpu_buffer_rsrc_t lr = make_rsrc(p.lo, (uint32_t)((int64_t)p.T * p.topk * p.I * 2));
  v4f acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int it = wave; it < items; it += WS * U) {
    Weights<FMT> qw[U];
    v4i H[U][RT][4], L[U][RT][4];
    v4f sw[U];
    float ls[U];
    uint32_t tokens[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(it + WS * u, items - 1);     // past the end: loaded again, not used
      const int sl = i / KB, kb = i - sl * KB, left = p.I - 128 * kb;
      const MoeSlot slot = p.slots[sl];
      const Rows<FMT> w(p.w2, p.s2, slot.e, p.H, n0, p.I, p.G2, l16, g);
      qw[u] = w.load(kb, left, g);
      sw[u] = w.sum_scale(kb, p.kg2);
      tokens[u] = slot.tokens;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int t = 16 * r + l16;
        const bool has = slot.tokens >> t & 1;
        const uint32_t row = (uint32_t)((int64_t)(slot.row0 + __popc(slot.tokens & ((1u << t) - 1))) * p.I * 2);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = piece_column<FMT>(g, c);
          const uint32_t off = has && col < left ? row + 2 * col : kPast;
          H[u][r][c] = __builtin_amdgcn_raw_buffer_load_b128(hr, off, 256u * (uint32_t)kb, 0);
          L[u][r][c] = __builtin_amdgcn_raw_buffer_load_b128(lr, off, 256u * (uint32_t)kb, 0);
        }
      }
      ls[u] = w.lane_scale(qw[u], g);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (it + WS * u >= items) break;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (!(tokens[u] >> (16 * r) & 0xFFFFu)) continue;
        v4f d = v4f{0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT == kInt4) {
          const int m8 = (int)0xC100C100;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            d = mfma16<false>(bf(v4i{m8, m8, m8, m8}), bf(piece<FMT>(L[u][r], c)), d);
            d = mfma16<false>(bf(v4i{m8, m8, m8, m8}), bf(piece<FMT>(H[u][r], c)), d);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const v8bf a = decode<FMT, false>(qw[u], c, ls[u]);
          d = mfma16<false>(a, bf(piece<FMT>(L[u][r], c)), d);
          d = mfma16<false>(a, bf(piece<FMT>(H[u][r], c)), d);
        }
        // a token that did not choose this expert takes nothing of it, not even NaN
        const bool has = tokens[u] >> (16 * r + l16) & 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = FMT == kMx ? acc[r][q] + d[q] : fmaf(d[q], sw[u][q], acc[r][q]);
          acc[r][q] = has ? v : acc[r][q];
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) red[wave][r][lane] = acc[r];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int t = 16 * r + l16;
    if (t >= p.T) break;
    v4f v = red[0][r][lane];
#pragma unroll
    for (int w = 1; w < WS; ++w) v += red[w][r][lane];
    const int64_t at = (int64_t)t * p.H + n0 + 4 * g;
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (p.add) v[q] += F16OUT ? f16_to_f32(p.add[at + q]) : bf16_to_f32(p.add[at + q]);
      o[q] = F16OUT ? f32_to_f16_rne(v[q]) : f32_to_bf16_rne(v[q]);
    }
    *reinterpret_cast<v2i*>(p.out + at) = v2i{(int)(o[0] | o[1] << 16), (int)(o[2] | o[3] << 16)};
  }
}

// ---- workspace: the list of experts, the middle, then (not routed inline) the route's own
static size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

struct MoeSpace {
  size_t slots, hi, lo, ids, weights, row_token, offsets, row_of, end;
};
static MoeSpace moe_space(int64_t T, int64_t E, int64_t topk, int64_t I) {
  const size_t R = (size_t)(T * topk);
  MoeSpace s;
  s.slots = 16;
  s.hi = s.slots + sizeof(MoeSlot) * (size_t)(E < (int64_t)R ? E : (int64_t)R);
  s.lo = s.hi + up16(R * (size_t)I * 2);
  s.ids = s.lo + up16(R * (size_t)I * 2);
  s.weights = s.ids + up16(R * 4);
  s.row_token = s.weights + up16(R * 4);
  s.offsets = s.row_token + up16(R * 4);
  s.row_of = s.offsets + up16((size_t)(E + 1) * 4);
  s.end = s.row_of + up16(R * 4);
  return s;
}

size_t moe_workspace(int64_t T, int64_t E, int64_t topk, int64_t I) {
  return T == 0 ? 0 : moe_space(T, E, topk, I).end;
}

hipError_t launch_route(const void* x, int dt, int64_t T, int64_t E, int64_t ld, int score, const float* bias,
                        int64_t G, int64_t topk_groups, int64_t group_top, int64_t topk, bool renorm, double scale,
                        int32_t* ids, float* weights, int32_t* row_token, int32_t* offsets, int32_t* row_of,
                        void* ws, hipStream_t stream);

template <int FMT, bool F16, int RT>
static hipError_t moe_go(MoeArgs& p, hipStream_t stream) {
  constexpr int WU = 4, WD = 8;
  const int64_t R = (int64_t)p.T * p.topk;
  p.NT = p.I / 16;
  const int64_t blocks = p.inl ? (R < p.E ? R : p.E) * p.NT : grouped_blocks(p.E, R, p.I, 16 * RT, 16);
  hipLaunchKernelGGL((moe_up_kernel<FMT, F16, RT, WU, 2>), dim3((unsigned)blocks), dim3(64 * WU), 0, stream, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<FMT, F16, RT, WD, RT == 1 ? 2 : 1>), dim3((unsigned)(p.H / 16)), dim3(64 * WD), 0,
                     stream, p);
  return hipGetLastError();
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
  p.nslots = reinterpret_cast<int32_t*>(base);
  p.slots = reinterpret_cast<MoeSlot*>(base + sp.slots);
  p.hi = reinterpret_cast<uint16_t*>(base + sp.hi);
  p.lo = reinterpret_cast<uint16_t*>(base + sp.lo);
  RouteArgs& a = p.route;
  a.x = logits; a.bias = bias; a.T = T; a.ld = ld; a.dt = dt;
  a.E = (int)E; a.topk = (int)topk; a.G = (int)G; a.per_group = (int)(E / G);
  a.topk_groups = (int)topk_groups; a.group_top = (int)group_top; a.score = score; a.renorm = renorm ? 1 : 0;
  a.scale = scale;
  a.ids = reinterpret_cast<int32_t*>(base + sp.ids);
  a.weights = reinterpret_cast<float*>(base + sp.weights);
  a.row_token = reinterpret_cast<int32_t*>(base + sp.row_token);
  a.offsets = reinterpret_cast<int32_t*>(base + sp.offsets);
  a.row_of = reinterpret_cast<int32_t*>(base + sp.row_of);
  p.inl = T <= kInline && E <= kInlineE;
  if (!p.inl) {
    const hipError_t e = launch_route(logits, dt, T, E, ld, score, bias, G, topk_groups, group_top, topk, renorm, scale,
                                      a.ids, a.weights, a.row_token, a.offsets, a.row_of, nullptr, stream);
    if (e != hipSuccess) return e;
  }
  auto by_rows = [&](auto f, auto h) {
    constexpr int F = decltype(f)::value;
    constexpr bool X = decltype(h)::value;
    return T <= 16 ? moe_go<F, X, 1>(p, stream) : moe_go<F, X, 2>(p, stream);
  };
  auto by_type = [&](auto f) { return f16 ? by_rows(f, std::true_type{}) : by_rows(f, std::false_type{}); };
  if (fmt == kFp8) return by_type(std::integral_constant<int, kFp8>{});
  if (fmt == kMx) return by_type(std::integral_constant<int, kMx>{});
  return by_type(std::integral_constant<int, kInt4>{});
}

}  // namespace w4
