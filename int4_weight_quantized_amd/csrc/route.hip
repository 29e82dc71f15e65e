// Routing of tokens to experts, and the row plan the grouped products read.
//
// Per token, in fp64 (the choice is between near values):
//   s = softmax(x) or 1 / (1 + exp(-x)); NaN and -inf logits are closed,
//       +inf counts as the largest fp32
//   c = s + bias;  key = x without a bias, c with one
//   groups of E / G consecutive experts: a group's value is the sum of its
//   group_top best c; the topk_groups best groups stay open
//   ids = the topk largest open keys, lowest index first among equals; -1
//   where none is left;  weight = s [/ sum of the chosen s] * scale
// The plan orders the rows (token, slot) by expert, then token:
//   offsets[e] .. offsets[e+1] are expert e's rows, row_token names each
//   row's token (-1 past the last), row_of is the inverse (-1 for none).
//
// Up to 256 experts, 16 lanes route one token (a wave four), each holding V
// consecutive experts: the argmax rounds exchange within a row of 16 lanes,
// by DPP, and all 64 tokens of a block go through at once. More experts, and
// groups that do not fall on whole lanes, take one wave per token, expert
// j * 64 + lane in register j. 16384 tokens of 256 experts in 8 groups take 32
// us (26 and, for the plan's kernel, 7): 256 blocks run through once, about 8
// us of it their latency, 10 the fp64 scores (own exponentials over several
// experts at a time spilled and gained nothing), 8 the argmax rounds. 8192 of
// 64 experts take 11.2. One wave per token: 16384 of 512 experts 54 us, of 1024
// 72; with a bias and sigmoid scores 384 experts 68 us, 1024 124 (its 16 keys
// in fp64 spill 69 registers).
// A block takes kTok = 64 tokens, so that a token is one bit of a 64-bit mask
// per expert: the rank of (token, expert) inside the block is the number of
// lower bits set, which needs no sort and no order of atomics. One block does
// the whole plan up to 64 tokens; above, it leaves its counts per expert (a
// byte each) and a second kernel places the rows: each of its blocks adds up
// all blocks' counts, which are few and lie in the L2. Where that square of
// reads passes 128 MiB a kernel between them scans the counts (64 experts: 16384
// tokens 12 us summed, 18 scanned, 65536 36 and 52; 256 experts: 32768 tokens
// 36 and 42, 65536 79 and 73, 131072 210 and 140).
#include "w4_device.h"

namespace w4 {

constexpr int kTok = 64;                 // tokens per block
constexpr int kRThreads = 1024;
constexpr int kRWaves = kRThreads / kWave;
constexpr int kMaxE = 1024;

struct RouteArgs {
  const void* x;
  const float* bias;
  int64_t T, ld;
  int E, topk, G, per_group, topk_groups, group_top, score, renorm;
  double scale;
  int32_t *ids, *row_token, *offsets, *row_of;
  float* weights;
  uint8_t* counts;                       // [blocks][ceil(E / 4) * 4]; null: one block
  int32_t* prefix;                       // where the counts are scanned: those before each block [blocks][E], totals [E]
  int vec;                               // rows of logits are aligned for whole-lane loads
};

// All lanes' best of L consecutive lanes (16: DPP inside a row of 16; 64: two
// exchanges more), op(own, other).
template <int CTRL>
__device__ __forceinline__ int dpp(int v) { return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false); }
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)dpp<CTRL>((int)b), hi = (uint32_t)dpp<CTRL>((int)(b >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) { return __int_as_float(dpp<CTRL>(__float_as_int(v))); }

template <int L, typename T, typename F>
__device__ __forceinline__ T lanes_reduce(T v, F op) {
  v = op(v, dpp<0xB1>(v));               // lane ^ 1
  v = op(v, dpp<0x4E>(v));               // lane ^ 2
  v = op(v, dpp<0x141>(v));              // mirror of 8 lanes: the other four
  v = op(v, dpp<0x140>(v));              // mirror of 16: the other eight
  if constexpr (L == 64) {
    v = op(v, __shfl_xor(v, 16, kWave));
    v = op(v, __shfl_xor(v, 32, kWave));
  }
  return v;
}
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
  return lanes_reduce<L>(v, [](double a, double b) { return a + b; });
}

// The best (largest key, then lowest id) of the wave.
template <int CTRL>
__device__ __forceinline__ void best_step(double& key, int& id) {
  const double o = dpp<CTRL>(key);
  const int oi = dpp<CTRL>(id);
  if (o > key || (o == key && oi < id)) {
    key = o;
    id = oi;
  }
}
__device__ __forceinline__ void wave_best(double& key, int& id) {
  best_step<0xB1>(key, id);
  best_step<0x4E>(key, id);
  best_step<0x141>(key, id);
  best_step<0x140>(key, id);
#pragma unroll
  for (int off = 16; off <= 32; off <<= 1) {
    const double o = __shfl_xor(key, off, kWave);
    const int oi = __shfl_xor(id, off, kWave);
    if (o > key || (o == key && oi < id)) {
      key = o;
      id = oi;
    }
  }
}

constexpr float kF32Max = 3.40282347e38f;

template <int DT>
__device__ __forceinline__ float load_logit(const void* x, int64_t i) {
  if constexpr (DT == 2) return static_cast<const float*>(x)[i];
  const uint16_t v = static_cast<const uint16_t*>(x)[i];
  return DT == 0 ? bf16_to_f32(v) : f16_to_f32(v);
}

// Inclusive sum over the wave.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int o = __shfl_up(v, off, kWave);
    if (lane >= off) v += o;
  }
  return v;
}

// Exclusive sum over the block's threads (one value each); returns the total
// through `total`. red: kRWaves ints of LDS.
__device__ __forceinline__ int block_scan(int v, int* red, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int inc = wave_scan(v, lane);
  if (lane == 63) red[wave] = inc;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kRWaves; ++w) {
    const int r = red[w];
    if (w < wave) before += r;
    sum += r;
  }
  __syncthreads();
  total = sum;
  return before + inc - v;
}

__device__ __forceinline__ double score_of(float x, int score, float top) {
  return score == 0 ? exp((double)x - (double)top) : 1.0 / (1.0 + exp(-(double)x));
}

// Place the rows of this block's tokens. mask[e]: the block's tokens that
// chose e; base[e]: the plan row of the first of them.
__device__ __forceinline__ void place_rows(const RouteArgs& a, int64_t t0, int tokens, const int32_t* ids,
                                           const unsigned long long* mask, const int* base, int total) {
  const int items = tokens * a.topk;
  for (int i = threadIdx.x; i < items; i += kRThreads) {
    const int tl = i / a.topk;
    const int64_t at = t0 * a.topk + i;
    const int e = ids[i];
    int row = -1;
    if (e >= 0) {
      row = base[e] + __popcll(mask[e] & ((1ull << tl) - 1));
      a.row_token[row] = (int32_t)(t0 + tl);
    }
    a.row_of[at] = row;
    if (at >= total) a.row_token[at] = -1;
  }
}

// The end of a routing block: its counts, or (one block) the plan itself.
__device__ __forceinline__ void finish_block(const RouteArgs& a, int64_t t0, int tokens, const int32_t* s_ids,
                                             const unsigned long long* mask, int* base, int* red) {
  const int tid = threadIdx.x;
  __syncthreads();
  const int cnt = tid < a.E ? __popcll(mask[tid]) : 0;
  if (a.counts) {
    const int ep = (a.E + 3) & ~3;
    if (tid < ep) a.counts[(int64_t)blockIdx.x * ep + tid] = (uint8_t)cnt;
    return;
  }
  int total;
  const int start = block_scan(cnt, red, total);
  if (tid < a.E) {
    base[tid] = start;
    a.offsets[tid] = start;
  }
  if (tid == 0) a.offsets[a.E] = total;
  __syncthreads();
  place_rows(a, t0, tokens, s_ids, mask, base, total);
}

__device__ __forceinline__ float max_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double max_of(double a, double b) { return fmax(a, b); }
// A chosen key: below every open one (their magnitude is an fp32's). Of a
// double only the high word is written.
__device__ __forceinline__ float shut(float) { return -__builtin_inff(); }
__device__ __forceinline__ double shut(double v) { return __hiloint2double((int)0xFFEFFFFFu, __double2loint(v)); }
template <typename K>
__device__ __forceinline__ K shut_below() { return sizeof(K) == 8 ? (K)-1e300 : -(K)__builtin_inff(); }

// 16 lanes per token, V consecutive experts per lane (E <= 16 V). K: the key,
// float (the logit) or double (a bias or groups). Groups cover GL = per_group
// / V whole lanes, a power of two.
template <int DT, int V, typename K>
__global__ __launch_bounds__(kRThreads) void route_rows_kernel(RouteArgs a) {
  constexpr bool GENERAL = sizeof(K) == 8;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem);
  int32_t* s_ids = reinterpret_cast<int32_t*>(mask + a.E);
  int* base = s_ids + kTok * a.topk;
  int* red = base + a.E;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, tl = tid >> 4;
  for (int e = tid; e < a.E; e += kRThreads) mask[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTok, t = t0 + tl;
  const int tokens = (int)min((int64_t)kTok, a.T - t0);
  const bool real = tl < tokens;
  const int e0 = l16 * V;
  constexpr float kClosed = -__builtin_inff();
  const K kLow = -(K)__builtin_inff();

  float x[V];
  if (a.vec && real && e0 + V <= a.E) {
    if constexpr (DT == 2) {
      const float* q = static_cast<const float*>(a.x) + t * a.ld + e0;
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const v4f v = *reinterpret_cast<const v4f*>(q + j);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[j + c] = v[c];
      }
    } else {
      const uint16_t* q = static_cast<const uint16_t*>(a.x) + t * a.ld + e0;
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const v2i v = *reinterpret_cast<const v2i*>(q + j);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint16_t h = (uint16_t)((uint32_t)v[c / 2] >> (16 * (c % 2)));
          x[j + c] = DT == 0 ? bf16_to_f32(h) : f16_to_f32(h);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = real && e0 + j < a.E ? load_logit<DT>(a.x, t * a.ld + e0 + j) : kClosed;
  }
  float top = kClosed;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    x[j] = x[j] > kClosed ? fminf(x[j], kF32Max) : kClosed;   // NaN: closed
    top = fmaxf(top, x[j]);
  }
  if (a.score == 0) top = lanes_reduce<16>(top, [](float p, float q) { return fmaxf(p, q); });
  if (!(top > kClosed)) top = 0.f;                   // every expert closed: no score is used
  K key[V];
  double sum = 1.0;
  if (GENERAL || (a.score == 0 && !a.renorm)) {
    double part = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double p = x[j] > kClosed ? score_of(x[j], a.score, top) : 0.0;
      if constexpr (GENERAL) key[j] = p;
      part += p;
    }
    if (a.score == 0) sum = fmax(lanes_sum<16>(part), 1e-300);
  }
  if constexpr (GENERAL) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double c = (a.score == 0 ? key[j] / sum : key[j]) +
                       (double)(a.bias && e0 + j < a.E ? a.bias[e0 + j] : 0.f);
      key[j] = (x[j] > kClosed && c > kLow) ? c : kLow;   // a NaN or -inf bias closes its expert
    }
    if (a.G > 1) {
      const int GL = a.per_group / V;                // lanes per group
      double b0 = kLow, b1 = kLow;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        b1 = fmax(b1, fmin(b0, key[j]));
        b0 = fmax(b0, key[j]);
      }
      for (int off = 1; off < GL; off <<= 1) {
        const double o0 = __shfl_xor(b0, off, kWave), o1 = __shfl_xor(b1, off, kWave);
        b1 = fmax(fmax(b1, o1), fmin(b0, o0));
        b0 = fmax(b0, o0);
      }
      const double value = (a.group_top == 2 && b1 > kLow) ? b0 + b1 : b0;
      const int g = l16 / GL;
      int before = 0;                                // groups that rank before this lane's
      for (int h = 0; h < a.G; ++h) {
        const double o = __shfl(value, (lane & 48) + h * GL, kWave);
        before += (o > value || (o == value && h < g)) ? 1 : 0;
      }
      if (before >= a.topk_groups) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = kLow;
      }
    }
    if (!a.bias) {                                   // the key is the logit itself
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = key[j] > kLow ? (double)x[j] : kLow;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = x[j];
  }

  // topk rounds of argmax; lane i of the token's 16 keeps choices i, 16 + i, ..
  int mine[4] = {-1, -1, -1, -1};
  double part = 0.0;
  double w[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    for (int i = 16 * q; i < min(a.topk, 16 * q + 16); ++i) {
      K best = key[0];
#pragma unroll
      for (int j = 1; j < V; ++j) best = max_of(best, key[j]);
      best = lanes_reduce<16>(best, [](K p, K q) { return max_of(p, q); });
      int id = 0x7FFFFFFF;
#pragma unroll
      for (int j = V - 1; j >= 0; --j) id = key[j] == best ? e0 + j : id;
      id = lanes_reduce<16>(id, [](int p, int q) { return min(p, q); });
      if (best > shut_below<K>()) {                  // the same in all 16 lanes
        if (l16 == i - 16 * q) mine[q] = id;
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = id == e0 + j ? shut(key[j]) : key[j];
      }
    }
    if (mine[q] >= 0) {
      w[q] = score_of(fminf(load_logit<DT>(a.x, t * a.ld + mine[q]), kF32Max), a.score, top) / sum;
      atomicOr(&mask[mine[q]], 1ull << tl);
    }
    part += w[q];
    if (16 * q + 16 >= a.topk) break;
  }
  const double norm = a.renorm ? fmax(lanes_sum<16>(part), 1e-300) : 1.0;
  if (real) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = 16 * q + l16;
      if (i >= a.topk) break;
      a.ids[t * a.topk + i] = mine[q];
      a.weights[t * a.topk + i] = (float)(w[q] / norm * a.scale);
      s_ids[tl * a.topk + i] = mine[q];
    }
  }
  finish_block(a, t0, tokens, s_ids, mask, base, red);
}

// V: experts per lane (E <= 64 V).  GENERAL: keys in fp64 (a bias or groups).
template <int DT, int V, bool GENERAL>
__global__ __launch_bounds__(kRThreads) void route_kernel(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  // [E] masks, [kTok * topk] ids, [E] bases, scan scratch, then (GENERAL) the waves' choice values
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem);
  int32_t* s_ids = reinterpret_cast<int32_t*>(mask + a.E);
  int* base = s_ids + kTok * a.topk;
  int* red = base + a.E;
  double* s_c = reinterpret_cast<double*>(smem + ((8 * a.E + 4 * kTok * a.topk + 4 * a.E + 4 * kRWaves + 15) & ~15));
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < a.E; e += kRThreads) mask[e] = 0;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int tokens = (int)min((int64_t)kTok, a.T - t0);
  const double kLow = -__builtin_inf();

  float bias[V];
  int group[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * 64 + lane;
    bias[j] = (GENERAL && a.bias && e < a.E) ? a.bias[e] : 0.f;
    group[j] = GENERAL ? e / a.per_group : 0;
  }
  for (int tl = wave; tl < tokens; tl += kRWaves) {
    const int64_t t = t0 + tl;
    float x[V];
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 64 + lane;
      const float v = e < a.E ? load_logit<DT>(a.x, t * a.ld + e) : -__builtin_inff();
      x[j] = v > -__builtin_inff() ? fminf(v, kF32Max) : -__builtin_inff();   // NaN: closed
      top = fmaxf(top, x[j]);
    }
    top = wave_max(top);
    if (!(top > -__builtin_inff())) top = 0.f;         // every expert closed: no p is used
    double sum = 1.0;
    double key[V];
    if (GENERAL || (a.score == 0 && !a.renorm)) {
      double part = 0.0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const double p = x[j] > -__builtin_inff() ? score_of(x[j], a.score, top) : 0.0;
        key[j] = p;
        part += p;
      }
      if (a.score == 0) sum = fmax(lanes_sum<64>(part), 1e-300);
    }
    if constexpr (GENERAL) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const double c = key[j] / sum + (double)bias[j];
        key[j] = (x[j] > -__builtin_inff() && c > kLow) ? c : kLow;    // a NaN or -inf bias closes its expert
      }
      if (a.G > 1) {
        // lane group g of LG lanes takes expert group g
        double* mine = s_c + wave * a.E;
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (j * 64 + lane < a.E) mine[j * 64 + lane] = key[j];
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_s_waitcnt(0xC07F);
        int LG = 1;
        while (2 * LG * a.G <= 64) LG *= 2;
        const int g = lane / LG;
        double b0 = kLow, b1 = kLow;
        if (g < a.G)
          for (int i = lane & (LG - 1); i < a.per_group; i += LG) {
            const double c = mine[g * a.per_group + i];
            b1 = fmax(b1, fmin(b0, c));
            b0 = fmax(b0, c);
          }
        for (int off = 1; off < LG; off <<= 1) {
          const double o0 = __shfl_xor(b0, off, kWave), o1 = __shfl_xor(b1, off, kWave);
          b1 = fmax(fmax(b1, o1), fmin(b0, o0));
          b0 = fmax(b0, o0);
        }
        const double value = (a.group_top == 2 && b1 > kLow) ? b0 + b1 : b0;
        int before = 0;                                  // groups that rank before this lane's
        for (int h = 0; h < a.G; ++h) {
          const double o = __shfl(value, h * LG, kWave);
          before += (o > value || (o == value && h < g)) ? 1 : 0;
        }
        const unsigned long long kept = __ballot(g < a.G && before < a.topk_groups);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (group[j] < a.G && !((kept >> (group[j] * LG)) & 1)) key[j] = kLow;
      }
      if (!a.bias) {                                     // the key is the logit itself
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = key[j] > kLow ? (double)x[j] : kLow;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = (double)x[j];
    }
    // topk rounds of argmax; lane i keeps the i-th choice
    int my_id = -1;
    for (int i = 0; i < a.topk; ++i) {
      double best = kLow;
      int id = 0x7FFFFFFF;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (key[j] > best) {
          best = key[j];
          id = j * 64 + lane;
        }
      wave_best(best, id);
      if (!(best > kLow)) break;                         // nothing left (uniform)
      if (lane == i) my_id = id;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (id == j * 64 + lane) key[j] = kLow;
    }
    double w = 0.0;
    if (my_id >= 0) {
      const float xi = fminf(load_logit<DT>(a.x, t * a.ld + my_id), kF32Max);
      w = score_of(xi, a.score, top) / sum;
      atomicOr(&mask[my_id], 1ull << tl);
    }
    if (a.renorm) w = w / fmax(lanes_sum<64>(w), 1e-300);
    if (lane < a.topk) {
      a.ids[t * a.topk + lane] = my_id;
      a.weights[t * a.topk + lane] = (float)(w * a.scale);
      s_ids[tl * a.topk + lane] = my_id;
    }
  }
  finish_block(a, t0, tokens, s_ids, mask, base, red);
}

// Per expert, the exclusive sums of the blocks' counts and the total: 64
// experts per block (lane), the blocks' range cut over the waves.
__global__ __launch_bounds__(kRThreads) void route_scan_kernel(const uint8_t* __restrict__ counts,
                                                               int32_t* __restrict__ prefix, int E, int blocks) {
  const int ep = (E + 3) & ~3;
  __shared__ int part[kRWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int per = (blocks + kRWaves - 1) / kRWaves;
  const int b0 = min(wave * per, blocks), b1 = min(b0 + per, blocks);
  int s = 0;
  if (e < E)
    for (int b = b0; b < b1; ++b) s += counts[(int64_t)b * ep + e];
  part[wave][lane] = s;
  __syncthreads();
  int run = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kRWaves; ++w) {
    const int v = part[w][lane];
    if (w < wave) run += v;
    total += v;
  }
  if (e >= E) return;
  for (int b = b0; b < b1; ++b) {
    const int v = counts[(int64_t)b * ep + e];
    prefix[(int64_t)b * E + e] = run;
    run += v;
  }
  if (wave == 0) prefix[(int64_t)blocks * E + e] = total;
}

__global__ __launch_bounds__(kRThreads) void route_place_kernel(RouteArgs a, int blocks) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem);
  int32_t* s_ids = reinterpret_cast<int32_t*>(mask + a.E);
  int* base = s_ids + kTok * a.topk;
  int* red = base + a.E;
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * kTok;
  const int tokens = (int)min((int64_t)kTok, a.T - t0);
  if (tid < a.E) mask[tid] = 0;
  int sum = 0, mine = 0;                             // rows of expert tid, in all and in the blocks before
  if (a.prefix) {
    if (tid < a.E) {
      sum = a.prefix[(int64_t)blocks * a.E + tid];
      mine = a.prefix[(int64_t)blockIdx.x * a.E + tid];
    }
  } else {
    // thread (row group, 4 experts): two sums of the counts' bytes, joined in LDS
    int* s_sum = red + kRWaves;
    int* s_mine = s_sum + ((a.E + 3) & ~3);
    const int words = (a.E + 3) >> 2, groups = kRThreads / words, q = tid % words, rg = tid / words;
    for (int e = tid; e < 2 * 4 * words; e += kRThreads) s_sum[e] = 0;
    __syncthreads();
    if (rg < groups) {
      int all[4] = {0, 0, 0, 0}, low[4] = {0, 0, 0, 0};
#pragma unroll 4
      for (int b = rg; b < blocks; b += groups) {
        const uint32_t v = reinterpret_cast<const uint32_t*>(a.counts)[(int64_t)b * words + q];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = (int)((v >> (8 * c)) & 0xFFu);
          all[c] += n;
          low[c] += b < (int)blockIdx.x ? n : 0;
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        atomicAdd(&s_sum[4 * q + c], all[c]);
        atomicAdd(&s_mine[4 * q + c], low[c]);
      }
    }
    __syncthreads();
    if (tid < a.E) {
      sum = s_sum[tid];
      mine = s_mine[tid];
    }
  }
  int total;
  const int start = block_scan(sum, red, total);
  if (tid < a.E) {
    base[tid] = start + mine;
    if (blockIdx.x == 0) a.offsets[tid] = start;
  }
  if (blockIdx.x == 0 && tid == 0) a.offsets[a.E] = total;
  for (int i = tid; i < tokens * a.topk; i += kRThreads) {
    const int e = a.ids[t0 * a.topk + i];
    s_ids[i] = e;
    if (e >= 0) atomicOr(&mask[e], 1ull << (i / a.topk));
  }
  __syncthreads();
  place_rows(a, t0, tokens, s_ids, mask, base, total);
}

int64_t route_blocks(int64_t T) { return (T + kTok - 1) / kTok; }

static size_t counts_bytes(int64_t nb, int64_t E) { return ((size_t)nb * (size_t)((E + 3) & ~3) + 15) & ~(size_t)15; }

static bool scans(int64_t nb, int64_t E) { return nb * nb * E > ((int64_t)1 << 27); }

size_t route_workspace(int64_t T, int64_t E) {
  const int64_t nb = route_blocks(T);
  if (nb <= 1) return 0;
  return counts_bytes(nb, E) + (scans(nb, E) ? (size_t)(nb + 1) * (size_t)E * 4 : 0);
}

hipError_t launch_route(const void* x, int dt, int64_t T, int64_t E, int64_t ld, int score, const float* bias,
                        int64_t G, int64_t topk_groups, int64_t group_top, int64_t topk, bool renorm, double scale,
                        int32_t* ids, float* weights, int32_t* row_token, int32_t* offsets, int32_t* row_of,
                        void* ws, hipStream_t stream) {
  const int64_t nb = route_blocks(T);
  RouteArgs a;
  a.x = x; a.bias = bias; a.T = T; a.ld = ld;
  a.E = (int)E; a.topk = (int)topk; a.G = (int)G; a.per_group = (int)(E / G);
  a.topk_groups = (int)topk_groups; a.group_top = (int)group_top; a.score = score; a.renorm = renorm ? 1 : 0;
  a.scale = scale;
  a.ids = ids; a.row_token = row_token; a.offsets = offsets; a.row_of = row_of; a.weights = weights;
  a.counts = nb <= 1 ? nullptr : static_cast<uint8_t*>(ws);
  a.prefix = !scans(nb, E) ? nullptr : reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + counts_bytes(nb, E));
  const int64_t unit = dt == 2 ? 4 : 8;              // elements per 16 bytes
  a.vec = ld % unit == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
  const bool general = bias || G > 1;
  const size_t lds = (size_t)((8 * E + 4 * kTok * topk + 4 * E + 4 * kRWaves + 15) & ~15);
  const dim3 grid((unsigned)(nb > 0 ? nb : 1)), block(kRThreads);
  const int V = E <= 64 ? 4 : (E <= 128 ? 8 : 16);   // experts per lane with 16 lanes
  const int64_t lanes = a.per_group / V;             // lanes per group
  const bool rows = E <= 256 && (G == 1 || (lanes > 0 && a.per_group % V == 0 && (lanes & (lanes - 1)) == 0));
  auto by_dt = [&](auto f) {
    if (dt == 0) f(std::integral_constant<int, 0>{});
    else if (dt == 1) f(std::integral_constant<int, 1>{});
    else f(std::integral_constant<int, 2>{});
  };
  if (rows) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, stream, a); };
    by_dt([&](auto d) {
      constexpr int D = decltype(d)::value;
      if (V == 4) general ? go(route_rows_kernel<D, 4, double>) : go(route_rows_kernel<D, 4, float>);
      else if (V == 8) general ? go(route_rows_kernel<D, 8, double>) : go(route_rows_kernel<D, 8, float>);
      else general ? go(route_rows_kernel<D, 16, double>) : go(route_rows_kernel<D, 16, float>);
    });
  } else {
    const size_t need = lds + (G > 1 ? (size_t)8 * E * kRWaves : 0);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, need, stream, a); };
    by_dt([&](auto d) {
      constexpr int D = decltype(d)::value;
      if (!general) E <= 512 ? go(route_kernel<D, 8, false>) : go(route_kernel<D, 16, false>);
      else if (E <= 256) go(route_kernel<D, 4, true>);
      else if (E <= 512) go(route_kernel<D, 8, true>);
      else go(route_kernel<D, 16, true>);
    });
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || nb <= 1) return e;
  if (a.prefix) {
    hipLaunchKernelGGL(route_scan_kernel, dim3((unsigned)((E + 63) / 64)), block, 0, stream, a.counts, a.prefix, (int)E,
                       (int)nb);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const size_t place = lds + (size_t)8 * (size_t)((E + 3) & ~3);
  hipLaunchKernelGGL(route_place_kernel, grid, block, place, stream, a, (int)nb);
  return hipGetLastError();
}

}  // namespace w4
