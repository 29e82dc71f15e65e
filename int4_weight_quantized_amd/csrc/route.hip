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
// One wave routes one token, expert j * 64 + lane in register j. A block
// takes kTok = 64 tokens, so that a token is one bit of a 64-bit mask per
// expert: the rank of (token, expert) inside the block is the number of lower
// bits set, which needs no sort and no order of atomics. One block does the
// whole plan up to 64 tokens; above, a second kernel scans the blocks' counts
// per expert and a third places the rows.
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
  int32_t* counts;                       // [blocks][E], then totals [E]; null: one block
};

template <int DT>
__device__ __forceinline__ float load_logit(const void* x, int64_t i) {
  if constexpr (DT == 2) return static_cast<const float*>(x)[i];
  const uint16_t v = static_cast<const uint16_t*>(x)[i];
  return DT == 0 ? bf16_to_f32(v) : f16_to_f32(v);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
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
      x[j] = v > -__builtin_inff() ? fminf(v, 3.40282347e38f) : -__builtin_inff();   // NaN: closed
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
      if (a.score == 0) sum = fmax(wave_sum(part), 1e-300);
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
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const double o = __shfl_xor(best, off, kWave);
        const int oi = __shfl_xor(id, off, kWave);
        if (o > best || (o == best && oi < id)) {
          best = o;
          id = oi;
        }
      }
      if (!(best > kLow)) break;                         // nothing left (uniform)
      if (lane == i) my_id = id;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (id == j * 64 + lane) key[j] = kLow;
    }
    double w = 0.0;
    if (my_id >= 0) {
      const float xi = fminf(load_logit<DT>(a.x, t * a.ld + my_id), 3.40282347e38f);
      w = score_of(xi, a.score, top) / sum;
      atomicOr(&mask[my_id], 1ull << tl);
    }
    if (a.renorm) w = w / fmax(wave_sum(w), 1e-300);
    if (lane < a.topk) {
      a.ids[t * a.topk + lane] = my_id;
      a.weights[t * a.topk + lane] = (float)(w * a.scale);
      s_ids[tl * a.topk + lane] = my_id;
    }
  }
  __syncthreads();
  const int cnt = tid < a.E ? __popcll(mask[tid]) : 0;
  if (a.counts) {
    if (tid < a.E) a.counts[(int64_t)blockIdx.x * a.E + tid] = cnt;
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

// Per expert, the exclusive sums of the blocks' counts (in place) and the
// total: 64 experts per block (lane), the blocks' range cut over the waves.
__global__ __launch_bounds__(kRThreads) void route_scan_kernel(int32_t* __restrict__ counts, int E, int blocks) {
  __shared__ int part[kRWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int per = (blocks + kRWaves - 1) / kRWaves;
  const int b0 = min(wave * per, blocks), b1 = min(b0 + per, blocks);
  int s = 0;
  if (e < E)
    for (int b = b0; b < b1; ++b) s += counts[(int64_t)b * E + e];
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
    const int v = counts[(int64_t)b * E + e];
    counts[(int64_t)b * E + e] = run;
    run += v;
  }
  if (wave == 0) counts[(int64_t)blocks * E + e] = total;
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
  int total;
  const int start = block_scan(tid < a.E ? a.counts[(int64_t)blocks * a.E + tid] : 0, red, total);
  if (tid < a.E) {
    base[tid] = start + a.counts[(int64_t)blockIdx.x * a.E + tid];
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

size_t route_workspace(int64_t T, int64_t E) {
  const int64_t nb = route_blocks(T);
  return nb <= 1 ? 0 : (size_t)(nb + 1) * (size_t)E * 4;
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
  a.counts = nb <= 1 ? nullptr : static_cast<int32_t*>(ws);
  const bool general = bias || G > 1;
  size_t lds = (size_t)((8 * E + 4 * kTok * topk + 4 * E + 4 * kRWaves + 15) & ~15);
  const size_t place_lds = lds;
  if (G > 1) lds += (size_t)8 * E * kRWaves;
  const dim3 grid((unsigned)(nb > 0 ? nb : 1)), block(kRThreads);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, lds, stream, a); };
  auto by_v = [&](auto dtc, auto gen) {
    constexpr int D = decltype(dtc)::value;
    constexpr bool Gn = decltype(gen)::value;
    if (E <= 64) go(route_kernel<D, 1, Gn>);
    else if (E <= 128) go(route_kernel<D, 2, Gn>);
    else if (E <= 256) go(route_kernel<D, 4, Gn>);
    else if (E <= 512) go(route_kernel<D, 8, Gn>);
    else go(route_kernel<D, 16, Gn>);
  };
  auto by_dt = [&](auto gen) {
    if (dt == 0) by_v(std::integral_constant<int, 0>{}, gen);
    else if (dt == 1) by_v(std::integral_constant<int, 1>{}, gen);
    else by_v(std::integral_constant<int, 2>{}, gen);
  };
  if (general) by_dt(std::true_type{});
  else by_dt(std::false_type{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || nb <= 1) return e;
  hipLaunchKernelGGL(route_scan_kernel, dim3((unsigned)((E + 63) / 64)), block, 0, stream, a.counts, (int)E, (int)nb);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(route_place_kernel, grid, block, place_lds, stream, a, (int)nb);
  return hipGetLastError();
}

}  // namespace w4
