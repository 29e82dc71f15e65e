// Routing of one token by one wave (its mathematics: route.hip), shared by the
// router and by the kernel that runs a few tokens through the whole layer.
#pragma once

#include "w4_device.h"

namespace w4 {

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
  int dt;                                // type of the logits: 0 bf16, 1 fp16, 2 fp32
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

// The wave's largest key, the same in every lane: within rows of 16 lanes by DPP, the four rows' through scalar registers.
__device__ __forceinline__ double wave_max64(double v) {
  v = lanes_reduce<16>(v, [](double a, double b) { return fmax(a, b); });
  const long long b = __double_as_longlong(v);
  double r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)b, 16 * i), hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), 16 * i);
    r[i] = __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
  }
  return fmax(fmax(r[0], r[1]), fmax(r[2], r[3]));
}

constexpr float kF32Max = 3.40282347e38f;

// DT as above.
template <int DT>
__device__ __forceinline__ float load_logit(const void* x, int64_t i) {
  if constexpr (DT == 2) return static_cast<const float*>(x)[i];
  const uint16_t v = static_cast<const uint16_t*>(x)[i];
  return DT == 0 ? bf16_to_f32(v) : f16_to_f32(v);
}

// DT 3: the type is looked up (for kernels that route few tokens on the side).
template <int DT>
__device__ __forceinline__ float logit_of(const RouteArgs& a, int64_t i) {
  if constexpr (DT < 3) return load_logit<DT>(a.x, i);
  if (a.dt == 2) return load_logit<2>(a.x, i);
  const uint16_t v = static_cast<const uint16_t*>(a.x)[i];
  return a.dt == 0 ? bf16_to_f32(v) : f16_to_f32(v);
}

// A lane's V logits of token t, -inf past the last expert.
template <int DT, int V>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int lane, float (&x)[V]) {
  constexpr float kClosed = -__builtin_inff();
  if constexpr (DT < 3) {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = j * 64 + lane < a.E ? load_logit<DT>(a.x, t * a.ld + j * 64 + lane) : kClosed;
  } else if (a.dt == 2) {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = j * 64 + lane < a.E ? load_logit<2>(a.x, t * a.ld + j * 64 + lane) : kClosed;
  } else {
    uint16_t h[V];                                   // all loads, then one look at the type
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = j * 64 + lane < a.E ? static_cast<const uint16_t*>(a.x)[t * a.ld + j * 64 + lane] : 0;
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = j * 64 + lane < a.E ? (a.dt == 0 ? bf16_to_f32(h[j]) : f16_to_f32(h[j])) : kClosed;
  }
}

__device__ __forceinline__ double score_of(float x, int score, float top) {
  return score == 0 ? exp((double)x - (double)top) : 1.0 / (1.0 + exp(-(double)x));
}

// What a wave keeps of the experts that its lanes hold: expert j * 64 + lane in
// register j, V of them (E <= 64 V).
template <int V, bool GENERAL>
struct LaneExperts {
  float bias[V];
  int group[V];
  __device__ __forceinline__ LaneExperts(const RouteArgs& a, int lane) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 64 + lane;
      bias[j] = (GENERAL && a.bias && e < a.E) ? a.bias[e] : 0.f;
      group[j] = GENERAL ? e / a.per_group : 0;
    }
  }
};

// Routes token t: lane i gets the i-th choice and its weight before the scale
// (-1 and 0: none). GENERAL: keys in fp64 (a bias or groups); mine: E doubles of
// LDS of the wave's own where there are groups.
template <int DT, int V, bool GENERAL>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int lane, const LaneExperts<V, GENERAL>& own,
                                            double* mine, int& my_id, double& w) {
  const double kLow = -__builtin_inf();
  float x[V];
  load_logits<DT>(a, t, lane, x);
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float v = x[j];
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
      const double c = key[j] / sum + (double)own.bias[j];
      key[j] = (x[j] > -__builtin_inff() && c > kLow) ? c : kLow;    // a NaN or -inf bias closes its expert
    }
    if (a.G > 1) {
      // lane group g of LG lanes takes expert group g
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
        if (own.group[j] < a.G && !((kept >> (own.group[j] * LG)) & 1)) key[j] = kLow;
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
  my_id = -1;
  for (int i = 0; i < a.topk; ++i) {
    double best = kLow;
#pragma unroll
    for (int j = 0; j < V; ++j) best = fmax(best, key[j]);
    best = wave_max64(best);
    if (!(best > kLow)) break;                         // nothing left (uniform)
    int id = 0;                                        // the lowest expert that holds it
#pragma unroll
    for (int j = V - 1; j >= 0; --j) {
      const unsigned long long hit = __ballot(key[j] == best);
      id = hit ? j * 64 + __ffsll(hit) - 1 : id;
    }
    if (lane == i) my_id = id;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (id == j * 64 + lane) key[j] = kLow;
  }
  w = 0.0;
  if (my_id >= 0) {
    const float xi = fminf(logit_of<DT>(a, t * a.ld + my_id), kF32Max);
    w = score_of(xi, a.score, top) / sum;
  }
  if (a.renorm) w = w / fmax(lanes_sum<64>(w), 1e-300);
}

}  // namespace w4
