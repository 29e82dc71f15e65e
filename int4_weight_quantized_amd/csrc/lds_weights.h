// Weights of few-row products on their way through LDS: each wave has room for a step of its own there, which LDS DMA fills,
// so that no wave waits for another and what is on its way costs no registers. Loading straight into the matrix unit's
// layout (lane = row + 16 * column group) would touch 64 cache lines per load and cost the address unit 60 clocks where a
// DMA of 8 rows' full lines costs 16 (measured); it bound such kernels at 2 to 4 TB/s. One step of room is enough: a wave
// takes it into registers and asks for the next before it computes. More room per wave means fewer waves, which costs more
// than it hides: two steps took 131 us instead of 115 for the gate and up products of 8 tokens (64 experts, 7168 x 2048,
// MXFP4) and 69 instead of 64 for a grouped product of 8 tokens' 64 rows; three (the former in blocks of two waves) 151 and 85.
#pragma once
#include "mxfp4.h"

namespace w4 {

enum { kFp8 = 0, kMx = 1, kInt4 = 2 };               // formats of weights

// An LDS address as the instructions take it, uniform over the wave.
__device__ __forceinline__ uint32_t lds_address(const void* at) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)at);
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

// 16 rows n .. n + 15 of weight matrix e, [N, K] (rows: those that there are): 2 KiB of LDS per step, by two DMAs.
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
  __device__ __forceinline__ void open(const uint8_t* base, int64_t e, int64_t N, int64_t n, int64_t K, int rows = 16) {
    if constexpr (FMT == kInt4) {
      const int64_t tk = K / kTileK, tiles = (N + kTileN - 1) / kTileN * tk;
      w = make_rsrc(base + (e * tiles + n / kTileN * tk) * kTileBytes, (uint32_t)(tk * kTileBytes));
    } else {
      const int64_t bytes = FMT == kFp8 ? K : K / 2;
      w = make_rsrc(base + (e * N + n) * bytes, (uint32_t)(rows * bytes));
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

// The scales of MATS sets of 16 rows (the second `gap` rows after the first). FP8 and MXFP4: of 8 steps at a time, with the
// first of them (a step's own few bytes would ask eight times for a cache line, mostly while it is still on its way; the down
// products of 8 tokens, 7168 x 2048 MXFP4, took 83 us so and 77 us now): FP8 8 floats of each set; MXFP4 64 bytes of each row,
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
  __device__ __forceinline__ void open(const void* base, int64_t e, int64_t N_, int64_t n, int64_t gap, int64_t K, int G,
                                              int rows = 16) {
    const uint8_t* b = static_cast<const uint8_t*>(base);
    if constexpr (FMT == kFp8) {
      const int64_t size = (K + 127) / 128 * ((N_ + 127) / 128) * 4;
      s = make_rsrc(b + e * size, (uint32_t)size);
    } else if constexpr (FMT == kMx) {
      const int64_t ks = mx_scale_bytes(K);
      s = make_rsrc(b + (e * N_ + n) * ks, (uint32_t)(((MATS - 1) * gap + rows) * ks));
    } else {
      s = make_rsrc(b + e * G * N_ * 2, (uint32_t)(G * N_ * 2));
    }
  }
  // begins: whether a step's scales come with it (a run's first step, and every kSteps)
  static __device__ __forceinline__ bool begins(int k) { return k % kSteps == 0; }
  __device__ __forceinline__ void fetch(int k, uint32_t dst, int lane) const {
    k = __builtin_amdgcn_readfirstlane(k);           // (the compiler does not see everywhere that they are uniform)
    dst = __builtin_amdgcn_readfirstlane(dst);
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
  // MXFP4: a lane's scale code of half q of step k; left: the columns from the step's first to the end
  static __device__ __forceinline__ uint32_t code(const uint8_t* at, int k, int m, int q, int left, int l16, int g) {
    const int piece = (k & 7) >> 1 ^ (l16 >> 2 & 3);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(at + 1024 * m + 64 * l16 + 16 * piece + 8 * (k & 1) + 4 * q);
    return 128 * q + 32 * g < left ? w >> (8 * g) & 0xFF : 0u;   // past K: the padding, or the next row's
  }
  static __device__ __forceinline__ float block(const uint8_t* at, int k, int m, int q, int left, int l16, int g) {
    const uint32_t c = code(at, k, m, q, left, l16, g);
    return c == kMxNan ? __uint_as_float(0x7FC00000u) : mx_scale_value(c);
  }
};

}  // namespace w4
