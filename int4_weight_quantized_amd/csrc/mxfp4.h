// The MXFP4 format (4-bit E2M1 elements, one E8M0 power of two per 32 of
// them along K), shared by its quantizer and products.
//
// A matrix is [rows][K / 2] bytes, the lower column in the low nibble, and
// [rows][4 * ceil(K / 128)] scale bytes: one per 32 columns, each row padded
// to whole blocks of 128 columns. The padding is never used.
#pragma once

#include "fp8_block.h"

namespace w4 {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr uint32_t kMxNan = 255;                     // E8M0's NaN

__host__ __device__ inline int64_t mx_scale_bytes(int64_t K) { return (K + 127) / 128 * 4; }

// The scale code of a block whose largest magnitude has the fp32 bits `amax`:
// 2^(floor(log2 amax) - 2), so that the largest element lies in [4, 8) and
// saturates at 6 from there; at least 2^-127. Infinities and NaN give NaN.
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255 ? kMxNan : (e < 2 ? 0u : e - 2);
}

// The power of two itself, in fp32 (2^-127 is subnormal there); not for NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t code) {
  return __uint_as_float(code ? code << 23 : 0x00400000u);
}

// Largest magnitude of 2 W values of 16 bits in W words, as fp32 bits. Positive
// bf16 and fp16 numbers order as their bits do.
template <bool BF16, int W>
__device__ __forceinline__ uint32_t mx_amax16(const int (&raw)[W]) {
  typedef unsigned short v2u __attribute__((ext_vector_type(2)));
  v2u m = {0, 0};
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const v2u a = __builtin_bit_cast(v2u, raw[i] & 0x7FFF7FFF);
    m = __builtin_elementwise_max(m, a);
  }
  const uint16_t h = m[0] > m[1] ? m[0] : m[1];
  return BF16 ? (uint32_t)h << 16 : __float_as_uint(f16_to_f32(h));
}

// 2 W values of 16 bits to 2 W codes, nearest even, saturating.
template <bool BF16, int W>
__device__ __forceinline__ void mx_encode16(const int (&raw)[W], float scale, int (&codes)[W / 4]) {
#pragma unroll
  for (int w = 0; w < W / 4; ++w) {
    uint32_t c = 0;
    if constexpr (BF16) {
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, raw[4 * w]), scale, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, raw[4 * w + 1]), scale, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, raw[4 * w + 2]), scale, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(v2bf, raw[4 * w + 3]), scale, 3);
    } else {
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(v2h, raw[4 * w]), scale, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(v2h, raw[4 * w + 1]), scale, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(v2h, raw[4 * w + 2]), scale, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(v2h, raw[4 * w + 3]), scale, 3);
    }
    codes[w] = (int)c;
  }
}

struct MxArgs {
  const uint8_t* a;                                  // codes; in the linear form of few rows: 16-bit activations
  const uint8_t* a_scale;
  const int32_t* row_token;                          // grouped: null = rows in segment order
  const int32_t* offsets;                            // grouped: [E + 1]
  const uint8_t* w;
  const uint8_t* w_scale;
  const void* bias;                                  // dense
  void* out;                                         // splits > 1: fp32 [splits][M][N]
  int64_t M;                                         // dense rows, or activation rows (T) of the grouped form
  int64_t R;                                         // output rows
  int E, N, K, KS, KT, NT, splits;                   // KS: scale bytes of a row; KT: steps of 256 along K
  int64_t tiles;                                     // dense: row tiles * NT
};

// XQ: 0 codes, 1 bf16 activations, 2 fp16 ones (dense only)
hipError_t launch_mx_stream(const MxArgs& p, int xq, int out_dt, hipStream_t stream);
// Threads that it takes: dense (E = 0) or grouped.
int64_t mx_stream_threads(int64_t M, int64_t N, int64_t E, int64_t R);

}  // namespace w4
