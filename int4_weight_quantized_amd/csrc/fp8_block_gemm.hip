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
#include "w4_device.h"

namespace w4 {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// 8 E4M3 bytes (words w, w + 1 of a fragment) as fp16
__device__ __forceinline__ v8h e4m3_to_f16(const v8i& f, int w) {
  v8h h;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const v2h lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[w + q], 1.0f, false);
    const v2h hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[w + q], 1.0f, true);
    h[4 * q] = lo[0];
    h[4 * q + 1] = lo[1];
    h[4 * q + 2] = hi[0];
    h[4 * q + 3] = hi[1];
  }
  return h;
}

// One scale block: 16 weight rows x 16 activation rows x 128.
template <bool F16>
__device__ __forceinline__ v4f block_product(const v8i& w, const v8i& a) {
  const v4f z = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (F16) {
    v4f d = z;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      d = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3_to_f16(w, 2 * c), e4m3_to_f16(a, 2 * c), d, 0, 0, 0);
    return d;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, z, 0, 0, 0, 0, 0, 0);
  }
}

constexpr int kFK = 128;                             // K step: one scale block

struct Fp8Args {
  const uint8_t* a;
  const float* a_scale;
  const int32_t* row_token;                          // grouped: null = rows in segment order
  const int32_t* offsets;                            // grouped: [E + 1]
  const uint8_t* w;
  const float* w_scale;
  const void* bias;
  void* out;                                         // splits > 1: fp32 [splits][M][N]
  int64_t M;                                         // dense rows, or activation rows (T) of the grouped form
  int64_t R;                                         // grouped: output rows
  int E, N, K, KB, NT, NBLK, splits;                 // NBLK: ceil(N / 128)
  int64_t tiles;                                     // dense: row tiles * NT
};

// Wave tile 16 MI rows of activations x 16 NJ columns, WM x WN waves.
template <int MI, int NJ, int WM, int WN, bool GROUPED, int OUT>   // OUT: 0 bf16, 1 fp16, 2 fp32
__global__ __launch_bounds__(64 * WM * WN) void fp8_tile_kernel(Fp8Args p) {
  constexpr int TH = 64 * WM * WN, BM = 16 * MI * WM, BN = 16 * NJ * WN;
  constexpr int RA = BM * 8 / TH, RB = BN * 8 / TH;  // LDS DMAs per thread and K step
  constexpr int NB = BN > 128 ? BN / 128 : 1;        // weight scale rows per tile
  static_assert(RA * TH == BM * 8 && RB * TH == BN * 8, "whole DMAs");
  __shared__ __attribute__((aligned(16))) uint8_t sA0[BM * kFK], sA1[BM * kFK], sB0[BN * kFK], sB1[BN * kFK];
  __shared__ __attribute__((aligned(16))) float sS[2][4][NB][BM];   // sa * sw of 4 K steps, two chunks

  // ---- work item
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, l16 = lane & 15;
  int e = 0, tn, split = 0;
  int64_t r0, row_end, out0 = 0;                     // first row and end of this tile's rows (segment-local if grouped)
  if constexpr (GROUPED) {
    // row tiles of the experts, 64 experts per round (one per lane)
    int total = 0;
    for (int c = 0; c < p.E; c += 64) {
      int mt = 0;
      if (c + lane < p.E) mt = (p.offsets[c + lane + 1] - p.offsets[c + lane] + BM - 1) / BM;
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) mt += __shfl_xor(mt, off, kWave);
      total += mt;
    }
    total = __builtin_amdgcn_readfirstlane(total) * p.NT;
    // block ids go to the 8 XCDs in turn: XCD x takes the x-th eighth of the items
    const int per = (total + 7) / 8, xi = (int)(blockIdx.x / 8);
    if (xi >= per) return;
    const int t = (int)(blockIdx.x % 8) * per + xi;
    if (t >= total) return;
    const int want = t / p.NT;                       // row tile, over all experts
    tn = t - want * p.NT;
    int cum = 0, mt = 0;
    e = -1;
    int seg0 = 0, cnt = 0;
    for (int c = 0; c < p.E && e < 0; c += 64) {
      int o0 = 0, o1 = 0;
      if (c + lane < p.E) {
        o0 = p.offsets[c + lane];
        o1 = p.offsets[c + lane + 1];
      }
      const int n = (o1 - o0 + BM - 1) / BM;
      int inc = n;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(inc, off, kWave);
        if (lane >= off) inc += o;
      }
      const unsigned long long hit = __ballot(want < cum + inc);
      if (hit) {
        const int src = __ffsll(hit) - 1;
        e = c + src;
        mt = want - cum - (__shfl(inc, src, kWave) - __shfl(n, src, kWave));
        seg0 = __shfl(o0, src, kWave);
        cnt = __shfl(o1, src, kWave) - seg0;
      }
      cum += __shfl(inc, 63, kWave);
    }
    if (e < 0) return;
    e = __builtin_amdgcn_readfirstlane(e);
    r0 = (int64_t)__builtin_amdgcn_readfirstlane(mt) * BM;
    out0 = __builtin_amdgcn_readfirstlane(seg0);
    row_end = __builtin_amdgcn_readfirstlane(cnt);
    if (out0 + row_end > p.R) row_end = p.R - out0;  // offsets past the output rows
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
  constexpr uint32_t kOut = 0x80000000u;
  const int lrow = lane >> 3, lchunk = lane & 7;
  const int64_t abase = (GROUPED && p.row_token) ? 0 : (out0 + r0) * p.K;
  const int64_t aspan = (GROUPED && p.row_token) ? p.M * p.K : min((int64_t)BM, (GROUPED ? p.M : p.M) - out0 - r0) * p.K;
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
    a_off[i] = t >= 0 ? (uint32_t)(t * p.K + 16 * c) : kOut;
    if (16 * c >= klast) a_dead |= 1u << i;
  }
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int r = (TH / 8) * i + 8 * wave + lrow;
    const int c = lchunk ^ ((r & 3) + 4 * ((r / (4 * NJ)) & 1));
    b_off[i] = n0 + r < p.N ? (uint32_t)((int64_t)r * p.K + 16 * c) : kOut;
    if (16 * c >= klast) b_dead |= 1u << i;
  }
  auto gload = [&](int tk, uint8_t* sa, uint8_t* sb) {
    const bool last = tk == p.KB - 1;
    const uint32_t ks = (uint32_t)tk * kFK;
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const uint32_t off = (last && ((a_dead >> i) & 1)) ? kOut : a_off[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          arsrc, (__attribute__((address_space(3))) void*)(sa + ((TH / 8) * i + 8 * wave) * kFK), 16, off, ks, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const uint32_t off = (last && ((b_dead >> i) & 1)) ? kOut : b_off[i];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wrsrc, (__attribute__((address_space(3))) void*)(sb + ((TH / 8) * i + 8 * wave) * kFK), 16, off, ks, 0, 0);
    }
  };

  // ---- scales: products sa * sw of 4 K steps at a time, thread (row, weight
  // block); LDS row order [wave row][16][MI], so a lane reads its MI in a run
  constexpr int RS = (BM * NB + TH - 1) / TH;
  auto load_scales = [&](int tk, float (&s)[RS][4]) {
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      const int u = tid + TH * i, r = u % BM, nb = u / BM;
      const int64_t t = u < BM * NB ? token(r) : -1;
      const int64_t arow = (GROUPED && p.row_token) ? t : out0 + r0 + t;
      const int wb = n0 / 128 + nb;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = t >= 0 && tk + j < k1 && wb < p.NBLK;
        s[i][j] = in ? p.a_scale[arow * p.KB + tk + j] * p.w_scale[((int64_t)e * p.NBLK + wb) * p.KB + tk + j] : 0.f;
      }
    }
  };
  auto store_scales = [&](int buf, const float (&s)[RS][4]) {
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      const int u = tid + TH * i, r = u % BM, nb = u / BM;
      if (u >= BM * NB) break;
      const int at = (r / (16 * MI)) * 16 * MI + (r % 16) * MI + (r / 16) % MI;
#pragma unroll
      for (int j = 0; j < 4; ++j) sS[buf][j][nb][at] = s[i][j];
    }
  };

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // ---- fragments: lane group g takes logical chunks g and g + 4 of its row.
  // Row rho of weight block j is column 4 NJ (rho / 4) + 4 j + rho % 4 of the
  // wave's 16 NJ, so a lane's results are 4 NJ consecutive columns.
  const int ar = 16 * MI * wm + l16;                 // + 16 i; 16 i leaves f unchanged
  const int a_ro = ar * kFK + 16 * (g ^ (ar & 7)), a_rx = ar * kFK + 16 * ((g + 4) ^ (ar & 7));
  const int br = 16 * NJ * wn + 4 * NJ * (l16 >> 2) + (l16 & 3);
  const int bpar = (l16 >> 2) & 1;                   // parity of br / (4 NJ): + 4 j stays inside the run of 4 NJ
  const int b_ro = br * kFK + 16 * (g ^ ((br & 3) + 4 * bpar)), b_rx = br * kFK + 16 * ((g + 4) ^ ((br & 3) + 4 * bpar));
  const int snb = (16 * NJ * wn) / 128 % NB;

  auto kstep = [&](int tk, const uint8_t* sa, const uint8_t* sb) {
    const int rel = tk - k0;
    float s[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) s[i] = sS[(rel >> 2) & 1][rel & 3][snb][16 * MI * wm + l16 * MI + i];
    v8i bf[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const v4i x0 = *reinterpret_cast<const v4i*>(sb + b_ro + 4 * j * kFK);
      const v4i x1 = *reinterpret_cast<const v4i*>(sb + b_rx + 4 * j * kFK);
      bf[j] = v8i{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const v4i x0 = *reinterpret_cast<const v4i*>(sa + a_ro + 16 * i * kFK);
      const v4i x1 = *reinterpret_cast<const v4i*>(sa + a_rx + 16 * i * kFK);
      const v8i af = v8i{x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const v4f d = block_product<OUT == 2>(bf[j], af);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(d[r], s[i], acc[i][j][r]);
      }
    }
  };

  if (k0 < k1) {
    float sc[RS][4];
    load_scales(k0, sc);
    gload(k0, sA0, sB0);
    store_scales(0, sc);
    __syncthreads();
    for (int tk = k0; tk < k1; tk += 2) {
      const int rel = tk - k0;
      const bool fetch = (rel & 3) == 0 && tk + 4 < k1;
      if (fetch) load_scales(tk + 4, sc);
      if (tk + 1 < k1) gload(tk + 1, sA1, sB1);
      kstep(tk, sA0, sB0);
      if (fetch) store_scales(((rel >> 2) + 1) & 1, sc);
      __syncthreads();
      if (tk + 1 >= k1) break;
      if (tk + 2 < k1) gload(tk + 2, sA0, sB0);
      kstep(tk + 1, sA1, sB1);
      __syncthreads();
    }
  }

  // ---- output: lane's row per i, 4 NJ consecutive columns
  const int nw = n0 + 16 * NJ * wn + 4 * NJ * g;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t r = r0 + 16 * MI * wm + 16 * i + l16;
    if (r >= row_end) continue;
    const int64_t orow = (out0 + r + (int64_t)split * p.M) * p.N;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int n = nw + 4 * j;
      if (n >= p.N) continue;
      float f[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) f[c] = acc[i][j][c];
      if (!GROUPED && p.bias && p.splits == 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          f[c] += OUT == 2 ? static_cast<const float*>(p.bias)[n + c]
                           : (OUT == 0 ? bf16_to_f32(static_cast<const uint16_t*>(p.bias)[n + c])
                                       : f16_to_f32(static_cast<const uint16_t*>(p.bias)[n + c]));
      }
      if constexpr (OUT == 2) {
        *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + orow + n) = v4f{f[0], f[1], f[2], f[3]};
      } else {
        uint32_t h[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) h[c] = OUT == 0 ? f32_to_bf16_rne(f[c]) : f32_to_f16_rne(f[c]);
        *reinterpret_cast<v2i*>(static_cast<uint16_t*>(p.out) + orow + n) =
            v2i{(int)(h[0] | (h[1] << 16)), (int)(h[2] | (h[3] << 16))};
      }
    }
  }
}

size_t fp8_block_gemm_workspace(int64_t M, int64_t N, int64_t K) { return 0; }

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
  p.splits = 1;
  constexpr int BM = 64, BN = 64;
  p.NT = (int)((N + BN - 1) / BN);
  p.tiles = (M + BM - 1) / BM * p.NT;
  const dim3 grid((unsigned)p.tiles), block(256);
  if (out_dt == 0) hipLaunchKernelGGL((fp8_tile_kernel<2, 2, 2, 2, false, 0>), grid, block, 0, stream, p);
  else if (out_dt == 1) hipLaunchKernelGGL((fp8_tile_kernel<2, 2, 2, 2, false, 1>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((fp8_tile_kernel<2, 2, 2, 2, false, 2>), grid, block, 0, stream, p);
  return hipGetLastError();
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
  constexpr int BM = 64, BN = 64;
  p.NT = (int)((N + BN - 1) / BN);
  const int64_t upper = (R / BM + (E < R ? E : R)) * p.NT;
  const dim3 grid((unsigned)((upper + 7) / 8 * 8)), block(256);
  if (out_dt == 0) hipLaunchKernelGGL((fp8_tile_kernel<2, 2, 2, 2, true, 0>), grid, block, 0, stream, p);
  else if (out_dt == 1) hipLaunchKernelGGL((fp8_tile_kernel<2, 2, 2, 2, true, 1>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((fp8_tile_kernel<2, 2, 2, 2, true, 2>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace w4
