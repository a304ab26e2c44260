// Bias, activation and residual behind the QLoRA linear, and their gradients.
//
//   z = x W'^T + s (x A^T) B^T + bias,   y = act(z) + residual     (one rounding, to bf16, at the end)
//   dz = dY * act'(z),   dbias = sum over tokens of dz             (the residual's gradient is dY)
//
// Activations, all in fp32:
//   relu       max(z, 0)
//   silu       z p,          p = 1 / (1 + e^-z)                  slope p + z p (1 - p)
//   gelu       z Phi(z),     Phi(z) = erfc(-z / sqrt 2) / 2       slope Phi(z) + z phi(z), phi the normal density
//   gelu_tanh  z p(2 u),     u = sqrt(2 / pi) (z + 0.044715 z^3)  slope p + z p (1 - p) 2 u'
// The tanh form uses (1 + tanh u) / 2 = 1 / (1 + e^-2u), and the erf form erfc: neither loses its
// small results for negative z to a cancellation against 1.
// Slopes at an infinite z (what bf16 makes of a saved z above 3.39e38, too) are their limits, 0 or 1:
// the term z p (1 - p) would be infinity times 0.  Values there are the formulas': act(-inf) is NaN but for ReLU.
#pragma once

#include "gemm.h"
#include "rmsnorm.cuh"

namespace qnf4 {

enum Act : int32_t { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kSqrt2OverPi = 0.79788456080286536f, kSqrtHalf = 0.70710678118654752f,
                kInvSqrt2Pi = 0.39894228040143268f, kGeluCubic = 0.044715f;

// 1 / (1 + e^-v) by the approximate exponential and reciprocal instructions, each within a few units
// of the 23rd bit, far below the bf16 rounding that follows.  Subnormal results are flushed: p is 0
// below 2^-126.
__device__ __forceinline__ float logistic_ftz(float v) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// Phi(-x) = erfc(x / sqrt 2) / 2 for x >= 0, two values at a time: the Chebyshev fit of Press et al.,
// Numerical Recipes (erfcc): erfc(y) = t exp(-y^2 + P(t)), t = 1 / (1 + y / 2), of fractional error
// below 1.2e-7 everywhere, so that the far negative tail of z Phi(z) keeps its leading bits.  (The
// library's erfcf took three times the instructions.)
__device__ __forceinline__ uint64_t upper_tail2(uint64_t x) {
  const uint64_t y = f32x2_mul(x, f32_pair(kSqrtHalf, kSqrtHalf));
  const uint64_t d = f32x2_fma(y, f32_pair(0.5f, 0.5f), f32_pair(1.0f, 1.0f));
  float t0, t1;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(pair_lo(d)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(pair_hi(d)));
  const uint64_t t = f32_pair(t0, t1);
  uint64_t s = f32_pair(0.17087277f, 0.17087277f);
  s = f32x2_fma(s, t, f32_pair(-0.82215223f, -0.82215223f));
  s = f32x2_fma(s, t, f32_pair(1.48851587f, 1.48851587f));
  s = f32x2_fma(s, t, f32_pair(-1.13520398f, -1.13520398f));
  s = f32x2_fma(s, t, f32_pair(0.27886807f, 0.27886807f));
  s = f32x2_fma(s, t, f32_pair(-0.18628806f, -0.18628806f));
  s = f32x2_fma(s, t, f32_pair(0.09678418f, 0.09678418f));
  s = f32x2_fma(s, t, f32_pair(0.37409196f, 0.37409196f));
  s = f32x2_fma(s, t, f32_pair(1.00002368f, 1.00002368f));
  s = f32x2_fma(s, t, f32_pair(-1.26551223f, -1.26551223f));
  s = f32x2_fma(f32x2_mul(x, f32_pair(-0.5f, -0.5f)), x, s);    // - y^2 = - x^2 / 2
  float e0, e1;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(pair_lo(s) * 1.4426950408889634f));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(pair_hi(s) * 1.4426950408889634f));
  return f32x2_mul(f32x2_mul(t, f32_pair(0.5f, 0.5f)), f32_pair(e0, e1));
}

// act(z) for two values at a time
template <int ACT>
__device__ __forceinline__ uint64_t act_value2(uint64_t z) {
  const float z0 = pair_lo(z), z1 = pair_hi(z);
  if constexpr (ACT == kActRelu) return f32_pair(z0 < 0.0f ? 0.0f : z0, z1 < 0.0f ? 0.0f : z1);   // a NaN stays one
  if constexpr (ACT == kActSilu) return f32x2_mul(z, f32_pair(logistic_ftz(z0), logistic_ftz(z1)));
  if constexpr (ACT == kActGelu) {
    const uint64_t s = upper_tail2(f32_pair(fabsf(z0), fabsf(z1)));
    return f32x2_mul(z, f32_pair(z0 > 0.0f ? 1.0f - pair_lo(s) : pair_lo(s), z1 > 0.0f ? 1.0f - pair_hi(s) : pair_hi(s)));
  }
  if constexpr (ACT == kActGeluTanh) {
    constexpr float c = 2.0f * kSqrt2OverPi;
    const uint64_t v = f32x2_mul(z, f32x2_fma(f32x2_mul(z, z), f32_pair(c * kGeluCubic, c * kGeluCubic), f32_pair(c, c)));
    return f32x2_mul(z, f32_pair(logistic_ftz(pair_lo(v)), logistic_ftz(pair_hi(v))));
  }
  return z;
}

// The nearest finite value (of a NaN any: it meets the NaN of its logistic)
__device__ __forceinline__ float nearest_finite(float v) {
  float r;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(3.402823466e38f));   // the smaller magnitude, v's sign
  return r;
}

// dy * act'(z) for two values at a time
template <int ACT>
__device__ __forceinline__ uint64_t act_grad2(uint64_t dy, uint64_t z) {
  const float z0 = pair_lo(z), z1 = pair_hi(z);
  if constexpr (ACT == kActRelu) return f32_pair(z0 <= 0.0f ? 0.0f : pair_lo(dy), z1 <= 0.0f ? 0.0f : pair_hi(dy));
  const uint64_t one = f32_pair(1.0f, 1.0f), minus = f32_pair(-1.0f, -1.0f);
  if constexpr (ACT == kActSilu) {
    const uint64_t p = f32_pair(logistic_ftz(z0), logistic_ftz(z1)), v = f32_pair(nearest_finite(z0), nearest_finite(z1));
    return f32x2_mul(dy, f32x2_fma(f32x2_mul(v, p), f32x2_fma(p, minus, one), p));
  }
  if constexpr (ACT == kActGelu) {
    // Abramowitz & Stegun 7.1.26: erfc(x) = t (a1 + t (a2 + ...)) e^-x^2 with t = 1 / (1 + p x), x >= 0,
    // within 1.5e-7; with x = |z| / sqrt 2 its exponential is also the density's.  (Through erfcf the
    // call took twice the time: 251 us at 8192 x 13824 against 104 us of HBM traffic.)
    const float x0 = fabsf(z0), x1 = fabsf(z1);
    const uint64_t x = f32_pair(x0, x1);
    const uint64_t q = f32x2_mul(x, f32x2_mul(x, f32_pair(-0.72134752044448171f, -0.72134752044448171f)));
    const uint64_t d = f32x2_fma(x, f32_pair(0.23164188f, 0.23164188f), one);
    float e0, e1, t0, t1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(pair_lo(q)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(pair_hi(q)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(pair_lo(d)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(pair_hi(d)));
    const uint64_t t = f32_pair(t0, t1), e = f32_pair(e0, e1);
    uint64_t s = f32_pair(0.5307027145f, 0.5307027145f);   // the five coefficients, halved
    s = f32x2_fma(s, t, f32_pair(-0.7265760135f, -0.7265760135f));
    s = f32x2_fma(s, t, f32_pair(0.7107068705f, 0.7107068705f));
    s = f32x2_fma(s, t, f32_pair(-0.142248368f, -0.142248368f));
    s = f32x2_fma(s, t, f32_pair(0.127414796f, 0.127414796f));
    s = f32x2_mul(f32x2_mul(s, t), e);                       // Phi(-|z|)
    // z phi(z); 0 where the density has vanished (z may be infinite there)
    const float g0 = e0 == 0.0f ? 0.0f : z0 * e0 * kInvSqrt2Pi, g1 = e1 == 0.0f ? 0.0f : z1 * e1 * kInvSqrt2Pi;
    const float c0 = z0 > 0.0f ? 1.0f - pair_lo(s) : pair_lo(s), c1 = z1 > 0.0f ? 1.0f - pair_hi(s) : pair_hi(s);
    return f32x2_mul(dy, f32_pair(c0 + g0, c1 + g1));
  }
  if constexpr (ACT == kActGeluTanh) {
    constexpr float c = 2.0f * kSqrt2OverPi;
    const uint64_t zz = f32x2_mul(z, z);
    // 2 u = z (c + c 0.044715 z^2) and its slope c + 3 c 0.044715 z^2
    const uint64_t cc = f32_pair(c, c), c1 = f32_pair(c * kGeluCubic, c * kGeluCubic),
                   c3 = f32_pair(3.0f * c * kGeluCubic, 3.0f * c * kGeluCubic);
    const uint64_t v = f32x2_mul(z, f32x2_fma(zz, c1, cc)), slope = f32x2_fma(zz, c3, cc);
    const uint64_t p = f32_pair(logistic_ftz(pair_lo(v)), logistic_ftz(pair_hi(v)));
    const uint64_t q = f32x2_mul(f32x2_mul(z, p), f32x2_fma(p, minus, one));
    // p has saturated long before the slope of u overflows; q is 0 there, or infinity times 0
    const float inf = __uint_as_float(0x7F800000u);
    const float t0 = pair_lo(slope) == inf ? 0.0f : pair_lo(q) * pair_lo(slope);
    const float t1 = pair_hi(slope) == inf ? 0.0f : pair_hi(q) * pair_hi(slope);
    return f32x2_mul(dy, f32_pair(pair_lo(p) + t0, pair_hi(p) + t1));
  }
  return dy;
}

// act over n values; `act` is the same for the whole grid
template <int ACT, int N>
__device__ __forceinline__ void act_apply_t(float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t v = act_value2<ACT>(f32_pair(z[i], z[i + 1]));
    z[i] = pair_lo(v);
    z[i + 1] = pair_hi(v);
  }
}
template <int N>
__device__ __forceinline__ void act_apply(float (&z)[N], int act) {
  switch (act) {
    case kActRelu: act_apply_t<kActRelu>(z); break;
    case kActSilu: act_apply_t<kActSilu>(z); break;
    case kActGelu: act_apply_t<kActGelu>(z); break;
    case kActGeluTanh: act_apply_t<kActGeluTanh>(z); break;
    default: break;
  }
}

// ---------------------------------------------------------------------------------------
// the epilogue over split-K partials: one thread per 8 features of a token
// ---------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) reduce_splits_epilogue_kernel(const float* __restrict__ ws, int splits,
                                                                     int64_t split_stride, int64_t n8, int64_t features8,
                                                                     const EpiArgs e, uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n8) return;
  float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < splits; ++s) {
    const float4* p = reinterpret_cast<const float4*>(ws + (int64_t)s * split_stride) + 2 * i;
    const float4 a = p[0], b = p[1];
    f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
    f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
  }
  float q[8];
  if (e.bias) {
    unpack8(reinterpret_cast<const uint4*>(e.bias)[i % features8], q);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += q[j];
  }
  if (e.z) reinterpret_cast<uint4*>(e.z)[i] = pack8(f);
  act_apply(f, e.act);
  if (e.residual) {
    unpack8(reinterpret_cast<const uint4*>(e.residual)[i], q);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += q[j];
  }
  reinterpret_cast<uint4*>(out)[i] = pack8(f);
}

static cudaError_t launch_reduce_splits_epilogue(const float* ws, int splits, int64_t split_stride, int64_t tokens,
                                                 int64_t features, const EpiArgs& e, uint16_t* out, cudaStream_t st) {
  const int64_t n8 = tokens * features / 8;
  reduce_splits_epilogue_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, st>>>(ws, splits, split_stride, n8,
                                                                              features / 8, e, out);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------------------
// gradient of the activation, and the bias's
// ---------------------------------------------------------------------------------------
// Block (32 lanes along the features, 8 each) x (8 warps along the tokens); blockIdx.x tiles the
// features by 256, blockIdx.y the tokens.  A thread keeps its 8 columns' sums of dz (before their
// rounding to bf16) in registers; the 8 warps' sums are joined in shared memory and left as one
// row of partial sums per token block.  An HBM stream: 8192 x 13824, SiLU, with the bias's gradient 115
// us, 0.90 of the memory rate, without it 111 us.
constexpr int kEbCols = 256, kEbWarps = 8, kEbRows = 4;

struct EpiBwdArgs {
  const uint16_t* dy;
  const uint16_t* z;         // bf16 pre-activation, or
  const uint8_t* z_codes;    // its 8-bit checkpoint
  const uint8_t* z_scales;
  int64_t M, N;
  int64_t rows_per_block;
  uint16_t* dz;
  float* partial;            // [gridDim.y][N] or NULL
};

// (Four blocks per SM hide the loads better than the three of 66 to 80 registers: 115 against 121 us for
// SiLU.  An 8-bit z needs more for its decoding: three blocks, 112 us; two 128 us; spills at four cost 7 %.)
template <int ACT, bool Z8>
__global__ void __launch_bounds__(256, Z8 ? 3 : 4) epilogue_bwd_kernel(const EpiBwdArgs a) {
  __shared__ float sums[kEbWarps][kEbCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * kEbCols + 8 * lane;
  const int64_t m0 = (int64_t)blockIdx.y * a.rows_per_block + warp;
  const int rows = (int)(min(m0 - warp + a.rows_per_block, a.M) - m0);   // tokens m0, m0 + 8, ... below m0 + rows
  const int64_t ld = a8_ld(a.N), G = a8_groups(a.N);
  const int64_t step = (int64_t)kEbWarps * a.N;
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
  if (n < a.N) {
    const uint16_t* dy = a.dy + m0 * a.N + n;
    const uint16_t* zp = a.z + m0 * a.N + n;
    const uint8_t* zc = a.z_codes + m0 * ld + n;
    const uint8_t* zs = a.z_scales + m0 * G + (n >> 5);
    uint16_t* dz = a.dz + m0 * a.N + n;
    for (int r0 = 0; r0 < rows; r0 += kEbRows * kEbWarps) {
      // kEbRows tokens' loads first, then their arithmetic and stores
      uint4 dv[kEbRows], zv[Z8 ? 1 : kEbRows];
      uint2 qv[Z8 ? kEbRows : 1];
      uint32_t byte[Z8 ? kEbRows : 1];
#pragma unroll
      for (int i = 0; i < kEbRows; ++i, dy += step) {
        dv[i] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (Z8) {
          qv[i] = make_uint2(0u, 0u);
          byte[i] = 127u;
        } else {
          zv[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (r0 + i * kEbWarps < rows) {
          dv[i] = __ldcs(reinterpret_cast<const uint4*>(dy));
          if constexpr (ACT != kActNone && Z8) {
            qv[i] = __ldcs(reinterpret_cast<const uint2*>(zc));
            byte[i] = __ldg(zs);
          } else if constexpr (ACT != kActNone) {
            zv[i] = __ldcs(reinterpret_cast<const uint4*>(zp));
          }
        }
        if constexpr (Z8) {
          zc += kEbWarps * ld;
          zs += kEbWarps * G;
        } else {
          zp += step;
        }
      }
#pragma unroll
      for (int i = 0; i < kEbRows; ++i, dz += step) {
        uint64_t d[4];
        unpack8_pairs(dv[i], d);
        if constexpr (ACT != kActNone) {
          uint64_t z[4];
          if constexpr (Z8) {
            const float s = a8_scale(byte[i]);
            const float2 f0 = a8_decode2(qv[i].x, s), f1 = a8_decode2(qv[i].x >> 16, s), f2 = a8_decode2(qv[i].y, s),
                         f3 = a8_decode2(qv[i].y >> 16, s);
            z[0] = f32_pair(f0.x, f0.y);
            z[1] = f32_pair(f1.x, f1.y);
            z[2] = f32_pair(f2.x, f2.y);
            z[3] = f32_pair(f3.x, f3.y);
          } else {
            unpack8_pairs(zv[i], z);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = act_grad2<ACT>(d[j], z[j]);
          if (r0 + i * kEbWarps < rows)
            *reinterpret_cast<uint4*>(dz) =
                make_uint4(pack_bf16x2(pair_lo(d[0]), pair_hi(d[0])), pack_bf16x2(pair_lo(d[1]), pair_hi(d[1])),
                           pack_bf16x2(pair_lo(d[2]), pair_hi(d[2])), pack_bf16x2(pair_lo(d[3]), pair_hi(d[3])));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x2_add(acc[j], d[j]);   // tokens past the end hold zeros
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    sums[warp][8 * lane + 2 * j] = pair_lo(acc[j]);
    sums[warp][8 * lane + 2 * j + 1] = pair_hi(acc[j]);
  }
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * kEbCols + threadIdx.x;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kEbWarps; ++w) s += sums[w][threadIdx.x];
  if (col < a.N) a.partial[(int64_t)blockIdx.y * a.N + col] = s;
}

// Token blocks of the backward: enough blocks to fill the GPU several times over, at least 32
// tokens each.
static int64_t epi_bwd_parts(int64_t M, int64_t N) {
  const int64_t tiles = (N + kEbCols - 1) / kEbCols;
  int64_t parts = (148 * 8 + tiles - 1) / tiles;
  const int64_t cap = (M + 31) / 32;
  if (parts > cap) parts = cap;
  return parts < 1 ? 1 : parts;
}

template <bool Z8>
static cudaError_t launch_epilogue_bwd_z(EpiBwdArgs a, int act, dim3 grid, cudaStream_t st) {
  switch (act) {
    case kActRelu: epilogue_bwd_kernel<kActRelu, Z8><<<grid, 256, 0, st>>>(a); break;
    case kActSilu: epilogue_bwd_kernel<kActSilu, Z8><<<grid, 256, 0, st>>>(a); break;
    case kActGelu: epilogue_bwd_kernel<kActGelu, Z8><<<grid, 256, 0, st>>>(a); break;
    case kActGeluTanh: epilogue_bwd_kernel<kActGeluTanh, Z8><<<grid, 256, 0, st>>>(a); break;
    default: epilogue_bwd_kernel<kActNone, false><<<grid, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

// dz (unless act is none, where it equals dy) and dbias (or NULL).
static cudaError_t launch_epilogue_bwd(EpiBwdArgs a, int act, uint16_t* dbias, cudaStream_t st) {
  constexpr int64_t kStep = kEbRows * kEbWarps;
  const int64_t most = epi_bwd_parts(a.M, a.N);
  a.rows_per_block = ((a.M + most - 1) / most + kStep - 1) / kStep * kStep;
  const int64_t parts = (a.M + a.rows_per_block - 1) / a.rows_per_block;
  if (!dbias) a.partial = nullptr;
  const dim3 grid((unsigned)((a.N + kEbCols - 1) / kEbCols), (unsigned)parts);
  cudaError_t e = a.z_codes ? launch_epilogue_bwd_z<true>(a, act, grid, st) : launch_epilogue_bwd_z<false>(a, act, grid, st);
  if (e != cudaSuccess || !dbias) return e;
  return launch_column_sum(a.partial, (int)parts, a.N, dbias, st);
}

}  // namespace qnf4
