// Bias, activation and residual behind the QLoRA linear, and their gradients.
//
//   z = x W'^T + s (x A^T) B^T + bias,   y = act(z) + residual     (one rounding, to bf16, at the end)
//   dz = dY * act'(z),   dbias = sum over tokens of dz             (the residual's gradient is dY)
//
// Activations, all in fp32:
//   relu       max(z, 0)
//   silu       z p,          p = 1 / (1 + e^-z)                  slope p + z p (1 - p)
//   gelu       z Phi(z),     Phi(z) = erfc(-z / sqrt 2) / 2       slope Phi(z) + z phi(z)
//   gelu_tanh  z p(2 u),     u = sqrt(2 / pi) (z + 0.044715 z^3)  slope p + z p (1 - p) 2 u'
// The tanh form uses (1 + tanh u) / 2 = 1 / (1 + e^-2u), and the erf form erfc: neither loses its
// small results for negative z to a cancellation against 1.
#pragma once

#include "gemm.h"
#include "rmsnorm.cuh"

namespace qnf4 {

enum Act : int32_t { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kSqrt2OverPi = 0.79788456080286536f, kSqrtHalf = 0.70710678118654752f,
                kInvSqrt2Pi = 0.39894228040143268f, kGeluCubic = 0.044715f;

// 1 / (1 + e^-v): the approximate exponential and reciprocal instructions, each within a few
// units of the 23rd bit, far below the bf16 rounding that follows.  e^-v = inf gives 0.
__device__ __forceinline__ float logistic(float v) {
  float r;
  const float d = 1.0f + __expf(-v);
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;    // a NaN stays one
  if constexpr (ACT == kActSilu) return z * logistic(z);
  if constexpr (ACT == kActGelu) return 0.5f * z * erfcf(-kSqrtHalf * z);
  if constexpr (ACT == kActGeluTanh) return z * logistic(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad(float dy, float z) {
  if constexpr (ACT == kActRelu) return z <= 0.0f ? 0.0f : dy;
  if constexpr (ACT == kActSilu) {
    const float p = logistic(z);
    return dy * fmaf(z * p, 1.0f - p, p);
  }
  if constexpr (ACT == kActGelu) return dy * (0.5f * erfcf(-kSqrtHalf * z) + z * kInvSqrt2Pi * __expf(-0.5f * z * z));
  if constexpr (ACT == kActGeluTanh) {
    const float p = logistic(2.0f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
    const float q = z * p * (1.0f - p);
    // q is 0 where p has saturated; the slope of u may have overflowed there
    const float t = q == 0.0f ? 0.0f : q * (2.0f * kSqrt2OverPi) * fmaf(3.0f * kGeluCubic * z, z, 1.0f);
    return dy * (p + t);
  }
  return dy;
}

// act over 8 values; `act` is the same for the whole grid
__device__ __forceinline__ void act_apply8(float (&z)[8], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = act_value<kActRelu>(z[i]);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = act_value<kActSilu>(z[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = act_value<kActGelu>(z[i]);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = act_value<kActGeluTanh>(z[i]);
      break;
    default:
      break;
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
  act_apply8(f, e.act);
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
// row of partial sums per token block.
constexpr int kEbCols = 256, kEbWarps = 8;

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

template <int ACT, bool Z8>
__global__ void __launch_bounds__(256) epilogue_bwd_kernel(const EpiBwdArgs a) {
  __shared__ float sums[kEbWarps][kEbCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * kEbCols + 8 * lane;
  const int64_t m0 = (int64_t)blockIdx.y * a.rows_per_block;
  const int64_t m1 = min(m0 + a.rows_per_block, a.M);
  const int64_t ld = a8_ld(a.N), G = a8_groups(a.N);
  float acc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (n < a.N) {
    for (int64_t m = m0 + warp; m < m1; m += kEbWarps) {
      float d[8], z[8];
      unpack8(*reinterpret_cast<const uint4*>(a.dy + m * a.N + n), d);
      if constexpr (ACT != kActNone) {
        if constexpr (Z8) {
          const uint2 q = *reinterpret_cast<const uint2*>(a.z_codes + m * ld + n);
          const float s = a8_scale(a.z_scales[m * G + (n >> 5)]);
          const float2 f0 = a8_decode2(q.x, s), f1 = a8_decode2(q.x >> 16, s), f2 = a8_decode2(q.y, s),
                       f3 = a8_decode2(q.y >> 16, s);
          z[0] = f0.x; z[1] = f0.y; z[2] = f1.x; z[3] = f1.y; z[4] = f2.x; z[5] = f2.y; z[6] = f3.x; z[7] = f3.y;
        } else {
          unpack8(*reinterpret_cast<const uint4*>(a.z + m * a.N + n), z);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = act_grad<ACT>(d[i], z[i]);
        *reinterpret_cast<uint4*>(a.dz + m * a.N + n) = pack8(d);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += d[i];
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[warp][8 * lane + i] = acc[i];
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
  const int64_t parts = epi_bwd_parts(a.M, a.N);
  a.rows_per_block = (a.M + parts - 1) / parts;
  if (!dbias) a.partial = nullptr;
  const dim3 grid((unsigned)((a.N + kEbCols - 1) / kEbCols), (unsigned)parts);
  cudaError_t e = a.z_codes ? launch_epilogue_bwd_z<true>(a, act, grid, st) : launch_epilogue_bwd_z<false>(a, act, grid, st);
  if (e != cudaSuccess || !dbias) return e;
  return launch_column_sum(a.partial, (int)parts, a.N, dbias, st);
}

}  // namespace qnf4
