// Root-mean-square norm of the hidden states in front of a QLoRA linear, with the residual
// stream's addition and an 8-bit checkpoint of its output, and its gradients.
//
//   v = x + residual                       (fp32; v = x without a residual)
//   h = bf16(v)                            (the residual stream handed on)
//   rstd = 1 / sqrt(mean_k v^2 + eps)      (fp32)
//   y = bf16(v * rstd * w)                 (read by the linears' forward)
//   y8 = the 8-bit checkpoint of y         (act8.cuh; read by the linears' backward)
//
// y is formed from the unrounded sum; y8 from y's bf16 values, so that it is bit for bit what
// quantizing y would give.  Gradients, with n = h * rstd and g = dy * w:
//   dx = dh + rstd * (g - n * mean_k(g * n)),   dw = sum over tokens of dy * n.
// All sums are fp32.
#pragma once

#include "act8.cuh"

namespace qnf4 {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf_lo(v.x); f[1] = bf_hi(v.x); f[2] = bf_lo(v.y); f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z); f[5] = bf_hi(v.z); f[6] = bf_lo(v.w); f[7] = bf_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Sum over the block (any multiple of 32 threads up to 1024); every thread gets the result.
// `slots` holds one float per warp; the same order of additions in every launch.
__device__ __forceinline__ float block_sum(float v, float* slots) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = (int)(threadIdx.x & 31) < warps ? slots[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  __syncthreads();   // `slots` may be written again
  return s;
}

struct NormFwdArgs {
  const uint16_t* x;
  const uint16_t* res;    // or NULL
  const uint16_t* w;
  int64_t M, K;
  float eps;
  uint16_t* y;
  uint16_t* h;            // NULL without a residual
  float* rstd;
  uint8_t* codes;         // NULL: no 8-bit output
  uint8_t* scales;
};

// One block per token; the row is read twice (the second time from L1 / L2).
__global__ void __launch_bounds__(512) rmsnorm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float slots[32];
  const int64_t m = blockIdx.x;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + m * a.K);
  const uint4* r = a.res ? reinterpret_cast<const uint4*>(a.res + m * a.K) : nullptr;
  const int64_t n8 = a.K / 8;
  float ss = 0.0f;
  for (int64_t c = threadIdx.x; c < n8; c += blockDim.x) {
    float f[8], q[8];
    unpack8(x[c], f);
    if (r) {
      unpack8(r[c], q);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += q[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
  }
  ss = block_sum(ss, slots);
  const float rstd = 1.0f / sqrtf(ss / (float)a.K + a.eps);
  if (threadIdx.x == 0) a.rstd[m] = rstd;
  const int64_t ld = a8_ld(a.K), G = a8_groups(a.K);
  // with an 8-bit output the loop covers whole groups of 32 features, so that the four lanes of a
  // group stay together
  const int64_t end = a.codes ? 4 * G : n8;
  const int64_t span = (end + blockDim.x - 1) / blockDim.x * blockDim.x;
  for (int64_t c = threadIdx.x; c < span; c += blockDim.x) {
    uint4 yv = make_uint4(0u, 0u, 0u, 0u);
    if (c < n8) {
      float f[8], q[8];
      unpack8(x[c], f);
      if (r) {
        unpack8(r[c], q);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += q[i];
        reinterpret_cast<uint4*>(a.h + m * a.K)[c] = pack8(f);
      }
      unpack8(reinterpret_cast<const uint4*>(a.w)[c], q);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * q[i];
      yv = pack8(f);
      reinterpret_cast<uint4*>(a.y + m * a.K)[c] = yv;
    }
    if (a.codes) {
      uint2 q8;
      const uint32_t byte = a8_encode8(yv, q8);
      if (8 * c < ld) *reinterpret_cast<uint2*>(a.codes + m * ld + 8 * c) = q8;
      if (c < n8 && (c & 3) == 0) a.scales[m * G + (c >> 2)] = (uint8_t)byte;
    }
  }
}

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* dh;     // or NULL
  const uint16_t* h;
  const uint16_t* w;
  const float* rstd;
  int64_t M, K;
  uint16_t* dx;
  float* partial;         // [gridDim.x][K] sums of dy * n, or NULL
};

// Block b takes the tokens b, b + gridDim.x, ...
__global__ void __launch_bounds__(512) rmsnorm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float slots[32];
  const int64_t n8 = a.K / 8;
  const uint4* w = reinterpret_cast<const uint4*>(a.w);
  float* part = a.partial ? a.partial + (int64_t)blockIdx.x * a.K : nullptr;
  if (part)
    for (int64_t c = threadIdx.x; c < n8; c += blockDim.x)
      for (int i = 0; i < 8; ++i) part[8 * c + i] = 0.0f;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const uint4* dy = reinterpret_cast<const uint4*>(a.dy + m * a.K);
    const uint4* h = reinterpret_cast<const uint4*>(a.h + m * a.K);
    const float rstd = a.rstd[m];
    float dot = 0.0f;
    for (int64_t c = threadIdx.x; c < n8; c += blockDim.x) {
      float d[8], hh[8], ww[8];
      unpack8(dy[c], d);
      unpack8(h[c], hh);
      unpack8(w[c], ww);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = hh[i] * rstd;
        dot = fmaf(d[i] * ww[i], n, dot);
        if (part) part[8 * c + i] += d[i] * n;
      }
    }
    dot = block_sum(dot, slots) / (float)a.K;
    for (int64_t c = threadIdx.x; c < n8; c += blockDim.x) {
      float d[8], hh[8], ww[8], o[8];
      unpack8(dy[c], d);
      unpack8(h[c], hh);
      unpack8(w[c], ww);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (d[i] * ww[i] - hh[i] * rstd * dot);
      if (a.dh) {
        float e[8];
        unpack8(reinterpret_cast<const uint4*>(a.dh + m * a.K)[c], e);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += e[i];
      }
      reinterpret_cast<uint4*>(a.dx + m * a.K)[c] = pack8(o);
    }
  }
}

// out[k] = bf16(sum_p partial[p][k]), added in the order p = 0 .. parts - 1.
__global__ void __launch_bounds__(256) column_sum_bf16_kernel(const float* __restrict__ partial, int parts, int64_t n,
                                                              uint16_t* __restrict__ out) {
  const int64_t k = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (k >= n) return;
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += partial[(int64_t)p * n + k];
  out[k] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
}

static int norm_threads(int64_t k) {
  const int64_t t = (k / 8 + 31) / 32 * 32;
  return (int)(t > 512 ? 512 : t);
}

// Blocks of the backward pass: every token has one, up to two per SM when the weight's gradient
// is wanted (each block leaves one row of partial sums).
static int norm_bwd_blocks(int64_t M, bool dweight) {
  const int64_t cap = dweight ? 2 * 148 : (1ll << 31) - 1;
  return (int)(M < cap ? M : cap);
}

static cudaError_t launch_rmsnorm_fwd(const NormFwdArgs& a, cudaStream_t st) {
  rmsnorm_fwd_kernel<<<(unsigned)a.M, norm_threads(a.K), 0, st>>>(a);
  return cudaGetLastError();
}

static cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, uint16_t* dweight, cudaStream_t st) {
  const int blocks = norm_bwd_blocks(a.M, dweight != nullptr);
  rmsnorm_bwd_kernel<<<blocks, norm_threads(a.K), 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dweight) return e;
  column_sum_bf16_kernel<<<(unsigned)((a.K + 255) / 256), 256, 0, st>>>(a.partial, blocks, a.K, dweight);
  return cudaGetLastError();
}

}  // namespace qnf4
