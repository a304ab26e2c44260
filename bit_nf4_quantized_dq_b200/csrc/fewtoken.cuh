// The linear's forward for a few tokens (decoding): y = act(x W'^T + t B^T + bias) + residual with
// W' streamed once from its 4-bit codes, t = s x A^T.
//
// Work: 0.516 bytes of codes and scales per weight from HBM, against about 3 instructions per weight
// to expand them; the products themselves are nothing.  So the kernel is built around the stream:
//  - A block owns 16 rows of W (the 16 rows of a warp-level m16n8k16 bf16 product, fp32 sums) and
//    its warps share the columns in units of 256: 4 lanes x 64 weights per row, so a lane expands
//    whole blocks of 64 through one 16-entry table per block (nf4_device.cuh) straight into the
//    product's A registers.  The order of the columns inside a product does not matter as long
//    as x is taken in the same order, so lane c of a row group takes columns 64 c .. 64 c + 63.
//  - tcgen05 would need the tile staged in shared or tensor memory for 128 rows and at least 16
//    tokens; the same rows as 16-token tiles of the fused GEMM (with its K splits and a reduction)
//    took 62 us at 13824 x 5120 and one token.
//  - The next unit's codes and scales are on their way while one is expanded.
//  - The warps' sums are joined in shared memory, in the order of the warps, and the epilogue is
//    applied there.  W' is exactly the dequantized bf16 weight, as everywhere else.
#pragma once

#include "epilogue.cuh"
#include "gemm.h"

namespace qnf4 {

constexpr int kFewTokens = 16;    // most tokens of this path
constexpr int kFewRows = 16;

struct FewTokenParams {
  const uint16_t* x;       // [M][K]
  int32_t M;
  int64_t K, N;
  const uint8_t* codes;
  const uint8_t* scale_codes;
  const float* scales;
  const float* mean;
  int32_t scale_fp32;
  Codebook cb;
  const float* t;          // [M][r] or NULL
  const uint16_t* B;       // [N][r]
  int32_t r;
  EpiArgs post;
  uint16_t* y;             // [M][N]
};

// t[m][j] = s sum_k x[m][k] A[j][k]: one block per rank column, all tokens.
struct FewTokenDownParams {
  const uint16_t* x;
  const uint16_t* A;
  int32_t M, r;
  int64_t K;
  float s;
  float* t;
};

template <int TOK>
__global__ void __launch_bounds__(128) few_token_down_kernel(const FewTokenDownParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the product may start streaming W
  __shared__ float sums[4][TOK];
  const int j = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n8 = p.K / 8;
  const uint4* a = reinterpret_cast<const uint4*>(p.A + (int64_t)j * p.K);
  uint64_t acc[TOK];
#pragma unroll
  for (int m = 0; m < TOK; ++m) acc[m] = 0ull;
  for (int64_t c = threadIdx.x; c < n8; c += 128) {
    uint64_t av[4];
    unpack8_pairs(__ldg(a + c), av);
#pragma unroll
    for (int m = 0; m < TOK; ++m) {
      if (m >= p.M) break;
      uint64_t xv[4];
      unpack8_pairs(__ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)m * p.K) + c), xv);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m] = f32x2_fma(av[i], xv[i], acc[m]);
    }
  }
#pragma unroll
  for (int m = 0; m < TOK; ++m) {
    float v = pair_lo(acc[m]) + pair_hi(acc[m]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) sums[warp][m] = v;
  }
  __syncthreads();
  if (threadIdx.x < TOK && (int)threadIdx.x < p.M)
    p.t[(int64_t)threadIdx.x * p.r + j] =
        p.s * (((sums[0][threadIdx.x] + sums[1][threadIdx.x]) + sums[2][threadIdx.x]) + sums[3][threadIdx.x]);
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One row's 64 columns as fetched: the codes, the scale of their block and, where a block boundary
// lies inside (K % 64 != 0), the next block's and the number of 8-code words before the boundary.
// Columns past K and rows past N have zero scales, so they expand to zeros.
template <bool GENERIC>
struct FewUnit {
  uint32_t w[8];
  float s0, s1;
  int32_t split;
};

template <bool GENERIC>
__device__ __forceinline__ void few_fetch(const FewTokenParams& p, int64_t n, int64_t kcol, float mean,
                                          FewUnit<GENERIC>& u) {
  auto scale = [&](int64_t blk) {
    if (p.scale_fp32) return __ldg(p.scales + blk);
    return dq_block_scale(__ldg(p.scale_codes + blk), __ldg(p.scales + (blk >> 8)), mean);
  };
  u.s0 = u.s1 = 0.0f;
  u.split = 8;
#pragma unroll
  for (int j = 0; j < 8; ++j) u.w[j] = 0u;
  if (n >= p.N || kcol >= p.K) return;
  const int64_t f0 = n * p.K + kcol, blk = f0 >> 6;
  u.s0 = scale(blk);
  if constexpr (!GENERIC) {
    const uint4* src = reinterpret_cast<const uint4*>(p.codes + (f0 >> 1));
    const uint4 a = __ldg(src), b = __ldg(src + 1);
    u.w[0] = a.x; u.w[1] = a.y; u.w[2] = a.z; u.w[3] = a.w;
    u.w[4] = b.x; u.w[5] = b.y; u.w[6] = b.z; u.w[7] = b.w;
  } else {
    const int valid = (int)min((p.K - kcol) >> 3, (int64_t)8);
    u.split = (int)((64 - (f0 & 63)) >> 3);
    // the second block exists whenever a valid word lies in it
    if (u.split < valid) u.s1 = scale(blk + 1);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(p.codes + (f0 >> 1));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) u.w[j] = __ldg(src + j);
  }
}

// NT groups of 8 tokens; WARPS warps share the columns.
template <int NT, int WARPS, bool GENERIC>
__global__ void __launch_bounds__(32 * WARPS) few_token_kernel(const __grid_constant__ FewTokenParams p) {
  __shared__ float red[WARPS][kFewRows][8 * NT + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * kFewRows;
  const float mean = p.scale_fp32 ? 0.0f : __ldg(p.mean);
  const int64_t step = 256 * WARPS;
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;

  FewUnit<GENERIC> u0, u1;
  int64_t kcol = 256 * (int64_t)warp + 64 * c;
  few_fetch<GENERIC>(p, n0 + g, kcol, mean, u0);
  few_fetch<GENERIC>(p, n0 + g + 8, kcol, mean, u1);
  // the loop's bound is the warp's: a lane whose columns lie past K takes zeros
  for (int64_t kw = 256 * (int64_t)warp; kw < p.K; kw += step, kcol += step) {
    const FewUnit<GENERIC> v0 = u0, v1 = u1;
    few_fetch<GENERIC>(p, n0 + g, kcol + step, mean, u0);
    few_fetch<GENERIC>(p, n0 + g + 8, kcol + step, mean, u1);
    Nf4Lut L0, L1, M0, M1;
    nf4_lut_build(v0.s0, L0, p.cb);
    nf4_lut_build(v1.s0, L1, p.cb);
    if constexpr (GENERIC) {
      nf4_lut_build(v0.s1, M0, p.cb);
      nf4_lut_build(v1.s1, M1, p.cb);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint4 xv[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tok = 8 * t + g;
        xv[t] = make_uint4(0u, 0u, 0u, 0u);
        if (tok < p.M && kcol + 8 * j < p.K)
          xv[t] = __ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)tok * p.K + kcol + 8 * j));
      }
      uint32_t a[4], b[4];
      nf4_expand8(v0.w[j], (GENERIC && j >= v0.split) ? M0 : L0, a);
      nf4_expand8(v1.w[j], (GENERIC && j >= v1.split) ? M1 : L1, b);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_bf16_16816(acc[t], a[0], b[0], a[1], b[1], xv[t].x, xv[t].y);
        mma_bf16_16816(acc[t], a[2], b[2], a[3], b[3], xv[t].z, xv[t].w);
      }
    }
  }
  // accumulator i of lane (g, c): row g + 8 (i / 2), token 2 c + i % 2
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][g + 8 * (i >> 1)][8 * t + 2 * c + (i & 1)] = acc[t][i];
  __syncthreads();
  if (p.t) asm volatile("griddepcontrol.wait;" ::: "memory");   // t comes from the grid before
  for (int o = threadIdx.x; o < kFewRows * 8 * NT; o += 32 * WARPS) {
    const int row = o % kFewRows, tok = o / kFewRows;
    const int64_t n = n0 + row;
    if (n >= p.N || tok >= p.M) continue;
    float z = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) z += red[w][row][tok];
    if (p.t) {
      const uint4* b = reinterpret_cast<const uint4*>(p.B + n * p.r);
      const float4* t = reinterpret_cast<const float4*>(p.t + (int64_t)tok * p.r);
      float d = 0.0f;
      for (int j = 0; j < p.r / 8; ++j) {
        float bv[8];
        unpack8(__ldg(b + j), bv);
        const float4 t0 = t[2 * j], t1 = t[2 * j + 1];
        d = fmaf(bv[0], t0.x, d); d = fmaf(bv[1], t0.y, d); d = fmaf(bv[2], t0.z, d); d = fmaf(bv[3], t0.w, d);
        d = fmaf(bv[4], t1.x, d); d = fmaf(bv[5], t1.y, d); d = fmaf(bv[6], t1.z, d); d = fmaf(bv[7], t1.w, d);
      }
      z += d;
    }
    if (p.post.bias) z += __uint_as_float((uint32_t)p.post.bias[n] << 16);
    const int64_t at = (int64_t)tok * p.N + n;
    if (p.post.z) p.post.z[at] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
    float v[8] = {z, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    act_apply8(v, p.post.act);
    if (p.post.residual) v[0] += __uint_as_float((uint32_t)p.post.residual[at] << 16);
    p.y[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
  }
}

template <int NT, int WARPS>
static cudaError_t launch_few_token_w(const FewTokenParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.N + kFewRows - 1) / kFewRows));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.t ? 1 : 0;   // with adapters the grid before is the one that makes t
  return p.K % 64 ? cudaLaunchKernelEx(&cfg, few_token_kernel<NT, WARPS, true>, p)
                  : cudaLaunchKernelEx(&cfg, few_token_kernel<NT, WARPS, false>, p);
}

static cudaError_t launch_few_token(const FewTokenParams& p, cudaStream_t st) {
  // 8 warps per 16 rows; 16 where the rows alone leave most SMs with one block or none
  const bool wide = (p.N + kFewRows - 1) / kFewRows < 2 * 148;
  if (p.M <= 8) return wide ? launch_few_token_w<1, 16>(p, st) : launch_few_token_w<1, 8>(p, st);
  return wide ? launch_few_token_w<2, 16>(p, st) : launch_few_token_w<2, 8>(p, st);
}

static cudaError_t launch_few_token_down(const FewTokenDownParams& p, cudaStream_t st) {
  if (p.M == 1) few_token_down_kernel<1><<<p.r, 128, 0, st>>>(p);
  else if (p.M <= 4) few_token_down_kernel<4><<<p.r, 128, 0, st>>>(p);
  else few_token_down_kernel<kFewTokens><<<p.r, 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace qnf4
