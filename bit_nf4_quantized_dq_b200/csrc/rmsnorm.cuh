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

#include <algorithm>

#include "act8.cuh"

namespace qnf4 {

// Sum over the block (any multiple of 32 threads up to 1024); every thread gets the result, added in
// the same order in every launch.  `slots` holds one float per warp; a loop alternates between two
// sets of slots, so that one barrier per sum is enough.
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
  return s;
}

// 16 bytes global -> shared, asynchronous (past L1), in groups that the issuing thread waits for.
__device__ __forceinline__ void cp_async16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

// One block per token, each thread with up to VPT units of 8 features in registers, so that x and
// the residual are read once: an HBM stream of 4 to 9 bytes per value and a block-wide sum between
// its loads and its stores (several resident blocks cover one another's sums).  8192 x 5120 with residual
// and 8-bit output: 61 us, 0.95 of the memory rate.
template <int VPT, bool RES, bool A8>
__global__ void __launch_bounds__(512) rmsnorm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float slots[32];
  const int64_t m = blockIdx.x;
  const int n8 = (int)(a.K / 8), T = blockDim.x;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + m * a.K);
  uint4 xv[VPT], rv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * T + threadIdx.x;
    xv[i] = rv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < n8) {
      xv[i] = __ldcs(x + c);
      if constexpr (RES) rv[i] = __ldcs(reinterpret_cast<const uint4*>(a.res + m * a.K) + c);
    }
  }
  float f[VPT][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * T + threadIdx.x;
    unpack8(xv[i], f[i]);
    if constexpr (RES) {
      float q[8];
      unpack8(rv[i], q);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] += q[j];
      if (c < n8) reinterpret_cast<uint4*>(a.h + m * a.K)[c] = pack8(f[i]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[i][j], f[i][j], ss);
  }
  ss = block_sum(ss, slots);
  const float rstd = 1.0f / sqrtf(ss / (float)a.K + a.eps);
  if (threadIdx.x == 0) a.rstd[m] = rstd;
  const int64_t ld = a8_ld(a.K), G = a8_groups(a.K);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * T + threadIdx.x;
    uint4 yv = make_uint4(0u, 0u, 0u, 0u);
    if (c < n8) {
      float q[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(a.w) + c), q);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] *= f[i][j] * rstd;
      yv = pack8(q);
      reinterpret_cast<uint4*>(a.y + m * a.K)[c] = yv;
    }
    if constexpr (A8) {
      // the block covers whole groups of 32 features: units past K encode zeros
      uint2 q8;
      const uint32_t byte = a8_encode8(yv, q8);
      if (8 * (int64_t)c < ld) *reinterpret_cast<uint2*>(a.codes + m * ld + 8 * (int64_t)c) = q8;
      if (c < n8 && (c & 3) == 0) a.scales[m * G + (c >> 2)] = (uint8_t)byte;
    }
  }
}

// Rows too long for the registers of one block: the same, with the row read twice (the second time
// from L2).
__global__ void __launch_bounds__(512) rmsnorm_fwd_long_kernel(const NormFwdArgs a) {
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
  const int64_t end = a.codes ? 4 * G : n8;   // whole groups: a group's four lanes stay together
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
      for (int i = 0; i < 8; ++i) q[i] *= f[i] * rstd;
      yv = pack8(q);
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

// A block takes a run of tokens (every gridDim.x-th token instead read the same bytes 10 to 25 % slower:
// 64.6 against 58.6 us for 8192 x 5120 with both optional parts); a thread owns up to VPT units of 8
// features, the same ones for every token, so the weight's gradient accumulates in its registers and leaves as
// one row of partial sums per block.  The rows of dy, h and dh of the next S - 1 tokens are on their
// way into shared memory meanwhile: a thread copies and reads only its own units, so the ring
// needs no barrier, and a token costs one barrier, that of its sum.
// (96 registers at VPT = 2: two blocks of 320 threads per SM at K = 5120.)
template <int VPT, int S, bool DH, bool DW>
__global__ void __maxnreg__(VPT <= 2 ? 96 : 128) rmsnorm_bwd_kernel(const NormBwdArgs a) {
  extern __shared__ uint4 ring[];   // [stage][dy, h (, dh)][VPT][threads]
  __shared__ float slots[2][32];
  constexpr int kRows = DH ? 3 : 2;
  constexpr bool kKeep = VPT <= 2;   // g and n stay in registers across the sum, else they are formed again
  const int n8 = (int)(a.K / 8), T = blockDim.x;
  const float inv_k = 1.0f / (float)a.K;
  uint4* mine = ring + threadIdx.x;
  auto slot = [&](int stage, int row, int i) { return mine + ((stage * kRows + row) * VPT + i) * T; };
  auto load = [&](int64_t m, int stage, int64_t end) {
    if (m < end) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = i * T + threadIdx.x;
        if (c < n8) {
          cp_async16(slot(stage, 0, i), reinterpret_cast<const uint4*>(a.dy + m * a.K) + c);
          cp_async16(slot(stage, 1, i), reinterpret_cast<const uint4*>(a.h + m * a.K) + c);
          if constexpr (DH) cp_async16(slot(stage, 2, i), reinterpret_cast<const uint4*>(a.dh + m * a.K) + c);
        }
      }
    }
    cp_async_commit();
  };
  const int64_t per = a.M / gridDim.x, extra = a.M - per * gridDim.x;
  const int64_t first = blockIdx.x * per + min((int64_t)blockIdx.x, extra), last = first + per + (blockIdx.x < extra ? 1 : 0);
#pragma unroll
  for (int s = 0; s < S; ++s) load(first + s, s, last);
  // pairs of fp32 values throughout: the paired instructions halve the arithmetic
  uint64_t w2[VPT][4], acc[DW ? VPT : 1][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = i * T + threadIdx.x;
    unpack8_pairs(c < n8 ? __ldg(reinterpret_cast<const uint4*>(a.w) + c) : make_uint4(0u, 0u, 0u, 0u), w2[i]);
    if constexpr (DW) {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
    }
  }
  int stage = 0, flip = 0;
  for (int64_t m = first; m < last; ++m) {
    const float rstd = __ldg(a.rstd + m);
    const uint64_t r2 = f32_pair(rstd, rstd);
    cp_async_wait<S - 1>();
    uint64_t g2[kKeep ? VPT : 1][4], n2[kKeep ? VPT : 1][4], dot2 = 0ull;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (i * T + (int)threadIdx.x >= n8) continue;
      const int k = kKeep ? i : 0;
      uint64_t d[4];
      unpack8_pairs(*slot(stage, 0, i), d);
      unpack8_pairs(*slot(stage, 1, i), n2[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n2[k][j] = f32x2_mul(n2[k][j], r2);
        g2[k][j] = f32x2_mul(d[j], w2[i][j]);
        dot2 = f32x2_fma(g2[k][j], n2[k][j], dot2);
        if constexpr (DW) acc[i][j] = f32x2_fma(d[j], n2[k][j], acc[i][j]);
      }
    }
    const float dot = block_sum(pair_lo(dot2) + pair_hi(dot2), slots[flip]) * inv_k;
    flip ^= 1;
    const uint64_t c2 = f32_pair(-rstd * dot, -rstd * dot);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * T + threadIdx.x;
      if (c >= n8) continue;
      const int k = kKeep ? i : 0;
      uint64_t e[4] = {0ull, 0ull, 0ull, 0ull};
      if constexpr (!kKeep) {
        unpack8_pairs(*slot(stage, 0, i), g2[0]);
        unpack8_pairs(*slot(stage, 1, i), n2[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          n2[0][j] = f32x2_mul(n2[0][j], r2);
          g2[0][j] = f32x2_mul(g2[0][j], w2[i][j]);
        }
      }
      if constexpr (DH) unpack8_pairs(*slot(stage, 2, i), e);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = f32x2_fma(n2[k][j], c2, f32x2_fma(g2[k][j], r2, e[j]));
      reinterpret_cast<uint4*>(a.dx + m * a.K)[c] =
          make_uint4(pack_bf16x2(pair_lo(e[0]), pair_hi(e[0])), pack_bf16x2(pair_lo(e[1]), pair_hi(e[1])),
                     pack_bf16x2(pair_lo(e[2]), pair_hi(e[2])), pack_bf16x2(pair_lo(e[3]), pair_hi(e[3])));
    }
    load(m + S, stage, last);   // every value of this stage has been used
    if (++stage == S) stage = 0;
  }
  if constexpr (DW) {
    float* part = a.partial + (int64_t)blockIdx.x * a.K;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = i * T + threadIdx.x;
      if (c < n8) {
        reinterpret_cast<ulonglong2*>(part)[2 * c] = make_ulonglong2(acc[i][0], acc[i][1]);
        reinterpret_cast<ulonglong2*>(part)[2 * c + 1] = make_ulonglong2(acc[i][2], acc[i][3]);
      }
    }
  }
}

// Rows too long for the registers of one block: dy and h are read twice, the partial sums of the
// weight's gradient accumulate in memory.
__global__ void __launch_bounds__(512) rmsnorm_bwd_long_kernel(const NormBwdArgs a) {
  __shared__ float slots[2][32];
  int flip = 0;
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
    dot = block_sum(dot, slots[flip]) / (float)a.K;
    flip ^= 1;
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

// out[k] = bf16(sum_p partial[p][k]).  A block owns 32 columns; warp w takes the parts w, w + 32, ...,
// and the warps' sums are added in the order of the warps, so the order of additions is fixed.  (With
// 8 warps the 1480 parts of a 560-wide norm took 8 us, three quarters of its gradient's time.)
constexpr int kColumnWarps = 32;

// (`partial` is not __restrict__: the grid before may still write it when this one starts, and a promise of
// unchanging memory would let its loads move in front of the wait.)
__global__ void __launch_bounds__(32 * kColumnWarps) column_sum_bf16_kernel(const float* partial, int parts, int64_t n,
                                                                            uint16_t* out) {
  __shared__ float sums[kColumnWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts come from the grid before
  if (k < n) {
#pragma unroll 8
    for (int p = warp; p < parts; p += kColumnWarps) s += partial[(int64_t)p * n + k];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && k < n) {
    float t = sums[0][lane];
#pragma unroll
    for (int w = 1; w < kColumnWarps; ++w) t += sums[w][lane];
    out[k] = __bfloat16_as_ushort(__float2bfloat16_rn(t));
  }
}

static cudaError_t launch_column_sum(const float* partial, int parts, int64_t n, uint16_t* out, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((n + 31) / 32));
  cfg.blockDim = dim3(32 * kColumnWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, column_sum_bf16_kernel, partial, parts, n, out);
}

// Threads for `units` row units of 8 values, `vpt` per thread.
static int norm_threads(int64_t units, int vpt) { return (int)(((units + vpt - 1) / vpt + 31) / 32 * 32); }

// Units per thread of the backward kernel, and its blocks: one per token up to what keeps about 640
// threads per SM busy (2 to 16 blocks), then each block walks over its share of the tokens.
static int norm_bwd_vpt(int64_t units) { return units > 1024 ? 4 : units > 64 ? 2 : 1; }
static int norm_bwd_blocks(int64_t M, int64_t K) {
  const int64_t units = K / 8;
  const int64_t per_sm = std::min<int64_t>(16, std::max<int64_t>(2, 640 / norm_threads(units, norm_bwd_vpt(units))));
  return (int)std::min<int64_t>(M, 148 * per_sm);
}

constexpr int64_t kNormUnits = 4 * 512;       // row units that one forward block's registers hold
// Row units of which the backward's ring holds three tokens' dy, h and dh (216 KB of the 227 KB a
// block may have); above, up to kNormUnits, it holds two.
constexpr int64_t kNormBwdUnits3 = 4 * 384;
constexpr int kNormRingMax = 3 * 3 * 16 * (int)kNormBwdUnits3;
static_assert(2 * 3 * 16 * kNormUnits <= kNormRingMax && kNormRingMax <= 227 * 1024 - 1024, "ring size");

template <int VPT>
static void launch_rmsnorm_fwd_v(const NormFwdArgs& a, int threads, cudaStream_t st) {
  const unsigned g = (unsigned)a.M;
  if (a.res) {
    if (a.codes) rmsnorm_fwd_kernel<VPT, true, true><<<g, threads, 0, st>>>(a);
    else rmsnorm_fwd_kernel<VPT, true, false><<<g, threads, 0, st>>>(a);
  } else {
    if (a.codes) rmsnorm_fwd_kernel<VPT, false, true><<<g, threads, 0, st>>>(a);
    else rmsnorm_fwd_kernel<VPT, false, false><<<g, threads, 0, st>>>(a);
  }
}

static cudaError_t launch_rmsnorm_fwd(const NormFwdArgs& a, cudaStream_t st) {
  const int64_t units = 4 * a8_groups(a.K);
  if (units > kNormUnits) rmsnorm_fwd_long_kernel<<<(unsigned)a.M, 512, 0, st>>>(a);
  else if (units > 512) launch_rmsnorm_fwd_v<4>(a, norm_threads(units, 4), st);
  else if (units > 64) launch_rmsnorm_fwd_v<2>(a, norm_threads(units, 2), st);
  else launch_rmsnorm_fwd_v<1>(a, norm_threads(units, 1), st);
  return cudaGetLastError();
}

template <int VPT, int S, bool DH, bool DW>
static cudaError_t launch_rmsnorm_bwd_t(const NormBwdArgs& a, int blocks, int threads, cudaStream_t st) {
  const int smem = S * (DH ? 3 : 2) * VPT * threads * 16;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = enable_smem_once(rmsnorm_bwd_kernel<VPT, S, DH, DW>, kNormRingMax, configured);
  if (e != cudaSuccess) return e;
  rmsnorm_bwd_kernel<VPT, S, DH, DW><<<blocks, threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int VPT, int S>
static cudaError_t launch_rmsnorm_bwd_v(const NormBwdArgs& a, int blocks, int threads, cudaStream_t st) {
  if (a.partial)
    return a.dh ? launch_rmsnorm_bwd_t<VPT, S, true, true>(a, blocks, threads, st)
                : launch_rmsnorm_bwd_t<VPT, S, false, true>(a, blocks, threads, st);
  return a.dh ? launch_rmsnorm_bwd_t<VPT, S, true, false>(a, blocks, threads, st)
              : launch_rmsnorm_bwd_t<VPT, S, false, false>(a, blocks, threads, st);
}

static cudaError_t launch_rmsnorm_bwd(const NormBwdArgs& a, uint16_t* dweight, cudaStream_t st) {
  const int blocks = norm_bwd_blocks(a.M, a.K);
  const int64_t units = a.K / 8;
  const int vpt = norm_bwd_vpt(units), threads = norm_threads(units, vpt);
  cudaError_t e;
  if (units > kNormUnits) {
    rmsnorm_bwd_long_kernel<<<blocks, 512, 0, st>>>(a);
    e = cudaGetLastError();
  } else if (vpt == 4) {
    e = units > kNormBwdUnits3 ? launch_rmsnorm_bwd_v<4, 2>(a, blocks, threads, st)
                               : launch_rmsnorm_bwd_v<4, 3>(a, blocks, threads, st);
  } else if (vpt == 2) {
    e = launch_rmsnorm_bwd_v<2, 3>(a, blocks, threads, st);
  } else {
    e = launch_rmsnorm_bwd_v<1, 3>(a, blocks, threads, st);
  }
  if (e != cudaSuccess || !dweight) return e;
  return launch_column_sum(a.partial, blocks, a.K, dweight, st);
}

}  // namespace qnf4
