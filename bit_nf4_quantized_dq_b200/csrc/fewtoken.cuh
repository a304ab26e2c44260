// The linear's forward for a few tokens (decoding): y = act(x W'^T + t B^T + bias) + residual with
// W' streamed once from its 4-bit codes, t = s x A^T.
//
// Work: 0.516 bytes of codes and scales per weight from HBM; the products are nothing, and what has
// to be kept small is the expansion of the codes.  Byte permutes (nf4_device.cuh, two per weight on a
// pipe of half rate) took 28 us at 13824 x 5120, five times the HBM time.  Here a byte of two codes
// looks up its two fp32 levels in shared memory: a table of 256 level pairs, one copy per lane, so
// that a warp's 64-bit reads never share a bank, and the address is one byte permute.  The pair is
// then scaled and rounded by paired arithmetic, bf16(fp32(level * scale)), exactly the dequantized
// weight of every other path.
//  - One block of 16 warps per SM (the table is 64 KB).  A tile is 8 rows of W, the n side of the
//    warp-level m16n8k16 bf16 product (fp32 sums), with up to 16 tokens on its m side.  A work item
//    is 8 rows x 256 columns: lane (g, c) holds row g, columns 64 c .. 64 c + 63, whole blocks with
//    one scale each; the order of the columns inside a product is free as long as x follows it.
//  - A block's share of the tiles makes one list of items, columns outermost, cut evenly over its
//    warps: a warp keeps the x of its 256 columns in registers and walks down the tiles.  Each
//    item's sums go to shared memory and are added over the columns in order, so results do not
//    depend on timing; the epilogue is applied there.
//  - The codes and scales of the next two items are on their way while one is expanded.
//  - tcgen05 would need the tile staged for 128 rows and at least 16 tokens; as 16-token tiles of the
//    fused GEMM (with its K splits and a reduction) the same layer takes 52 us, here 24 us.
#pragma once

#include "epilogue.cuh"
#include "gemm.h"

namespace qnf4 {

constexpr int kFewTokens = 16;    // most tokens of this path
constexpr int kFewRows = 8;       // rows of W per tile
constexpr int kFewCols = 256;     // columns per work item
constexpr int kFewWarps = 16;
// The table sits at shared address 65536, so that its address bytes are (lane * 8, code byte, 1, 0):
// one permute of the codes and a lane constant.  The items' sums lie behind it.
constexpr uint32_t kFewTableAddr = 65536, kFewTableBytes = 65536;
constexpr int kFewSumBytes = 96 * 1024;
constexpr int kFewSmemBytes = (int)(kFewTableAddr + kFewTableBytes) + kFewSumBytes;
static_assert(kFewSmemBytes <= 227 * 1024, "shared memory of one block");
// item sums that fit: kFewRows x (8 or 16 tokens) floats each
__host__ __device__ constexpr int few_slots(bool two) { return kFewSumBytes / ((two ? 16 : 8) * kFewRows * 4); }

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

// t[m][j] = s sum_k x[m][k] A[j][k]: one block per rank column and kFewDownTokens tokens.
constexpr int kFewDownTokens = 4;
struct FewTokenDownParams {
  const uint16_t* x;
  const uint16_t* A;
  int32_t M, r;
  int64_t K;
  float s;
  float* t;
};

template <int TOK>
__global__ void __launch_bounds__(256) few_token_down_kernel(const FewTokenDownParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the product may start streaming W
  __shared__ float sums[8][TOK];
  const int j = blockIdx.x, m0 = blockIdx.y * TOK, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n8 = p.K / 8;
  const uint4* a = reinterpret_cast<const uint4*>(p.A + (int64_t)j * p.K);
  uint64_t acc[TOK];
#pragma unroll
  for (int m = 0; m < TOK; ++m) acc[m] = 0ull;
#pragma unroll 2
  for (int64_t c = threadIdx.x; c < n8; c += 256) {
    uint64_t av[4];
    unpack8_pairs(__ldg(a + c), av);
#pragma unroll
    for (int m = 0; m < TOK; ++m) {
      uint64_t xv[4];   // tokens past M repeat the last one, unread
      unpack8_pairs(__ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)min(m0 + m, p.M - 1) * p.K) + c), xv);
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
  if (threadIdx.x < TOK && m0 + (int)threadIdx.x < p.M) {
    float v = sums[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) v += sums[w][threadIdx.x];
    p.t[(int64_t)(m0 + threadIdx.x) * p.r + j] = p.s * v;
  }
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (a, b) as bf16 pairs: hi = bf16(v), lo = bf16(v - hi)
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(a - bf_lo(hi), b - bf_hi(hi));
}

// One row's 64 columns as fetched, nothing computed yet (a use of a loaded value would hold the warp
// until it arrives): the codes, the stored scale of their block and, where a block boundary lies
// inside (K % 64 != 0), the next block's and the number of 8-code words before the boundary.
struct FewScale {
  uint32_t code;   // E4M3 scale code (double quantization)
  float value;     // its group constant, or the fp32 scale itself
};
template <bool GENERIC>
struct FewUnit {
  uint32_t w[8];
  FewScale s0, s1;
  int32_t split;
};

__device__ __forceinline__ FewScale few_scale(const FewTokenParams& p, uint32_t blk) {
  if (p.scale_fp32) return FewScale{0u, __ldg(p.scales + blk)};
  return FewScale{__ldg(p.scale_codes + blk), __ldg(p.scales + (blk >> 8))};
}

// `src` addresses the unit's codes, `blk` is its first block, `in_blk` the words of its first block
// (8 where K % 64 == 0), `valid` its number of 8-code words before K.  Columns past K take codes
// before them: x is zero there.
template <bool GENERIC>
__device__ __forceinline__ void few_fetch(const FewTokenParams& p, const uint8_t* src, uint32_t blk, int in_blk,
                                          int valid, FewUnit<GENERIC>& u) {
  u.s0 = few_scale(p, blk);
  if constexpr (GENERIC) {
    u.split = in_blk;
    u.s1 = few_scale(p, in_blk < valid ? blk + 1 : blk);   // the next block exists where a valid word lies in it
#pragma unroll
    for (int j = 0; j < 8; ++j) u.w[j] = __ldg(reinterpret_cast<const uint32_t*>(src) + (j < valid ? j : 0));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(src)), b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    u.w[0] = a.x; u.w[1] = a.y; u.w[2] = a.z; u.w[3] = a.w;
    u.w[4] = b.x; u.w[5] = b.y; u.w[6] = b.z; u.w[7] = b.w;
  }
}

// TWO: more than 8 tokens.
template <bool TWO, bool GENERIC>
__global__ void __launch_bounds__(32 * kFewWarps, 1) few_token_kernel(const __grid_constant__ FewTokenParams p) {
  constexpr int kTok = TWO ? 16 : 8;
  constexpr int kSlot = kTok * kFewRows;
  extern __shared__ __align__(16) uint8_t few_smem[];
  uint8_t* const at65536 = few_smem + (kFewTableAddr - smem_u32(few_smem));
  float* sums = reinterpret_cast<float*>(at65536 + kFewTableBytes);      // [tile][quad][kTok][kFewRows]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const float mean = p.scale_fp32 ? 0.0f : __ldg(p.mean);
  const int quads = (int)((p.K + kFewCols - 1) / kFewCols);
  const int64_t tiles = p.N / kFewRows;
  const int64_t t_begin = tiles * blockIdx.x / gridDim.x, t_end = tiles * (blockIdx.x + 1) / gridDim.x;
  // rounds of tiles whose sums fit, of even sizes
  const int most = few_slots(TWO) / (quads + 1);
  const int rounds = (int)((t_end - t_begin + most - 1) / most);
  const int per_round = (int)((t_end - t_begin + rounds - 1) / rounds);
  const uint16_t* x0 = p.x + (int64_t)min(g, p.M - 1) * p.K;       // rows past M repeat the last one, unread
  const uint16_t* x1 = p.x + (int64_t)min(g + 8, p.M - 1) * p.K;

  if (threadIdx.x == 0) {
#pragma unroll
    for (int j = 0; j < 16; ++j) sums[j] = p.cb.q[j];
  }
  __syncthreads();
  for (int b = warp; b < 256; b += kFewWarps)
    *reinterpret_cast<float2*>(at65536 + b * 256 + lane * 8) = make_float2(sums[b & 15], sums[b >> 4]);
  __syncthreads();
  // behind the barrier, and opaque: every lookup's address depends on it
  uint32_t lane_addr = kFewTableAddr + (uint32_t)lane * 8u;
  asm volatile("" : "+r"(lane_addr)::"memory");

  for (int64_t t0 = t_begin; t0 < t_end; t0 += per_round) {
    const int nt = (int)min(t_end - t0, (int64_t)per_round);
    const int items = nt * quads;
    const int i0 = (int)((int64_t)items * warp / kFewWarps), i1 = (int)((int64_t)items * (warp + 1) / kFewWarps);
    // the item whose codes are fetched next
    int f_quad = i0 / nt, f_tile = i0 - f_quad * nt, f_valid = 0, f_in = 8;
    const uint8_t* f_src = nullptr;
    uint32_t f_blk = 0;
    int64_t f_at = 0;   // flat index of the unit's first weight
    auto locate = [&]() {
      f_src = p.codes + (f_at >> 1);
      f_blk = (uint32_t)(f_at >> 6);
      f_in = GENERIC ? (int)((64 - (f_at & 63)) >> 3) : 8;
    };
    auto place = [&]() {
      int64_t kcol = (int64_t)f_quad * kFewCols + 64 * c;
      f_valid = kcol >= p.K ? 0 : (int)min((p.K - kcol) >> 3, (int64_t)8);
      if (f_valid == 0) kcol = p.K - 8 * (f_valid = GENERIC ? 1 : 8);
      f_at = ((t0 + f_tile) * kFewRows + g) * p.K + kcol;
      locate();
    };
    auto fetch = [&](FewUnit<GENERIC>& u) {
      few_fetch<GENERIC>(p, f_src, f_blk, f_in, f_valid, u);
      if (++f_tile == nt) {
        f_tile = 0;
        if (++f_quad < quads) place();
      } else if constexpr (GENERIC) {
        f_at += kFewRows * p.K;
        locate();
      } else {
        f_src += kFewRows / 2 * p.K;
        f_blk += (uint32_t)(p.K >> 3);   // 8 rows of K / 64 blocks
      }
    };
    int quad = f_quad, tile = f_tile;
    FewUnit<GENERIC> u0, u1;
    if (i0 < i1) {
      place();
      fetch(u0);
    }
    if (i0 + 1 < i1) fetch(u1);
    for (int i = i0; i < i1; ++quad, tile = 0) {
      // this warp's tiles of one quad of columns: x stays in registers
      uint4 xa[8], xb[TWO ? 8 : 1];
      const int64_t kcol = (int64_t)quad * kFewCols + 64 * c;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xa[j] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (TWO) xb[j] = xa[j];
        if (kcol + 8 * j < p.K) {
          xa[j] = __ldg(reinterpret_cast<const uint4*>(x0 + kcol + 8 * j));
          if constexpr (TWO) xb[j] = __ldg(reinterpret_cast<const uint4*>(x1 + kcol + 8 * j));
        }
      }
      const int stop = min(i1, i + nt - tile);
      float* out = sums + (tile * quads + quad) * kSlot + g * kFewRows + 2 * c;
#pragma unroll 2
      for (; i < stop; ++i, out += quads * kSlot) {
        const FewUnit<GENERIC> v = u0;
        u0 = u1;
        if (i + 2 < i1) fetch(u1);
        const float s0 = p.scale_fp32 ? v.s0.value : dq_block_scale(v.s0.code, v.s0.value, mean);
        const float s1 = !GENERIC ? s0 : p.scale_fp32 ? v.s1.value : dq_block_scale(v.s1.code, v.s1.value, mean);
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float sc = (GENERIC && j >= v.split) ? s1 : s0;
          uint32_t b[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t at = prmt(v.w[j], lane_addr, 0x7604u | ((uint32_t)h << 4));
            uint64_t q;
            asm("ld.shared.b64 %0, [%1];" : "=l"(q) : "r"(at));   // the table does not change any more
            q = f32x2_mul(q, f32_pair(sc, sc));
            b[h] = pack_bf16x2(pair_lo(q), pair_hi(q));
          }
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          const uint4& y = TWO ? xb[j] : zero;
          mma_bf16_16816(acc, xa[j].x, y.x, xa[j].y, y.y, b[0], b[1]);
          mma_bf16_16816(acc, xa[j].z, y.z, xa[j].w, y.w, b[2], b[3]);
        }
        // accumulators: token g (and g + 8), rows 2 c and 2 c + 1
        *reinterpret_cast<float2*>(out) = make_float2(acc[0], acc[1]);
        if constexpr (TWO) *reinterpret_cast<float2*>(out + 8 * kFewRows) = make_float2(acc[2], acc[3]);
      }
    }
    if (p.t) {
      // t B^T: t as bf16 hi + lo (16 significant bits), one more slot of sums per tile
      asm volatile("griddepcontrol.wait;" ::: "memory");   // t comes from the grid before
      const float* ta = p.t + (int64_t)min(g, p.M - 1) * p.r;
      const float* tb = p.t + (int64_t)min(g + 8, p.M - 1) * p.r;
      for (int tl = warp; tl < nt; tl += kFewWarps) {
        const uint16_t* brow = p.B + ((t0 + tl) * kFewRows + g) * p.r;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 4 * c; j < p.r + 4 * c; j += 16) {   // 16 rank columns a step: lane c takes 4 of them
          float4 va = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vb = va;
          uint2 bv = make_uint2(0u, 0u);
          if (j < p.r) {
            va = *reinterpret_cast<const float4*>(ta + j);
            if constexpr (TWO) vb = *reinterpret_cast<const float4*>(tb + j);
            bv = __ldg(reinterpret_cast<const uint2*>(brow + j));
          }
          uint32_t ha0, la0, ha1, la1, hb0, lb0, hb1, lb1;
          split_bf16x2(va.x, va.y, ha0, la0);
          split_bf16x2(va.z, va.w, ha1, la1);
          split_bf16x2(vb.x, vb.y, hb0, lb0);
          split_bf16x2(vb.z, vb.w, hb1, lb1);
          mma_bf16_16816(acc, ha0, hb0, ha1, hb1, bv.x, bv.y);
          mma_bf16_16816(acc, la0, lb0, la1, lb1, bv.x, bv.y);
        }
        float* out = sums + (nt * quads + tl) * kSlot + g * kFewRows + 2 * c;
        *reinterpret_cast<float2*>(out) = make_float2(acc[0], acc[1]);
        if constexpr (TWO) *reinterpret_cast<float2*>(out + 8 * kFewRows) = make_float2(acc[2], acc[3]);
      }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < nt * kFewRows * p.M; o += 32 * kFewWarps) {
      const int row = o % kFewRows, rest = o / kFewRows, tl = rest % nt, tok = rest / nt;
      const int64_t n = (t0 + tl) * kFewRows + row;
      float z = 0.0f;
      const float* part = sums + tl * quads * kSlot + tok * kFewRows + row;
#pragma unroll 8
      for (int w = 0; w < quads; ++w) z += part[w * kSlot];
      if (p.t) z += sums[(nt * quads + tl) * kSlot + tok * kFewRows + row];
      if (p.post.bias) z += __uint_as_float((uint32_t)p.post.bias[n] << 16);
      const int64_t at = (int64_t)tok * p.N + n;
      if (p.post.z) p.post.z[at] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
      float v[2] = {z, 0.0f};
      act_apply(v, p.post.act);
      if (p.post.residual) v[0] += __uint_as_float((uint32_t)p.post.residual[at] << 16);
      p.y[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
    __syncthreads();   // the sums are free for the next round
  }
}

// Whether this path takes the shape: few tokens, a row's items fit the sums, block numbers 32 bits.
// Nine to sixteen tokens double the registers of x and the sums of an item, and with long rows the
// fused GEMM's 16-token tiles are then faster: at 16 tokens 72 against 58 us for 5120 x 13824, but 53
// against 55 us for 13824 x 5120, 27 against 34 us for 5120 x 5120 and 19 against 27 us for 4096 x
// 4096.  Up to 8 tokens this path takes 0.35 to 0.6 of the tiles' time.
static bool few_token_fits(int64_t M, int64_t K, int64_t N) {
  if (M > 8 && K > 8192) return false;
  return M <= kFewTokens && (K + kFewCols - 1) / kFewCols < few_slots(M > 8) && N * K < (1ll << 37);
}

template <bool TWO, bool GENERIC>
static cudaError_t launch_few_token_t(const FewTokenParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = enable_smem_once(few_token_kernel<TWO, GENERIC>, kFewSmemBytes, configured);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, p.N / kFewRows));
  cfg.blockDim = dim3(32 * kFewWarps);
  cfg.dynamicSmemBytes = kFewSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.t ? 1 : 0;   // with adapters the grid before is the one that makes t
  return cudaLaunchKernelEx(&cfg, few_token_kernel<TWO, GENERIC>, p);
}

static cudaError_t launch_few_token(const FewTokenParams& p, cudaStream_t st) {
  if (p.M <= 8) return p.K % 64 ? launch_few_token_t<false, true>(p, st) : launch_few_token_t<false, false>(p, st);
  return p.K % 64 ? launch_few_token_t<true, true>(p, st) : launch_few_token_t<true, false>(p, st);
}

static cudaError_t launch_few_token_down(const FewTokenDownParams& p, cudaStream_t st) {
  if (p.M == 1) few_token_down_kernel<1><<<p.r, 256, 0, st>>>(p);
  else few_token_down_kernel<kFewDownTokens><<<dim3(p.r, (p.M + kFewDownTokens - 1) / kFewDownTokens), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace qnf4
