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
//  - One block of 16 warps per SM (the table is 64 KB).  A work item is 16 rows of W (the m side of the
//    warp-level m16n8k16 bf16 product, fp32 sums, with 8 or 16 tokens on its n side) x 256 columns:
//    lane (g, c) holds rows g and g + 8, columns 64 c .. 64 c + 63, whole blocks with one scale each;
//    the order of the columns inside a product is free as long as x follows it.
//  - A block's share of the 16-row tiles makes one list of items, columns outermost, cut evenly over
//    its warps: a warp keeps the x of its 256 columns in registers and walks down the tiles.  Each
//    item's sums go to shared memory and are added over the columns in order, so results do not
//    depend on timing; the epilogue is applied there.
//  - The codes come by TMA, 2 KB per item, three items ahead in a ring of each warp: 96 KB on their way
//    per SM.  (With 2 KB ahead in a thread's registers or 48 KB in all, the stream alone took 9 us
//    more than an empty loop, at 36 MB.)  The 128-byte swizzle lets the lanes read them without bank
//    conflicts.  The scales are one item ahead in registers.
//  - tcgen05 would need the tile staged for 128 rows and at least 16 tokens; as 16-token tiles of the
//    fused GEMM (with its K splits and a reduction) the same layer takes 54 us, here 21 us.
// With K % 64 != 0 code rows are only 4-byte aligned and blocks span rows: a kernel of its own reads
// the codes into registers, in tiles of 8 rows.
#pragma once

#include <algorithm>

#include "epilogue.cuh"
#include "gemm.h"

namespace qnf4 {

constexpr int kFewTokens = 16;    // most tokens of this path
constexpr int kFewCols = 256;     // columns per work item
constexpr int kFewWarps = 16;
constexpr int kFewBlocks = 148;   // one per SM
// Shared memory.  The table sits at shared address 65536, so that its address bytes are (lane * 8, code
// byte, 1, 0): one permute of the codes and a lane constant.  The items' sums lie in front of it, from
// the start of the block's part on, the warps' rings of codes behind it.
constexpr uint32_t kFewTableAddr = 65536, kFewRingAddr = 131072;
constexpr int kFewRing = 3;       // items on their way per warp
constexpr int kFewItemBytes = 16 * kFewCols / 2;
constexpr int kFewRingBytes = kFewWarps * kFewRing * kFewItemBytes;
constexpr int kFewSmemBytes = (int)kFewRingAddr + kFewRingBytes + kFewWarps * kFewRing * 8 + 16;
static_assert(kFewSmemBytes <= 227 * 1024, "shared memory of one block");
constexpr int kFewStageBytes = 4 * kFewCols * 2;   // x of four tokens
constexpr int kFewRaggedSmemBytes = (int)kFewRingAddr + kFewWarps * kFewStageBytes;
static_assert(kFewStageBytes <= kFewItemBytes, "a slot of the ring hands over x");
// Room for sums: the block's part of shared memory starts 1 KB up (checked at the launch).
constexpr int kFewReservedBytes = 1024, kFewSumBytes = (int)kFewTableAddr - kFewReservedBytes;

struct FewTokenParams {
  CUtensorMap map;         // codes [N][K / 2], boxes of 16 rows x 128 bytes, 128-byte swizzle (K % 64 == 0)
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
  float* part;             // [quads of columns + 1][M][N] sums of the items (flat list), or NULL
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
__global__ void __maxnreg__(TOK == 1 ? 32 : 64) few_token_down_kernel(const FewTokenDownParams p) {
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

// The stored scale of a block as fetched, nothing computed yet (a use of a loaded value would hold
// the warp until it arrives).
struct FewScale {
  uint32_t code;   // E4M3 scale code (double quantization)
  float value;     // its group constant, or the fp32 scale itself
};
__device__ __forceinline__ FewScale few_scale(const FewTokenParams& p, uint32_t blk) {
  if (p.scale_fp32) return FewScale{0u, __ldg(p.scales + blk)};
  return FewScale{__ldg(p.scale_codes + blk), __ldg(p.scales + (blk >> 8))};
}
__device__ __forceinline__ float few_scale_value(const FewTokenParams& p, const FewScale& s, float mean) {
  return p.scale_fp32 ? s.value : dq_block_scale(s.code, s.value, mean);
}

// Fills the table: warp w writes the pairs of the bytes w, w + 16, ..., whose low code is w.  Returns the
// lane's table address, which every lookup's address depends on (opaque, so that no lookup moves in
// front of the barrier).
__device__ __forceinline__ uint32_t few_fill_table(const FewTokenParams& p, uint8_t* table) {
  static_assert(kFewWarps == 16, "one warp per low code");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float low = p.cb.q[warp];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    *reinterpret_cast<float2*>(table + (16 * i + warp) * 256 + lane * 8) = make_float2(low, p.cb.q[i]);
  __syncthreads();
  uint32_t lane_addr = kFewTableAddr + (uint32_t)lane * 8u;
  asm volatile("" : "+r"(lane_addr)::"memory");
  return lane_addr;
}
// Brings `bytes` bytes into L2, a line per thread.  What the end of a block reads (the adapter's rows, bias,
// residual) is fetched from its start on: read on demand it cost 1 to 2 us there, of 10.
__device__ __forceinline__ void few_prefetch(const void* base, int64_t bytes, int index, int threads) {
  const char* at = static_cast<const char*>(base);
  if (bytes <= 0) return;
  for (int64_t o = (int64_t)index * 128; o < bytes + 127; o += (int64_t)threads * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(at + (o < bytes ? o : bytes - 1)));
}
__device__ __forceinline__ void few_prefetch_rows(const FewTokenParams& p, int64_t n0, int64_t n1, bool outputs) {
  if (p.t) few_prefetch(p.B + n0 * p.r, (n1 - n0) * p.r * 2, threadIdx.x, 32 * kFewWarps);
  if (!outputs) return;
  if (p.post.bias && threadIdx.x < 32) few_prefetch(p.post.bias + n0, (n1 - n0) * 2, threadIdx.x, 32);
  if (p.post.residual)
    for (int tok = threadIdx.x >> 5; tok < p.M; tok += kFewWarps)
      few_prefetch(p.post.residual + tok * p.N + n0, (n1 - n0) * 2, threadIdx.x & 31, 32);
}
// Eight codes -> the four level pairs; and those times the scale, as bf16 pairs of the dequantized weight.
__device__ __forceinline__ void few_lookup8(uint32_t w, uint32_t lane_addr, uint64_t (&q)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t at = prmt(w, lane_addr, 0x7604u | ((uint32_t)k << 4));
    asm("ld.shared.b64 %0, [%1];" : "=l"(q[k]) : "r"(at));   // the table does not change any more
  }
}
__device__ __forceinline__ void few_round8(const uint64_t (&q)[4], uint64_t scale, uint32_t (&o)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t v = f32x2_mul(q[k], scale);
    o[k] = pack_bf16x2(pair_lo(v), pair_hi(v));
  }
}
__device__ __forceinline__ void few_expand8(uint32_t w, float scale, uint32_t lane_addr, uint32_t (&o)[4]) {
  uint64_t q[4];
  few_lookup8(w, lane_addr, q);
  few_round8(q, f32_pair(scale, scale), o);
}

// A block's share of `tiles`.
struct FewShare {
  int begin, end;
};
__device__ __forceinline__ FewShare few_share(int tiles) {
  const int base = tiles / (int)gridDim.x, extra = tiles - base * (int)gridDim.x;
  FewShare s;
  s.begin = (int)blockIdx.x * base + min((int)blockIdx.x, extra);
  s.end = s.begin + base + ((int)blockIdx.x < extra ? 1 : 0);
  return s;
}
// The tiles of a round: rounds of even sizes whose sums (`slot` floats per item, `quads` items per tile and one more
// for the adapter term) fit between the start of shared memory and the table.
__device__ __forceinline__ int few_per_round(int tiles, int quads, int slot) {
  const int one = 4 * slot * (quads + 1);
  if ((int64_t)tiles * one <= kFewSumBytes) return tiles;   // (the divisions are not free at the start of a short kernel)
  const int most = kFewSumBytes / one, rounds = (tiles + most - 1) / most;
  return (tiles + rounds - 1) / rounds;
}

// This lane's 64 columns (64 c .. 64 c + 63 of the quad) of its tokens g and, with NT = 2, g + 8, zeros
// past K.  Read directly, an instruction asks for 16 bytes of 32 different lines; so the warp reads whole
// rows of 512 bytes, four tokens at a time, and hands them over through 2 KB of shared memory: 16-byte
// piece j of lane column c of row i lies at j ^ (c + 4 i), so that neither side meets a bank conflict.
// 13824 x 5120, 8 tokens: 24.6 us, direct 26.6; 5120 x 13816 (ragged), 8 tokens 41.7 and 51.8, 16 tokens
// 68.8 and 103.  Tokens past M keep what the buffer held; nothing reads their sums.
template <int NT>
__device__ __forceinline__ void few_load_x(const FewTokenParams& p, int quad, uint8_t* stage, uint4 (&xv)[NT][8]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t col = (int64_t)quad * kFewCols + 8 * lane;
  const uint16_t* src = p.x + col;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint4 raw[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 8 * t + 4 * k + i;
        raw[k][i] = make_uint4(0u, 0u, 0u, 0u);
        if (tok < p.M && col < p.K) raw[k][i] = __ldg(reinterpret_cast<const uint4*>(src + tok * p.K));
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (8 * t + 4 * k >= p.M) break;
      __syncwarp();   // the buffer's last readers are done
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(stage + i * 512 + (((lane & 24) | ((lane & 7) ^ (((lane >> 3) + 4 * i) & 7))) << 4)) =
            raw[k][i];
      __syncwarp();
      if ((g >> 2) == k) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          xv[t][j] = *reinterpret_cast<const uint4*>(stage + (g & 3) * 512 + ((8 * c + (j ^ ((c + 4 * g) & 7))) << 4));
      }
    }
  }
}

// The outputs of a round's tiles: the items' sums added over the columns in order (and the adapter
// term, in slot nt * quads + tile), bias, activation, residual.  `at(row, token)` is a sum's place in
// its slot.
template <int ROWS, class At>
__device__ __forceinline__ void few_finish(const FewTokenParams& p, const float* sums, int slot, int t0, int nt, int quads,
                                           At at) {
  for (int o = threadIdx.x; o < nt * ROWS * p.M; o += 32 * kFewWarps) {
    const int row = o % ROWS, rest = o / ROWS, tl = rest % nt, tok = rest / nt;
    const int64_t n = (int64_t)(t0 + tl) * ROWS + row;
    if (n >= p.N) continue;
    const float* part = sums + at(row, tok);
    float z = 0.0f;
#pragma unroll 8
    for (int w = 0; w < quads; ++w) z += part[(tl * quads + w) * slot];
    if (p.t) z += part[(nt * quads + tl) * slot];
    if (p.post.bias) z += __uint_as_float((uint32_t)p.post.bias[n] << 16);
    const int64_t to = (int64_t)tok * p.N + n;
    if (p.post.z) p.post.z[to] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
    float v[2] = {z, 0.0f};
    act_apply(v, p.post.act);
    if (p.post.residual) v[0] += __uint_as_float((uint32_t)p.post.residual[to] << 16);
    p.y[to] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
  }
}

// K % 64 == 0.  TWO: more than 8 tokens.
// FLAT: the blocks share one list of all items, columns outermost, whatever tile they cut; every item
// leaves its sums in p.part for few_token_join_kernel.
// Registers: 128 are what 16 warps can have.  With 112, and as much of the SM set aside for shared memory
// by the down-projection, a block of that fits beside one of this: 8 % for one token of 5120 x 13824 as a
// flat list (25.1 us); the tile form does not gain.
template <bool TWO, bool FLAT>
__global__ void __maxnreg__(TWO || !FLAT ? 128 : 112) few_token_kernel(const __grid_constant__ FewTokenParams p) {
  constexpr int kRows = 16, NT = TWO ? 2 : 1, kSlot = NT * kRows * 8;   // sums [group of 8 tokens][row][token]
  extern __shared__ __align__(16) uint8_t few_smem[];
  uint8_t* const smem0 = few_smem - smem_u32(few_smem);                // shared address 0
  float* const sums = reinterpret_cast<float*>(few_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  uint8_t* const ring = smem0 + kFewRingAddr + warp * kFewRing * kFewItemBytes;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem0 + kFewRingAddr + kFewRingBytes);
  uint64_t* const full = bars + warp * kFewRing;
  volatile uint32_t* const abort_word = reinterpret_cast<uint32_t*>(bars + kFewWarps * kFewRing);
  if (threadIdx.x == 0) tma_prefetch_desc(&p.map);
  if (lane == 0) {   // a warp's ring is its own: no barrier of the block
    for (int k = 0; k < kFewRing; ++k) mbar_init(&full[k], 1);
    mbar_fence_init();
  }
  if (threadIdx.x == 0) *abort_word = 0u;
  __syncwarp();

  const int quads = (int)((p.K + kFewCols - 1) / kFewCols);
  const int tiles = (int)((p.N + kRows - 1) / kRows);
  const FewShare share = FLAT ? FewShare{0, tiles} : few_share(tiles);
  const float mean = p.scale_fp32 ? 0.0f : __ldg(p.mean);
  int slot = 0, pending = 0;     // the ring's slot read next, and its loads on their way
  uint32_t phase = 0u;
  bool ok = true;
  // FLAT: an item's sums of rows g and g + 8, tokens 2 c and 2 c + 1 of group t
  auto store_flat = [&](int at_quad, int at_tile, int t, const float (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int tok = 8 * t + 2 * c + (k & 1);
      const int64_t n = (int64_t)at_tile * kRows + g + 8 * (k >> 1);
      if (tok < p.M && n < p.N) p.part[((int64_t)at_quad * p.M + tok) * p.N + n] = v[k];
    }
  };
  const int t0 = share.begin, nt = share.end - share.begin;   // with tiles, all of their sums fit (few_token_plan)
  const int items = nt * quads;
  int i0 = items * warp / kFewWarps, i1 = items * (warp + 1) / kFewWarps;
  if constexpr (FLAT) {
    const int64_t parts = (int64_t)gridDim.x * kFewWarps, part = (int64_t)blockIdx.x * kFewWarps + warp;
    i0 = (int)(items * part / parts);
    i1 = (int)(items * (part + 1) / parts);
  }
  int quad = i0 / nt, tile = i0 - quad * nt;
  // the item whose codes are loaded next
  int c_quad = quad, c_tile = tile, c_left = i1 - i0;
  auto load_codes = [&](int s) {
    if (c_left == 0) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[s], kFewItemBytes);
      tma_load_2d(ring + s * kFewItemBytes, &p.map, c_quad * (kFewCols / 2), (t0 + c_tile) * kRows, &full[s]);
    }
    --c_left;
    ++pending;
    if (++c_tile == nt) {
      c_tile = 0;
      ++c_quad;
    }
  };
  // The first loads go out as one instruction of as many lanes (an instruction holds its thread for
  // hundreds of cycles, whatever the number of its lanes).
  {
    const int ahead = min(kFewRing - 1, c_left);   // the last slot hands over x first
    int my_quad = c_quad, my_tile = c_tile;
    for (int k = 0; k < ahead; ++k) {
      if (k == lane) {
        my_quad = c_quad;
        my_tile = c_tile;
      }
      if (++c_tile == nt) {
        c_tile = 0;
        ++c_quad;
      }
    }
    if (lane < ahead) {
      mbar_arrive_expect_tx(&full[lane], kFewItemBytes);
      tma_load_2d(ring + lane * kFewItemBytes, &p.map, my_quad * (kFewCols / 2), (t0 + my_tile) * kRows, &full[lane]);
    }
    c_left -= ahead;
    pending = ahead;
    __syncwarp();
  }
  // The scales of the next item.  Columns past K (whose codes arrive as zeros, and where x is zero) and
  // rows past N (N is a multiple of 8; their sums are not used) take the scales before them.
  int f_quad = quad, f_tile = tile;
  uint32_t f_blk[2] = {0u, 0u};
  auto place = [&]() {
    const int64_t col = min((int64_t)f_quad * kFewCols + 64 * c, p.K - 64);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = (int64_t)(t0 + f_tile) * kRows + g + 8 * h;
      f_blk[h] = (uint32_t)((min(n, p.N - 1) * p.K + col) >> 6);
    }
  };
  FewScale next[2];
  auto fetch = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) next[h] = few_scale(p, f_blk[h]);
    ++f_tile;
    if (f_tile == nt) {
      f_tile = 0;
      ++f_quad;
    }
    if (f_tile == 0 || f_tile == nt - 1) {   // (the last tile's second half may lie past N)
      place();
    } else {
      f_blk[0] += (uint32_t)(p.K >> 2);      // 16 rows of K / 64 blocks
      f_blk[1] += (uint32_t)(p.K >> 2);
    }
  };
  if (i0 < i1) {
    place();
    fetch();
  }
  uint4 xv[NT][8];
  // x by way of a free slot of the ring, which then takes its codes; with two groups of tokens each lane
  // reads its own (their registers leave no room for rows on their way: 44.8 us instead of 42.8 for 16
  // tokens of 13824 x 5120)
  auto load_x = [&](int s) {
    if constexpr (TWO) {
      load_codes(s);
      const int64_t col = (int64_t)quad * kFewCols + 64 * c;
#pragma unroll
      for (int t = 0; t < NT; ++t) {   // tokens past M repeat the last one, unread
        const uint4* src = reinterpret_cast<const uint4*>(p.x + (int64_t)min(8 * t + g, p.M - 1) * p.K + col);
#pragma unroll
        for (int j = 0; j < 8; ++j) xv[t][j] = col < p.K ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
      }
    } else {
      few_load_x<NT>(p, quad, ring + s * kFewItemBytes, xv);
      fence_proxy_async_smem();
      __syncwarp();
      load_codes(s);
    }
  };
  if (i0 < i1) load_x(kFewRing - 1);
  const uint32_t lane_addr = few_fill_table(p, smem0 + kFewTableAddr);   // while the codes arrive
  if constexpr (FLAT) {
    const int64_t tile16 = (int64_t)blockIdx.x * kFewWarps;
    few_prefetch_rows(p, min(tile16 * kRows, p.N), min((tile16 + kFewWarps) * kRows, p.N), false);
  } else {
    few_prefetch_rows(p, (int64_t)share.begin * kRows, min((int64_t)share.end * kRows, p.N), true);
  }
  for (int i = i0; i < i1 && ok;) {
    // this warp's tiles of one quad of columns
    const int stop = min(i1, i + nt - tile);
    float* out = sums + (tile * quads + quad) * kSlot + g * 8 + 2 * c;
    for (; i < stop; ++i, out += quads * kSlot) {
      const FewScale s0 = next[0], s1 = next[1];
      if (i + 1 < i1) fetch();
      if (!mbar_try_wait(&full[slot], phase) && !mbar_wait_thread(&full[slot], phase, abort_word, kErrWaitTma)) ok = false;
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      // rows g and g + 8: their 16-byte chunks 2 c and 2 c + 1 lie at (chunk ^ g), a phase of 8 lanes (two
      // rows) reads 8 different bank groups
      const uint8_t* row = ring + slot * kFewItemBytes + g * 128;
      const float f0 = few_scale_value(p, s0, mean), f1 = few_scale_value(p, s1, mean);
      float acc[NT][2][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[t][0][k] = acc[t][1][k] = 0.0f;
      uint4 qa[2], qb[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        qa[h] = *reinterpret_cast<const uint4*>(row + (((2 * c + h) ^ g) << 4));
        qb[h] = *reinterpret_cast<const uint4*>(row + 1024 + (((2 * c + h) ^ g) << 4));
      }
      const uint32_t wa[8] = {qa[0].x, qa[0].y, qa[0].z, qa[0].w, qa[1].x, qa[1].y, qa[1].z, qa[1].w};
      const uint32_t wb[8] = {qb[0].x, qb[0].y, qb[0].z, qb[0].w, qb[1].x, qb[1].y, qb[1].z, qb[1].w};
      const uint64_t v0 = f32_pair(f0, f0), v1 = f32_pair(f1, f1);
      // the lookups of the next 8 columns are on their way while these are rounded and multiplied
      uint64_t la[2][4], lb[2][4];
      few_lookup8(wa[0], lane_addr, la[0]);
      few_lookup8(wb[0], lane_addr, lb[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j < 7) {
          few_lookup8(wa[j + 1], lane_addr, la[(j + 1) & 1]);
          few_lookup8(wb[j + 1], lane_addr, lb[(j + 1) & 1]);
        }
        uint32_t a[4], b[4];
        few_round8(la[j & 1], v0, a);
        few_round8(lb[j & 1], v1, b);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4& x = xv[t][j];
          mma_bf16_16816(acc[t][0], a[0], b[0], a[1], b[1], x.x, x.y);
          mma_bf16_16816(acc[t][1], a[2], b[2], a[3], b[3], x.z, x.w);
        }
      }
      --pending;
      __syncwarp();   // every lane has used its codes: the slot takes the item kFewRing ahead
      const int used = slot;
      const bool turn = i + 1 == stop && stop < i1;   // to the next quad of columns
      if (!turn) load_codes(used);
      if (++slot == kFewRing) {
        slot = 0;
        phase ^= 1u;
      }
      // sums of rows g and g + 8, tokens 2 c and 2 c + 1 of each group
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (FLAT) {
          const float both[4] = {acc[t][0][0] + acc[t][1][0], acc[t][0][1] + acc[t][1][1],
                                 acc[t][0][2] + acc[t][1][2], acc[t][0][3] + acc[t][1][3]};
          store_flat(quad, tile, t, both);
        } else {
          *reinterpret_cast<float2*>(out + t * 128) =
              make_float2(acc[t][0][0] + acc[t][1][0], acc[t][0][1] + acc[t][1][1]);
          *reinterpret_cast<float2*>(out + t * 128 + 64) =
              make_float2(acc[t][0][2] + acc[t][1][2], acc[t][0][3] + acc[t][1][3]);
        }
      }
      if constexpr (FLAT) ++tile;
      if (turn) {
        ++quad;
        load_x(used);
      }
    }
    tile = 0;
  }
  if (p.t) {
    // t B^T: t as bf16 hi + lo (16 significant bits), one more slot of sums per tile
    asm volatile("griddepcontrol.wait;" ::: "memory");   // t comes from the grid before
    constexpr int kSteps = TWO ? 2 : 4;
    const int first = FLAT ? (int)blockIdx.x * kFewWarps + warp : warp, step = FLAT ? (int)gridDim.x * kFewWarps : kFewWarps;
    for (int tl = first; tl < nt; tl += step) {
      const int64_t n0 = (int64_t)(t0 + tl) * kRows + g, n1 = min(n0 + 8, p.N - 1);
      float acc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[t][k] = 0.0f;
      for (int j0 = 4 * c; j0 < p.r + 4 * c; j0 += 16 * kSteps) {
        // 16 rank columns a step, lane c takes 4 of them; the loads of several steps go out together (one
        // by one they took 1 us at rank 64)
        uint2 b0[4], b1[kSteps];
        float4 tv[NT][kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int j = j0 + 16 * k;
          b0[k] = b1[k] = make_uint2(0u, 0u);
          if (j < p.r) {
            b0[k] = __ldg(reinterpret_cast<const uint2*>(p.B + n0 * p.r + j));
            b1[k] = __ldg(reinterpret_cast<const uint2*>(p.B + n1 * p.r + j));
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            tv[t][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (j < p.r) tv[t][k] = *reinterpret_cast<const float4*>(p.t + (int64_t)min(8 * t + g, p.M - 1) * p.r + j);
          }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          if (j0 + 16 * k >= p.r + 4 * c) break;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint32_t h0, l0, h1, l1;
            split_bf16x2(tv[t][k].x, tv[t][k].y, h0, l0);
            split_bf16x2(tv[t][k].z, tv[t][k].w, h1, l1);
            mma_bf16_16816(acc[t], b0[k].x, b1[k].x, b0[k].y, b1[k].y, h0, h1);
            mma_bf16_16816(acc[t], b0[k].x, b1[k].x, b0[k].y, b1[k].y, l0, l1);
          }
        }
      }
      float* out = sums + (nt * quads + tl) * kSlot + g * 8 + 2 * c;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (FLAT) {
          store_flat(quads, tl, t, acc[t]);
        } else {
          *reinterpret_cast<float2*>(out + t * 128) = make_float2(acc[t][0], acc[t][1]);
          *reinterpret_cast<float2*>(out + t * 128 + 64) = make_float2(acc[t][2], acc[t][3]);
        }
      }
    }
  }
  __syncthreads();
  if (!FLAT && !*abort_word)   // the same for every thread: all waits are over
    few_finish<kRows>(p, sums, kSlot, t0, nt, quads, [](int row, int tok) { return (tok >> 3) * 128 + row * 8 + (tok & 7); });
  if (*abort_word && lane == 0) {
    // a wait ran out: let the copies in flight land before the block's shared memory goes away
    for (int k = 0; k < pending; ++k) {
      const int s = slot + k < kFewRing ? slot + k : slot + k - kFewRing;
      const uint32_t ph = slot + k < kFewRing ? phase : phase ^ 1u;
      for (int i = 0; i < (1 << 20) && !mbar_try_wait(&full[s], ph); ++i) {}
    }
  }
}

// Joins a flat list's `parts` sums per output (the quads of columns and, behind them, the adapter term):
// y of 32 features of one token per block.  Warp w adds the parts w, w + 8, ...; the warps' sums are
// added in their order.
__global__ void __launch_bounds__(256) few_token_join_kernel(const __grid_constant__ FewTokenParams p, int parts) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tok = blockIdx.y;
  const int64_t n = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f, bias = 0.0f, res = 0.0f;
  const int64_t to = (int64_t)tok * p.N + n;
  if (n < p.N) {   // inputs of the call, not of the grid before
    if (p.post.bias) bias = __uint_as_float((uint32_t)p.post.bias[n] << 16);
    if (p.post.residual) res = __uint_as_float((uint32_t)p.post.residual[to] << 16);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n < p.N) {
    const float* part = p.part + to;
#pragma unroll 8
    for (int w = warp; w < parts; w += 8) v += part[(int64_t)w * p.M * p.N];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || n >= p.N) return;
  float z = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) z += sums[w][lane];
  z += bias;
  if (p.post.z) p.post.z[to] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
  float a[2] = {z, 0.0f};
  act_apply(a, p.post.act);
  p.y[to] = __bfloat16_as_ushort(__float2bfloat16_rn(p.post.residual ? a[0] + res : a[0]));
}

// K % 64 != 0: what a lane holds of its row's 64 columns in the next item.
struct FewUnit {
  FewScale s0, s1;   // of the block of its first column and of the next
  int32_t split;     // 8-code words before the boundary between them
  uint32_t w[8];
};

// K % 64 != 0.  Tiles of 8 rows on the n side of the product, the tokens on its m side; lane (g, c) holds
// row g, columns 64 c .. 64 c + 63.  TWO: more than 8 tokens.
template <bool TWO>
__global__ void __launch_bounds__(32 * kFewWarps, 1) few_token_ragged_kernel(const __grid_constant__ FewTokenParams p) {
  constexpr int kRows = 8, kSlot = (TWO ? 16 : 8) * kRows;   // sums [token][row]
  extern __shared__ __align__(16) uint8_t few_smem[];
  float* const sums = reinterpret_cast<float*>(few_smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int quads = (int)((p.K + kFewCols - 1) / kFewCols);
  const FewShare share = few_share((int)(p.N / kRows));
  const int per_round = few_per_round(share.end - share.begin, quads, kSlot);
  const float mean = p.scale_fp32 ? 0.0f : __ldg(p.mean);
  uint8_t* const stage = few_smem + (kFewRingAddr - smem_u32(few_smem)) + warp * kFewStageBytes;   // hands over x
  few_prefetch_rows(p, (int64_t)share.begin * kRows, (int64_t)share.end * kRows, true);
  const uint32_t lane_addr = few_fill_table(p, few_smem + (kFewTableAddr - smem_u32(few_smem)));

  for (int t0 = share.begin; t0 < share.end; t0 += per_round) {
    const int nt = min(share.end - t0, per_round);
    const int items = nt * quads;
    const int i0 = items * warp / kFewWarps, i1 = items * (warp + 1) / kFewWarps;
    int quad = i0 / nt, tile = i0 - quad * nt;
    // the item fetched next: the flat index of the lane's first weight and its 8-code words before K
    // (columns past K, where x is zero, take the last word before them)
    int f_quad = quad, f_tile = tile, f_valid = 0;
    int64_t f_at = 0;
    auto place = [&]() {
      int64_t col = (int64_t)f_quad * kFewCols + 64 * c;
      f_valid = col >= p.K ? 1 : (int)min((p.K - col) >> 3, (int64_t)8);
      if (col >= p.K) col = p.K - 8;
      f_at = ((int64_t)(t0 + f_tile) * kRows + g) * p.K + col;
    };
    FewUnit u;
    auto fetch = [&]() {
      const uint32_t blk = (uint32_t)(f_at >> 6);
      u.split = (int)((64 - (f_at & 63)) >> 3);
      u.s0 = few_scale(p, blk);
      u.s1 = few_scale(p, u.split < f_valid ? blk + 1 : blk);   // the next block exists where a valid word lies in it
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.codes + (f_at >> 1));
#pragma unroll
      for (int j = 0; j < 8; ++j) u.w[j] = __ldg(src + (j < f_valid ? j : 0));
      f_at += kRows * p.K;
      if (++f_tile == nt) {
        f_tile = 0;
        ++f_quad;
        place();
      }
    };
    if (i0 < i1) {
      place();
      fetch();
    }
    for (int i = i0; i < i1; ++quad, tile = 0) {
      // this warp's tiles of one quad of columns: x stays in registers
      uint4 xv[TWO ? 2 : 1][8];
      few_load_x<TWO ? 2 : 1>(p, quad, stage, xv);
      const uint4(&xa)[8] = xv[0];
      const uint4(&xb)[8] = xv[TWO ? 1 : 0];
      const int stop = min(i1, i + nt - tile);
      float* out = sums + (tile * quads + quad) * kSlot + g * kRows + 2 * c;
      for (; i < stop; ++i, out += quads * kSlot) {
        const FewUnit v = u;
        if (i + 1 < i1) fetch();
        const float s0 = few_scale_value(p, v.s0, mean), s1 = few_scale_value(p, v.s1, mean);
        float acc0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, acc1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t b[4];
          few_expand8(v.w[j], j >= v.split ? s1 : s0, lane_addr, b);
          if constexpr (TWO) {
            mma_bf16_16816(acc0, xa[j].x, xb[j].x, xa[j].y, xb[j].y, b[0], b[1]);
            mma_bf16_16816(acc1, xa[j].z, xb[j].z, xa[j].w, xb[j].w, b[2], b[3]);
          } else {
            // The four x registers as they were loaded are the A operand of both products (any other
            // order would have to be moved together each time).  Rows 0-7 then hold columns 0, 1, 4, 5
            // of the 8 and rows 8-15 columns 2, 3, 6, 7: with the weights of the former the upper
            // half of the sums is the tokens', with those of the latter the lower half.
            mma_bf16_16816(acc0, xa[j].x, xa[j].y, xa[j].z, xa[j].w, b[0], b[2]);
            mma_bf16_16816(acc1, xa[j].x, xa[j].y, xa[j].z, xa[j].w, b[1], b[3]);
          }
        }
        // sums of token g (and g + 8), rows 2 c and 2 c + 1
        if constexpr (TWO) {
          *reinterpret_cast<float2*>(out) = make_float2(acc0[0] + acc1[0], acc0[1] + acc1[1]);
          *reinterpret_cast<float2*>(out + 8 * kRows) = make_float2(acc0[2] + acc1[2], acc0[3] + acc1[3]);
        } else {
          *reinterpret_cast<float2*>(out) = make_float2(acc0[0] + acc1[2], acc0[1] + acc1[3]);
        }
      }
    }
    if (p.t) {
      // t B^T: t as bf16 hi + lo (16 significant bits), one more slot of sums per tile
      asm volatile("griddepcontrol.wait;" ::: "memory");   // t comes from the grid before
      const float* ta = p.t + (int64_t)min(g, p.M - 1) * p.r;
      const float* tb = p.t + (int64_t)min(g + 8, p.M - 1) * p.r;
      for (int tl = warp; tl < nt; tl += kFewWarps) {
        const uint16_t* brow = p.B + ((int64_t)(t0 + tl) * kRows + g) * p.r;
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
        float* out = sums + (nt * quads + tl) * kSlot + g * kRows + 2 * c;
        *reinterpret_cast<float2*>(out) = make_float2(acc[0], acc[1]);
        if constexpr (TWO) *reinterpret_cast<float2*>(out + 8 * kRows) = make_float2(acc[2], acc[3]);
      }
    }
    __syncthreads();
    few_finish<kRows>(p, sums, kSlot, t0, nt, quads, [](int row, int tok) { return tok * kRows + row; });
    __syncthreads();   // the sums are free for the next round
  }
}

// How this path takes a shape.  Whole tiles join their sums in the block that owns them, where all of
// a block's sums fit and the tiles load the SMs evenly.  Otherwise a flat list of the items over all
// blocks loads them evenly and a second kernel joins, 1 to 3 us more: with adapters and one token 23.8
// against 20.7 us for 13824 x 5120 and 12.7 against 10.6 us for 4096 x 4096.  The rule's bound, 12 items more on
// the fullest SM than on average, lies between 4096 x 11008 (12 items; 1 token 17.9 us as tiles, 19.3 as a list, 8
// tokens 21.7 and 20.8) and 5120 x 5120 (17 items; 1 token 13.9 and 14.9, 16 tokens 25.6 and 24.4).
// With K % 64 != 0 the other side is 16-token tiles of the fused GEMM with the same epilogue (SiLU, residual, rank
// 64): 1 token 26.6 against 85 us for 13824 x 5112, 11.2 against 31 for 4000 x 3000, 18 against 43 for 128 x
// 30008; 16 tokens 45.5 against 85, 16.8 against 31 and 39 against 42.  Rows of thousands of columns in two and more
// rounds come near at 16 tokens (70 against 90 us for 5120 x 13816, 99.4 against 99.8 for 4096 x 20008) and lose 2
// to 6 % at the longest (144 against 141 for 4096 x 30008, 270 against 256 for 13824 x 18008).  Without adapters the
// tiles need two launches less: 59.8 against 77 us for 5120 x 13816, but 32.9 against 26.9 for 128 x 30008.  A bound on
// K would give away more at 9 tokens (66 against 84 us for 2048 x 30008) than it gains there.
enum FewPlan : int { kFewNo = 0, kFewTiles = 1, kFewFlat = 2 };
static FewPlan few_token_plan(int64_t M, int64_t K, int64_t N) {
  if (M > kFewTokens || N * K >= (1ll << 37)) return kFewNo;
  const int64_t quads = (K + kFewCols - 1) / kFewCols, tokens = M > 8 ? 16 : 8;
  if (K % 64) return (quads + 1) * tokens * 8 * 4 <= kFewSumBytes ? kFewTiles : kFewNo;
  const int64_t tiles = (N + 15) / 16, most = (tiles + kFewBlocks - 1) / kFewBlocks;   // tiles of the fullest SM
  const bool fits = most * (quads + 1) * tokens * 16 * 4 <= kFewSumBytes;
  return fits && most * quads - tiles * quads / kFewBlocks <= 12 ? kFewTiles : kFewFlat;
}

// The blocks are those that few_token_plan counts on, one per SM of the whole GPU (a partition of it runs them in turn).
static cudaError_t launch_few_token_k(void (*kernel)(const FewTokenParams), std::atomic<uint64_t>& configured, int smem,
                                      int64_t blocks, const FewTokenParams& p, cudaStream_t st) {
  int dev = 0, reserved = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e == cudaSuccess && reserved > kFewReservedBytes) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess) e = enable_smem_once(kernel, smem, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(kFewBlocks, blocks));
  cfg.blockDim = dim3(32 * kFewWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.t ? 1 : 0;   // with adapters the grid before is the one that makes t
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

static cudaError_t launch_few_token(const FewTokenParams& p, FewPlan plan, cudaStream_t st) {
  static std::atomic<uint64_t> configured[6] = {{0}, {0}, {0}, {0}, {0}, {0}};
  const int64_t tiles = (p.N + 15) / 16, quads = (p.K + kFewCols - 1) / kFewCols;
  if (p.K % 64)
    return p.M <= 8 ? launch_few_token_k(few_token_ragged_kernel<false>, configured[0], kFewRaggedSmemBytes, p.N / 8, p, st)
                    : launch_few_token_k(few_token_ragged_kernel<true>, configured[1], kFewRaggedSmemBytes, p.N / 8, p, st);
  if (plan == kFewTiles)
    return p.M <= 8 ? launch_few_token_k(few_token_kernel<false, false>, configured[2], kFewSmemBytes, tiles, p, st)
                    : launch_few_token_k(few_token_kernel<true, false>, configured[3], kFewSmemBytes, tiles, p, st);
  cudaError_t e = p.M <= 8
                      ? launch_few_token_k(few_token_kernel<false, true>, configured[4], kFewSmemBytes, tiles * quads, p, st)
                      : launch_few_token_k(few_token_kernel<true, true>, configured[5], kFewSmemBytes, tiles * quads, p, st);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.N + 31) / 32), (unsigned)p.M);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_token_join_kernel, p, (int)quads + (p.t ? 1 : 0));
}

// The small kernels beside the product run with its split of the SM's memory, whatever they use of it.
static cudaError_t few_same_split_once() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (e != cudaSuccess || (bit && (done.load(std::memory_order_acquire) & bit))) return e;
  void (*down[2])(const FewTokenDownParams) = {few_token_down_kernel<1>, few_token_down_kernel<kFewDownTokens>};
  for (auto* k : down)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(few_token_join_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

static cudaError_t launch_few_token_down(const FewTokenDownParams& p, cudaStream_t st) {
  cudaError_t e = few_same_split_once();
  if (e != cudaSuccess) return e;
  if (p.M == 1) few_token_down_kernel<1><<<p.r, 256, 0, st>>>(p);
  else few_token_down_kernel<kFewDownTokens><<<dim3(p.r, (p.M + kFewDownTokens - 1) / kFewDownTokens), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace qnf4
