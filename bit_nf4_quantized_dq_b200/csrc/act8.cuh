// 8-bit activation checkpoints: a bf16 tensor x [M][K] held as E4M3 codes with one power-of-two
// scale per token and 32 features, for the tensors that only the backward pass reads again.
//
//   amax_g  = max |x| over the group (one token, features 32 g .. 32 g + 31, fewer at the end)
//   e_g     = the smallest integer with amax_g <= 448 * 2^e_g, clamped to [-117, 120]
//   code    = E4M3 round-to-nearest-even of x * 2^-e_g     (the scaling is exact: a power of two)
//   value   = code * 2^e_g
//
// The power-of-two scale costs nothing in precision (E4M3 keeps 4 significant bits wherever the
// value lies between 2^-6 and 448 of its group's scale, so a relative error of at most 2^-4 over
// a range of 2^14), and it makes every decoded value exact in bf16: 4 significant bits, and the
// clamp keeps 2^-9 * 2^e a normal number.  Decoding therefore rounds nothing.  Groups with e = 120
// (amax above 1.75 * 2^127) saturate at code value 240: 256 * 2^120 would be infinite in bf16.
// A group with an infinity or a NaN has the scale byte 255 and decodes to NaN as a whole, so that
// a diverged step does not look like a large finite one.
//
// Decoding takes any code and scale byte (a checkpoint may come from elsewhere): E4M3(code) *
// 2^(byte - 127), NaN for the codes 0x7F and 0xFF and for the byte 255.  Bytes outside [10, 247], which
// the quantizer does not write, give values that bf16 may have to round to a subnormal or infinity.
//
// Stored: codes uint8 [M][ld], ld = K rounded up to 16 (so that tile loads keep their 16-byte
// row pitch; the pad holds zero codes); scales uint8 [M][ceil(K / 32)], byte e + 127.
// 8.25 bits per value instead of 16.
#pragma once

#include "nf4_device.cuh"

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

// Two fp32 values in one 64-bit register pair, for the paired arithmetic of sm_100.
__device__ __forceinline__ uint64_t f32_pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float pair_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float pair_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void unpack8_pairs(const uint4& v, uint64_t (&p)[4]) {
  p[0] = f32_pair(bf_lo(v.x), bf_hi(v.x));
  p[1] = f32_pair(bf_lo(v.y), bf_hi(v.y));
  p[2] = f32_pair(bf_lo(v.z), bf_hi(v.z));
  p[3] = f32_pair(bf_lo(v.w), bf_hi(v.w));
}

constexpr int kA8Group = 32;
constexpr uint32_t kA8NanScale = 255u;
constexpr uint32_t kA8MinScale = 10u;   // byte of e = -117
constexpr uint32_t kA8TopScale = 247u;  // byte of e = 120

__host__ __device__ __forceinline__ int64_t a8_ld(int64_t k) { return (k + 15) / 16 * 16; }
__host__ __device__ __forceinline__ int64_t a8_groups(int64_t k) { return (k + kA8Group - 1) / kA8Group; }

// Scale byte of a group from the bits of its largest magnitude (bf16, finite): with amax = 1.f *
// 2^p, amax <= 448 * 2^e means e >= p - 8 while 1.f <= 1.75, else p - 7.  Zeros and subnormals
// (p < -126) fall under the clamp.
__device__ __forceinline__ uint32_t a8_scale_byte(uint32_t amax_bits) {
  const int b = (int)(amax_bits >> 7) - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);
  return (uint32_t)max(b, (int)kA8MinScale);
}
// 2^-e of a scale byte: exponent field 127 - e = 254 - byte, in [7, 244].
__device__ __forceinline__ float a8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^e of a scale byte (2^-127, subnormal, of the byte 0); NaN for the byte 255.
__device__ __forceinline__ float a8_scale(uint32_t byte) {
  return __uint_as_float(byte == kA8NanScale ? 0x7FC00000u : max(byte << 23, 0x00400000u));
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One thread's 8 features (four bf16 pairs) of a group that four neighbouring lanes share: the
// group's scale byte and this thread's 8 codes.  All lanes of the warp call it.
__device__ __forceinline__ uint32_t a8_encode8(const uint4& v, uint2& codes) {
  const uint32_t mk = 0x7FFF7FFFu;
  uint32_t m = max_u16x2(max_u16x2(v.x & mk, v.y & mk), max_u16x2(v.z & mk, v.w & mk));
  m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const uint32_t amax = max(m & 0xFFFFu, m >> 16);
  uint32_t byte = a8_scale_byte(amax);
  if (amax >= 0x7F80u) byte = kA8NanScale;
  const float inv = a8_inv_scale(byte == kA8NanScale ? 127u : byte);
  uint64_t f[4];
  unpack8_pairs(v, f);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = f32x2_mul(f[i], f32_pair(inv, inv));
    c[i] = e4m3x2_encode_hw(pair_lo(f[i]), pair_hi(f[i]));
  }
  if (byte == kA8TopScale) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3x2_encode_hw(fminf(fmaxf(pair_lo(f[i]), -240.0f), 240.0f),
                              fminf(fmaxf(pair_hi(f[i]), -240.0f), 240.0f));
  }
  codes.x = c[0] | (c[1] << 16);
  codes.y = c[2] | (c[3] << 16);
  return byte;
}

// Two codes (bits 0-7 and 8-15) -> two fp32 values times `scale`.
__device__ __forceinline__ float2 a8_decode2(uint32_t pair, float scale) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(pair & 0xFFFFu));
  const __half2 hh = *reinterpret_cast<const __half2*>(&h);
  const float2 f = __half22float2(hh);
  return make_float2(f.x * scale, f.y * scale);
}

// 16 codes -> 16 bf16 values as eight pairs, with integer operations and one paired bf16 product
// per two values.  A code's exponent and mantissa bits (eeee mmm), moved to the low end of a
// bf16's exponent and the top of its mantissa, read as the code's value times 2^-120 (the
// exponent biases differ by 120; subnormal codes become subnormal bf16 values of the same ratio),
// so one product with 2^(120 + e) restores it, exact for every scale that the quantizer writes.
// Scales above 2^7 would overflow that factor and take a second product.  The NaN codes 0x7F and
// 0xFF read as 480: a carry into their top bit finds them, and the call returns whether there are any, for
// the caller to mark (a branch in here, between the units of a caller, cost dA 6 % of its time).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t a8_decode16(const uint4& q, uint32_t byte, uint32_t (&o)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  const int e = (int)byte - 127;
  const uint32_t f = byte == kA8NanScale ? 0x7FC0u : (uint32_t)(247 + min(e, 7)) << 7;
  const uint32_t f2 = f | (f << 16);
  uint32_t nan = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    nan |= (w[i] & 0x7F7F7F7Fu) + 0x01010101u;
    const uint32_t a = prmt(w[i], 0u, 0x1404u), b = prmt(w[i], 0u, 0x3424u);
    o[2 * i] = mul_bf16x2((a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), f2);
    o[2 * i + 1] = mul_bf16x2((b & 0x80008000u) | ((b >> 4) & 0x07F007F0u), f2);
  }
  if (e > 7 && byte != kA8NanScale) {
    const uint32_t g = (uint32_t)(127 + e - 7) << 7, g2 = g | (g << 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = mul_bf16x2(o[i], g2);
  }
  return nan & 0x80808080u;
}
// NaN in the places of the NaN codes of q.
__device__ __forceinline__ void a8_mark_nan16(const uint4& q, uint32_t (&o)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    const uint32_t a = prmt(m, 0u, 0x1404u), b = prmt(m, 0u, 0x3424u);   // 0x8000 per NaN code
    o[2 * i] |= a - (a >> 9);                                            // 0x7FC0
    o[2 * i + 1] |= b - (b >> 9);
  }
}

// Threads (x along the features, 8 each; y along the tokens); each takes kA8Rows tokens at a time,
// `batches` times, and loads all of them first, so that enough bytes are in flight.  blockDim.x is a
// multiple of 4, so a group's four lanes sit in one warp and in one row.
constexpr int kA8Rows = 4;

__global__ void __launch_bounds__(256) act8_quantize_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                            int batches, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const int64_t ld = a8_ld(K), G = a8_groups(K);
  const int by = (int)blockDim.y, per_block = kA8Rows * by * batches;
  const int64_t m0 = (int64_t)blockIdx.x * per_block + threadIdx.y;
  const int rows = (int)min(M - m0, (int64_t)(per_block - threadIdx.y));   // tokens m0, m0 + by, ... below m0 + rows
  for (int64_t c0 = (int64_t)blockIdx.y * blockDim.x; c0 < 4 * G; c0 += (int64_t)gridDim.y * blockDim.x) {
    const int64_t k = 8 * (c0 + threadIdx.x);
    const uint16_t* src = x + m0 * K + k;
    uint8_t* dst = codes + m0 * ld + k;
    uint8_t* sdst = scales + m0 * G + (k >> 5);
    const int in = k < K ? rows : 0, out = k < ld ? rows : 0, mark = (threadIdx.x & 3) == 0 ? in : 0;
    for (int r = 0; r < per_block; r += kA8Rows * by) {
      uint4 v[kA8Rows];
#pragma unroll
      for (int i = 0; i < kA8Rows; ++i, src += by * K) {
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r + i * by < in) v[i] = __ldcs(reinterpret_cast<const uint4*>(src));
      }
#pragma unroll
      for (int i = 0; i < kA8Rows; ++i, dst += by * ld, sdst += by * G) {
        uint2 q;
        const uint32_t byte = a8_encode8(v[i], q);
        if (r + i * by < out) *reinterpret_cast<uint2*>(dst) = q;
        if (r + i * by < mark) *sdst = (uint8_t)byte;
      }
    }
  }
}

__global__ void __launch_bounds__(256) act8_dequant_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t M, int64_t K,
                                                           uint16_t* __restrict__ out) {
  const int64_t ld = a8_ld(K), G = a8_groups(K);
  const int64_t m0 = (int64_t)blockIdx.x * blockDim.y * kA8Rows + threadIdx.y;
  for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < K / 8; c += (int64_t)gridDim.y * blockDim.x) {
    uint2 q[kA8Rows];
    uint32_t byte[kA8Rows];
#pragma unroll
    for (int i = 0; i < kA8Rows; ++i) {
      const int64_t m = m0 + i * blockDim.y;
      if (m < M) {
        q[i] = __ldcs(reinterpret_cast<const uint2*>(codes + m * ld + 8 * c));
        byte[i] = __ldg(scales + m * G + (c >> 2));
      }
    }
#pragma unroll
    for (int i = 0; i < kA8Rows; ++i) {
      const int64_t m = m0 + i * blockDim.y;
      if (m >= M) break;
      const float s = a8_scale(byte[i]);
      const float2 f0 = a8_decode2(q[i].x, s), f1 = a8_decode2(q[i].x >> 16, s), f2 = a8_decode2(q[i].y, s),
                   f3 = a8_decode2(q[i].y >> 16, s);
      *reinterpret_cast<uint4*>(out + m * K + 8 * c) =
          make_uint4(pack_bf16x2(f0.x, f0.y), pack_bf16x2(f1.x, f1.y), pack_bf16x2(f2.x, f2.y), pack_bf16x2(f3.x, f3.y));
    }
  }
}

// Block shape of a kernel whose threads take 8 features each of rows of `chunks` such units: as
// many threads along the row as it has units (a power of two, 4 .. 256), the rest along tokens.
static void a8_launch_shape(int64_t M, int64_t chunks, dim3* grid, dim3* block, int* batches = nullptr) {
  int bx = 4;
  while (bx < 256 && bx < chunks) bx *= 2;
  const int by = 256 / bx;
  *block = dim3((unsigned)bx, (unsigned)by);
  int64_t gy = (chunks + bx - 1) / bx;
  if (gy > 65535) gy = 65535;
  int64_t gx = (M + kA8Rows * by - 1) / (kA8Rows * by);
  if (batches) {   // up to four batches per block while the grid keeps eight blocks per SM
    *batches = 1;
    while (*batches < 4 && gx * gy >= 2 * 8 * 148) {
      *batches *= 2;
      gx = (M + kA8Rows * by * *batches - 1) / (kA8Rows * by * *batches);
    }
  }
  *grid = dim3((unsigned)gx, (unsigned)gy);
}

// Rows of whole groups make one flat run of values, codes and scales: where that cuts into rows of 2048, one
// block wide, the blocks read whole rows (8192 x 13824: 56 us, as it stands 61).
static void a8_flatten(int64_t* M, int64_t* K) {
  constexpr int64_t kRow = 2048;
  if (*K % kA8Group || *M * *K % kRow || *M * *K / kRow >= (1ll << 31)) return;
  *M = *M * *K / kRow;
  *K = kRow;
}

static cudaError_t launch_act8_quantize(const uint16_t* x, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales,
                                        cudaStream_t st) {
  dim3 grid, block;
  int batches;
  a8_flatten(&M, &K);
  a8_launch_shape(M, 4 * a8_groups(K), &grid, &block, &batches);
  act8_quantize_kernel<<<grid, block, 0, st>>>(x, M, K, batches, codes, scales);
  return cudaGetLastError();
}

static cudaError_t launch_act8_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, uint16_t* out,
                                       cudaStream_t st) {
  dim3 grid, block;
  a8_flatten(&M, &K);
  a8_launch_shape(M, K / 8, &grid, &block);
  act8_dequant_kernel<<<grid, block, 0, st>>>(codes, scales, M, K, out);
  return cudaGetLastError();
}

}  // namespace qnf4
