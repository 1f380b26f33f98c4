// The 4-bit cache format on the device: tile layout and row quantization.
//
// A (block, KV head) tile of a 4-bit cache is 16 (d/2 + 4) bytes: 8 d bytes of
// codes, then 16 pairs (scale, mid) of halves, one per token. A row element is
// mid + (code - 7.5) scale.
//   keys    row t is the d/2 bytes at t d/2; dimension 2i is the low nibble of
//           byte i, 2i + 1 the high one.
//   values  the bytes of tokens 2p and 2p + 1 interleave by 16 bits. With
//           W = d/32, dimension x of token t lies in byte
//             (((p / 4) 32 + (x / 4W) 4 + p % 4) W + (x / 4) % W) 4 + 2 (t % 2) + (x % 4) / 2,
//           p = t / 2, nibble x % 2. A warp's lane then finds the codes it feeds
//           to a matrix instruction in W consecutive words, and the warp reads
//           512 (d = 128) or 256 contiguous bytes at a time without bank conflicts.
#pragma once

#include "pa_device.cuh"

namespace pa {

// Tag type of a 4-bit cache.
struct Int4 {};

__host__ __device__ constexpr int int4_row_bytes(int d) { return d / 2 + 4; }
__host__ __device__ constexpr int int4_tile_bytes(int d) { return kBlockSize * int4_row_bytes(d); }

// Byte of a value tile that holds dimensions x, x + 1 (x even) of token t.
template <int D>
__device__ __forceinline__ int int4_value_byte(int t, int x) {
  constexpr int W = D / 32;
  const int p = t >> 1;
  return ((((p >> 2) * 32 + (x / (4 * W)) * 4 + (p & 3)) * W + (x >> 2) % W) << 2) +
         ((t & 1) << 1) + ((x >> 1) & 1);
}

// What int4_value_byte grows by from dimensions 16u to 16u + 4q, q < 4.
template <int D>
__device__ __forceinline__ constexpr int int4_value_step(int q) {
  return D == 128 ? 4 * q : 32 * (q >> 1) + 4 * (q & 1);
}

// min / max that return NaN when an operand is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Quantizes a row of 16 LANES elements held by LANES adjacent lanes (16 each;
// every lane of the warp must call it). codes[0] takes elements 0-7, codes[1]
// 8-15, element e in bits 4(e % 8). Returns (scale, mid) as two halves. All
// steps are single fp32 operations rounded to nearest, so that the codes are
// reproducible bit for bit:
//   x clamped to +-65504 (the range of the two halves), mx, mn over the row,
//   scale = half((mx - mn) / 15), mid = half((mx + mn) * 0.5),
//   inv = scale > 0 ? 1 / scale : 0, code = clamp(rint((x - mid) * inv + 7.5), 0, 15).
// (Clamping before rint gives the same code, since the bounds are whole numbers.)
// A row holding a NaN gets NaN parameters (it reads back as NaN) and codes 0.
template <int LANES>
__device__ __forceinline__ uint32_t int4_quantize_row(float (&f)[16], uint32_t (&codes)[2]) {
  float mx = f[0], mn = f[0];
#pragma unroll
  for (int e = 1; e < 16; ++e) {
    mx = max_nan(mx, f[e]);
    mn = min_nan(mn, f[e]);
  }
#pragma unroll
  for (int mask = 1; mask < LANES; mask <<= 1) {
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, mask));
    mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, mask));
  }
  if (mx > 65504.f || mn < -65504.f) {  // rare: clamp the elements (and a NaN stays one)
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = min_nan(max_nan(f[e], -65504.f), 65504.f);
    mx = min_nan(mx, 65504.f);
    mx = max_nan(mx, -65504.f);
    mn = max_nan(mn, -65504.f);
    mn = min_nan(mn, 65504.f);
  }
  const __half scale = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.f));
  const __half mid = __float2half_rn(__fmul_rn(__fadd_rn(mx, mn), 0.5f));
  const float s = __half2float(scale), minus_c = -__half2float(mid);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  // rint by adding 1.5 2^23, whose unit is 1: the code is then the low bits of the float,
  // under the constant kMagic; the eight of a word join by multiplications by 16, which
  // move the constants' sum to kRest
  constexpr uint32_t kMagic = 0x4b400000u;  // 1.5 2^23
  constexpr uint32_t kRest = kMagic * 0x11111111u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0u;
#pragma unroll
    for (int e = 6; e >= 0; e -= 2) {
      float u = f[8 * h + e], v = f[8 * h + e + 1];
      fadd2(u, v, minus_c, minus_c);
      u = __fmul_rn(u, inv);  // (packed multiplications were fused with the next addition)
      v = __fmul_rn(v, inv);
      fadd2(u, v, 7.5f, 7.5f);
      u = fminf(fmaxf(u, 0.f), 15.f);  // NaN: 0
      v = fminf(fmaxf(v, 0.f), 15.f);
      fadd2(u, v, 12582912.f, 12582912.f);
      w = w * 16u + __float_as_uint(v);
      w = w * 16u + __float_as_uint(u);
    }
    codes[h] = w - kRest;
  }
  return (uint32_t)__half_as_ushort(scale) | ((uint32_t)__half_as_ushort(mid) << 16);
}

}  // namespace pa
