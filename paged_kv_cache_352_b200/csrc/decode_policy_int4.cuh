// Tensor-core arithmetic policy of the paged-decode kernel over 4-bit caches.
#pragma once

#include <cuda.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "decode_policies.cuh"
#include "int4_cache.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// Int4TensorPolicy (any G) attends to values mid_t + (n - 7.5) s_t, n the 4-bit
// codes of token t's row, s_t and mid_t its half-precision scale and midpoint:
//   score_t = sm_scale (s_t (q . n_t - 7.5 sum q) + mid_t sum q)
//   out     = (sum_t w_t n_t - 7.5 sum_t w_t + sum_t p_t mid_t) / sum_t p_t,
//   w_t = p_t s_t
// so codes enter the products as they are and each token's two parameters are
// applied to one score, not to d elements. A 4-bit tile carries 4 codes per two
// bytes of the memory stream, so the instructions spent per code decide whether
// the stream keeps up: every product runs on mma.sync (also for one query head
// per KV head, whose 7 padding rows cost nothing the tensor pipe lacks), and a
// code becomes an operand with half an instruction. The contraction has G rows
// of work per code byte, far too few for a 128-row tcgen05 tile.
//
// Codes as subnormal halves. The low four bits of a half with a zero exponent
// are worth n 2^-24 and the next four n 2^-20, both exact. So of one 32-bit word
// (eight codes) w & 0x000f000f and w & 0x00f000f0 are operand registers as they
// stand, and the same masks of w >> 8 give the other four codes: 5 instructions
// for 8 codes. The powers of two are taken back in the query operand (a factor
// 1/16 at the dimensions of the high nibbles) and in the fp32 results.
//
// k-slots of K (lane = 4g + c holds slots 2c, 2c+1, 2c+8, 2c+9 of A and B): lane
// c takes dimensions 8W c .. 8W c + 8W - 1 of a row (W = d/32 words). Word j
// gives two steps: dimensions 8j+0, +4 | +1, +5 and 8j+2, +6 | +3, +7. S column
// n of n-tile nt is token n + 8nt, so lane (g, c) ends up with tokens 2c, 2c+1,
// 2c+8, 2c+9 of head g, which is the B fragment of P^T.
//
// O^T = V^T P^T. A value tile interleaves the bytes of token pairs (int4_cache.cuh),
// so a word holds four dimensions of tokens 2p, 2p+1 and the same masks yield the
// A registers: word q of pair c gives a0 (dimension 4Wg + 4q) and a1 (+1), of
// pair c + 4 a2 and a3; shifted, dimensions +2 and +3 for the next m-tile.
//
// Precision. Products are exact, sums are fp32. q is brought below 2^15 by a
// power of two (exact in half unless 2^29 below the row's largest element). The
// weights w are rounded to half precision relative to the largest value scale
// seen (a power of two S, raised when a larger scale comes, as the softmax
// reference is), and -7.5 sum w is taken over the rounded weights, so that their
// errors multiply the centred codes. For half outputs the rounding residual of
// w joins the product too: with at most 4 query heads per KV head heads repeat
// in columns 4-7, whose lanes feed the residual (no cost); with 8 it is a second
// product. For bf16 outputs the weights' 2^-11 is 1/8 of the output's own step.
template <typename T, int D, int G>
struct Int4TensorPolicy {
  static constexpr int W = D / 32;   // words of codes a lane reads per row / per pair
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;
  static constexpr int QV = D / 32;  // 16-byte query chunks a lane reads
  static constexpr int kCodeBytes = kBS * D / 2;
  static constexpr int kTileBytes = int4_tile_bytes(D);
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kAlign = 128;
  static constexpr int kScratchBytes = 0;
  static constexpr bool kTensorCores = true;
  static constexpr bool kTma2D = false;
  static constexpr bool kFp8Cache = false;
  static constexpr int kMinCtasPerSm = 4;
  static constexpr bool kResidual = std::is_same<T, __half>::value;
  static constexpr bool kRepeat = kResidual && G <= 4;  // columns 4-7 repeat heads 0-3
  static_assert(D == 64 || D == 128, "unsupported head_dim");
  static_assert(kTileBytes % 16 == 0, "bulk copies take multiples of 16 bytes");

  int g, c, lane_;
  uint4 qraw[QV];
  uint32_t qa[KSTEPS][2];
  float m, l, row_scale, qsum;
  float sumw, pmid;   // sum of (rounded) weights, sum of p mid
  float vmax, vinv;   // S and 2^7 / S (both 0 until a positive scale comes)
  float o[MT][4];

  __device__ __forceinline__ void init(int lane) {
    lane_ = lane;
    g = lane >> 2;
    c = lane & 3;
  }
  __device__ __forceinline__ int head() const { return kRepeat ? (g & 3) : g; }

  __device__ __forceinline__ void prefetch_q(const DecodeArgs& a, int s, int kvh) {
    const uint4* row = reinterpret_cast<const uint4*>(
        reinterpret_cast<const T*>(a.q) +
        ((size_t)s * a.num_q_heads + (size_t)kvh * G + head()) * D + 8 * W * c);
#pragma unroll
    for (int i = 0; i < QV; ++i) qraw[i] = head() < G ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
  }

  __device__ __forceinline__ void begin(float scale_log2) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      float f[8];
      Storage<T>::to_f32(qraw[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^-k brings the row's largest element to [2^14, 2^15)
    int k = amax > 0.f && amax < INFINITY ? ilogbf(amax) - 14 : 0;
    if (k < -100) k = -100;
    const float down = exp2f((float)-k);
    row_scale = scale_log2 * exp2f((float)k);
    float qs = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float f[8];
      Storage<T>::to_f32(qraw[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= down;
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // low nibbles: dimensions 2r, 2r + 4; high: one more
        const __half2 lo = __floats2half2_rn(f[2 * r], f[2 * r + 4]);
        const __half2 hi = __floats2half2_rn(f[2 * r + 1] * 0.0625f, f[2 * r + 5] * 0.0625f);
        const float2 fl = __half22float2(lo), fh = __half22float2(hi);
        qs += (fl.x + fl.y) + 16.f * (fh.x + fh.y);
        memcpy(&qa[2 * j + r][0], &lo, 4);
        memcpy(&qa[2 * j + r][1], &hi, 4);
      }
    }
    qs += __shfl_xor_sync(0xffffffffu, qs, 1);
    qs += __shfl_xor_sync(0xffffffffu, qs, 2);
    qsum = qs;
    m = -INFINITY;
    l = sumw = pmid = vmax = vinv = 0.f;
#pragma unroll
    for (int t = 0; t < MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
  }

  static __device__ __forceinline__ void issue(const DecodeArgs& a, const CUtensorMap*,
                                               const CUtensorMap*, unsigned char* dst,
                                               uint64_t* bar, int phys, int kvh) {
    const size_t off = ((size_t)phys * a.num_kv_heads + kvh) * kTileBytes;
    mbar_arrive_expect_tx(bar, kStageBytes);
    bulk_copy_g2s(dst, static_cast<const unsigned char*>(a.k_cache) + off, kTileBytes, bar);
    bulk_copy_g2s(dst + kTileBytes, static_cast<const unsigned char*>(a.v_cache) + off, kTileBytes,
                  bar);
  }

  static __device__ __forceinline__ void load_words(const unsigned char* p, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    }
  }

  // (scale, mid) of the lane's tokens 2c, 2c+1, 2c+8, 2c+9
  __device__ __forceinline__ void load_params(const unsigned char* tile, float2 (&p)[4]) const {
    const uint2 a = *reinterpret_cast<const uint2*>(tile + kCodeBytes + 8 * c);
    const uint2 b = *reinterpret_cast<const uint2*>(tile + kCodeBytes + 32 + 8 * c);
    p[0] = half2_bits_to_float2(a.x);
    p[1] = half2_bits_to_float2(a.y);
    p[2] = half2_bits_to_float2(b.x);
    p[3] = half2_bits_to_float2(b.y);
  }

  __device__ __forceinline__ void block(unsigned char* stage, int valid, unsigned char*) {
    constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;
    const unsigned char* Ks = stage;
    const unsigned char* Vs = stage + kTileBytes;
    // ---- S = Q K^T
    uint32_t kw[2][W];
    load_words(Ks + g * (D / 2) + c * (4 * W), kw[0]);
    load_words(Ks + (g + 8) * (D / 2) + c * (4 * W), kw[1]);
    float2 kp[4], vp[4];
    load_params(Ks, kp);
    load_params(Vs, vp);
    float sacc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t w = kw[nt][j], u = w >> 8;
        MmaOps<__half>::run(sacc[nt], qa[2 * j][0], qa[2 * j][1], w & kLo, w & kHi);
        MmaOps<__half>::run(sacc[nt], qa[2 * j + 1][0], qa[2 * j + 1][1], u & kLo, u & kHi);
      }
    }
    // ---- online softmax; element i is token 2c + (i & 1) + 8 (i >> 1) of head g
    float x[4];
    bool ok[4];
    float bmax = -INFINITY;
    const float q75 = 7.5f * qsum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ok[i] = head() < G && 2 * c + (i & 1) + 8 * (i >> 1) < valid;
      const float dot = fmaf(sacc[i >> 1][i & 1], 16777216.f, -q75);
      x[i] = ok[i] ? fmaf(kp[i].x, dot, kp[i].y * qsum) * row_scale : -INFINITY;
      bmax = fmaxf(bmax, x[i]);
    }
    bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, 1));
    bmax = fmaxf(bmax, __shfl_xor_sync(0xffffffffu, bmax, 2));
    float alpha;
    const float mref = lazy_reference(m, bmax, alpha);
    // parameters of slots past the context may be any bits: they are read as 0
    float smax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = 2 * c + (i & 1) + 8 * (i >> 1) < valid;
      vp[i].x = in ? vp[i].x : 0.f;
      vp[i].y = in ? vp[i].y : 0.f;
      smax = fmaxf(smax, vp[i].x);
    }
    if (__any_sync(0xffffffffu, alpha != 1.f || smax > vmax)) {
      // a softmax reference or the value-scale reference S moved: bring the sums
      // to the new ones. Lane (g, c)'s outputs are columns 2c and 2c + 1, whose
      // factors live in lanes 4(2c) and 4(2c + 1).
      smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, 1));
      smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, 2));
      float f = 1.f;
      if (smax > vmax) {
        // the power of two at or above smax (a half: exact here)
        const float s2 = __uint_as_float((__float_as_uint(smax) + 0x007fffffu) & 0x7f800000u);
        f = vmax / s2;
        vmax = s2;
        vinv = 128.f / s2;
      }
      const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * c) * f;
      const float a1 = __shfl_sync(0xffffffffu, alpha, 8 * c + 4) * f;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        o[t][0] *= a0;
        o[t][1] *= a1;
        o[t][2] *= a0;
        o[t][3] *= a1;
      }
      l *= alpha;
      pmid *= alpha;
      sumw *= alpha * f;
    }
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = exp2f(x[i] - mref);
      l += p;
      pmid = fmaf(p, vp[i].y, pmid);
      w[i] = p * (vp[i].x * vinv);  // at most 2^8 2^7 (the reference is lazy by 2^8)
    }
    uint32_t pb0, pb1, lo0 = 0u, lo1 = 0u;
    {
      const __half2 h0 = __floats2half2_rn(w[0], w[1]), h1 = __floats2half2_rn(w[2], w[3]);
      const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
      memcpy(&pb0, &h0, 4);
      memcpy(&pb1, &h1, 4);
      if constexpr (kResidual) {
        sumw += (w[0] + w[1]) + (w[2] + w[3]);
        const __half2 r0 = __floats2half2_rn(w[0] - f0.x, w[1] - f0.y);
        const __half2 r1 = __floats2half2_rn(w[2] - f1.x, w[3] - f1.y);
        memcpy(&lo0, &r0, 4);
        memcpy(&lo1, &r1, 4);
        if constexpr (kRepeat) {
          pb0 = g < 4 ? pb0 : lo0;
          pb1 = g < 4 ? pb1 : lo1;
        }
      } else {
        sumw += (f0.x + f0.y) + (f1.x + f1.y);
      }
    }
    // ---- O^T += V^T P^T
    uint32_t va[W], vb[W];
    load_words(Vs + lane_ * (4 * W), va);
    load_words(Vs + (32 + lane_) * (4 * W), vb);
#pragma unroll
    for (int q = 0; q < W; ++q) {
      const uint32_t a = va[q], b = vb[q], a8 = a >> 8, b8 = b >> 8;
      mma_full<__half>(o[2 * q], a & kLo, a & kHi, b & kLo, b & kHi, pb0, pb1);
      mma_full<__half>(o[2 * q + 1], a8 & kLo, a8 & kHi, b8 & kLo, b8 & kHi, pb0, pb1);
      if constexpr (kResidual && !kRepeat) {
        mma_full<__half>(o[2 * q], a & kLo, a & kHi, b & kLo, b & kHi, lo0, lo1);
        mma_full<__half>(o[2 * q + 1], a8 & kLo, a8 & kHi, b8 & kLo, b8 & kHi, lo0, lo1);
      }
    }
  }

  __device__ __forceinline__ void to_red(float* red_m, float* red_l, float* red_acc, int warp,
                                         int) {
#pragma unroll
    for (int mask = 1; mask <= 2; mask <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, mask);
      sumw += __shfl_xor_sync(0xffffffffu, sumw, mask);
      pmid += __shfl_xor_sync(0xffffffffu, pmid, mask);
    }
    if (g < G && c == 0) {
      red_m[warp * G + g] = m;
      red_l[warp * G + g] = l;
    }
    if constexpr (kRepeat) {  // columns 4-7 hold the residual's share of heads 0-3
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] += __shfl_xor_sync(0xffffffffu, o[t][e], 2);
    }
    const float back = vmax * 0.0078125f;  // 1 / vinv
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 2 * c + e;
      const float sw = __shfl_sync(0xffffffffu, sumw, 8 * c + 4 * e);
      const float pm = __shfl_sync(0xffffffffu, pmid, 8 * c + 4 * e);
      if (h < G) {
        float* dst = red_acc + (warp * G + h) * D + 4 * W * g;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          dst[2 * t] = fmaf(fmaf(o[t][e], 16777216.f, -7.5f * sw), back, pm);
          dst[2 * t + 1] = fmaf(fmaf(o[t][2 + e], 1048576.f, -7.5f * sw), back, pm);
        }
      }
    }
  }
};

}  // namespace pa
