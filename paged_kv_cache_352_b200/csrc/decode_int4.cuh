// Paged decode over 4-bit caches: kernel template and launcher, instantiated per
// (query type, head_dim) in paged_decode_<type>_d<dim>_int4.cu.
//
// Values are mid_t + (n - 7.5) s_t, n the 4-bit codes of token t's row, s_t and
// mid_t its half-precision scale and midpoint, so
//   score_t = sm_scale (s_t (q . n_t - 7.5 sum q) + mid_t sum q)
//   out     = (sum_t w_t n_t - 7.5 sum_t w_t + sum_t p_t mid_t) / sum_t p_t,
//   w_t = p_t s_t:
// codes enter the products as they are, and a token's two parameters are applied
// to one score instead of d elements.
//
// What bounds it. A (block, KV head) takes 16 (d + 8) bytes, of which an SM's share
// of the memory stream brings one every 95 cycles (d = 128, 1.9 GHz); its four
// schedulers then have 380 issue slots a tile. The loop takes about 215 instructions a
// tile, 88 of them turning codes into operands and 17 products, and a warp some 1500 more
// around it (ncu: issue 63 %, ALU 54 %, DRAM 56 %; the largest stalls are fixed latencies
// and warps not selected: no pipe is full, and 16 warps an SM leave chains uncovered).
// It is built for few instructions:
//   - every product runs on mma.sync, also for one query head per KV head (the
//     padding columns cost tensor time that is not short: 8 cycles per instruction,
//     17 a tile). The contraction has G columns of work, far too few for tcgen05;
//   - codes are operands as they lie: the low four bits of a half with zero
//     exponent are worth n 2^-24, the next four n 2^-20, both exact. Of a word of
//     eight key codes, w & 0x000f000f and w & 0x00f000f0 are operand registers, and
//     the same masks of w >> 8 give the rest: 5 instructions for 8 codes; value codes
//     take two bits more (w << 2 and w >> 6), see Precision. The powers of two are taken
//     back in the query operand (1/16 at the dimensions of high nibbles) and in the fp32
//     results. (Value codes could do with 4, whole bytes and high nibbles whose sums are
//     subtracted at the end; but the bytes' sums are 16 times as large and a long context's
//     mean is what is left of them: the error over 32k-131k tokens grew from 0.17% to 0.52%);
//   - the cache layout (int4_cache.cuh) gives each lane the 16 bytes it feeds to
//     its own registers, so lanes copy their own chunks by cp.async: no barrier,
//     no lane that issues for the others, 9 copies per two blocks;
//   - codes are the 16-row A operand of both products, so no operand is padding
//     that has to be cleared, and a lane's scores belong to the same two heads as
//     its output columns: sums and references need no exchange between lanes
//     unless a reference moves;
//   - a step takes two blocks: one vote, one wait for 32 tokens, and two
//     independent chains of products.
//
// Measured: 64 sequences of 128-2048 tokens, 32 heads, d = 128, f16 (337 MB): 69 us,
// 4.9 TB/s, in short bursts, 77 us in a loop of seconds (power limit, lower clock); the other
// caches' loop over these tiles took 105.5 us, the same loads without arithmetic take
// 53.9 us, a copy of the bytes 52.1 us. 8 sequences of 32768-131072 tokens, 64 query and 8
// KV heads, bf16: 160 and 182 us (loads alone 114).
//
// S = K Q^T. Lane 4g + c holds k-slots 2c, 2c+1, 2c+8, 2c+9 of A (rows g, g + 8)
// and of B (column g). It takes dimensions 8W c .. 8W c + 8W - 1 (W = d/32 words a
// row) of tokens g and g + 8, and of query head g: word j of a row gives two
// products, dimensions 8j+0, +4 | +1, +5 and 8j+2, +6 | +3, +7. The result is
// tokens g, g + 8 of heads 2c, 2c + 1; movmatrix turns the weights into the B
// operand of
// O^T = V^T P^T. A value word holds four dimensions of tokens 2p, 2p+1: word q of
// pair c gives a0 (dimension 4Wg + 4q) and a1 (+1), of pair c + 4 a2 and a3;
// shifted, dimensions +2 and +3 for the next m-tile. The result's columns are
// heads 2c, 2c + 1 again. One more product with ones for V gives sum w, from which the
// others start.
//
// Precision. Products are exact, sums are fp32. The matrix instruction, though, cuts its
// addends (towards zero) at about 2^-24 of the largest, and takes a subnormal code's size from
// its exponent field: n 2^-24 counts as 2^-14. What a token loses is of one sign for all
// dimensions. So value codes are shifted to 2^-22 and 2^-18 (one shift more per word), a step's
// products start from -7.5 sum w and end near 0, and they join the running sums by ordinary fp32
// additions, rounded to nearest. With running sums as the accumulator and codes at 2^-24 and
// 2^-20, half outputs over 131072 tokens of normal scores were off by 2.4e-4 of their norm
// beside their rounding's 2.1e-4; now by 7e-6 (scores twice as wide: 5.7e-4, 7e-5). It costs
// 3.5 to 4 %. q is brought below 2^15 by a
// power of two (exact in half unless 2^28 below the row's largest element, or 2^24 at the
// dimensions of high nibbles, whose operand is q / 16: 2^-35 of that element is lost). The
// weights w are rounded to half precision in units that put the largest at 2^6 to 2^7 when
// the reference moves; it moves when a weight reaches 2^15, 1/2 of half's range (one
// test on the packed halves), and follows the largest w = p s, not p and s apart: behind
// constant rows (s = 0) of high scores, or beside a large row of none, weights keep their bits.
// 7.5 sum w is taken over the rounded weights, so that their errors multiply the
// centred codes. What the rounding leaves of w joins the products too, rounded to half
// again (2^-22 of w in all): with at most 4 query heads per KV head heads repeat in
// columns 4-7, whose lanes feed it; with 8 it is a second product with sums of its own (in
// one chain with the weights' it would be cut at their size). Without it bf16 outputs over
// these contexts differ from 32-bit sums by 8e-4 to 1e-3 of their norm, with it by 1e-4; it
// costs 3 % (4 heads) and 14 % (8; 160 -> 182 us for the long contexts, 138 -> 160 in a burst).
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <atomic>

#include "decode_common.cuh"
#include "decode_merge.cuh"
#include "int4_cache.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kInt4Warps = 4;
constexpr int kInt4Stages = 3;
constexpr int kInt4CtasPerSm = 4;  // 128 registers a thread

// A lane's four chunks of a block's codes: two of K, two of V.
template <int CB>
__device__ __forceinline__ void copy_block(uint32_t dst, const unsigned char* k,
                                           const unsigned char* v) {
  cp_async<CB>(dst, k);
  cp_async<CB, 32 * CB, 32 * CB>(dst, k);
  cp_async<CB, 64 * CB>(dst, v);
  cp_async<CB, 96 * CB, 32 * CB>(dst, v);
}
// d += A B, m16n8k16, half operands, fp32 sums
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = c + A B: a chain's first product, its start kept in other registers
__device__ __forceinline__ void mma_16816_from(float (&d)[4], const float (&c)[4], uint32_t a0,
                                               uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}

// Transposes an 8 x 8 matrix of halves spread over the warp (row lane / 4).
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <int W>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// Largest magnitude of eight 16-bit elements.
template <typename T>
struct Amax;
template <>
struct Amax<__half> {
  static __device__ __forceinline__ float of(const uint4& u) {
    const __half2* h = reinterpret_cast<const __half2*>(&u);
    const __half2 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])),
                              __hmax2(__habs2(h[2]), __habs2(h[3])));
    const float2 f = __half22float2(m);
    return fmaxf(f.x, f.y);
  }
};
template <>
struct Amax<__nv_bfloat16> {
  static __device__ __forceinline__ float of(const uint4& u) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])),
                                     __hmax2(__habs2(h[2]), __habs2(h[3])));
    const float2 f = __bfloat1622float2(m);
    return fmaxf(f.x, f.y);
  }
};

// One warp's running softmax state over 4-bit tiles.
template <typename T, int D, int G>
struct Int4State {
  static constexpr int W = D / 32;  // words of codes a lane reads per row / per pair
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;
  static constexpr int kCodeBytes = kBlockSize * D / 2;
  static constexpr int kTileBytes = int4_tile_bytes(D);
  static constexpr bool kRepeat = G <= 4;  // columns 4-7 repeat heads 0-3
  static constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;

  int g, c, lane;
  uint4 qraw[W];
  uint32_t qb[KSTEPS][2];           // head g's operand
  // Of heads 2c, 2c + 1. Everything accumulated is in units of 2^ref (-inf before the
  // first step). l and pmid are this lane's share (tokens g, g + 8).
  float ref[2], l[2], pmid[2], row_scale[2], qsum[2];
  float centre[4];  // -7.5 qsum, where the products of a tile start
  float o[MT][4];   // sum w (n - 7.5), in the products' units

  // the head of column h
  static __device__ __forceinline__ int head(int h) { return kRepeat ? (h & 3) : h; }

  __device__ __forceinline__ void prefetch_q(const DecodeArgs& a, int s, int kvh, int lane_) {
    lane = lane_;
    g = lane >> 2;
    c = lane & 3;
    const uint4* row = reinterpret_cast<const uint4*>(
        reinterpret_cast<const T*>(a.q) +
        ((size_t)s * a.num_q_heads + (size_t)kvh * G + head(g)) * D + 8 * W * c);
#pragma unroll
    for (int i = 0; i < W; ++i) qraw[i] = head(g) < G ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
  }

  __device__ __forceinline__ void begin(float scale_log2) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) amax = fmaxf(amax, Amax<T>::of(qraw[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^-k brings the row's largest element to [2^14, 2^15)
    int k = amax > 0.f && amax < INFINITY ? ilogbf(amax) - 14 : 0;
    if (k < -100) k = -100;
    const float down = exp2f((float)-k);
    // The products are in units of 2^-24. The cap keeps the factor finite for rows
    // past 2^117, whose scores lie more than 2^50 apart with or without it.
    const float rs = scale_log2 * exp2f((float)(k + 24 < 125 ? k + 24 : 125));
    float qs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float f[8];
      Storage<T>::to_f32(qraw[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= down;
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // low nibbles: dimensions 2r, 2r + 4; high: one more
        const __half2 lo = __floats2half2_rn(f[2 * r], f[2 * r + 4]);
        const __half2 hi = __hmul2(__floats2half2_rn(f[2 * r + 1], f[2 * r + 5]),
                                   __float2half2_rn(0.0625f));
        memcpy(&qb[2 * j + r][0], &lo, 4);
        memcpy(&qb[2 * j + r][1], &hi, 4);
        // sum q as the product with codes of 1, in the layout of the scores
        mma_16816(qs, 0x00010001u, 0x00010001u, 0x00100010u, 0x00100010u, qb[2 * j + r][0],
                  qb[2 * j + r][1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qsum[e] = qs[e];
      row_scale[e] = __shfl_sync(0xffffffffu, rs, 8 * c + 4 * e);
      centre[e] = centre[2 + e] = -7.5f * qsum[e];
      ref[e] = -INFINITY;
      l[e] = pmid[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int t = 0; t < MT; ++t) o[t][e] = 0.f;
  }

  // (scale, mid) of token t
  static __device__ __forceinline__ float2 param(const unsigned char* p, int t) {
    return half2_bits_to_float2(*reinterpret_cast<const uint32_t*>(p + 4 * t));
  }

  // Weights of a step: t the scores over row_scale, in the references' units.
  struct Weights {
    float p[2];         // sum of p per head, this lane's tokens
    float pm[2];        // sum of p mid
    float w[2][2][2];   // [block][i][e]
    uint32_t h[2][2];   // the same as halves
    // Whether a weight leaves the range: some w at or past 2^15 (or inf or NaN, which a
    // reference of -inf gives too), or p past 2^60 (the reference leaves 2^31 at most).
    __device__ __forceinline__ bool out_of_range() const {
      const uint32_t m = __vmaxu2(__vmaxu2(h[0][0], h[0][1]), __vmaxu2(h[1][0], h[1][1]));
      return ((m + 0x08000800u) & 0x80008000u) != 0u || !(p[0] + p[1] <= 1.15e18f);
    }
  };

  template <bool kMask>
  __device__ __forceinline__ void weigh(const float (&t)[2][4], const float2 (&vp)[2][2],
                                        int valid0, int valid1, Weights& r) const {
    r.p[0] = r.p[1] = r.pm[0] = r.pm[1] = 0.f;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool in = !kMask || g + 8 * i < (b ? valid1 : valid0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float z = fmaf(t[b][2 * i + e], row_scale[e], -ref[e]);
          if (!in) z = -INFINITY;
          const float p = fast_exp2(z);
          r.p[e] += p;
          r.pm[e] = fmaf(p, vp[b][i].y, r.pm[e]);
          r.w[b][i][e] = p * vp[b][i].x;
        }
        const __half2 h = __floats2half2_rn(r.w[b][i][0], r.w[b][i][1]);
        memcpy(&r.h[b][i], &h, 4);
      }
  }

  // Moves the references to cover a step whose weights left the range (the first step
  // among them), and brings what has accumulated to the new ones, which are the same in
  // every lane of a column. A token's weight counts with its own scale, so that the largest
  // w of the step is put at 2^6 to 2^7 whatever the other tokens' scales are, a constant
  // row's (0) as the smallest half: p is 2^31 at most.
  template <bool kMask>
  __device__ __forceinline__ void move(const float (&t)[2][4], const float2 (&vp)[2][2],
                                       int valid0, int valid1) {
    float bmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (!kMask || g + 8 * i < (b ? valid1 : valid0)) {
          // log2 of the power of two at or above the scale (exact: a half has 11 bits)
          const uint32_t s = __float_as_uint(fmaxf(vp[b][i].x, 5.9604644775390625e-8f));
          const float up = (float)((int)((s + 0x007fffffu) >> 23) - 127);
          bmax[0] = fmaxf(bmax[0], fmaf(t[b][2 * i], row_scale[0], up));
          bmax[1] = fmaxf(bmax[1], fmaf(t[b][2 * i + 1], row_scale[1], up));
        }
#pragma unroll
    for (int mask = 4; mask <= 16; mask <<= 1) {
      bmax[0] = fmaxf(bmax[0], __shfl_xor_sync(0xffffffffu, bmax[0], mask));
      bmax[1] = fmaxf(bmax[1], __shfl_xor_sync(0xffffffffu, bmax[1], mask));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool first = ref[e] == -INFINITY;  // nothing of this head has accumulated
      // (scores of NaN or -inf alone leave a first reference at 0, a number to the merges)
      const float to = bmax[e] == -INFINITY ? (first ? 0.f : ref[e]) : fmaxf(ref[e], bmax[e] - 7.f);
      const float alpha = first ? 1.f : fast_exp2(ref[e] - to);
      ref[e] = to;
      l[e] *= alpha;
      pmid[e] *= alpha;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        o[i][e] *= alpha;
        o[i][2 + e] *= alpha;
      }
    }
  }

  // Two blocks, `codes` and `par` as Int4Stage lays them out. kMask: block i has
  // valid<i> tokens inside the context (0: not copied); what lies in the others'
  // slots may be any bits.
  template <bool kMask>
  __device__ __forceinline__ void step(const unsigned char* codes, const unsigned char* par,
                                       int valid0, int valid1) {
    // ---- S = K Q^T
    float t[2][4];  // [block][2 i + e]: token g + 8 i, head 2c + e
    float2 vp[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const unsigned char* kc = codes + b * 2 * kCodeBytes + lane * (4 * W);
      uint32_t ka[W], kb[W];
      load_words<W>(kc, ka);
      load_words<W>(kc + kCodeBytes / 2, kb);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t u = ka[j], v = kb[j], u8 = u >> 8, v8 = v >> 8;
        if (j == 0)
          mma_16816_from(t[b], centre, u & kLo, v & kLo, u & kHi, v & kHi, qb[0][0], qb[0][1]);
        else
          mma_16816(t[b], u & kLo, v & kLo, u & kHi, v & kHi, qb[2 * j][0], qb[2 * j][1]);
        mma_16816(t[b], u8 & kLo, v8 & kLo, u8 & kHi, v8 & kHi, qb[2 * j + 1][0],
                  qb[2 * j + 1][1]);
      }
    }
    // ---- scores over row_scale: s (q . n - 7.5 sum q) + mid sum q
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 kp = param(par + b * 128, g + 8 * i);
        vp[b][i] = param(par + b * 128 + 64, g + 8 * i);
        if (kMask && g + 8 * i >= (b ? valid1 : valid0)) vp[b][i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          t[b][2 * i + e] = fmaf(kp.x, t[b][2 * i + e], kp.y * qsum[e]);
      }
    Weights r;
    weigh<kMask>(t, vp, valid0, valid1, r);
    if (__any_sync(0xffffffffu, r.out_of_range())) {
      move<kMask>(t, vp, valid0, valid1);
      weigh<kMask>(t, vp, valid0, valid1, r);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += r.p[e];
      pmid[e] += r.pm[e];
    }
    // ---- O^T += V^T P^T - 7.5 sum w
    uint32_t pb[2][2], lo[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 f = half2_bits_to_float2(r.h[b][i]);
        const __half2 rl = __floats2half2_rn(r.w[b][i][0] - f.x, r.w[b][i][1] - f.y);
        memcpy(&lo[b][i], &rl, 4);
        pb[b][i] = r.h[b][i];
        if constexpr (kRepeat) pb[b][i] = c < 2 ? pb[b][i] : lo[b][i];
        else lo[b][i] = transpose8(lo[b][i]);
        pb[b][i] = transpose8(pb[b][i]);
      }
    constexpr uint32_t kOnes = 0x3c003c00u;
    float sw[4] = {0.f, 0.f, 0.f, 0.f};
    mma_16816(sw, kOnes, kOnes, kOnes, kOnes, pb[0][0], pb[0][1]);
    mma_16816(sw, kOnes, kOnes, kOnes, kOnes, pb[1][0], pb[1][1]);
    if constexpr (!kRepeat) {
      float sl[4] = {0.f, 0.f, 0.f, 0.f};
      mma_16816(sl, kOnes, kOnes, kOnes, kOnes, lo[0][0], lo[0][1]);
      mma_16816(sl, kOnes, kOnes, kOnes, kOnes, lo[1][0], lo[1][1]);
      sw[0] += sl[0];
      sw[1] += sl[1];
    }
    // -7.5 sum w in the products' units (2^-22 at low nibbles, 2^-18 at high ones)
    const float start[4] = {sw[0] * -1.7881393432617188e-06f, sw[1] * -1.7881393432617188e-06f,
                            sw[0] * -2.86102294921875e-05f, sw[1] * -2.86102294921875e-05f};
    uint32_t va[2][W], vb[2][W];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const unsigned char* vc = codes + b * 2 * kCodeBytes + kCodeBytes + lane * (4 * W);
      load_words<W>(vc, va[b]);
      load_words<W>(vc + kCodeBytes / 2, vb[b]);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float d[4];
      uint32_t a[2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t x = t & 1 ? va[b][t >> 1] >> 6 : va[b][t >> 1] << 2;
        const uint32_t y = t & 1 ? vb[b][t >> 1] >> 6 : vb[b][t >> 1] << 2;
        a[b][0] = x & 4 * kLo, a[b][1] = x & 4 * kHi, a[b][2] = y & 4 * kLo, a[b][3] = y & 4 * kHi;
      }
      mma_16816_from(d, start, a[0][0], a[0][1], a[0][2], a[0][3], pb[0][0], pb[0][1]);
      if constexpr (!kRepeat) {  // two chains: the residuals' own, joined below
        float r[4] = {0.f, 0.f, 0.f, 0.f};
        mma_16816(r, a[0][0], a[0][1], a[0][2], a[0][3], lo[0][0], lo[0][1]);
        mma_16816(d, a[1][0], a[1][1], a[1][2], a[1][3], pb[1][0], pb[1][1]);
        mma_16816(r, a[1][0], a[1][1], a[1][2], a[1][3], lo[1][0], lo[1][1]);
        fadd2(d[0], d[1], r[0], r[1]);
        fadd2(d[2], d[3], r[2], r[3]);
      } else {
        mma_16816(d, a[1][0], a[1][1], a[1][2], a[1][3], pb[1][0], pb[1][1]);
      }
      fadd2(o[t][0], o[t][1], d[0], d[1]);
      fadd2(o[t][2], o[t][3], d[2], d[3]);
    }
  }

  // Sums the lanes' shares of l and pmid.
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int mask = 4; mask <= 16; mask <<= 1) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], mask);
        pmid[e] += __shfl_xor_sync(0xffffffffu, pmid[e], mask);
      }
    if constexpr (kRepeat) {  // columns 4-7 repeat the heads for the residual alone
      pmid[0] = c < 2 ? pmid[0] : 0.f;
      pmid[1] = c < 2 ? pmid[1] : 0.f;
    }
  }

  // Unnormalised outputs (in units of 2^ref) of head 2c + e: dimensions
  // 4W g + 4q .. + 3.
  __device__ __forceinline__ float4 row4(int e, int q) const {
    return make_float4(fmaf(o[2 * q][e], 4194304.f, pmid[e]),
                       fmaf(o[2 * q][2 + e], 262144.f, pmid[e]),
                       fmaf(o[2 * q + 1][e], 4194304.f, pmid[e]),
                       fmaf(o[2 * q + 1][2 + e], 262144.f, pmid[e]));
  }
};

// A stage of a warp's ring: per block the K codes and the V codes (each as in
// the tile), then per block the parameters of K and of V (64 bytes each).
template <int D>
struct Int4Stage {
  static constexpr int kCodeBytes = kBlockSize * D / 2;
  static constexpr int kParOff = 4 * kCodeBytes;
  static constexpr int kBytes = kParOff + 2 * 128;
};

// Grid (KV head, partition or group of kInt4Warps partitions, sequence), as the
// other decode kernels'. In the one-CTA-per-partition mode warp w takes the pairs
// of blocks w, w + 4, ... of the CTA's partition; with a.warp_parts it takes
// partition 4 y + w whole, and merge_partitions_kernel follows.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kInt4Warps * 32, kInt4CtasPerSm)
    paged_decode_int4_kernel(const DecodeArgs a) {
  using St = Int4State<T, D, G>;
  using Stage = Int4Stage<D>;
  constexpr int WARPS = kInt4Warps, STAGES = kInt4Stages;
  constexpr int CB = D / 8;  // bytes of a lane's chunk (16 or 8)
  grid_dependency_wait();
  allow_dependents();
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.x;
  const int s = a.seq_order ? __ldg(a.seq_order + blockIdx.z) : (int)blockIdx.z;
  if ((unsigned)s >= (unsigned)a.num_seqs) {
    if (blockIdx.y == 0 && kvh == 0 && threadIdx.x == 0)
      report(a.dev_error, PA_DEVERR_CONTEXT_RANGE);
    return;
  }
  const int part = a.warp_parts ? blockIdx.y * WARPS + warp : blockIdx.y;
  // the warp's blocks: pairs from `first`, `stride` blocks apart
  const int first = part * a.part_blocks + (a.warp_parts ? 0 : 2 * warp);
  const int stride = a.warp_parts ? 2 : 2 * WARPS;
  const int32_t* table = a.block_tables + (size_t)s * a.max_blocks_per_seq;
  // Independent loads first, so that their latencies overlap: the context length,
  // the first 32 table entries of the warp (lane i: block i & 1 of pair i / 2;
  // entries past the sequence are padding, never used) and q.
  int ctx = __ldg(a.context_lens + s);
  int raw_entry = -1;
  {
    const long long b = first + (long long)(lane >> 1) * stride + (lane & 1);
    if (b < a.max_blocks_per_seq) raw_entry = __ldg(table + b);
  }
  St st;
  st.prefetch_q(a, s, kvh, lane);
  if (ctx < 0 || ctx > a.max_blocks_per_seq * kBlockSize || ctx > a.max_context_len) {
    if (blockIdx.y == 0 && kvh == 0 && threadIdx.x == 0)
      report(a.dev_error, PA_DEVERR_CONTEXT_RANGE);
    ctx = 0;  // flagged; the sequence yields a zero output
  }
  const int nblk = (ctx + kBlockSize - 1) / kBlockSize;
  const int nparts = (nblk + a.part_blocks - 1) / a.part_blocks;
  T* out_rows = reinterpret_cast<T*>(a.out) + ((size_t)s * a.num_q_heads + (size_t)kvh * G) * D;
  if (nblk == 0) {
    if (blockIdx.y == 0 && !a.warp_parts)
      for (int i = threadIdx.x; i < G * D; i += blockDim.x) out_rows[i] = Storage<T>::from_f32(0.f);
    return;  // the merge kernel writes the zero row of a sequence without states
  }
  if ((a.warp_parts ? (int)blockIdx.y * WARPS : part) >= nparts) return;  // the whole CTA
  const int last = min(nblk, (part + 1) * a.part_blocks);  // blocks end here
  const int pairs = last > first ? (last - first + stride - 1) / stride : 0;

  // Entry of the table as the place of its tile: offset / 64 (tiles are multiples
  // of 64 bytes; 2^38 bytes of pool), kNone past the warp's blocks, kBad outside
  // the pool. Lane i holds block i & 1 of pair base + i / 2.
  constexpr uint32_t kNone = 0xfffffffeu, kBad = 0xffffffffu;
  static_assert(St::kTileBytes % 64 == 0, "tile places are counted in 64 bytes");
  const uint32_t block_units = (uint32_t)a.num_kv_heads * (St::kTileBytes / 64);
  auto in_range = [&](int base) {
    const int pair = base + (lane >> 1);
    return pair < pairs && first + pair * stride + (lane & 1) < last;
  };
  auto place = [&](int e) -> uint32_t {
    return (unsigned)e < (unsigned)a.num_blocks ? (uint32_t)e * block_units : kBad;
  };
  auto entries = [&](int base) -> uint32_t {
    return in_range(base) ? place(__ldg(table + first + (base + (lane >> 1)) * stride + (lane & 1)))
                          : kNone;
  };
  uint32_t win = in_range(0) ? place(raw_entry) : kNone;
  uint32_t win_next = entries(16);

  // shared-memory places of this lane's chunks in stage 0, and their sources less
  // the tile's offset; lanes 0-15 copy the parameters: 16 bytes (lane & 3) of K or V
  // (lane & 4) of block lane / 8
  const uint32_t ring = smem_addr(smem) + warp * STAGES * Stage::kBytes;
  const unsigned char* kt = static_cast<const unsigned char*>(a.k_cache) +
                            (size_t)kvh * St::kTileBytes + lane * CB;
  const unsigned char* vt = static_cast<const unsigned char*>(a.v_cache) +
                            (size_t)kvh * St::kTileBytes + lane * CB;
  const unsigned char* par_src = ((lane & 4) ? vt : kt) - lane * CB + St::kCodeBytes +
                                 16 * (lane & 3);
  const uint32_t par_dst = Stage::kParOff + 16 * (lane & 15);
  uint32_t skipped = 0;  // bits 2 st, 2 st + 1: block 0 or 1 of stage st was not copied
  auto issue = [&](int jp, int stg) {
    if (jp < pairs) {
      if ((jp & 15) == 0 && jp > 0) {
        win = win_next;
        win_next = entries(jp + 16);
      }
      const uint32_t e0 = __shfl_sync(0xffffffffu, win, 2 * (jp & 15));
      const uint32_t e1 = __shfl_sync(0xffffffffu, win, 2 * (jp & 15) + 1);
      const uint32_t dst = ring + stg * Stage::kBytes;
      const uint64_t off0 = (uint64_t)e0 * 64u, off1 = (uint64_t)e1 * 64u;
      if (max(e0, e1) < kNone) {
        copy_block<CB>(dst + lane * CB, kt + off0, vt + off0);
        copy_block<CB>(dst + (128 + lane) * CB, kt + off1, vt + off1);
        if (lane < 16) cp_async<16>(dst + par_dst, par_src + (lane < 8 ? off0 : off1));
        if (skipped) skipped &= ~(3u << (2 * stg));
      } else {  // the last block of an odd count, or a bad entry
        const bool ok0 = e0 < kNone, ok1 = e1 < kNone;
        if (ok0) copy_block<CB>(dst + lane * CB, kt + off0, vt + off0);
        if (ok1) copy_block<CB>(dst + (128 + lane) * CB, kt + off1, vt + off1);
        if (lane < 16 && (lane < 8 ? ok0 : ok1))
          cp_async<16>(dst + par_dst, par_src + (lane < 8 ? off0 : off1));
        skipped = (skipped & ~(3u << (2 * stg))) | ((ok0 ? 0u : 1u) | (ok1 ? 0u : 2u)) << (2 * stg);
        if ((e0 == kBad || e1 == kBad) && lane == 0) report(a.dev_error, PA_DEVERR_BLOCK_RANGE);
      }
    }
    cp_async_commit();  // a group per step, also an empty one: the waits count groups
  };
  for (int j = 0; j < STAGES - 1; ++j) issue(j, j);
  st.begin(a.scale_log2);

  int stg = 0;
  const int limit = ctx - first * kBlockSize;  // tokens from the warp's first block on
  for (int j = 0; j < pairs; ++j) {
    cp_async_wait<STAGES - 2>();
    // publishes the parameters that other lanes copied, and orders this step's
    // copies behind every lane's reads of the stage they go to (step j - 1's)
    __syncwarp();
    issue(j + STAGES - 1, stg == 0 ? STAGES - 1 : stg - 1);
    const unsigned char* codes = smem + (warp * STAGES + stg) * Stage::kBytes;
    const int v0 = limit - j * stride * kBlockSize;
    const uint32_t miss = (skipped >> (2 * stg)) & 3u;
    if (v0 >= 2 * kBlockSize && miss == 0)
      st.template step<false>(codes, codes + Stage::kParOff, 0, 0);
    else if (miss != 3u)
      st.template step<true>(codes, codes + Stage::kParOff, (miss & 1u) ? 0 : v0,
                             (miss & 2u) ? 0 : v0 - kBlockSize);
    stg = stg == STAGES - 1 ? 0 : stg + 1;
  }
  cp_async_wait<0>();

  // ---- merge the warps. Every warp has the same layout of outputs, so each scales
  // its own to the common reference and leaves them by lane: no bank conflicts, and
  // the thread that adds up a float4 already holds its heads' sums.
  st.close();
  __shared__ float red_m[WARPS][8], red_l[WARPS][8];
  if (st.g == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      red_m[warp][2 * st.c + e] = st.ref[e];
      red_l[warp][2 * st.c + e] = st.l[e];
    }
  }
  __syncthreads();  // (and every warp is done with its ring)
  constexpr int W = St::W, POS = 2 * W;  // float4 positions of a lane: (e, q)
  float4* red_acc = reinterpret_cast<float4*>(smem);  // [WARPS][POS][32]
  float M[2], L[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int h = 2 * st.c + e;
    M[e] = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M[e] = fmaxf(M[e], red_m[w][h]);
    // finite unless every block of the partition was skipped as out of range
    const float mr = M[e] == -INFINITY ? 0.f : M[e];
    L[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) L[e] = fmaf(fast_exp2(red_m[w][h] - mr), red_l[w][h], L[e]);
    const float sc = fast_exp2(red_m[warp][h] - mr);
    if (St::head(h) < G) {
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const float4 v = st.row4(e, q);
        red_acc[(warp * POS + e * W + q) * 32 + lane] =
            make_float4(v.x * sc, v.y * sc, v.z * sc, v.w * sc);
      }
    }
  }
  __syncthreads();
  const bool split = a.warp_parts || nparts > 1;
  const size_t row0 = (((size_t)s * a.num_kv_heads + kvh) * a.max_parts + blockIdx.y) * G;
#pragma unroll
  for (int i = 0; i < POS / WARPS; ++i) {
    const int pos = warp * (POS / WARPS) + i;
    const int e = pos / W, q = pos % W;
    const int h = 2 * st.c + e;
    if (h >= G) continue;
    float4 v = red_acc[pos * 32 + lane];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      const float4 u = red_acc[(w * POS + pos) * 32 + lane];
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    if constexpr (St::kRepeat) {  // the residual's share, from the lane of column h + 4
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 u = red_acc[(w * POS + pos) * 32 + (lane ^ 2)];
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
    }
    const int dim = 4 * W * st.g + 4 * q;
    const float Mh = e ? M[1] : M[0], Lh = e ? L[1] : L[0];
    if (!split) {
      const float f = Lh > 0.f || Lh != Lh ? 1.f / Lh : 0.f;
      T r[4] = {Storage<T>::from_f32(v.x * f), Storage<T>::from_f32(v.y * f),
                Storage<T>::from_f32(v.z * f), Storage<T>::from_f32(v.w * f)};
      uint2 packed;
      memcpy(&packed, r, sizeof(packed));
      *reinterpret_cast<uint2*>(out_rows + h * D + dim) = packed;
    } else {
      *reinterpret_cast<float4*>(a.ws_acc + (row0 + h) * D + dim) = v;
      if (dim == 0) {
        a.ws_m[row0 + h] = Mh;
        a.ws_l[row0 + h] = Lh;
      }
    }
  }
  if (!split || a.warp_parts) return;
  merge_if_last<T, D, G, WARPS>(a, reinterpret_cast<float*>(smem), s, kvh, nparts, out_rows);
}

template <typename T, int D, int G>
cudaError_t launch_int4(const DecodeArgs& a, cudaStream_t stream) {
  constexpr int WARPS = kInt4Warps;
  const size_t ring = size_t(WARPS) * kInt4Stages * Int4Stage<D>::kBytes;
  const size_t red = size_t(WARPS) * 8 * D * sizeof(float);
  const size_t wts = (size_t)a.max_parts * G * sizeof(float);
  size_t smem = ring > red ? ring : red;
  if (smem < wts) smem = wts;
  constexpr size_t kLimit = 200 * 1024;
  if (smem > kLimit) return cudaErrorInvalidConfiguration;
  auto kern = paged_decode_int4_kernel<T, D, G>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int kMaxDev = 64;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  static std::atomic<bool> ready[kMaxDev];
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLimit);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  const int y = a.warp_parts == 1 ? (a.max_parts + WARPS - 1) / WARPS : a.max_parts;
  e = launch_dependent(kern, dim3(a.num_kv_heads, y, a.num_seqs), dim3(WARPS * 32), smem, stream,
                       a);
  if (e != cudaSuccess || !a.warp_parts) return e;
  return launch_dependent(merge_partitions_kernel<T, D, G, WARPS>,
                          dim3(a.num_kv_heads * G, a.num_seqs), dim3(kMergeThreads), 0, stream, a);
}

}  // namespace

// Launches the 4-bit decode for one query/output type T and head_dim.
template <typename T, int D>
cudaError_t launch_decode_int4_typed(const DecodeArgs& a, int group, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_int4<T, D, 1>(a, stream);
    case 2: return launch_int4<T, D, 2>(a, stream);
    case 4: return launch_int4<T, D, 4>(a, stream);
    case 8: return launch_int4<T, D, 8>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pa
