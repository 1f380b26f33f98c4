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
// schedulers then have 380 issue slots a tile. Half of them go to turning
// codes into operands and multiplying, so the loop is built for few instructions:
//   - every product runs on mma.sync, also for one query head per KV head (the
//     padding columns cost tensor time that is not short: 8 cycles per instruction,
//     17 a tile). The contraction has G columns of work, far too few for tcgen05;
//   - codes are operands as they lie: the low four bits of a half with zero
//     exponent are worth n 2^-24, the next four n 2^-20, both exact. Of a word of
//     eight codes, w & 0x000f000f and w & 0x00f000f0 are operand registers, and
//     the same masks of w >> 8 give the rest: 5 instructions for 8 codes. The
//     powers of two are taken back in the query operand (1/16 at the dimensions
//     of high nibbles) and in the fp32 results;
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
// S = K Q^T. Lane 4g + c holds k-slots 2c, 2c+1, 2c+8, 2c+9 of A (rows g, g + 8)
// and of B (column g). It takes dimensions 8W c .. 8W c + 8W - 1 (W = d/32 words a
// row) of tokens g and g + 8, and of query head g: word j of a row gives two
// products, dimensions 8j+0, +4 | +1, +5 and 8j+2, +6 | +3, +7. The result is
// tokens g, g + 8 of heads 2c, 2c + 1; movmatrix turns the weights into the B
// operand of
// O^T = V^T P^T. A value word holds four dimensions of tokens 2p, 2p+1: word q of
// pair c gives a0 (dimension 4Wg + 4q) and a1 (+1), of pair c + 4 a2 and a3;
// shifted, dimensions +2 and +3 for the next m-tile. The result's columns are
// heads 2c, 2c + 1 again. One more product with ones for V gives sum w.
//
// Precision. Products are exact, sums are fp32. q is brought below 2^15 by a
// power of two (exact in half unless 2^29 below the row's largest element). The
// weights w are rounded to half precision relative to the largest value scale
// seen (a power of two S, raised when a larger scale comes, as the softmax
// reference is), and 7.5 sum w is taken over the rounded weights, so that their
// errors multiply the centred codes. For half outputs the rounding residual of
// w joins the product too: with at most 4 query heads per KV head heads repeat
// in columns 4-7, whose lanes feed the residual (no cost); with 8 it is a second
// product. For bf16 outputs the weights' 2^-11 is 1/8 of the output's own step.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <atomic>
#include <type_traits>

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

// Copies BYTES (8 or 16) from global to shared memory asynchronously.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* smem, const void* gmem) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(gmem)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += A B, m16n8k16, half operands, fp32 sums
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// One warp's running softmax state over 4-bit tiles.
template <typename T, int D, int G>
struct Int4State {
  static constexpr int W = D / 32;  // words of codes a lane reads per row / per pair
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;
  static constexpr int kCodeBytes = kBlockSize * D / 2;
  static constexpr int kTileBytes = int4_tile_bytes(D);
  static constexpr bool kResidual = std::is_same<T, __half>::value;
  static constexpr bool kRepeat = kResidual && G <= 4;  // columns 4-7 repeat heads 0-3
  static constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;

  int g, c, lane;
  uint4 qraw[W];
  uint32_t qb[KSTEPS][2];           // head g's operand
  // of heads 2c, 2c + 1; l and pmid are this lane's share (tokens g, g + 8)
  float m[2], l[2], pmid[2], row_scale[2], qsum[2];
  float vmax, vinv;                 // S and 2^7 / S (both 0 until a positive scale comes)
  float o[MT][4], ow[4];

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
    for (int i = 0; i < W; ++i) {
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
    const float rs = scale_log2 * exp2f((float)k);
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
        memcpy(&qb[2 * j + r][0], &lo, 4);
        memcpy(&qb[2 * j + r][1], &hi, 4);
      }
    }
    qs += __shfl_xor_sync(0xffffffffu, qs, 1);
    qs += __shfl_xor_sync(0xffffffffu, qs, 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qsum[e] = __shfl_sync(0xffffffffu, qs, 8 * c + 4 * e);
      row_scale[e] = __shfl_sync(0xffffffffu, rs, 8 * c + 4 * e);
      m[e] = -INFINITY;
      l[e] = pmid[e] = 0.f;
    }
    vmax = vinv = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ow[e] = 0.f;
#pragma unroll
      for (int t = 0; t < MT; ++t) o[t][e] = 0.f;
    }
  }

  // (scale, mid) of token t
  static __device__ __forceinline__ float2 param(const unsigned char* p, int t) {
    return half2_bits_to_float2(*reinterpret_cast<const uint32_t*>(p + 4 * t));
  }

  // Two blocks, `codes` and `par` as Int4Stage lays them out. kMask: block i has
  // valid<i> tokens inside the context (0: not copied); what lies in the others'
  // slots may be any bits.
  template <bool kMask>
  __device__ __forceinline__ void step(const unsigned char* codes, const unsigned char* par,
                                       int valid0, int valid1) {
    auto in = [&](int b, int i) { return !kMask || g + 8 * i < (b ? valid1 : valid0); };
    // ---- S = K Q^T
    float x[2][4];  // [block][2 i + e]: token g + 8 i, head 2c + e
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      x[b][0] = x[b][1] = x[b][2] = x[b][3] = 0.f;
      const unsigned char* kc = codes + b * 2 * kCodeBytes + lane * (4 * W);
      uint32_t ka[W], kb[W];
      load_words<W>(kc, ka);
      load_words<W>(kc + kCodeBytes / 2, kb);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t u = ka[j], v = kb[j], u8 = u >> 8, v8 = v >> 8;
        mma_16816(x[b], u & kLo, v & kLo, u & kHi, v & kHi, qb[2 * j][0], qb[2 * j][1]);
        mma_16816(x[b], u8 & kLo, v8 & kLo, u8 & kHi, v8 & kHi, qb[2 * j + 1][0],
                  qb[2 * j + 1][1]);
      }
    }
    // ---- scores
    float bmax[2] = {-INFINITY, -INFINITY};
    float2 vp[2][2];
    float smax = 0.f;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 kp = param(par + b * 128, g + 8 * i);
        vp[b][i] = param(par + b * 128 + 64, g + 8 * i);
        if (!in(b, i)) vp[b][i] = make_float2(0.f, 0.f);
        smax = fmaxf(smax, vp[b][i].x);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& y = x[b][2 * i + e];
          const float dot = fmaf(y, 16777216.f, -7.5f * qsum[e]);
          y = fmaf(kp.x, dot, kp.y * qsum[e]) * row_scale[e];
          if (!in(b, i)) y = -INFINITY;
          bmax[e] = fmaxf(bmax[e], y);
        }
      }
    const bool moved =
        bmax[0] > m[0] + kLazyRescaleLog2 || bmax[1] > m[1] + kLazyRescaleLog2 || smax > vmax;
    if (__any_sync(0xffffffffu, moved)) {
      // a softmax reference or the value-scale reference S moves: bring the sums
      // to the new ones (the same in every lane of a column)
#pragma unroll
      for (int mask = 4; mask <= 16; mask <<= 1) {
        bmax[0] = fmaxf(bmax[0], __shfl_xor_sync(0xffffffffu, bmax[0], mask));
        bmax[1] = fmaxf(bmax[1], __shfl_xor_sync(0xffffffffu, bmax[1], mask));
        smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, mask));
      }
      float f = 1.f;
      if (smax > vmax) {
        // the power of two at or above smax (a half: exact here)
        const float s2 = __uint_as_float((__float_as_uint(smax) + 0x007fffffu) & 0x7f800000u);
        f = vmax / s2;
        vmax = s2;
        vinv = 128.f / s2;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float alpha;
        lazy_reference(m[e], bmax[e], alpha);
        l[e] *= alpha;
        pmid[e] *= alpha;
        alpha *= f;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          o[t][e] *= alpha;
          o[t][2 + e] *= alpha;
        }
        ow[e] *= alpha;
      }
    }
    const float mref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
    // ---- O^T += V^T P^T
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t pb[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float sv = vp[b][i].x * vinv;
        float w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = fast_exp2(x[b][2 * i + e] - mref[e]);
          l[e] += p;
          pmid[e] = fmaf(p, vp[b][i].y, pmid[e]);
          w[e] = p * sv;  // at most 2^8 2^7 (the reference is lazy by 2^8)
        }
        const __half2 h = __floats2half2_rn(w[0], w[1]);
        memcpy(&pb[i], &h, 4);
        if constexpr (kResidual) {
          const float2 r = __half22float2(h);
          const __half2 rl = __floats2half2_rn(w[0] - r.x, w[1] - r.y);
          memcpy(&lo[i], &rl, 4);
          if constexpr (kRepeat) pb[i] = c < 2 ? pb[i] : lo[i];
          else lo[i] = transpose8(lo[i]);
        }
        pb[i] = transpose8(pb[i]);
      }
      const unsigned char* vc = codes + b * 2 * kCodeBytes + kCodeBytes + lane * (4 * W);
      uint32_t va[W], vb[W];
      load_words<W>(vc, va);
      load_words<W>(vc + kCodeBytes / 2, vb);
      constexpr uint32_t kOnes = 0x3c003c00u;
      mma_16816(ow, kOnes, kOnes, kOnes, kOnes, pb[0], pb[1]);
      if constexpr (kResidual && !kRepeat)
        mma_16816(ow, kOnes, kOnes, kOnes, kOnes, lo[0], lo[1]);
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const uint32_t a = va[q], d = vb[q], a8 = a >> 8, d8 = d >> 8;
        mma_16816(o[2 * q], a & kLo, a & kHi, d & kLo, d & kHi, pb[0], pb[1]);
        mma_16816(o[2 * q + 1], a8 & kLo, a8 & kHi, d8 & kLo, d8 & kHi, pb[0], pb[1]);
        if constexpr (kResidual && !kRepeat) {
          mma_16816(o[2 * q], a & kLo, a & kHi, d & kLo, d & kHi, lo[0], lo[1]);
          mma_16816(o[2 * q + 1], a8 & kLo, a8 & kHi, d8 & kLo, d8 & kHi, lo[0], lo[1]);
        }
      }
    }
  }

  __device__ __forceinline__ void to_red(float* red_m, float* red_l, float* red_acc, int warp) {
    if constexpr (kRepeat) {  // columns 4-7 hold the residual's share of heads 0-3
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int t = 0; t < MT; ++t) o[t][e] += __shfl_xor_sync(0xffffffffu, o[t][e], 2);
        ow[e] += __shfl_xor_sync(0xffffffffu, ow[e], 2);
      }
    }
    const float back = vmax * 0.0078125f;  // 1 / vinv
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int mask = 4; mask <= 16; mask <<= 1) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], mask);
        pmid[e] += __shfl_xor_sync(0xffffffffu, pmid[e], mask);
      }
      const int h = 2 * c + e;
      if (h < G) {
        if (g == 0) {
          red_m[warp * G + h] = m[e];
          red_l[warp * G + h] = l[e];
        }
        float2* dst = reinterpret_cast<float2*>(red_acc + (warp * G + h) * D + 4 * W * g);
#pragma unroll
        for (int t = 0; t < MT; ++t)
          dst[t] = make_float2(fmaf(fmaf(o[t][e], 16777216.f, -7.5f * ow[e]), back, pmid[e]),
                               fmaf(fmaf(o[t][2 + e], 1048576.f, -7.5f * ow[e]), back, pmid[e]));
      }
    }
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
  int ctx = __ldg(a.context_lens + s);
  // lane i holds the table entry of block i & 1 of pair base + i / 2
  auto entries = [&](int base) {
    const long long b = first + (long long)(base + (lane >> 1)) * stride + (lane & 1);
    return b < a.max_blocks_per_seq ? __ldg(table + b) : -1;
  };
  int win = entries(0);
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

  unsigned char* ring = smem + (size_t)warp * STAGES * Stage::kBytes;
  const uint32_t block_stride = (uint32_t)a.num_kv_heads * St::kTileBytes;
  const unsigned char* kt = static_cast<const unsigned char*>(a.k_cache) +
                            (size_t)kvh * St::kTileBytes;
  const unsigned char* vt = static_cast<const unsigned char*>(a.v_cache) +
                            (size_t)kvh * St::kTileBytes;
  // lanes 0-15 copy the parameters: 16 bytes (lane & 3) of K or V (lane & 4) of block lane / 8
  const unsigned char* par_src = ((lane & 4) ? vt : kt) + St::kCodeBytes + 16 * (lane & 3);
  const int par_dst = Stage::kParOff + 16 * (lane & 15);

  int win_next = pairs > 16 ? entries(16) : -1;
  uint32_t copied = 0;  // bits 2 st, 2 st + 1: blocks 0 and 1 of stage st were copied
  auto issue = [&](int jp, int stg) {
    if (jp < pairs) {
      if ((jp & 15) == 0 && jp > 0) {
        win = win_next;
        win_next = jp + 16 < pairs ? entries(jp + 16) : -1;
      }
      const int b0 = first + jp * stride;
      const int e0 = __shfl_sync(0xffffffffu, win, 2 * (jp & 15));
      const int e1 = __shfl_sync(0xffffffffu, win, 2 * (jp & 15) + 1);
      const bool ok0 = (unsigned)e0 < (unsigned)a.num_blocks;
      const bool has1 = b0 + 1 < last;
      const bool ok1 = has1 && (unsigned)e1 < (unsigned)a.num_blocks;
      copied = (copied & ~(3u << (2 * stg))) | ((ok0 ? 1u : 0u) | (ok1 ? 2u : 0u)) << (2 * stg);
      if (!ok0 || (has1 && !ok1)) {
        if (lane == 0) report(a.dev_error, PA_DEVERR_BLOCK_RANGE);
      }
      unsigned char* dst = ring + stg * Stage::kBytes;
      const uint64_t off0 = (uint64_t)(uint32_t)e0 * block_stride;
      const uint64_t off1 = (uint64_t)(uint32_t)e1 * block_stride;
      if (ok0) {
        unsigned char* to = dst + lane * CB;
        cp_async<CB>(to, kt + off0 + lane * CB);
        cp_async<CB>(to + 32 * CB, kt + off0 + (32 + lane) * CB);
        cp_async<CB>(to + 64 * CB, vt + off0 + lane * CB);
        cp_async<CB>(to + 96 * CB, vt + off0 + (32 + lane) * CB);
      }
      if (ok1) {
        unsigned char* to = dst + (128 + lane) * CB;
        cp_async<CB>(to, kt + off1 + lane * CB);
        cp_async<CB>(to + 32 * CB, kt + off1 + (32 + lane) * CB);
        cp_async<CB>(to + 64 * CB, vt + off1 + lane * CB);
        cp_async<CB>(to + 96 * CB, vt + off1 + (32 + lane) * CB);
      }
      if (lane < 16 && (lane < 8 ? ok0 : ok1))
        cp_async<16>(dst + par_dst, par_src + (lane < 8 ? off0 : off1));
    }
    cp_async_commit();  // a group per step, also an empty one: the waits count groups
  };
  for (int j = 0; j < STAGES - 1; ++j) issue(j, j);
  st.begin(a.scale_log2);

  int stg = 0;
  for (int j = 0; j < pairs; ++j) {
    cp_async_wait<STAGES - 2>();
    // publishes the parameters that other lanes copied, and orders this step's
    // copies behind every lane's reads of the stage they go to (step j - 1's)
    __syncwarp();
    const int next = stg == 0 ? STAGES - 1 : stg - 1;
    issue(j + STAGES - 1, next);
    const unsigned char* codes = ring + stg * Stage::kBytes;
    const uint32_t got = (copied >> (2 * stg)) & 3u;
    const int b0 = first + j * stride;
    const int v0 = (got & 1u) ? ctx - b0 * kBlockSize : 0;
    const int v1 = (got & 2u) ? ctx - (b0 + 1) * kBlockSize : 0;
    if (v0 >= kBlockSize && v1 >= kBlockSize)
      st.template step<false>(codes, codes + Stage::kParOff, kBlockSize, kBlockSize);
    else if (got)
      st.template step<true>(codes, codes + Stage::kParOff, v0, v1);
    stg = stg == STAGES - 1 ? 0 : stg + 1;
  }
  cp_async_wait<0>();

  __syncthreads();
  float* red_m = reinterpret_cast<float*>(smem);  // [WARPS][G]
  float* red_l = red_m + WARPS * G;                // [WARPS][G]
  float* red_acc = red_l + WARPS * G;              // [WARPS][G][D]
  st.to_red(red_m, red_l, red_acc, warp);
  __syncthreads();
  if (a.warp_parts)
    store_cta_state<D, G, WARPS>(a, red_m, red_l, red_acc, s, kvh, blockIdx.y);
  else
    finish_partition<T, D, G, WARPS>(a, red_m, red_m, red_l, red_acc, s, kvh, part, nparts,
                                     out_rows);
}

template <typename T, int D, int G>
cudaError_t launch_int4(const DecodeArgs& a, cudaStream_t stream) {
  constexpr int WARPS = kInt4Warps;
  const size_t ring = size_t(WARPS) * kInt4Stages * Int4Stage<D>::kBytes;
  const size_t red = size_t(WARPS) * G * (D + 2) * sizeof(float);
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
  const int y = a.warp_parts ? (a.max_parts + WARPS - 1) / WARPS : a.max_parts;
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
