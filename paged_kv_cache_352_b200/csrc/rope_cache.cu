// Writing new tokens into a paged cache with the rotary position embedding
// applied on the way (sm_100a), writes into 4-bit caches, and the read-back of
// 4-bit rows.
//
// A token at position p turns the pairs (a, b) of the first R = rotary_dim
// elements of each query and key row by the angles of its row of the cos/sin
// table: a' = a cos - b sin, b' = b cos + a sin, pairs (i, i + R/2) or, when
// interleaved, (2i, 2i + 1). The rotated queries go to q_out, the rotated keys
// and the values as they are into the cache slots, so that keys are read and
// written once. fp32 throughout, every operation rounded by itself (no
// contraction): the bits of a cache then do not depend on how a compiler fuses.
//
// The call moves bytes: per token 2 d (2 Hq + 2 Hkv) of input and output rows
// plus the cache rows, against 3 flops per rotated element. A row is covered by
// d/16 lanes of two 8-element chunks: for half-split pairs a lane takes the
// chunks at 8u and R/2 + 8u, for adjacent pairs 16u and 16u + 8, and in both it
// needs the table entries 8u .. 8u + 7 of cos and of sin. Those are loaded once
// per lane and used for every row the lane turns. What costs time beside the bytes are
// the chains slot -> place and position -> angles -> row: the first rows are loaded before
// them, and further rows while the ones before are turned.
//
// Measured (inputs that rotate over four sets): 16384 tokens of 32 + 8 heads, d = 128, 16-bit:
// 67.6 us, 6.1 TB/s (94 % of a copy), into E4M3 76, into 4 bits 76; 4096 tokens 21.6 us
// (15.9 at the copy rate), into E4M3 25.1 (14.6; every element is divided by the scale,
// IEEE, as the format's codes are defined), into 4 bits 24.6 (14.0), written in 4 bits without
// queries 10.7 (3.3), read back 6.7 (3.3). 4096 tokens are 1536 CTAs, 1.7 to 2.1 times what is
// resident at once: every wave starts with the chain of lookups, and the last is part filled.
#include <cuda_runtime.h>

#include <type_traits>

#include "int4_cache.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kRopeThreads = 128;

// Rows of each token that a lane group holds at once (as many again are on their way), and
// CTAs per SM (96 or 80 registers). 4096 tokens of 32 + 8 heads, five and six CTAs, in one run
// (its figures are 5 % below those above): E4M3 24.9 and 23.7 us, 4 bits 23.7 and 23.2 us;
// 16-bit, 16384 tokens: 69.5 and 71.0 us. Four rows loaded at once and none ahead took 27.4,
// 25.1 and 69.1 us.
template <typename C>
struct RopeShape {
  static constexpr int kUnroll = 2, kCtasPerSm = 5;
};
template <>
struct RopeShape<E4M3> {
  static constexpr int kUnroll = 2, kCtasPerSm = 6;
};
template <>
struct RopeShape<Int4> {
  static constexpr int kUnroll = 2, kCtasPerSm = 6;
};

template <typename T>
__device__ __forceinline__ uint4 from_f32x8(const float* f) {
  T r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = Storage<T>::from_f32(f[e]);
  uint4 u;
  memcpy(&u, r, sizeof(u));
  return u;
}

__device__ __forceinline__ uint2 to_e4m3x8(const float* f, float scale) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float* g = f + 4 * i;
    const uint32_t p0 = f32x2_to_e4m3x2(__fdiv_rn(g[0], scale), __fdiv_rn(g[1], scale));
    const uint32_t p1 = f32x2_to_e4m3x2(__fdiv_rn(g[2], scale), __fdiv_rn(g[3], scale));
    w[i] = (p0 & 0xffffu) | (p1 << 16);
  }
  return make_uint2(w[0], w[1]);
}

// The pair (a, b) turned by an angle's (c, s); every operation rounded by itself.
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// T: type of q, key, value. C: cache element (T, E4M3 or Int4). A warp serves two
// neighbouring tokens: half of its d/16-lane groups the even one, half the odd one.
// `splits` warps share their rows (Hq query, Hkv key, Hkv value rows, in this order).
// Two tokens because of the 4-bit value tiles, which interleave the bytes of a slot
// pair: when the two tokens fill such a pair, as a prompt's do, their lanes exchange
// halves and each stores 8 bytes where one token alone would store 2 bytes in four
// places (4096 tokens of 8 heads: 15.4 -> 10.2 us).
template <typename T, typename C, int D>
__global__ void __launch_bounds__(kRopeThreads, RopeShape<C>::kCtasPerSm)
    rope_and_cache_kernel(const RopeArgs r, int splits, int rows_per_warp) {
  grid_dependency_wait();
  allow_dependents();
  constexpr int LANES = D / 16;        // lanes of a row
  constexpr int kUnroll = RopeShape<C>::kUnroll;
  constexpr int RPW = 32 / LANES / 2;  // rows of each token a warp handles at a time
  const int64_t warp = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int u = lane % LANES, sub = lane / LANES;
  const int64_t pair = warp / splits;
  if (2 * pair >= r.num_tokens) return;
  const int split = (int)(warp - pair * splits);
  const int rows = r.num_q_heads + 2 * r.num_kv_heads;
  const int row_begin = split * rows_per_warp;
  const int row_end = min(rows, row_begin + rows_per_warp);
  const int64_t t = 2 * pair + (sub & 1);
  const bool first_lane = split == 0 && u == 0 && sub < 2;  // of its token, to report

  const bool rot = u < r.rotary_dim / 16;
  const bool halves = rot && !r.interleaved;
  // the lane's chunks of a query or key row; of a value row they are 16u, 16u + 8
  const int off_a = halves ? 8 * u : 16 * u;
  const int off_b = halves ? r.rotary_dim / 2 + 8 * u : 16 * u + 8;
  auto fetch = [&](int base, uint4(&raw)[kUnroll][2]) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int row = base + i * RPW + (sub >> 1);
      raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= row_end || t >= r.num_tokens) continue;
      const T* src;
      int oa = off_a, ob = off_b;
      if (row < r.num_q_heads) {
        src = static_cast<const T*>(r.q) + t * r.q_stride + (int64_t)row * D;
      } else {
        const int h = row - r.num_q_heads;
        if (h < r.num_kv_heads) {
          src = static_cast<const T*>(r.key) + t * r.key_stride + (int64_t)h * D;
        } else {
          src = static_cast<const T*>(r.value) + t * r.value_stride +
                (int64_t)(h - r.num_kv_heads) * D;
          oa = 16 * u;
          ob = 16 * u + 8;
        }
      }
      raw[i][0] = *reinterpret_cast<const uint4*>(src + oa);
      raw[i][1] = *reinterpret_cast<const uint4*>(src + ob);
    }
  };
  // the first rows are on their way while slot, position and angles are looked up
  uint4 raw[kUnroll][2];
  fetch(row_begin, raw);

  bool live = t < r.num_tokens;  // whether anything of this lane's token is written
  const int64_t slot = live ? __ldg(r.slot_mapping + t) : -1;
  bool store = slot >= 0;  // whether its rows are cached
  if (slot >= r.num_slots) {
    store = false;
    if (first_lane) report(r.dev_error, PA_DEVERR_SLOT_RANGE);
  }

  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (r.rotary_dim > 0 && live) {
    const int64_t p = __ldg(r.positions + t);
    if (p < 0 || p >= r.num_positions) {  // nothing of this token is written
      if (first_lane) report(r.dev_error, PA_DEVERR_POSITION);
      live = store = false;
    } else if (rot) {
      const float* row = r.cos_sin + p * r.rotary_dim + 8 * u;
      const float4 c0 = __ldg(reinterpret_cast<const float4*>(row));
      const float4 c1 = __ldg(reinterpret_cast<const float4*>(row) + 1);
      const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + r.rotary_dim / 2));
      const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + r.rotary_dim / 2) + 1);
      cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
      cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
      sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
      sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }
  }
  const int64_t block = store ? slot / kBlockSize : 0;
  const int tok = store ? (int)(slot - block * kBlockSize) : 0;
  // whether the two tokens fill slots 2i and 2i + 1 (of one block, then): uniform
  bool paired = false;
  if constexpr (std::is_same<C, Int4>::value) {
    const int64_t other = __shfl_xor_sync(0xffffffffu, store ? slot : -4, LANES);
    paired = __all_sync(0xffffffffu, store && (slot ^ 1) == other && (int)(slot & 1) == (sub & 1));
  }
  // places inside a 4-bit tile: this token's key row, its values' first two bytes, and the
  // 8 bytes of the pair that this lane stores when both tokens are there
  const int odd8 = (sub & 1) ? 8 : 0;
  const int k_place = tok * (D / 2);
  const int v_place = int4_value_byte<D>(tok, 16 * u);
  const int pair_place = int4_value_byte<D>(tok & ~1, 16 * u + odd8);

  for (int base = row_begin; base < row_end; base += RPW * kUnroll) {
    uint4 next[kUnroll][2];
    if (base + RPW * kUnroll < row_end) fetch(base + RPW * kUnroll, next);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int first = base + i * RPW;
      if (first >= row_end) break;  // uniform across the warp
      const int row = first + (sub >> 1);
      const bool in = live && row < row_end;
      const bool is_q = row < r.num_q_heads;
      const bool is_v = row >= r.num_q_heads + r.num_kv_heads;
      float f[16];
      Storage<T>::to_f32(raw[i][0], *reinterpret_cast<float(*)[8]>(&f[0]));
      Storage<T>::to_f32(raw[i][1], *reinterpret_cast<float(*)[8]>(&f[8]));
      if (rot && !is_v) {
        if (halves) {
#pragma unroll
          for (int e = 0; e < 8; ++e) rotate(f[e], f[8 + e], cs[e], sn[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) rotate(f[2 * e], f[2 * e + 1], cs[e], sn[e]);
        }
      }
      if (in && is_q) {
        T* dst = static_cast<T*>(r.q_out) + t * r.q_out_stride + (int64_t)row * D;
        *reinterpret_cast<uint4*>(dst + off_a) = from_f32x8<T>(f);
        *reinterpret_cast<uint4*>(dst + off_b) = from_f32x8<T>(f + 8);
      }
      if (first + RPW <= r.num_q_heads) continue;  // the warp holds query rows only
      const int h = row - r.num_q_heads - (is_v ? r.num_kv_heads : 0);
      const int64_t tile = block * r.num_kv_heads + h;
      const int oa = is_v ? 16 * u : off_a, ob = is_v ? 16 * u + 8 : off_b;
      const bool write = in && !is_q && store;
      if constexpr (std::is_same<C, Int4>::value) {
        uint32_t codes[2];
        const uint32_t par = int4_quantize_row<LANES>(f, codes);
        // the even token's lane takes the pair's first 8 dimensions, the odd one's the other 8
        const bool odd = sub & 1;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? codes[0] : codes[1], LANES);
        if (write) {
          unsigned char* dst =
              static_cast<unsigned char*>(is_v ? r.v_cache : r.k_cache) + tile * int4_tile_bytes(D);
          if (is_v && paired) {
            const uint32_t even_codes = odd ? got : codes[0], odd_codes = odd ? codes[1] : got;
            *reinterpret_cast<uint2*>(dst + pair_place) =
                make_uint2(__byte_perm(even_codes, odd_codes, 0x5410),
                           __byte_perm(even_codes, odd_codes, 0x7632));
          } else if (is_v) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint16_t*>(dst + v_place + int4_value_step<D>(q)) =
                  (uint16_t)(codes[q >> 1] >> (16 * (q & 1)));
          } else {
            *reinterpret_cast<uint32_t*>(dst + k_place + oa / 2) = codes[0];
            *reinterpret_cast<uint32_t*>(dst + k_place + ob / 2) = codes[1];
          }
          if (u == 0) *reinterpret_cast<uint32_t*>(dst + 8 * D + 4 * tok) = par;
        }
      } else if constexpr (std::is_same<C, E4M3>::value) {
        if (write) {
          unsigned char* dst = static_cast<unsigned char*>(is_v ? r.v_cache : r.k_cache) +
                               (tile * kBlockSize + tok) * D;
          const float scale = is_v ? r.v_scale : r.k_scale;
          *reinterpret_cast<uint2*>(dst + oa) = to_e4m3x8(f, scale);
          *reinterpret_cast<uint2*>(dst + ob) = to_e4m3x8(f + 8, scale);
        }
      } else {
        if (write) {
          T* dst = static_cast<T*>(is_v ? r.v_cache : r.k_cache) + (tile * kBlockSize + tok) * D;
          // value rows and elements past rotary_dim keep their bits
          *reinterpret_cast<uint4*>(dst + oa) = rot && !is_v ? from_f32x8<T>(f) : raw[i][0];
          *reinterpret_cast<uint4*>(dst + ob) = rot && !is_v ? from_f32x8<T>(f + 8) : raw[i][1];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      raw[i][0] = next[i][0];
      raw[i][1] = next[i][1];
    }
  }
}

// One lane group of d/16 lanes per (token, KV head, K or V) row: 16 codes a lane.
template <typename T, int D>
__global__ void __launch_bounds__(256)
    read_slots_int4_kernel(T* key, T* value, int64_t key_stride, int64_t value_stride,
                           const unsigned char* __restrict__ k_cache,
                           const unsigned char* __restrict__ v_cache,
                           const int64_t* __restrict__ slot_mapping, int64_t total,
                           int num_kv_heads, int64_t num_slots, int* dev_error) {
  grid_dependency_wait();
  allow_dependents();
  constexpr int LANES = D / 16;
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= total) return;
  const int u = (int)(idx % LANES);
  const int64_t row = idx / LANES;
  const int64_t t = row / (2 * num_kv_heads);
  int h = (int)(row - t * 2 * num_kv_heads);
  const int64_t slot = __ldg(slot_mapping + t);
  if (slot < 0) return;
  if (slot >= num_slots) {
    if (u == 0 && h == 0) report(dev_error, PA_DEVERR_SLOT_RANGE);
    return;
  }
  const bool is_v = h >= num_kv_heads;
  if (is_v) h -= num_kv_heads;
  const int64_t block = slot / kBlockSize;
  const int tok = (int)(slot - block * kBlockSize);
  const unsigned char* tile =
      (is_v ? v_cache : k_cache) + (block * num_kv_heads + h) * int4_tile_bytes(D);
  uint32_t w[2];
  if (is_v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = *reinterpret_cast<const uint16_t*>(
          tile + int4_value_byte<D>(tok, 16 * u + 8 * i));
      const uint32_t hi = *reinterpret_cast<const uint16_t*>(
          tile + int4_value_byte<D>(tok, 16 * u + 8 * i + 4));
      w[i] = lo | (hi << 16);
    }
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(tile + tok * (D / 2) + 8 * u);
    w[0] = v.x;
    w[1] = v.y;
  }
  const float2 p =
      half2_bits_to_float2(*reinterpret_cast<const uint32_t*>(tile + 8 * D + 4 * tok));
  float f[16];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    f[e] = fmaf((float)((w[e >> 3] >> (4 * (e & 7))) & 15u) - 7.5f, p.x, p.y);
  T* dst = is_v ? value + t * value_stride : key + t * key_stride;
  uint4* out = reinterpret_cast<uint4*>(dst + (int64_t)h * D + 16 * u);
  out[0] = from_f32x8<T>(f);
  out[1] = from_f32x8<T>(f + 8);
}

template <typename T, typename C, int D>
cudaError_t launch_rope_typed(const RopeArgs& r, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16) / 2;
  const int rows = r.num_q_heads + 2 * r.num_kv_heads;
  if (r.num_tokens == 0 || rows == 0) return cudaSuccess;
  // Warps that share a token pair's rows: one per RPW rows while the tokens alone do
  // not give the 148 SMs 32 warps each, fewer as tokens grow (a warp that keeps
  // a pair's rows looks up its slot, position and angles once). With 64 and 48 instead:
  // 16384 tokens, 16-bit, 70.1 and 67.7 us against 67.7; 1237 tokens into E4M3 6.0 and 6.0
  // us against 5.1.
  const int groups = (rows + RPW - 1) / RPW;
  const long long pairs = ((long long)r.num_tokens + 1) / 2;
  const long long target = 148 * 32;
  long long splits = (target + pairs - 1) / pairs;
  if (splits > groups) splits = groups;
  const int per = (int)((groups + splits - 1) / splits);
  const int used = (groups + per - 1) / per;
  const long long ctas = (pairs * used + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(rope_and_cache_kernel<T, C, D>, dim3((unsigned)ctas), dim3(kRopeThreads),
                          0, stream, r, used, per * RPW);
}

template <typename T, typename C>
cudaError_t launch_rope_d(const RopeArgs& r, int head_dim, cudaStream_t stream) {
  return head_dim == 64 ? launch_rope_typed<T, C, 64>(r, stream)
                        : launch_rope_typed<T, C, 128>(r, stream);
}

template <typename T>
cudaError_t launch_rope_t(const RopeArgs& r, int head_dim, int cache_dtype, cudaStream_t stream) {
  switch (cache_dtype) {
    case PA_INT4: return launch_rope_d<T, Int4>(r, head_dim, stream);
    case PA_FP8_E4M3: return launch_rope_d<T, E4M3>(r, head_dim, stream);
    default: return launch_rope_d<T, T>(r, head_dim, stream);
  }
}

template <typename T, int D>
cudaError_t launch_read_typed(void* key, void* value, int64_t key_stride, int64_t value_stride,
                              const void* k_cache, const void* v_cache,
                              const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                              int num_blocks, int* dev_error, cudaStream_t stream) {
  const int64_t total = (int64_t)num_tokens * 2 * num_kv_heads * (D / 16);
  if (total == 0) return cudaSuccess;
  const int64_t ctas = (total + 255) / 256;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_dependent(read_slots_int4_kernel<T, D>, dim3((unsigned)ctas), dim3(256), 0, stream,
                          static_cast<T*>(key), static_cast<T*>(value), key_stride, value_stride,
                          static_cast<const unsigned char*>(k_cache),
                          static_cast<const unsigned char*>(v_cache), slot_mapping, total,
                          num_kv_heads, (int64_t)num_blocks * kBlockSize, dev_error);
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeArgs& r, int head_dim, int dtype, int cache_dtype,
                                  cudaStream_t stream) {
  return dtype == PA_F16 ? launch_rope_t<__half>(r, head_dim, cache_dtype, stream)
                         : launch_rope_t<__nv_bfloat16>(r, head_dim, cache_dtype, stream);
}

cudaError_t launch_read_slots_int4(void* key, void* value, int64_t key_stride,
                                   int64_t value_stride, const void* k_cache, const void* v_cache,
                                   const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                                   int head_dim, int num_blocks, int dtype, int* dev_error,
                                   cudaStream_t stream) {
  auto fn = dtype == PA_F16
                ? (head_dim == 64 ? launch_read_typed<__half, 64> : launch_read_typed<__half, 128>)
                : (head_dim == 64 ? launch_read_typed<__nv_bfloat16, 64>
                                  : launch_read_typed<__nv_bfloat16, 128>);
  return fn(key, value, key_stride, value_stride, k_cache, v_cache, slot_mapping, num_tokens,
            num_kv_heads, num_blocks, dev_error, stream);
}

}  // namespace pa
