// Beam search's selection (sm_100a): the best continuations over the beams of a
// sequence and the vocabulary.
//
//   score[k][v] = beam_score[k] + x[k][v] - logsumexp_v x[k],
//   the N largest of the K V scores of a sequence, ties to the smallest k V + v.
//
// The logits are read once: 2 or 4 bytes each, against one exponential, a
// comparison and an addition. A row's ranking does not need its logsumexp, so one
// CTA takes a tile of a row (kept in registers) and leaves the tile's maximum, its
// sum of exponentials and its N largest logits in the workspace; then one CTA per
// sequence adds up the rows' sums and ranks K x tiles x N candidates. For little
// work that is the CTA that finishes the sequence's last tile (4 beams of 32000
// logits: 10.3 us a call instead of 12.9 us with a second launch); for much work it
// is a second launch, since every tile would wait for the release of its results
// (64 x 8 beams of 131072 logits: 41.8 us instead of 47.6 us).
//
// The N largest of a tile without sorting it: the N-th largest of the maxima of
// kGroups groups of elements bounds the N-th largest element from below, so the few
// elements at or above it are collected in shared memory and ranked by counting,
// for each, those before it. Where ties make too many (a tile of equal logits) the N
// are taken one by one instead; either way the order is (value descending, index
// ascending), and a result does not depend on the order of the atomics.
//
// Scores are formed and ranked in double precision: neighbouring candidates of
// different beams are often closer than fp32 scores resolve. The exponentials'
// sums are fp32 per thread (at most kPer terms), double from there on.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kGroups = 64;       // groups of a tile whose maxima bound the N-th largest
constexpr int kTileCap = 2048;    // candidates a tile ranks at once
constexpr int kMergeCap = 1024;   // candidates a sequence ranks at once

// Floats in the order of unsigned integers (NaN aside).
__device__ __forceinline__ uint32_t orderable(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_orderable(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// (value, index) as one key: larger is better, ties to the smaller index. 0 is
// below every candidate. -0 counts as 0.
__device__ __forceinline__ uint64_t make_key(float x, uint32_t index) {
  return ((uint64_t)orderable(__fadd_rn(x, 0.f)) << 32) | (uint32_t)~index;
}

// A 16-byte load of logits: kPerLoad of them, kept packed in registers (a tile of
// 64 16-bit logits a thread is 32 registers, and four CTAs fit an SM).
template <typename T>
struct Logits {
  static constexpr int kPerLoad = 8;
  static __device__ __forceinline__ void widen(const uint4& u, float (&f)[8]) {
    Storage<T>::to_f32(u, f);
  }
  static __device__ __forceinline__ float one(const T* p) { return static_cast<float>(*p); }
  // the largest (NaN ignored), two at a time
  static __device__ __forceinline__ float largest(const uint4& u) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                         __nv_bfloat162>::type;
    T2 h[4];
    memcpy(h, &u, sizeof(u));
    const T2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(static_cast<float>(m.x), static_cast<float>(m.y));
  }
  static __device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
    T r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = Storage<T>::from_f32(f[e]);
    uint4 u;
    memcpy(&u, r, sizeof(u));
    return u;
  }
};
template <>
struct Logits<float> {
  static constexpr int kPerLoad = 4;
  static __device__ __forceinline__ void widen(const uint4& u, float (&f)[4]) {
    memcpy(f, &u, sizeof(u));
  }
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ float largest(const uint4& u) {
    float f[4];
    widen(u, f);
    return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
  }
  static __device__ __forceinline__ uint4 narrow(const float (&f)[4]) {
    uint4 u;
    memcpy(&u, f, sizeof(u));
    return u;
  }
};

// The workspace's parts.
struct Work {
  int* done;       // [num_seqs] tiles finished, back to 0 after the merge (small tiles)
  float* max;      // [rows][tiles]
  float* sum;      // [rows][tiles]
  uint64_t* keys;  // [rows][tiles][select], best first, 0 past the candidates
};

// Candidates are ordered by score, ties to the smaller flat index.
__device__ __forceinline__ bool before(double s, int64_t f, double t, int64_t g) {
  return s > t || (s == t && f < g);
}

// Sequence b by one CTA: its rows' logsumexp, then its best candidates. `buffer`: shared
// memory of kMergeCap (double, int64) pairs. The tiles' results were written by other
// CTAs: they are read past L1.
template <int kMergeThreads>
__device__ __forceinline__ void merge_sequence(const BeamArgs& a, const Work& work, int tiles,
                                               int b, uint64_t* buffer) {
  constexpr int kWarps = kMergeThreads / 32;
  // a score is (x - largest) + offset: offset is the beam score less the logarithm of the
  // sum of exponentials relative to the row's largest logit, -inf for a dead beam
  __shared__ double offset[PA_BEAM_MAX];
  __shared__ float largest[PA_BEAM_MAX];
  double* cs = reinterpret_cast<double*>(buffer);
  int64_t* cf = reinterpret_cast<int64_t*>(buffer + kMergeCap);
  const int beams = a.num_beams, vocab = a.vocab, select = a.select;
  const float* tile_max = work.max;
  const float* tile_sum = work.sum;
  const uint64_t* tile_keys = work.keys;
  __shared__ double group_max[kGroups];
  __shared__ double warp_best[kWarps];
  __shared__ int count;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_beam = tiles * select;
  const int total = beams * per_beam;
  // this thread's first candidates, on their way while the rows' sums are added up
  constexpr int kAhead = 4;
  uint64_t ahead[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = threadIdx.x + j * kMergeThreads;
    ahead[j] = i < total ? __ldcg(tile_keys + (size_t)b * total + i) : 0;
  }
  for (int k = warp; k < beams; k += kWarps) {
    const size_t row = (size_t)b * beams + k;
    float M = -INFINITY;
    for (int t = lane; t < tiles; t += 32) M = fmaxf(M, __ldcg(tile_max + row * tiles + t));
#pragma unroll
    for (int mask = 16; mask > 0; mask >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, mask));
    double S = 0.0;
    for (int t = lane; t < tiles; t += 32) {
      const float m = __ldcg(tile_max + row * tiles + t), s = __ldcg(tile_sum + row * tiles + t);
      if (m > -INFINITY || s != s) S += (double)s * exp((double)m - (double)M);
    }
#pragma unroll
    for (int mask = 16; mask > 0; mask >>= 1) S += __shfl_xor_sync(0xffffffffu, S, mask);
    if (lane == 0) {
      const float beam = a.beam_scores[row];
      double o = -INFINITY;
      if (M > -INFINITY || S != S) o = M < INFINITY ? (double)beam - log(S) : NAN;
      if (o != o || o == INFINITY) {  // a NaN or +inf among the logits, or as beam score
        report(a.dev_error, PA_DEVERR_LOGITS);
        o = -INFINITY;
      }
      offset[k] = o;
      largest[k] = M;
    }
  }
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  auto score_key = [&](int i, uint64_t key, double& s, int64_t& f) {
    const int k = i / per_beam;
    s = -INFINITY;
    f = INT64_MAX;
    if (key != 0 && offset[k] > -INFINITY) {
      s = ((double)from_orderable((uint32_t)(key >> 32)) - (double)largest[k]) + offset[k];
      f = (int64_t)k * vocab + (uint32_t)~(uint32_t)key;
    }
  };
  auto score_of = [&](int i, double& s, int64_t& f) {
    score_key(i, __ldcg(tile_keys + (size_t)b * total + i), s, f);
  };
  // as in a tile: the select-th largest of 64 groups' maxima bounds the result from below
  double top = -INFINITY;
  double as[kAhead];
  int64_t af[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    as[j] = -INFINITY;
    const int i = threadIdx.x + j * kMergeThreads;
    if (i < total) score_key(i, ahead[j], as[j], af[j]);
    top = as[j] > top ? as[j] : top;
  }
  for (int i = threadIdx.x + kAhead * kMergeThreads; i < total; i += kMergeThreads) {
    double s;
    int64_t f;
    score_of(i, s, f);
    top = s > top ? s : top;
  }
  constexpr int kGroupLanes = kMergeThreads / kGroups;
#pragma unroll
  for (int mask = 1; mask < kGroupLanes; mask <<= 1)
    top = fmax(top, __shfl_xor_sync(0xffffffffu, top, mask));  // (never NaN)
  if (threadIdx.x % kGroupLanes == 0) group_max[threadIdx.x / kGroupLanes] = top;
  __syncthreads();
  {
    // kGroupLanes threads count for each group
    const double p = group_max[threadIdx.x / kGroupLanes];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kGroups / kGroupLanes; ++i)
      rank += group_max[i * kGroupLanes + threadIdx.x % kGroupLanes] >= p;
#pragma unroll
    for (int mask = 1; mask < kGroupLanes; mask <<= 1)
      rank += __shfl_xor_sync(0xffffffffu, rank, mask);
    double best = rank >= select ? p : -INFINITY;
#pragma unroll
    for (int mask = 16; mask >= kGroupLanes; mask >>= 1) {
      const double o = __shfl_xor_sync(0xffffffffu, best, mask);
      best = o > best ? o : best;
    }
    if (lane == 0) warp_best[warp] = best;
  }
  __syncthreads();
  double lowest = warp_best[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) lowest = warp_best[w] > lowest ? warp_best[w] : lowest;
  auto collect = [&](double s, int64_t f) {
    if (s > -INFINITY && s >= lowest) {
      const int at = atomicAdd(&count, 1);
      if (at < kMergeCap) {
        cs[at] = s;
        cf[at] = f;
      }
    }
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) collect(as[j], af[j]);
  for (int i = threadIdx.x + kAhead * kMergeThreads; i < total; i += kMergeThreads) {
    double s;
    int64_t f;
    score_of(i, s, f);
    collect(s, f);
  }
  __syncthreads();
  const int n = count;
  const size_t out = (size_t)b * select;
  auto put = [&](int rank, double s, int64_t f) {
    a.scores[out + rank] = (float)s;
    a.parents[out + rank] = s > -INFINITY ? (int32_t)(f / vocab) : -1;
    a.tokens[out + rank] = s > -INFINITY ? (int32_t)(f % vocab) : -1;
  };
  if (n <= kMergeCap) {
    for (int i = threadIdx.x; i < n; i += kMergeThreads) {
      const double s = cs[i];
      const int64_t f = cf[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += before(cs[j], cf[j], s, f);
      if (rank < select) put(rank, s, f);
    }
    for (int i = n + threadIdx.x; i < select; i += kMergeThreads) put(i, -INFINITY, 0);
    return;
  }
  // more equal candidates than the buffer holds: one at a time
  __shared__ double bs[kWarps];
  __shared__ int64_t bf[kWarps];
  double ls = INFINITY;
  int64_t lf = -1;
  for (int r = 0; r < select; ++r) {
    double s = -INFINITY;
    int64_t f = INT64_MAX;
    for (int i = threadIdx.x; i < total; i += kMergeThreads) {
      double t;
      int64_t g;
      score_of(i, t, g);
      if (t > -INFINITY && before(ls, lf, t, g) && before(t, g, s, f)) {
        s = t;
        f = g;
      }
    }
#pragma unroll
    for (int mask = 16; mask > 0; mask >>= 1) {
      const double t = __shfl_xor_sync(0xffffffffu, s, mask);
      const int64_t g = __shfl_xor_sync(0xffffffffu, f, mask);
      if (before(t, g, s, f)) {
        s = t;
        f = g;
      }
    }
    __syncthreads();
    if (lane == 0) {
      bs[warp] = s;
      bf[warp] = f;
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
      if (before(bs[w], bf[w], s, f)) {
        s = bs[w];
        f = bf[w];
      }
    if (threadIdx.x == 0) put(r, s, f);
    ls = s;
    lf = f;
  }
}

constexpr int kMergeThreads = 512;

__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const BeamArgs a, const Work work, int tiles) {
  grid_dependency_wait();
  allow_dependents();
  __shared__ uint64_t buffer[2 * kMergeCap];
  merge_sequence<kMergeThreads>(a, work, tiles, blockIdx.x, buffer);
}

// One tile of one row: kBeamThreads threads x LOADS 16-byte loads. MERGE: the CTA
// of a sequence's last tile merges it.
template <typename T, int LOADS, bool MERGE>
__global__ void __launch_bounds__(kBeamThreads, 4)
    beam_tile_kernel(const BeamArgs a, const Work work, int tiles) {
  grid_dependency_wait();
  allow_dependents();
  constexpr int EPL = Logits<T>::kPerLoad;
  constexpr int kPer = EPL * LOADS;
  constexpr int kWarps = kBeamThreads / 32;
  __shared__ __align__(16) uint32_t group_max[kGroups];
  __shared__ float warp_max[kWarps], warp_sum[kWarps];
  __shared__ uint64_t cand[kTileCap];
  __shared__ uint32_t threshold;
  __shared__ int count;
  const int row = blockIdx.x / tiles, tile = blockIdx.x - row * tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vocab = a.vocab, select = a.select;
  const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
  const int base = tile * kBeamThreads * kPer;
  // element e of load i of this thread: index base + (i * kBeamThreads + thread) EPL + e;
  // past the row: -inf, which is never a candidate and adds nothing
  auto load = [&](int at) {
    if (at + EPL <= vocab) return __ldg(reinterpret_cast<const uint4*>(x + at));
    float f[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) f[e] = at + e < vocab ? Logits<T>::one(x + at + e) : -INFINITY;
    return Logits<T>::narrow(f);
  };
  uint4 u[LOADS];
  if (base + kBeamThreads * kPer <= vocab) {  // the whole tile: one address, no tests
    const uint4* from = reinterpret_cast<const uint4*>(x + base) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) u[i] = __ldg(from + i * kBeamThreads);
  } else {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      u[i] = load(base + (i * kBeamThreads + (int)threadIdx.x) * EPL);
  }
  if (threadIdx.x == 0) {
    count = 0;
    threshold = 0;
  }
  float load_max[LOADS];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    load_max[i] = Logits<T>::largest(u[i]);
    mx = fmaxf(mx, load_max[i]);
  }
  // groups of four neighbouring lanes
  float gm = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
  if ((lane & 3) == 0) group_max[threadIdx.x >> 2] = orderable(gm);
  float wm = gm;
#pragma unroll
  for (int mask = 4; mask <= 16; mask <<= 1)
    wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, mask));
  __syncthreads();
  {
    // the select-th largest of the groups' maxima: the largest value with at least
    // `select` maxima at or above it; four threads count for each group
    const uint32_t g = group_max[threadIdx.x >> 2];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kGroups / 4; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(group_max + 4 * i + 4 * (lane & 3));
      rank += (v.x >= g) + (v.y >= g) + (v.z >= g) + (v.w >= g);
    }
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    const uint32_t best = __reduce_max_sync(0xffffffffu, rank >= select ? g : 0u);
    if (lane == 0) atomicMax(&threshold, best);
  }
  // sum of exponentials relative to the warp's maximum; a NaN makes it NaN
  const float ref = wm == -INFINITY ? 0.f : wm;
  constexpr float kLog2e = 1.4426950408889634f;
  float even = 0.f, odd = 0.f;  // summed in pairs by packed fp32 instructions
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    float f[EPL];
    Logits<T>::widen(u[i], f);
#pragma unroll
    for (int e = 0; e < EPL; e += 2) {
      // (x - ref) log2 e: the difference first, so that a row of the type's lowest or
      // largest values is as exact as another
      float p = f[e], q = f[e + 1];
      fadd2(p, q, -ref, -ref);
      fmul2(p, q, kLog2e);
      fadd2(even, odd, fast_exp2(p), fast_exp2(q));
    }
  }
  float sum = even + odd;
#pragma unroll
  for (int mask = 1; mask <= 16; mask <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, mask);
  if (lane == 0) {
    warp_max[warp] = wm;
    warp_sum[warp] = sum;
  }
  __syncthreads();
  const float lowest = from_orderable(threshold);
  // The few loads that hold candidates are read again (they are in L2): a loop over
  // them is a fraction of the code that 64 tests in registers unroll to, and the
  // instruction cache is what such code waits for.
  uint32_t hits = 0;
#pragma unroll
  for (int i = 0; i < LOADS; ++i) hits |= (load_max[i] >= lowest ? 1u : 0u) << i;
#pragma unroll 1
  while (hits) {
    const int i = __ffs(hits) - 1;
    hits &= hits - 1;
    const int at = base + (i * kBeamThreads + (int)threadIdx.x) * EPL;
    float f[EPL];
    Logits<T>::widen(load(at), f);
    uint32_t in = 0;
#pragma unroll
    for (int e = 0; e < EPL; ++e) in |= (f[e] >= lowest && f[e] > -INFINITY ? 1u : 0u) << e;
    int c = in ? atomicAdd(&count, __popc(in)) : 0;
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      if ((in >> e) & 1u) {
        if (c < kTileCap) cand[c] = make_key(f[e], at + e);
        ++c;
      }
  }
  const size_t out = (size_t)row * tiles + tile;
  if (threadIdx.x == 0) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, warp_max[w]);
    float S = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      S += warp_sum[w] * (warp_max[w] == -INFINITY
                              ? 1.f
                              : expf(warp_max[w] - M));
    work.max[out] = M;
    work.sum[out] = S;
  }
  __syncthreads();
  uint64_t* keys = work.keys + out * select;
  auto take_one_by_one = [&]() {
    // more ties than the buffer holds: one at a time, each the largest below the last
    uint64_t last = ~0ull;
    uint64_t* best = cand;  // [kWarps]
    const int end = min(vocab, base + kBeamThreads * kPer);
    for (int r = 0; r < select; ++r) {
      uint64_t k = 0;
#pragma unroll 4
      for (int at = base + (int)threadIdx.x; at < end; at += kBeamThreads) {
        const float f = Logits<T>::one(x + at);
        const uint64_t c = make_key(f, at);
        if (f > -INFINITY && c < last && c > k) k = c;
      }
#pragma unroll
      for (int mask = 16; mask > 0; mask >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, k, mask);
        k = o > k ? o : k;
      }
      __syncthreads();
      if (lane == 0) best[warp] = k;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) k = best[w] > k ? best[w] : k;
      if (threadIdx.x == 0) keys[r] = k;
      last = k;
    }
  };
  const int n = count;
  if (n <= kTileCap) {
    for (int i = threadIdx.x; i < n; i += kBeamThreads) {
      const uint64_t k = cand[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += cand[j] > k;
      if (rank < select) keys[rank] = k;
    }
    for (int i = n + threadIdx.x; i < select; i += kBeamThreads) keys[i] = 0;
  } else {
    take_one_by_one();
  }

  if constexpr (MERGE) {
    // as the split-KV merge of the decode: the barrier makes the CTA's stores visible to
    // thread 0, whose gpu-scope acq_rel add publishes them
    __shared__ bool last_tile;
    const int seq = row / a.num_beams;
    __syncthreads();
    if (threadIdx.x == 0) {
      last_tile = atom_add_acq_rel_gpu(work.done + seq, 1) == a.num_beams * tiles - 1;
      if (last_tile) work.done[seq] = 0;
    }
    __syncthreads();
    if (last_tile) merge_sequence<kBeamThreads>(a, work, tiles, seq, cand);
  }
}

// Elements of a tile: 64 per thread (16-bit) or 32 (fp32) for large work, a
// quarter for little.
template <typename T>
constexpr int tile_elems(bool large) {
  return kBeamThreads * Logits<T>::kPerLoad * (large ? 8 : 2);
}

constexpr int kLargeTiles = 148 * 2;

bool large_tiles(int64_t rows, int vocab, int elem) {
  // enough large tiles for every SM to hold two CTAs
  const int64_t big = elem == 4 ? tile_elems<float>(true) : tile_elems<__half>(true);
  return rows * ((vocab + big - 1) / big) >= kLargeTiles;
}

}  // namespace

void beam_layout(int num_seqs, int num_beams, int vocab, int select, int dtype, BeamLayout* lay) {
  const int elem = dtype == PA_F32 ? 4 : 2;
  const int64_t rows = (int64_t)num_seqs * num_beams;
  const bool large = large_tiles(rows, vocab, elem);
  const int64_t per = elem == 4 ? tile_elems<float>(large) : tile_elems<__half>(large);
  lay->large = large;
  lay->tiles = (int)((vocab + per - 1) / per);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t n = (size_t)rows * lay->tiles;
  // small tiles only come with fewer sequences than kLargeTiles; the counters have a place
  // of their own whatever the sizes, so that no call leaves results where another counts
  lay->max_off = up(kLargeTiles * sizeof(int));
  lay->sum_off = lay->max_off + up(n * sizeof(float));
  lay->key_off = lay->sum_off + up(n * sizeof(float));
  lay->bytes = lay->key_off + up(n * select * sizeof(uint64_t));
}

cudaError_t launch_beam_select(const BeamArgs& a, int dtype, cudaStream_t stream) {
  BeamLayout lay;
  beam_layout(a.num_seqs, a.num_beams, a.vocab, a.select, dtype, &lay);
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  Work work;
  work.done = reinterpret_cast<int*>(ws);
  work.max = reinterpret_cast<float*>(ws + lay.max_off);
  work.sum = reinterpret_cast<float*>(ws + lay.sum_off);
  work.keys = reinterpret_cast<uint64_t*>(ws + lay.key_off);
  const int64_t ctas = (int64_t)lay.tiles * a.num_seqs * a.num_beams;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto go = [&](auto kern) {
    return launch_dependent(kern, dim3((unsigned)ctas), dim3(kBeamThreads), 0, stream, a, work,
                            lay.tiles);
  };
  if (!lay.large) {
    return dtype == PA_F32   ? go(beam_tile_kernel<float, 2, true>)
           : dtype == PA_F16 ? go(beam_tile_kernel<__half, 2, true>)
                             : go(beam_tile_kernel<__nv_bfloat16, 2, true>);
  }
  const cudaError_t e = dtype == PA_F32   ? go(beam_tile_kernel<float, 8, false>)
                        : dtype == PA_F16 ? go(beam_tile_kernel<__half, 8, false>)
                                          : go(beam_tile_kernel<__nv_bfloat16, 8, false>);
  if (e != cudaSuccess) return e;
  return launch_dependent(beam_merge_kernel, dim3(a.num_seqs), dim3(kMergeThreads), 0, stream, a,
                          work, lay.tiles);
}

}  // namespace pa
