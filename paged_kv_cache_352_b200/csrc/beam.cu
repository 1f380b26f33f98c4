// Beam search's selection (sm_100a): the best continuations over the beams of a
// sequence and the vocabulary.
//
//   score[k][v] = beam_score[k] + x[k][v] - logsumexp_v x[k],
//   the N largest of the K V scores of a sequence, ties to the smallest k V + v.
//
// The logits are read once: 2 or 4 bytes each, against one exponential, a
// comparison and an addition. A row's ranking does not need its logsumexp, so a CTA
// takes a piece of a row and leaves the piece's maximum, its sum of exponentials and
// its N largest logits in the workspace; then one CTA per sequence adds up the rows'
// sums and ranks K x pieces x N candidates. For little work a piece is 8 or 16 logits a
// thread and the CTA that finishes the sequence's last piece merges it (4 beams of 32000
// logits: 8 us; a second launch cost 2.6 us more). For much work 4 CTAs an SM each walk
// an equal share of the rows laid end to end, as pieces of up to 16 chunks, and a second
// launch merges: its launch is cheaper than every CTA's wait for the release of its
// results. 64 x 8 beams of 131072 bf16 logits take 38 us, 31 of them reading (20.8 at
// the copy rate). Other forms, in one run with this one at 37.3 us: 41.1 with a CTA and a
// piece per 16384 logits, 41.3 and 42.5 with shares of at most 8 and 4 chunks, 40.9 with
// chunks copied two ahead through shared memory (fewer waits, more instructions), 43.2 with
// 3 CTAs an SM. No pipe is above half of its rate (exponentials 50 %, issue 45 %, DRAM
// 49 %); the largest stall is the wait for loads: a piece's last step loads the chunk that it
// has just taken once more, nothing is in flight while a piece is ranked, which most shares
// do twice, and SMs finish 10 % apart.
//
// The N largest of a piece without sorting it: the N-th largest of the maxima of
// kGroups groups of threads bounds the N-th largest element from below, so the few
// elements at or above it are collected in shared memory and ranked by counting,
// for each, those before it. Where ties make too many (a piece of equal logits) the N
// are taken one by one instead; either way the order is (value descending, index
// ascending), and a result does not depend on the order of the atomics.
//
// Scores are formed and ranked in double precision: neighbouring candidates of
// different beams are often closer than fp32 scores resolve. The exponentials' sums are
// fp32 per chunk and thread (at most 32 terms), per piece (at most 16 chunks) and CTA,
// double from there on: their rounding (a score within 8e-6 by the worst case; of 20000 rows
// of random, rising, falling and peaked logits none was off by more than 5.2e-7) depends on
// where the shares cut a row. So where candidates of different beams come closer than kNear,
// the merging CTA sums those rows again in double precision, in an order that depends on the
// row alone: the order of such candidates is exact, and beams that are copies of each other
// tie. It takes a row of 131072 logits again in 31 us, two rows for about one in a hundred
// calls of 64 sequences (8 beams, 16 places).
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stddef.h>
#include <string.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kGroups = 64;       // groups of a piece whose maxima bound the N-th largest
constexpr int kPieceCap = 2048;   // candidates a piece ranks at once
constexpr int kMergeCap = 1024;   // candidates a sequence ranks at once
constexpr int kMaxPer = 16;       // chunks of a CTA's share
constexpr double kNear = 1.9073486328125e-6;  // 2^-19

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

// A 16-byte load of logits: kPerLoad of them, kept packed in registers (two chunks of
// 16-bit logits, one taken and one on its way, are 32: four CTAs fit an SM).
template <typename T>
struct Logits {
  static constexpr int kPerLoad = 8;
  static __device__ __forceinline__ void widen(const uint4& u, float (&f)[8]) {
    Storage<T>::to_f32(u, f);
  }
  static __device__ __forceinline__ float one(const T* p) { return static_cast<float>(*p); }
  // the largest (NaN ignored), two at a time
  template <int N>
  static __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                         __nv_bfloat162>::type;
    T2 m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      T2 h[4];
      memcpy(h, &u[i], sizeof(u[i]));
      m[i] = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      if (i) m[0] = __hmax2(m[0], m[i]);
    }
    return fmaxf(static_cast<float>(m[0].x), static_cast<float>(m[0].y));
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
  template <int N>
  static __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[4];
      widen(u[i], f);
      m = fmaxf(m, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
    }
    return m;
  }
  static __device__ __forceinline__ uint4 narrow(const float (&f)[4]) {
    uint4 u;
    memcpy(&u, f, sizeof(u));
    return u;
  }
};

// The 16 bytes of logits at `at`, -inf past the row: the end of a row and what lies
// behind it in its last chunk.
template <typename T>
__device__ __noinline__ uint4 load_last(const T* x, int at, int vocab) {
  constexpr int EPL = Logits<T>::kPerLoad;
  float f[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) f[e] = at + e < vocab ? Logits<T>::one(x + at + e) : -INFINITY;
  return Logits<T>::narrow(f);
}

// The workspace's parts.
struct Work {
  int* done;       // [num_seqs] pieces finished, back to 0 after the merge (little work)
  float* max;      // [rows][pieces]
  float* sum;      // [rows][pieces], of the exponentials relative to max
  uint64_t* keys;  // [rows][pieces][select], best first, 0 past the candidates
};

// Candidates are ordered by score, ties to the smaller flat index.
__device__ __forceinline__ bool before(double s, int32_t f, double t, int32_t g) {
  return s > t || (s == t && f < g);
}

// Shared memory of a sequence's merge.
template <int kWarps>
struct MergeShared {
  // a score is (x - largest) + offset: offset is the beam score less the logarithm of the
  // sum of exponentials relative to the row's largest logit, -inf for a dead beam
  __align__(16) double offset[PA_BEAM_MAX];
  __align__(16) float largest[PA_BEAM_MAX];
  __align__(16) float beam[PA_BEAM_MAX];  // beam scores
  __align__(16) double group_max[kGroups];
  __align__(16) double warp_best[kWarps];
  __align__(16) double best_score[kWarps];
  __align__(16) int32_t best_index[kWarps];
  __align__(16) double top[PA_BEAM_MAX];  // the results in order
  __align__(16) int32_t top_index[PA_BEAM_MAX];
  __align__(16) unsigned long long near;  // beams whose sums are to be taken again
  __align__(16) int count;
};

// Logit `at` of a row, widened.
__device__ __forceinline__ float any_logit(const BeamArgs& a, size_t row, int at) {
  const int64_t i = (int64_t)row * a.row_stride + at;
  if (a.dtype == PA_F32) return __ldg(static_cast<const float*>(a.logits) + i);
  if (a.dtype == PA_F16) return __half2float(static_cast<const __half*>(a.logits)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[i]);
}

// This thread's share of the sum of exp(x - largest) over a row.
template <typename T, int kThreads>
__device__ __forceinline__ double exact_share(const T* x, int vocab, double largest) {
  constexpr int EPL = Logits<T>::kPerLoad;
  double s[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) s[e] = 0.0;
  for (int at = threadIdx.x * EPL; at < vocab; at += kThreads * EPL) {
    float f[EPL];
    Logits<T>::widen(at + EPL <= vocab ? __ldg(reinterpret_cast<const uint4*>(x + at))
                                       : load_last<T>(x, at, vocab),
                     f);
#pragma unroll
    for (int e = 0; e < EPL; ++e) s[e] += exp((double)f[e] - largest);
  }
#pragma unroll
  for (int e = 1; e < EPL; ++e) s[0] += s[e];
  return s[0];
}

// The sum of exp(x - largest) over a row by the whole CTA, in double precision and in an
// order that depends on the row and the CTA's threads alone. partial: [kThreads / 32] of
// shared memory.
template <int kThreads>
__device__ __forceinline__ double exact_sum(const BeamArgs& a, size_t row, float largest,
                                         double* partial) {
  const int64_t first = (int64_t)row * a.row_stride;
  double S;
  if (a.dtype == PA_F32)
    S = exact_share<float, kThreads>(static_cast<const float*>(a.logits) + first, a.vocab, largest);
  else if (a.dtype == PA_F16)
    S = exact_share<__half, kThreads>(static_cast<const __half*>(a.logits) + first, a.vocab,
                                      largest);
  else
    S = exact_share<__nv_bfloat16, kThreads>(static_cast<const __nv_bfloat16*>(a.logits) + first,
                                             a.vocab, largest);
#pragma unroll
  for (int mask = 16; mask > 0; mask >>= 1) S += __shfl_xor_sync(0xffffffffu, S, mask);
  __syncthreads();  // the row before is done with `partial`
  if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = S;
  __syncthreads();
  S = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) S += partial[w];
  return S;
}

// Result `rank` of sequence b.
__device__ __forceinline__ void put_result(const BeamArgs& a, int b, int rank, double s,
                                           int32_t f) {
  const size_t out = (size_t)b * a.select + rank;
  // (a finite score past the largest float stays one: -inf goes with no candidate)
  a.scores[out] = s > -INFINITY ? fmaxf((float)s, -FLT_MAX) : -INFINITY;
  a.parents[out] = s > -INFINITY ? f / a.vocab : -1;
  a.tokens[out] = s > -INFINITY ? f % a.vocab : -1;
}

// Takes the sums of the rows in sh.near again and, unless there were too many (n >
// kMergeCap), ranks the n collected candidates by them. A function of its own, so that
// the registers and the code of calls that need it are not others'.
template <int kThreads>
__device__ __noinline__ void rank_again(const BeamArgs& a, int b, int n,
                                        MergeShared<kThreads / 32>& sh, double* cs, int32_t* cf) {
  const unsigned long long near = sh.near;
  for (int k = 0; k < a.num_beams; ++k) {
    if (!(near >> k & 1)) continue;
    const size_t row = (size_t)b * a.num_beams + k;
    const double S = exact_sum<kThreads>(a, row, sh.largest[k], sh.warp_best);
    if (threadIdx.x == 0) sh.offset[k] = (double)sh.beam[k] - log(S);
  }
  __syncthreads();
  if (n > kMergeCap) return;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int k = cf[i] / a.vocab;
    const float x = any_logit(a, (size_t)b * a.num_beams + k, cf[i] % a.vocab);
    cs[i] = ((double)x - (double)sh.largest[k]) + sh.offset[k];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += before(cs[j], cf[j], cs[i], cf[i]);
    if (rank < a.select) put_result(a, b, rank, cs[i], cf[i]);
  }
}

// Sequence b by one CTA: its rows' logsumexp, then its best candidates. cs, cf: shared
// memory for kMergeCap candidates. The pieces' results were written by other CTAs: they
// are read past L1.
template <int kMergeThreads>
__device__ __forceinline__ void merge_sequence(const BeamArgs& a, const Work& work, int pieces,
                                               int b, MergeShared<kMergeThreads / 32>& sh,
                                               double* cs, int32_t* cf) {
  constexpr int kWarps = kMergeThreads / 32;
  const int beams = a.num_beams, vocab = a.vocab, select = a.select;
  const float* piece_max = work.max;
  const float* piece_sum = work.sum;
  const uint64_t* piece_keys = work.keys;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_beam = pieces * select;
  const int total = beams * per_beam;
  // this thread's first candidates, on their way while the rows' sums are added up
  constexpr int kAhead = 4;
  uint64_t ahead[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = threadIdx.x + j * kMergeThreads;
    ahead[j] = i < total ? __ldcg(piece_keys + (size_t)b * total + i) : 0;
  }
  for (int k = warp; k < beams; k += kWarps) {
    const size_t row = (size_t)b * beams + k;
    float m0 = -INFINITY, s0 = 0.f;  // the first 32 pieces stay in registers
    if (lane < pieces) {
      m0 = __ldcg(piece_max + row * pieces + lane);
      s0 = __ldcg(piece_sum + row * pieces + lane);
    }
    const float beam = lane == 0 ? a.beam_scores[row] : 0.f;
    float M = m0;
    for (int t = lane + 32; t < pieces; t += 32) M = fmaxf(M, __ldcg(piece_max + row * pieces + t));
#pragma unroll
    for (int mask = 16; mask > 0; mask >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, mask));
    double S = 0.0;
    auto add = [&](float m, float s) {
      if (m > -INFINITY || s != s) S += (double)s * exp((double)m - (double)M);
    };
    add(m0, s0);
    for (int t = lane + 32; t < pieces; t += 32)
      add(__ldcg(piece_max + row * pieces + t), __ldcg(piece_sum + row * pieces + t));
#pragma unroll
    for (int mask = 16; mask > 0; mask >>= 1) S += __shfl_xor_sync(0xffffffffu, S, mask);
    if (lane == 0) {
      double o = -INFINITY;
      if (!(beam < INFINITY)) o = NAN;  // also where every token is masked
      else if (M > -INFINITY || S != S) o = M < INFINITY ? (double)beam - log(S) : NAN;
      if (o != o || o == INFINITY) {  // a NaN or +inf among the logits, or as beam score
        report(a.dev_error, PA_DEVERR_LOGITS);
        o = -INFINITY;
      }
      sh.offset[k] = o;
      sh.largest[k] = M;
      sh.beam[k] = beam;
    }
  }
  if (threadIdx.x == 0) {
    sh.count = 0;
    sh.near = 0;
  }
  __syncthreads();
  auto score_key = [&](int i, uint64_t key, double& s, int32_t& f) {
    const int k = i / per_beam;
    s = -INFINITY;
    f = INT32_MAX;
    if (key != 0 && sh.offset[k] > -INFINITY) {
      s = ((double)from_orderable((uint32_t)(key >> 32)) - (double)sh.largest[k]) + sh.offset[k];
      f = k * vocab + (int32_t)~(uint32_t)key;  // below 2^30
    }
  };
  auto score_of = [&](int i, double& s, int32_t& f) {
    score_key(i, __ldcg(piece_keys + (size_t)b * total + i), s, f);
  };
  // as in a piece: the select-th largest of 64 groups' maxima bounds the result from below
  double top = -INFINITY;
  double as[kAhead];
  int32_t af[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    as[j] = -INFINITY;
    const int i = threadIdx.x + j * kMergeThreads;
    if (i < total) score_key(i, ahead[j], as[j], af[j]);
    top = as[j] > top ? as[j] : top;
  }
  for (int i = threadIdx.x + kAhead * kMergeThreads; i < total; i += kMergeThreads) {
    double s;
    int32_t f;
    score_of(i, s, f);
    top = s > top ? s : top;
  }
  constexpr int kGroupLanes = kMergeThreads / kGroups;
#pragma unroll
  for (int mask = 1; mask < kGroupLanes; mask <<= 1)
    top = fmax(top, __shfl_xor_sync(0xffffffffu, top, mask));  // (never NaN)
  if (threadIdx.x % kGroupLanes == 0) sh.group_max[threadIdx.x / kGroupLanes] = top;
  __syncthreads();
  {
    // kGroupLanes threads count for each group
    const double p = sh.group_max[threadIdx.x / kGroupLanes];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kGroups / kGroupLanes; ++i)
      rank += sh.group_max[i * kGroupLanes + threadIdx.x % kGroupLanes] >= p;
#pragma unroll
    for (int mask = 1; mask < kGroupLanes; mask <<= 1)
      rank += __shfl_xor_sync(0xffffffffu, rank, mask);
    double best = rank >= select ? p : -INFINITY;
#pragma unroll
    for (int mask = 16; mask >= kGroupLanes; mask >>= 1) {
      const double o = __shfl_xor_sync(0xffffffffu, best, mask);
      best = o > best ? o : best;
    }
    if (lane == 0) sh.warp_best[warp] = best;
  }
  __syncthreads();
  double lowest = sh.warp_best[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) lowest = sh.warp_best[w] > lowest ? sh.warp_best[w] : lowest;
  lowest -= kNear;  // what might belong above it
  auto collect = [&](double s, int32_t f) {
    if (s > -INFINITY && s >= lowest) {
      const int at = atomicAdd(&sh.count, 1);
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
    int32_t f;
    score_of(i, s, f);
    collect(s, f);
  }
  __syncthreads();
  const int n = sh.count;
  auto mark = [&](int k, int l) {
    if (k != l) atomicOr(&sh.near, 1ull << k | 1ull << l);
  };
  if (n <= kMergeCap) {
    for (int i = threadIdx.x; i < n; i += kMergeThreads) {
      const double s = cs[i];
      const int32_t f = cf[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += before(cs[j], cf[j], s, f);
      if (rank < select) {
        put_result(a, b, rank, s, f);
        sh.top[rank] = s;
        sh.top_index[rank] = f;
      }
    }
    for (int i = n + threadIdx.x; i < select; i += kMergeThreads)
      put_result(a, b, i, -INFINITY, 0);
    __syncthreads();
    // Beams whose candidates lie closer than their sums' rounding: neighbours in the order,
    // and what might still come to the last place.
    for (int i = threadIdx.x; i + 1 < min(n, select); i += kMergeThreads)
      if (sh.top[i] - sh.top[i + 1] <= kNear)
        mark(sh.top_index[i] / vocab, sh.top_index[i + 1] / vocab);
    if (n > select) {
      const double last = sh.top[select - 1];
      const int32_t index = sh.top_index[select - 1];
      for (int i = threadIdx.x; i < n; i += kMergeThreads)
        if (last - cs[i] <= kNear && before(last, index, cs[i], cf[i]))
          mark(index / vocab, cf[i] / vocab);
    }
  } else if (threadIdx.x < beams && sh.offset[threadIdx.x] > -INFINITY) {
    atomicOr(&sh.near, 1ull << threadIdx.x);  // too many to be compared
  }
  __syncthreads();
  const unsigned long long near = sh.near;
  // (one alone: a beam's order is its logits')
  if (near & (near - 1)) rank_again<kMergeThreads>(a, b, n, sh, cs, cf);
  if (n <= kMergeCap) return;
  // more equal candidates than the buffer holds: one at a time
  double ls = INFINITY;
  int32_t lf = -1;
  for (int r = 0; r < select; ++r) {
    double s = -INFINITY;
    int32_t f = INT32_MAX;
    for (int i = threadIdx.x; i < total; i += kMergeThreads) {
      double t;
      int32_t g;
      score_of(i, t, g);
      if (t > -INFINITY && before(ls, lf, t, g) && before(t, g, s, f)) {
        s = t;
        f = g;
      }
    }
#pragma unroll
    for (int mask = 16; mask > 0; mask >>= 1) {
      const double t = __shfl_xor_sync(0xffffffffu, s, mask);
      const int32_t g = __shfl_xor_sync(0xffffffffu, f, mask);
      if (before(t, g, s, f)) {
        s = t;
        f = g;
      }
    }
    __syncthreads();
    if (lane == 0) {
      sh.best_score[warp] = s;
      sh.best_index[warp] = f;
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
      if (before(sh.best_score[w], sh.best_index[w], s, f)) {
        s = sh.best_score[w];
        f = sh.best_index[w];
      }
    if (threadIdx.x == 0) put_result(a, b, r, s, f);
    ls = s;
    lf = f;
  }
}

constexpr int kMergeThreads = 512;

__global__ void __launch_bounds__(kMergeThreads, 1)
    beam_merge_kernel(const BeamArgs a, const Work work, int pieces) {
  grid_dependency_wait();
  allow_dependents();
  __shared__ struct {
    __align__(16) double cs[kMergeCap];
    __align__(16) int32_t cf[kMergeCap];
    MergeShared<kMergeThreads / 32> merge;
  } sh;
  merge_sequence<kMergeThreads>(a, work, pieces, blockIdx.x, sh.merge, sh.cs, sh.cf);
}

// Pieces of rows. A chunk is kBeamThreads threads x LOADS 16-byte loads of a row; a CTA
// takes `per` chunks of the rows laid end to end and leaves a result for every row among
// them, or with by_rows `per` chunks of one row. MERGE (one chunk a CTA): the CTA of a
// sequence's last piece merges it.
template <typename T, int LOADS, bool MERGE>
__global__ void __launch_bounds__(kBeamThreads, 4)
    beam_piece_kernel(const BeamArgs a, const Work work, int chunks, int per, int pieces,
                      bool by_rows) {
  grid_dependency_wait();
  allow_dependents();
  constexpr int EPL = Logits<T>::kPerLoad;
  constexpr int kChunk = kBeamThreads * EPL * LOADS;
  constexpr int kWarps = kBeamThreads / 32;
  constexpr float kLog2e = 1.4426950408889634f;
  struct Shared {
    __align__(16) uint64_t cand[kPieceCap];
    __align__(16) float chunk_max[MERGE ? 1 : kMaxPer][kBeamThreads];  // of each thread
    __align__(16) uint32_t group_max[kGroups];
    __align__(16) float warp_max[kWarps];
    __align__(16) float warp_sum[kWarps];
    __align__(16) uint32_t threshold;
    int count, last_piece;
  };
  __shared__ Shared sh;
  // every group has four threads, and its maximum is read 16 bytes at a time
  static_assert(kBeamThreads == 4 * kGroups, "groups of four neighbouring lanes");
  static_assert(offsetof(Shared, group_max) % 16 == 0 && alignof(Shared) % 16 == 0, "alignment");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vocab = a.vocab, select = a.select;
  const int total = a.num_seqs * a.num_beams * chunks;
  int at_chunk, end_chunk;
  if (by_rows) {
    const int row = blockIdx.x / pieces;
    at_chunk = row * chunks + ((int)blockIdx.x - row * pieces) * per;
    end_chunk = min(at_chunk + per, (row + 1) * chunks);
  } else {
    at_chunk = blockIdx.x * per;
    end_chunk = min(at_chunk + per, total);
  }
  while (at_chunk < end_chunk) {
    const int row = at_chunk / chunks, c0 = at_chunk - row * chunks;
    const int n_chunks = MERGE ? 1 : min(end_chunk - at_chunk, chunks - c0);
    const int piece = (int)blockIdx.x - (by_rows ? row * pieces : row * chunks / per);
    const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
    const int begin = c0 * kChunk;
    if (threadIdx.x == 0) {  // read behind the barriers below
      sh.count = 0;
      sh.threshold = 0;
    }
    // element e of load i of chunk j: index begin + j kChunk + (i kBeamThreads + thread) EPL
    // + e; past the row: -inf, which is never a candidate and adds nothing
    auto fetch = [&](uint4(&u)[LOADS], int j) {  // a chunk that the row covers
      const uint4* from = reinterpret_cast<const uint4*>(x + begin + j * kChunk) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) u[i] = __ldg(from + i * kBeamThreads);
    };
    auto fetch_bounded = [&](uint4(&u)[LOADS], int j) {
      const int base = begin + j * kChunk + (int)threadIdx.x * EPL;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int at = base + i * kBeamThreads * EPL;
        if (at + EPL <= vocab) u[i] = __ldg(reinterpret_cast<const uint4*>(x + at));
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int at = base + i * kBeamThreads * EPL;
        if (at + EPL > vocab) u[i] = load_last<T>(x, at, vocab);
      }
    };
    const int whole = min(n_chunks, vocab / kChunk - c0);  // the row's last may be short
    // the thread's largest logit and its sum of exponentials relative to it; a NaN makes
    // the sum NaN
    float mx = -INFINITY, sum = 0.f;
    auto take = [&](const uint4(&u)[LOADS], int j) {
      const float cm = Logits<T>::template largest<LOADS>(u);
      sh.chunk_max[j][threadIdx.x] = cm;
      const float to = fmaxf(mx, cm);
      const float ref = to == -INFINITY ? 0.f : to;
      const float keep = fast_exp2((mx - ref) * kLog2e);
      mx = to;
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
      sum = fmaf(sum, keep, even + odd);
    };
    // a chunk's loads are on their way while the one before is taken; no barriers, so that
    // warps drift apart and some always load
    uint4 ua[LOADS];
    if (whole > 0) {
      fetch(ua, 0);
      if constexpr (MERGE) {
        take(ua, 0);
      } else {
        uint4 ub[LOADS];
        for (int j = 0;;) {
          fetch(ub, min(j + 1, whole - 1));
          take(ua, j);
          if (++j == whole) break;
          fetch(ua, min(j + 1, whole - 1));
          take(ub, j);
          if (++j == whole) break;
        }
      }
    }
    if (whole < n_chunks) {
      fetch_bounded(ua, n_chunks - 1);
      take(ua, n_chunks - 1);
    }
    // groups of four neighbouring lanes
    float gm = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
    if ((lane & 3) == 0) sh.group_max[threadIdx.x >> 2] = orderable(gm);
    float wm = gm;
#pragma unroll
    for (int mask = 4; mask <= 16; mask <<= 1)
      wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, mask));
    if (mx > -INFINITY) sum *= fast_exp2((mx - wm) * kLog2e);
#pragma unroll
    for (int mask = 1; mask <= 16; mask <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, mask);
    if (lane == 0) {
      sh.warp_max[warp] = wm;
      sh.warp_sum[warp] = sum;
    }
    __syncthreads();
    {
      // the select-th largest of the groups' maxima: the largest value with at least
      // `select` maxima at or above it; four threads count for each group
      const uint32_t g = sh.group_max[threadIdx.x >> 2];
      int rank = 0;
#pragma unroll
      for (int i = 0; i < kGroups / 4; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(sh.group_max + 4 * i + 4 * (lane & 3));
        rank += (v.x >= g) + (v.y >= g) + (v.z >= g) + (v.w >= g);
      }
      rank += __shfl_xor_sync(0xffffffffu, rank, 1);
      rank += __shfl_xor_sync(0xffffffffu, rank, 2);
      const uint32_t best = __reduce_max_sync(0xffffffffu, rank >= select ? g : 0u);
      if (lane == 0) atomicMax(&sh.threshold, best);
    }
    __syncthreads();
    const size_t out = (size_t)row * pieces + piece;
    if (warp == kWarps - 1) {  // lane w: warp w's share
      const float m = lane < kWarps ? sh.warp_max[lane] : -INFINITY;
      float S = lane < kWarps ? sh.warp_sum[lane] : 0.f;
      float M = m;
#pragma unroll
      for (int mask = 1; mask < kWarps; mask <<= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, mask));
      if (m > -INFINITY) S *= expf(m - M);
#pragma unroll
      for (int mask = 1; mask < kWarps; mask <<= 1) S += __shfl_xor_sync(0xffffffffu, S, mask);
      if (lane == 0) {
        work.max[out] = M;
        work.sum[out] = S;
      }
    }
    const float lowest = from_orderable(sh.threshold);
    if constexpr (MERGE) {  // the one chunk is still in registers
      if (mx >= lowest && mx > -INFINITY) {
        uint32_t in = 0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          float f[EPL];
          Logits<T>::widen(ua[i], f);
#pragma unroll
          for (int e = 0; e < EPL; ++e)
            in |= (f[e] >= lowest && f[e] > -INFINITY ? 1u : 0u) << (i * EPL + e);
        }
        int c = atomicAdd(&sh.count, __popc(in));
        for (; in; in &= in - 1, ++c) {
          const int b = __ffs(in) - 1;
          const int at = begin + (b / EPL * kBeamThreads + (int)threadIdx.x) * EPL + b % EPL;
          if (c < kPieceCap) sh.cand[c] = make_key(Logits<T>::one(x + at), at);
        }
      }
    } else {
      // The few chunks of a thread that hold candidates are read again (from L2, mostly), the
      // LOADS x EPL elements of one by a warp at once, two on their way together.
      uint32_t hits = 0;
#pragma unroll 4
      for (int j = 0; j < n_chunks; ++j) {
        const float cm = sh.chunk_max[j][threadIdx.x];
        hits |= (cm >= lowest && cm > -INFINITY ? 1u : 0u) << j;
      }
      const int place = lane / EPL * kBeamThreads * EPL + lane % EPL;
      for (uint32_t m; (m = __ballot_sync(0xffffffffu, hits != 0)) != 0;) {
        const int first = __ffs(hits) - 1;  // -1 where there is none: not looked at
        int at[2];
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int from = m ? __ffs(m) - 1 : 0;
          const int j = __shfl_sync(0xffffffffu, first, from);
          at[h] = begin + j * kChunk + (warp * 32 + from) * EPL + place;
          f[h] = m != 0 && lane < LOADS * EPL && at[h] < vocab ? Logits<T>::one(x + at[h])
                                                               : -INFINITY;
          if (m != 0 && lane == from) hits &= hits - 1;
          m &= m - 1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (f[h] >= lowest && f[h] > -INFINITY) {
            const int c = atomicAdd(&sh.count, 1);
            if (c < kPieceCap) sh.cand[c] = make_key(f[h], at[h]);
          }
      }
    }
    __syncthreads();
    uint64_t* keys = work.keys + out * select;
    auto take_one_by_one = [&]() {
      // more ties than the buffer holds: one at a time, each the largest below the last
      uint64_t last = ~0ull;
      uint64_t* best = sh.cand;  // [kWarps]
      const int end = min(vocab, begin + n_chunks * kChunk);
      for (int r = 0; r < select; ++r) {
        uint64_t k = 0;
#pragma unroll 4
        for (int at = begin + (int)threadIdx.x; at < end; at += kBeamThreads) {
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
    const int n = sh.count;
    if (n <= kPieceCap) {
      for (int i = threadIdx.x; i < n; i += kBeamThreads) {
        const uint64_t k = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > k;
        if (rank < select) keys[rank] = k;
      }
      for (int i = n + threadIdx.x; i < select; i += kBeamThreads) keys[i] = 0;
    } else {
      take_one_by_one();
    }
    if (c0 + n_chunks == chunks) {  // the row's last piece: the places that it has no piece for
      for (int p = piece + 1; p < pieces; ++p) {
        const size_t none = (size_t)row * pieces + p;
        if (threadIdx.x == 0) {
          work.max[none] = -INFINITY;
          work.sum[none] = 0.f;
        }
        for (int i = threadIdx.x; i < select; i += kBeamThreads) work.keys[none * select + i] = 0;
      }
    }
    if constexpr (MERGE) {
      // as the split-KV merge of the decode: the barrier makes the CTA's stores visible to
      // thread 0, whose gpu-scope acq_rel add publishes them
      const int seq = row / a.num_beams;
      __syncthreads();
      if (threadIdx.x == 0) {
        sh.last_piece = atom_add_acq_rel_gpu(work.done + seq, 1) == a.num_beams * pieces - 1;
        if (sh.last_piece) work.done[seq] = 0;
      }
      __syncthreads();
      if (sh.last_piece) {
        static_assert(kPieceCap >= 2 * kMergeCap, "the merge takes the candidates' place");
        __shared__ MergeShared<kWarps> merge;
        merge_sequence<kBeamThreads>(a, work, pieces, seq, merge,
                                     reinterpret_cast<double*>(sh.cand),
                                     reinterpret_cast<int32_t*>(sh.cand + kMergeCap));
      }
      return;
    }
    at_chunk += n_chunks;
    __syncthreads();  // the next row's piece uses the same shared memory
  }
}

// Little work: a chunk of kSmallLoads loads a thread per CTA, merged in the same launch.
// Much: chunks of kLargeLoads, shared out evenly over the CTAs that the SMs hold at once.
constexpr int kSmallLoads = 2, kLargeLoads = 4;
constexpr int kResident = 148 * 4;
constexpr int kCounters = 512;  // sequences whose pieces are counted (little work)
static_assert(kLargeLoads * 8 <= 32, "a warp reads a thread's chunk at once");

int chunks_of(int vocab, int elem, int loads) {
  const int chunk = kBeamThreads * (16 / elem) * loads;
  return (vocab + chunk - 1) / chunk;
}

}  // namespace

void beam_layout(int num_seqs, int num_beams, int vocab, int select, int dtype, BeamLayout* lay) {
  const int elem = dtype == PA_F32 ? 4 : 2;
  const int64_t rows = (int64_t)num_seqs * num_beams;
  lay->chunks = chunks_of(vocab, elem, kLargeLoads);
  lay->large = rows * lay->chunks >= kResident || num_seqs > kCounters;
  lay->per = 1;
  if (lay->large) {
    const int64_t total = rows * lay->chunks, once = (int64_t)kResident * kMaxPer;
    const int64_t slots = (total + once - 1) / once * kResident;
    lay->per = (int)((total + slots - 1) / slots);
  } else {
    lay->chunks = chunks_of(vocab, elem, kSmallLoads);
  }
  lay->pieces = (lay->chunks + lay->per - 1) / lay->per;
  // Shares of one row each while they fit the SMs at once, too: a CTA then ends one piece, not
  // two (16 x 4 beams of 50257 fp32 logits: 9.3 us instead of 10.3 us).
  lay->by_rows = rows * lay->pieces <= kResident || !lay->large;
  if (!lay->by_rows) lay->pieces = (lay->chunks + lay->per - 2) / lay->per + 1;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t n = (size_t)rows * lay->pieces;
  // the counters have a place of their own whatever the sizes, so that no call leaves results
  // where another counts
  lay->max_off = up(kCounters * sizeof(int));
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
  const int64_t total = (int64_t)lay.chunks * a.num_seqs * a.num_beams;
  if (total > 0x7fff0000LL) return cudaErrorInvalidValue;
  auto go = [&](auto kern) {
    const int64_t ctas = lay.by_rows ? (int64_t)lay.pieces * a.num_seqs * a.num_beams
                                     : (total + lay.per - 1) / lay.per;
    return launch_dependent(kern, dim3((unsigned)ctas), dim3(kBeamThreads), 0, stream, a, work,
                            lay.chunks, lay.per, lay.pieces, lay.by_rows);
  };
  if (!lay.large) {
    return dtype == PA_F32   ? go(beam_piece_kernel<float, kSmallLoads, true>)
           : dtype == PA_F16 ? go(beam_piece_kernel<__half, kSmallLoads, true>)
                             : go(beam_piece_kernel<__nv_bfloat16, kSmallLoads, true>);
  }
  const cudaError_t e = dtype == PA_F32 ? go(beam_piece_kernel<float, kLargeLoads, false>)
                        : dtype == PA_F16
                            ? go(beam_piece_kernel<__half, kLargeLoads, false>)
                            : go(beam_piece_kernel<__nv_bfloat16, kLargeLoads, false>);
  if (e != cudaSuccess) return e;
  return launch_dependent(beam_merge_kernel, dim3(a.num_seqs), dim3(kMergeThreads), 0, stream, a,
                          work, lay.pieces);
}

}  // namespace pa
