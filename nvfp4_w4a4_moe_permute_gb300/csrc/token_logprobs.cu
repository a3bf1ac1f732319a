// minite_token_logprobs / minite_token_logprobs_backward: the log probability
// of a given token of each row of logits, the row's entropy and its top
// alternatives, and the gradient of the first two.
//
// With y = x / T over a row's V logits, M = max y, s = sum exp(y - M) and
// t = sum (y - M) exp(y - M):
//   log p_j = y_j - M - log s,  logprob = log p_i,  H = log s - t / s
// s is kept as r = s - 1, the sum without the maximum's own term, and log s =
// log1p(r): a token that is almost certain has a log probability of -r, which
// would be lost beside the 1 (r = 1e-4 to three digits).
//   dx_j = (1/T) (g_lp ([j = i] - p_j) - g_H p_j (log p_j + H))
// M (as a logit) and log s are kept apart for the backward: their sum would
// lose log s beside a large M.
// M, r and t come from one pass: a running maximum, with r and t moved to the
// new one when it grows (t <- c (t + d (r + 1)), r <- c (r + 1) for a shift d,
// c = exp d).
//
// The top alternatives cost the streaming loop nothing. Every thread's running
// maximum is the largest of the values it saw, so the k-th largest of the
// maxima of groups of four threads is a lower bound of the row's k-th largest
// logit, and only threads whose maximum reaches it can hold one of the top k:
// those threads' elements are read again, mostly from L2, and the few at or
// above the bound are ranked by counting (more than kCandidates of them by
// sorted lists in the lanes of warps). Equal logits rank by the lower index.
//
// Bound by HBM for learner batches: 4096 rows of 131072 BF16 175 us forward (161
// at the copy rate), 313 backward (321); the forward executes 9.1
// instructions an element (issue slots 61% busy). With 20 alternatives 229 us:
// the second reading fetches 16% more from HBM. A single row takes a cluster:
// 10.9 us for 131072 FP32 logits with 20 alternatives, 7.5 without, most of it
// latency.
#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace logprobs {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSegments = 8;        // a portable cluster's CTAs at most
constexpr int64_t kSegmentBytes = 131072;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.402823466e+38f;

struct Params {
  const void* logits;
  int64_t ld;
  int64_t V;
  const void* targets;      // int32 or int64 [N], or null
  int targets64;
  float inv_t;
  float k2;                 // log2(e) / temperature
  int fast;                 // fast_k(k2)
  int segments;             // of a row, a power of two
  int cluster;              // CTAs per row, a power of two up to segments
  float* logprob;
  float* entropy;
  float2* stats;            // [N] {largest logit, log s}, or null
  int k;
  int32_t* alt_ids;
  float* alt_lp;
  int32_t* status;
};

// 32 bytes of a row, one load of a thread.
struct Vec {
  uint4 lo, hi;
};

template <typename T> struct Elem;
template <> struct Elem<float> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float value(float x) { return x; }
  static __device__ __forceinline__ void unpack(const Vec& u, float (&x)[8]) {
    x[0] = __uint_as_float(u.lo.x); x[1] = __uint_as_float(u.lo.y);
    x[2] = __uint_as_float(u.lo.z); x[3] = __uint_as_float(u.lo.w);
    x[4] = __uint_as_float(u.hi.x); x[5] = __uint_as_float(u.hi.y);
    x[6] = __uint_as_float(u.hi.z); x[7] = __uint_as_float(u.hi.w);
  }
};
template <> struct Elem<uint16_t> {
  static constexpr int kVec = 16;
  static __device__ __forceinline__ float value(uint16_t x) {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
  }
  static __device__ __forceinline__ void unpack(const Vec& u, float (&x)[16]) {
    const uint32_t w[8] = {u.lo.x, u.lo.y, u.lo.z, u.lo.w, u.hi.x, u.hi.y, u.hi.z, u.hi.w};
    unpack_bf16x16(w, x);
  }
};

// A row as an unaligned head, 32-byte vectors and a tail.
template <typename T>
struct Row {
  const T* x;
  int64_t V;
  int head, tail;
  int64_t nv;
  __device__ __forceinline__ Row(const T* row, int64_t V_) : x(row), V(V_) {
    const uintptr_t off = (32 - (reinterpret_cast<uintptr_t>(row) & 31)) & 31;
    head = static_cast<int>(off / sizeof(T));
    if (head > V) head = static_cast<int>(V);
    nv = (V - head) / Elem<T>::kVec;
    tail = static_cast<int>(V - head - nv * Elem<T>::kVec);
  }
  __device__ __forceinline__ Vec vec(int64_t i) const {
    Vec v;
    // volatile and a memory clobber: to the compiler the load would else be a
    // function of its address alone, free to move ahead of pdl_wait()
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v.lo.x), "=r"(v.lo.y), "=r"(v.lo.z), "=r"(v.lo.w), "=r"(v.hi.x), "=r"(v.hi.y),
                   "=r"(v.hi.z), "=r"(v.hi.w)
                 : "l"(x + head + i * Elem<T>::kVec) : "memory");
    return v;
  }
  __device__ __forceinline__ int64_t tail0() const { return head + nv * Elem<T>::kVec; }
};

constexpr float kMask = -1.152921504606846976e+18f;   // -2^60, a BF16 value

// 2^x, within 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A vector's logits as float pairs, those below -2^60 (masked ones among
// them) raised to it, and their maximum.
__device__ __forceinline__ void pairs_of(const float*, const uint4& u, uint64_t* x, float& mx) {
  const float a = max_nan(__uint_as_float(u.x), kMask), b = max_nan(__uint_as_float(u.y), kMask);
  const float c = max_nan(__uint_as_float(u.z), kMask), d = max_nan(__uint_as_float(u.w), kMask);
  mx = fmaxf(fmaxf(a, b), fmaxf(c, d));
  x[0] = pair(a, b);
  x[1] = pair(c, d);
}
__device__ __forceinline__ void pairs_of(const uint16_t*, const uint4& u, uint64_t* x, float& mx) {
  constexpr uint32_t kMask2 = 0xDD80DD80u;   // -2^60 twice
  const uint32_t w0 = max_nan_bf16x2(u.x, kMask2), w1 = max_nan_bf16x2(u.y, kMask2);
  const uint32_t w2 = max_nan_bf16x2(u.z, kMask2), w3 = max_nan_bf16x2(u.w, kMask2);
  const uint32_t m = max_bf16x2(max_bf16x2(w0, w1), max_bf16x2(w2, w3));
  mx = fmaxf(bf16lo(m), bf16hi(m));
  x[0] = pair(bf16lo(w0), bf16hi(w0));
  x[1] = pair(bf16lo(w1), bf16hi(w1));
  x[2] = pair(bf16lo(w2), bf16hi(w2));
  x[3] = pair(bf16lo(w3), bf16hi(w3));
}

// Running (maximum, sum, weighted sum) of a set of logits in powers of two,
// with k = log2(e) / T and y = (x - m) k:  r = sum 2^y without one element at the
// maximum, t = sum y 2^y. The difference is taken before the product, so that y
// is exactly 0 at the maximum (a row with one token left has logprob 0 and
// entropy 0).
struct Stat {
  float m, r, t;
  __device__ __forceinline__ void raise(float nm, float k) {
    const float d = (m - nm) * k;
    const float c = ex2(d);
    const float s = r + 1.0f;
    t = c > 0.0f ? c * (t + d * s) : 0.0f;   // d * s may be infinite where c is 0
    r = c * s;
    m = nm;
  }
  __device__ __forceinline__ void merge(Stat o, float k) {
    if (o.m > m) raise(o.m, k);
    else if (o.m < m) o.raise(m, k);
    else o.r += 1.0f;   // one maximum of the two counts
    r += o.r;
    t += o.t;
  }
  // One logit, every special value looked at: for a row whose maximum lies
  // beyond +-2^59 (all of it masked, or infinite) or an extreme temperature.
  // m is -inf until there is a logit above it.
  __device__ __forceinline__ void add_any(float x, float k) {
    if (x > m) {
      raise(x, k);
      r += x - x;   // +inf: no probabilities
      return;
    }
    if (x == __int_as_float(0xFF800000)) return;   // masked: adds 0
    const float y = (x - m) * k;
    const float e = ex2(y);
    r += e;
    t += fmaxf(y, -1e30f) * e;   // y may be -inf, which adds 0, not -inf * 0
  }
};
// k in (2^-40, 2^13): a logit of -2^60 then has probability zero beside any
// maximum above -2^59 (2^-(2^59 k)), and no product with it comes near
// overflow.
__host__ __device__ inline bool fast_k(float k) { return k > 9.094947e-13f && k < 8192.0f; }
__device__ __forceinline__ bool fast_row(float m) { return fabsf(m) < 5.76460752303423488e+17f; }

__device__ __forceinline__ Stat shfl_xor(const Stat& a, int o) {
  Stat r;
  r.m = __shfl_xor_sync(0xffffffffu, a.m, o);
  r.r = __shfl_xor_sync(0xffffffffu, a.r, o);
  r.t = __shfl_xor_sync(0xffffffffu, a.t, o);
  return r;
}

// Order of the alternatives: larger logit first, then lower index.
__device__ __forceinline__ uint64_t rank_key(float x, int64_t i) {
  uint32_t b = __float_as_uint(x + 0.0f);   // -0 ranks as +0
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (static_cast<uint64_t>(b) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7FFFFFFFu) : ~b);
}
__device__ __forceinline__ int32_t key_index(uint64_t key) {
  return static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
}

// Insert a key into the warp's list (lane l: the l-th largest so far; 0 where
// there is none). Warp-collective, key uniform.
__device__ __forceinline__ void list_insert(uint64_t& mine, uint64_t key) {
  const int lane = threadIdx.x & 31;
  const int pos = __popc(__ballot_sync(0xffffffffu, mine > key));
  const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane == pos) mine = key;
  else if (lane > pos) mine = up;
}

// Join another warp's sorted list of k into this warp's. Warp-collective.
__device__ __forceinline__ void list_join(uint64_t& mine, const uint64_t* other, int k) {
  for (int l = 0; l < k; ++l) {
    const uint64_t cand = other[l];
    if (cand <= __shfl_sync(0xffffffffu, mine, k - 1)) break;
    list_insert(mine, cand);
  }
}

// Offer one value per lane (absent: x = -inf) to the warp's list of k.
__device__ __forceinline__ void list_offer(uint64_t& mine, int k, float x, int64_t i, float thr) {
  const float inf = __int_as_float(0x7F800000);
  uint64_t key = x >= thr && x > -inf ? rank_key(x, i) : 0;
  uint64_t worst = __shfl_sync(0xffffffffu, mine, k - 1);
  uint32_t todo = __ballot_sync(0xffffffffu, key > worst);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    const uint64_t cand = __shfl_sync(0xffffffffu, key, src);
    if (cand > __shfl_sync(0xffffffffu, mine, k - 1)) list_insert(mine, cand);
  }
}

constexpr int kGroups = kThreads / 4;   // threads whose maxima are compared for the threshold
constexpr int kCandidates = 512;

struct Shared {
  Stat stat[kMaxSegments][kWarps];
  Stat part[kMaxSegments];        // every segment's sums (the cluster's first CTA: all of the row)
  Stat row;
  alignas(16) float group_max[kGroups];   // read four at a time
  uint32_t thr;
  int n_sets, n_cand;
  uint8_t sets[kThreads];         // threads that hold candidates
  uint64_t cand[kCandidates];
  float thread_max[kThreads];     // more candidates than that: every thread's maximum,
  uint64_t list[kWarps][32];      // and each warp's best
  uint64_t best[32];              // the CTA's best, sorted, 0 where there is none
  uint64_t part_best[kMaxSegments][32];   // the cluster's first CTA: the others' best
};

// A row's segments [s0, s1) of `segs`: segment s holds the 32-byte vectors
// [begin(s), begin(s + 1)), thread t of it the vectors begin(s) + t + i kThreads.
struct Segments {
  int64_t nv;
  int segs, s0, s1;
  __device__ __forceinline__ int64_t begin(int s) const { return nv * s / segs; }
  __device__ __forceinline__ bool first() const { return s0 == 0; }
  __device__ __forceinline__ bool last() const { return s1 == segs; }
};

// A warp's stats, joined in a fixed order (on lane 0).
__device__ __forceinline__ Stat join_warp(Stat st, float k) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) st.merge(shfl_xor(st, o), k);
  return st;
}
// S.stat of n segments to S.part[s0 ...], one thread a segment, and, for the
// alternatives, the largest of the groups' maxima that at least k of them reach
// to S.thr. `mine` is the largest logit that this thread saw. Block-wide, with a
// barrier at both ends.
__device__ __forceinline__ void join_segments(Shared& S, int s0, int n, float k2, float mine, int k) {
  const int tid = threadIdx.x;
  if (k > 0) {
    float g = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((tid & 3) == 0) S.group_max[tid >> 2] = g;
    if (tid == 0) {
      S.thr = 0;
      S.n_sets = 0;
      S.n_cand = 0;
    }
    if (tid < 32) S.best[tid] = 0;
  }
  __syncthreads();
  if (tid < n) {
    Stat st = S.stat[tid][0];
    for (int w = 1; w < kWarps; ++w) st.merge(S.stat[tid][w], k2);
    S.part[s0 + tid] = st;
  }
  if (k > 0 && tid >= kThreads - kGroups) {
    const float own = S.group_max[tid - (kThreads - kGroups)];
    int reach = 0;
#pragma unroll
    for (int j = 0; j < kGroups / 4; ++j) {
      const float4 o = reinterpret_cast<const float4*>(S.group_max)[j];
      reach += (o.x >= own) + (o.y >= own) + (o.z >= own) + (o.w >= own);
    }
    if (reach >= k) atomicMax(&S.thr, static_cast<uint32_t>(rank_key(own, 0) >> 32));
  }
  __syncthreads();
}

// The k largest of n keys to best[0..k), by the number of larger ones (keys
// differ). Block-wide, without a barrier.
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, uint64_t* best, int k) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = keys[i];
    int larger = 0;
    for (int j = 0; j < n; ++j) larger += keys[j] > key;
    if (larger < k) best[larger] = key;
  }
}

// The k best of some segments (with the row's head if they are the first, its
// tail if the last) to S.best. `mine` is the largest logit that this thread saw
// in them: its vectors, head element tid, tail element tid. After join_segments;
// ends with a barrier.
template <typename T>
__device__ __forceinline__ void block_alternatives(Shared& S, const Row<T>& r, const Segments& sg,
                                                   float mine, int k) {
  constexpr int VEC = Elem<T>::kVec;
  const float inf = __int_as_float(0x7F800000);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool first = sg.first(), last = sg.last();
  float thr = key_value(static_cast<uint64_t>(S.thr) << 32);
  if (thr <= kMask) thr = -inf;   // what threads with masked logits only hold, or none
  auto offer = [&](float x, int64_t i) {
    if (x >= thr && x > -inf) {
      const int at = atomicAdd(&S.n_cand, 1);
      if (at < kCandidates) S.cand[at] = rank_key(x, i);
    }
  };
  if (mine >= thr) {
    S.sets[atomicAdd(&S.n_sets, 1)] = static_cast<uint8_t>(tid);
    if (first && tid < r.head) offer(Elem<T>::value(r.x[tid]), tid);
    if (last && tid < r.tail) offer(Elem<T>::value(r.x[r.tail0() + tid]), r.tail0() + tid);
  }
  __syncthreads();
  // all threads read the vectors of those sets again
  const int64_t per = (sg.nv / sg.segs + kThreads) / kThreads;   // vectors a thread has at most
  for (int s = sg.s0; s < sg.s1; ++s) {
    const int64_t v0 = sg.begin(s), v1 = sg.begin(s + 1);
    const int64_t todo = S.n_sets * per;
    for (int64_t q = tid; q < todo; q += kThreads) {
      const int64_t set = div_nonneg(q, per);
      const int64_t i = v0 + S.sets[set] + (q - set * per) * kThreads;
      if (i >= v1) continue;
      float v[VEC];
      Elem<T>::unpack(r.vec(i), v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) offer(v[j], r.head + i * VEC + j);
    }
  }
  __syncthreads();
  const int n = S.n_cand;
  if (n <= kCandidates) {
    rank_keys(S.cand, n, S.best, k);
    __syncthreads();
    return;
  }
  // Many equal logits: each warp keeps its k best in its lanes.
  S.thread_max[tid] = mine;
  __syncthreads();
  uint64_t list = 0;
  for (int j = warp; j < kThreads; j += kWarps) {
    if (!(S.thread_max[j] >= thr)) continue;
    float x = -inf;
    int64_t at = 0;
    if (lane == 0 && first && j < r.head) x = Elem<T>::value(r.x[at = j]);
    if (lane == 1 && last && j < r.tail) x = Elem<T>::value(r.x[at = r.tail0() + j]);
    if (first || last) list_offer(list, k, x, at, thr);
    for (int s = sg.s0; s < sg.s1; ++s) {
      const int64_t v1 = sg.begin(s + 1);
      for (int64_t i0 = sg.begin(s) + j; i0 < v1; i0 += 32 * kThreads) {
        const int64_t i = i0 + static_cast<int64_t>(lane) * kThreads;
        float v[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[q] = -inf;
        if (i < v1) Elem<T>::unpack(r.vec(i), v);
#pragma unroll
        for (int q = 0; q < VEC; ++q) list_offer(list, k, v[q], r.head + i * VEC + q, thr);
      }
    }
  }
  S.list[warp][lane] = list;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kWarps; ++w) list_join(list, S.list[w], k);
    if (lane < k) S.best[lane] = list;
  }
  __syncthreads();
}

// One row per cluster of CTAs (of one CTA where there are rows enough). A row is
// cut into segments by its length alone, a segment is summed by the 256 threads
// of one CTA, and the segments are joined in order by the cluster's first CTA:
// the results do not depend on how many CTAs shared a row. They do depend, in the
// last places, on the remainder of the row's address by 32 bytes: its vectors, and
// with them the threads' shares, start at a multiple of that.
// UNROLL 32-byte loads in flight per thread, CTAS CTAs per SM.
template <typename T, int UNROLL, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) logprobs_kernel(const Params p) {
  constexpr int VEC = Elem<T>::kVec;
  __shared__ Shared S;
  pdl_wait();
  const int tid = threadIdx.x;
  const int C = p.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t row = C > 1 ? blockIdx.x / static_cast<unsigned>(C) : blockIdx.x;
  int64_t target = -1;
  if (p.targets) {
    target = p.targets64 ? static_cast<const int64_t*>(p.targets)[row]
                         : static_cast<const int32_t*>(p.targets)[row];
    if (target < 0) {   // a row without a token to score: nothing is read
      if (rank != 0) return;
      if (tid == 0) {
        p.logprob[row] = 0.0f;
        if (p.entropy) p.entropy[row] = 0.0f;
        if (p.stats) p.stats[row] = make_float2(0.0f, 0.0f);
      }
      if (tid < p.k) {
        p.alt_ids[row * p.k + tid] = -1;
        p.alt_lp[row * p.k + tid] = __int_as_float(0xFF800000);
      }
      return;
    }
  }
  if (C > 1) cluster_arrive();
  const Row<T> r(static_cast<const T*>(p.logits) + row * p.ld, p.V);
  const Segments sg = {r.nv, p.segments, rank * (p.segments / C), (rank + 1) * (p.segments / C)};
  const float k2 = p.k2;
  Stat st;
  if (p.fast) {
    const uint64_t kk = pair(k2, k2);
    float mine = kMask;
    for (int seg = sg.s0; seg < sg.s1; ++seg) {
      // s2 sums all vectors but the one that holds the maximum; that one's sum
      // is `top` (with the maximum's 1), its index `at`.
      st = Stat{kMask, 0.0f, 0.0f};
      uint64_t s2 = 0, t2 = 0, m2 = pair(-kMask, -kMask);
      float top = 1.0f;
      int at = -1;
      auto up = [&](float mx) {   // a new maximum: rare after the first few vectors
        const float d = (st.m - mx) * k2;
        const float c = ex2(d);
        const uint64_t cc = pair(c, c), dd = pair(d, d);
        s2 = add2(s2, pair(top, 0.0f));
        t2 = c > 0.0f ? mul2(cc, fma2(dd, s2, t2)) : 0;
        s2 = mul2(cc, s2);
        st.m = mx;
        m2 = pair(-mx, -mx);
      };
      auto add = [&](const Vec& u, int64_t i) {
        uint64_t x[VEC / 2];
        float mx, mx2;
        pairs_of(static_cast<const T*>(nullptr), u.lo, &x[0], mx);
        pairs_of(static_cast<const T*>(nullptr), u.hi, &x[VEC / 4], mx2);
        mx = fmaxf(mx, mx2);
        const bool higher = mx > st.m;
        if (higher) {
          up(mx);
          at = static_cast<int>(i);
        }
        uint64_t v2 = 0;
#pragma unroll
        for (int q = 0; q < VEC / 2; ++q) {
          const uint64_t y = mul2(add2(x[q], m2), kk);
          float a, b;
          unpair(y, a, b);
          const uint64_t e = pair(ex2(a), ex2(b));
          v2 = add2(v2, e);
          t2 = fma2(y, e, t2);
        }
        if (higher) {
          float a, b;
          unpair(v2, a, b);
          top = a + b;
        } else {
          s2 = add2(s2, v2);
        }
      };
      auto single = [&](float x) {
        x = max_nan(x, kMask);
        if (x > st.m) {
          up(x);
          top = 1.0f;
          return;
        }
        float s, s1, t, t1;
        unpair(s2, s, s1);
        unpair(t2, t, t1);
        const float y = (x - st.m) * k2;
        const float e = ex2(y);
        s2 = pair(s + e, s1);
        t2 = pair(fmaf(y, e, t), t1);
      };
      if (seg == 0 && tid < r.head) single(Elem<T>::value(r.x[tid]));
      if (seg == p.segments - 1 && tid < r.tail) single(Elem<T>::value(r.x[r.tail0() + tid]));
      const int64_t v1 = sg.begin(seg + 1);
      int64_t i = sg.begin(seg) + tid;
      for (; i + (UNROLL - 1) * kThreads < v1; i += UNROLL * kThreads) {
        Vec u[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) u[j] = r.vec(i + j * kThreads);
#pragma unroll
        for (int j = 0; j < UNROLL; ++j) add(u[j], i + j * kThreads);
      }
#pragma unroll 1
      for (; i < v1; i += 2 * kThreads) {   // what is left, two in flight
        Vec u[2];
        u[0] = r.vec(i);
        if (i + kThreads < v1) u[1] = r.vec(i + kThreads);
        add(u[0], i);
        if (i + kThreads < v1) add(u[1], i + kThreads);
      }
      float a, b;
      unpair(s2, a, b);
      const float others = a + b;
      float rest = top - 1.0f;   // of the maximum's vector
      // Up to 16 roundings beside the 1 are 2^-20: where that is not small beside
      // the sum, the vector is summed again without its (first) maximum. Rare in
      // long rows, where one lane of a row whose token is almost certain does it.
      if (others + rest < 0.25f && at >= 0) {
        float v[VEC];
        Elem<T>::unpack(r.vec(at), v);
        rest = 0.0f;
        bool found = false;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float x = max_nan(v[j], kMask);
          const bool is = !found && x == st.m;
          found |= is;
          rest += is ? 0.0f : ex2((x - st.m) * k2);
        }
      }
      st.r = others + rest;
      unpair(t2, a, b);
      st.t = a + b;
      mine = fmaxf(mine, st.m);
      st = join_warp(st, k2);
      if ((tid & 31) == 0) S.stat[seg - sg.s0][tid >> 5] = st;
    }
    join_segments(S, sg.s0, sg.s1 - sg.s0, k2, mine, p.k);
    if (p.k > 0) block_alternatives<T>(S, r, sg, mine, p.k);
    if (C > 1) {
      cluster_wait();   // all CTAs run: their shared memory can be written
      if (rank != 0 && tid < 32) {
        if (tid < sg.s1 - sg.s0) {
          const Stat& o = S.part[sg.s0 + tid];
          const uint32_t to = mapa_shared(smem_u32(&o), 0);
          st_shared_cluster(to, __float_as_uint(o.m));
          st_shared_cluster(to + 4, __float_as_uint(o.r));
          st_shared_cluster(to + 8, __float_as_uint(o.t));
        }
        if (tid < p.k) {
          const uint32_t at = mapa_shared(smem_u32(&S.part_best[rank][tid]), 0);
          st_shared_cluster(at, static_cast<uint32_t>(S.best[tid]));
          st_shared_cluster(at + 4, static_cast<uint32_t>(S.best[tid] >> 32));
        }
        __syncwarp();
      }
      cluster_arrive();
      if (rank != 0) return;
      cluster_wait();
      if (p.k > 0) {   // the best of C sorted lists
        const int n = C * p.k;
        if (tid < p.k) S.part_best[0][tid] = S.best[tid];
        __syncthreads();
        if (tid < 32) S.best[tid] = 0;
        for (int i = tid; i < n; i += kThreads) {
          const int c = i / p.k;
          S.cand[i] = S.part_best[c][i - c * p.k];
        }
        __syncthreads();
        rank_keys(S.cand, n, S.best, p.k);
      }
    }
    if (tid == 0) {
      st = S.part[0];
      for (int s = 1; s < p.segments; ++s) st.merge(S.part[s], k2);
      S.row = st;
    }
    __syncthreads();
    st = S.row;
  }
  if (!p.fast || !fast_row(st.m)) {   // the first CTA does the whole row
    const Segments all = {r.nv, 1, 0, 1};
    st = Stat{__int_as_float(0xFF800000), 0.0f, 0.0f};
    if (tid < r.head) st.add_any(Elem<T>::value(r.x[tid]), k2);
    if (tid < r.tail) st.add_any(Elem<T>::value(r.x[r.tail0() + tid]), k2);
    for (int64_t i = tid; i < r.nv; i += kThreads) {
      float x[VEC];
      Elem<T>::unpack(r.vec(i), x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) st.add_any(x[j], k2);
    }
    const float mine = st.m;
    __syncthreads();   // S is written again
    st = join_warp(st, k2);
    if ((tid & 31) == 0) S.stat[0][tid >> 5] = st;
    join_segments(S, 0, 1, k2, mine, p.k);
    st = S.part[0];
    if (p.k > 0) block_alternatives<T>(S, r, all, mine, p.k);
  }
  const float inf = __int_as_float(0x7F800000);
  const bool none = st.m == -inf && st.r == st.r;   // every logit is -inf
  const float log_s = log1pf(st.r);
  if (tid == 0) {
    if (p.targets) {
      float lp;
      if (target >= p.V) {
        set_status(p.status, MINITE_ERR_BAD_TOKEN);
        lp = __int_as_float(0x7FC00000);
      } else {
        lp = none ? -inf : fmaf(Elem<T>::value(r.x[target]) - st.m, p.inv_t, -log_s);
      }
      p.logprob[row] = lp;
    }
    if (p.entropy) p.entropy[row] = none ? 0.0f : fmaf(-kLn2, st.t / (1.0f + st.r), log_s);
    if (p.stats) p.stats[row] = none ? make_float2(-inf, 0.0f) : make_float2(fmaxf(st.m, kLowest), log_s);
  }
  if (tid < p.k) {
    const uint64_t key = S.best[tid];
    const bool ok = key != 0 && st.r == st.r;   // a NaN or +inf logit: no ranking
    p.alt_ids[row * p.k + tid] = ok ? key_index(key) : -1;
    p.alt_lp[row * p.k + tid] =
        st.r != st.r ? st.r : (ok ? fmaf(key_value(key) - st.m, p.inv_t, -log_s) : -inf);
  }
}

struct BackParams {
  const void* logits;
  int64_t ld;
  int64_t V;
  const void* targets;
  int targets64;
  float inv_t;
  const float2* stats;
  const float* entropy;
  const float* g_lp;      // or null
  const float* g_ent;     // or null
  void* d;
  int64_t ldd;
  int32_t* status;
};

constexpr int kBackChunk = 8192;   // elements of a row per CTA

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_backward_kernel(const BackParams p) {
  constexpr int VEC = 16 / sizeof(T);
  pdl_wait();
  // last rows first: the forward read them last, so L2 still holds some
  const int64_t row = gridDim.y - 1 - blockIdx.y;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kBackChunk;
  const int64_t c1 = c0 + kBackChunk < p.V ? c0 + kBackChunk : p.V;
  T* d = static_cast<T*>(p.d) + row * p.ldd;
  const T* x = static_cast<const T*>(p.logits) + row * p.ld;
  int64_t target = -1;
  if (p.targets)
    target = p.targets64 ? static_cast<const int64_t*>(p.targets)[row]
                         : static_cast<const int32_t*>(p.targets)[row];
  const float2 st = p.stats[row];
  bool zero = p.targets && target < 0;
  if (p.targets && target >= p.V) {
    if (c0 == 0 && threadIdx.x == 0) set_status(p.status, MINITE_ERR_BAD_TOKEN);
    zero = true;
  }
  if (st.x == __int_as_float(0xFF800000)) zero = true;   // no logit left: nothing depends on them
  const float gl = p.g_lp && p.targets && !zero ? p.g_lp[row] : 0.0f;
  const float ge = p.g_ent && !zero ? p.g_ent[row] : 0.0f;
  const float h = p.g_ent && !zero ? p.entropy[row] : 0.0f;
  // d = q (a y + b) with y = log2 of the probability q
  const float k2 = p.inv_t * kLog2e;
  const float log2_s = st.y * kLog2e;
  const float a = -ge * kLn2 * p.inv_t, b = -fmaf(ge, h, gl) * p.inv_t;
  // At the target 1 - q is expm1's: the difference of g_lp and g_lp q would lose
  // it where q is almost 1.
  const float b_ent = -ge * h * p.inv_t, at_target = gl * p.inv_t;
  auto grad = [&](float v, int64_t j) {
    const float y = fmaf(v - st.x, k2, -log2_s);   // NaN stays in q
    const float q = ex2(y), finite = fmaxf(y, -1e30f);
    if (j != target) return q * fmaf(a, finite, b);
    return fmaf(q, fmaf(a, finite, b_ent), -at_target * expm1f(y * kLn2));
  };
  const uintptr_t ax = reinterpret_cast<uintptr_t>(x + c0) & 15, ad = reinterpret_cast<uintptr_t>(d + c0) & 15;
  auto put = [&](int64_t j, float g) {
    if constexpr (sizeof(T) == 2) d[j] = static_cast<T>(pack_bf16x2_rn(g, 0.0f));
    else d[j] = g;
  };
  int64_t va = c0, vb = c0;
  if (ax == ad) {   // 16-byte vectors over the part where both rows are aligned
    va = c0 + static_cast<int64_t>(((16 - ax) & 15) / sizeof(T));
    if (va > c1) va = c1;
    vb = va + (c1 - va) / VEC * VEC;
  }
  if (zero) {
    for (int64_t i = va + static_cast<int64_t>(threadIdx.x) * VEC; i < vb; i += kThreads * VEC)
      *reinterpret_cast<uint4*>(d + i) = make_uint4(0, 0, 0, 0);
  } else if (fast_row(st.x) && fast_k(k2)) {
    const uint64_t kk = pair(k2, k2), mm = pair(-st.x, -st.x), ll = pair(-log2_s, -log2_s);
    const uint64_t aa = pair(a, a), bb = pair(b, b);
    // The target's element is computed by the thread that writes its vector, before
    // the loop (d may be x) and written after it: inside, it cost 8 registers and
    // 11% of the BF16 kernel's time.
    const bool own = target >= va && target < vb &&
                     static_cast<int>((target - va) / VEC % kThreads) == static_cast<int>(threadIdx.x);
    const float owned = own ? grad(Elem<T>::value(x[target]), target) : 0.0f;
    auto one = [&](const uint4& u, int64_t i) {
      uint64_t v[VEC / 2];
      float mx, g[VEC];
      pairs_of(static_cast<const T*>(nullptr), u, v, mx);
#pragma unroll
      for (int q = 0; q < VEC / 2; ++q) {
        const uint64_t y = fma2(add2(v[q], mm), kk, ll);
        float y0, y1;
        unpair(y, y0, y1);
        unpair(mul2(pair(ex2(y0), ex2(y1)), fma2(aa, y, bb)), g[2 * q], g[2 * q + 1]);
      }
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint4*>(d + i) =
            make_uint4(pack_bf16x2_rn(g[0], g[1]), pack_bf16x2_rn(g[2], g[3]),
                       pack_bf16x2_rn(g[4], g[5]), pack_bf16x2_rn(g[6], g[7]));
      else
        *reinterpret_cast<float4*>(d + i) = make_float4(g[0], g[1], g[2], g[3]);
    };
    // four loads before the first store: d may be x, so the compiler keeps their order
    constexpr int UNROLL = 4;
    int64_t i = va + static_cast<int64_t>(threadIdx.x) * VEC;
    for (; i + (UNROLL - 1) * kThreads * VEC < vb; i += UNROLL * kThreads * VEC) {
      uint4 u[UNROLL];
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) u[j] = *reinterpret_cast<const uint4*>(x + i + j * kThreads * VEC);
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) one(u[j], i + j * kThreads * VEC);
    }
    for (; i < vb; i += kThreads * VEC) one(*reinterpret_cast<const uint4*>(x + i), i);
    if (own) put(target, owned);
  } else {
    vb = va;   // element by element
  }
  const int64_t rest = (va - c0) + (c1 - vb);
  for (int64_t i = threadIdx.x; i < rest; i += kThreads) {
    const int64_t j = i < va - c0 ? c0 + i : vb + (i - (va - c0));
    put(j, zero ? 0.0f : grad(Elem<T>::value(x[j]), j));
  }
}

template <typename T>
cudaError_t launch_forward(Params& p, int64_t N, cudaStream_t s) {
  // segments of about 128 KB; without the fast sums a row is summed as a whole
  p.segments = 1;
  while (p.fast && p.segments < kMaxSegments &&
         p.V * static_cast<int64_t>(sizeof(T)) > kSegmentBytes * p.segments)
    p.segments *= 2;
  // CTAs per row: up to one a segment while about two an SM suffice for all rows
  int c = p.segments;
  while (c > 1 && N * c > 2 * num_sms()) c /= 2;
  p.cluster = c;
  if (N > 0x7FFFFFFF / c) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(N * c));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(c);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = c > 1 ? 2 : 1;
  // Short rows: a CTA's time is latency (its start, the joins, the second look),
  // so eight CTAs an SM with one load in flight each; long ones, and few: four
  // with four. 4096 rows of 32000 BF16: 58 us against 66, with 20 alternatives 78
  // against 90; of 131072: 189 against 175, 237 against 229. 512 rows of 131072
  // with 20 alternatives: 45 against 39.
  if (p.V * static_cast<int64_t>(sizeof(T)) <= 65536 && N > 4 * num_sms())
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, 1, 8>, p);
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, 4, 4>, p);
}

}  // namespace logprobs
}  // namespace minite

using namespace minite;

extern "C" int minite_token_logprobs(const void* logits, int dtype, int64_t N, int64_t V,
                                     int64_t row_stride, const void* targets, int targets_int64,
                                     float temperature, float* logprob, float* entropy, float* stats,
                                     int32_t k, int32_t* alt_ids, float* alt_logprobs,
                                     int32_t* status, minite_stream_t stream) {
  using namespace logprobs;
  if (N == 0) return MINITE_OK;
  if (!logits || (dtype != MINITE_OUT_BF16 && dtype != MINITE_OUT_FP32) || (targets && !logprob) ||
      !(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.0f / temperature) ||
      k < 0 || (k > 0 && (!alt_ids || !alt_logprobs)))
    return MINITE_ERR_INVALID_ARG;
  if (N < 0 || N > 0x7FFFFFFF || V < 1 || V > 0x7FFFFFFF || row_stride < V || k > 32 || k > V)
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(logits, dtype == MINITE_OUT_FP32 ? 4 : 2) ||
      !aligned(targets, targets_int64 ? 8 : 4) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
      !aligned(stats, 8) || !aligned(alt_ids, 4) || !aligned(alt_logprobs, 4) || !aligned(status, 4))
    return MINITE_ERR_INVALID_ARG;
  Params p = {};
  p.logits = logits;
  p.ld = row_stride;
  p.V = V;
  p.targets = targets;
  p.targets64 = targets_int64;
  p.inv_t = 1.0f / temperature;
  p.k2 = p.inv_t * kLog2e;
  p.fast = fast_k(p.k2);
  p.logprob = logprob;
  p.entropy = entropy;
  p.stats = reinterpret_cast<float2*>(stats);
  p.k = k;
  p.alt_ids = alt_ids;
  p.alt_lp = alt_logprobs;
  p.status = status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MINITE_OUT_FP32 ? launch_forward<float>(p, N, s)
                                                 : launch_forward<uint16_t>(p, N, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

extern "C" int minite_token_logprobs_backward(const void* logits, int dtype, int64_t N, int64_t V,
                                              int64_t row_stride, const void* targets,
                                              int targets_int64, float temperature,
                                              const float* stats, const float* entropy,
                                              const float* grad_logprob, const float* grad_entropy,
                                              void* dlogits, int64_t dlogits_stride,
                                              int32_t* status, minite_stream_t stream) {
  using namespace logprobs;
  if (N == 0) return MINITE_OK;
  if (!logits || !dlogits || !stats || (dtype != MINITE_OUT_BF16 && dtype != MINITE_OUT_FP32) ||
      !(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.0f / temperature) ||
      (grad_entropy && !entropy) || (grad_logprob && !targets))
    return MINITE_ERR_INVALID_ARG;
  if (N < 0 || N > 0x7FFFFFFF || V < 1 || V > 0x7FFFFFFF || row_stride < V || dlogits_stride < V)
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  const uintptr_t ea = dtype == MINITE_OUT_FP32 ? 4 : 2;
  if (!aligned(logits, ea) || !aligned(dlogits, ea) || !aligned(targets, targets_int64 ? 8 : 4) ||
      !aligned(stats, 8) || !aligned(entropy, 4) || !aligned(grad_logprob, 4) ||
      !aligned(grad_entropy, 4) || !aligned(status, 4))
    return MINITE_ERR_INVALID_ARG;
  if (dlogits == logits && dlogits_stride != row_stride) return MINITE_ERR_INVALID_ARG;
  BackParams p = {};
  p.logits = logits;
  p.ld = row_stride;
  p.V = V;
  p.targets = targets;
  p.targets64 = targets_int64;
  p.inv_t = 1.0f / temperature;
  p.stats = reinterpret_cast<const float2*>(stats);
  p.entropy = entropy;
  p.g_lp = grad_logprob;
  p.g_ent = grad_entropy;
  p.d = dlogits;
  p.ldd = dlogits_stride;
  p.status = status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned chunks = static_cast<unsigned>((V + kBackChunk - 1) / kBackChunk);
  // a grid has at most 65535 rows
  for (int64_t r0 = 0; r0 < N;) {
    const int64_t rows = N - r0 < 65535 ? N - r0 : 65535;
    const dim3 grid(chunks, static_cast<unsigned>(rows));
    BackParams q = p;
    q.logits = static_cast<const char*>(logits) + r0 * row_stride * static_cast<int64_t>(ea);
    q.d = static_cast<char*>(dlogits) + r0 * dlogits_stride * static_cast<int64_t>(ea);
    if (targets) q.targets = static_cast<const char*>(targets) + r0 * (targets_int64 ? 8 : 4);
    q.stats = p.stats + r0;
    if (entropy) q.entropy = entropy + r0;
    if (grad_logprob) q.g_lp = grad_logprob + r0;
    if (grad_entropy) q.g_ent = grad_entropy + r0;
    const cudaError_t e =
        dtype == MINITE_OUT_FP32
            ? launch_pdl(logprobs_backward_kernel<float>, grid, dim3(kThreads), 0, s, q)
            : launch_pdl(logprobs_backward_kernel<uint16_t>, grid, dim3(kThreads), 0, s, q);
    if (e != cudaSuccess) return MINITE_ERR_CUDA;
    r0 += rows;
  }
  return cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}
