// minite_verify_drafts: drafted tokens verified against the target's
// probabilities, and the token that follows the ones that stand, from given
// random numbers (speculative sampling; Leviathan, Kalman and Matias, 2023, and
// Chen and others, 2023).
//
// With p = softmax(target / T) of a position and q = softmax(draft / T), draft x
// stands where u q(x) < p(x): with probability min(1, p(x) / q(x)) for uniform u.
// The first that falls is replaced by a sample of max(p - q, 0), and where all
// stand one more token is a sample of p, so that every token is distributed as p.
// A sample of weights r is argmax r_j / e_j for exponential variates e_j: the
// variates' race, which needs neither the weights' sum nor an order of additions.
//
// Two launches. stats_kernel streams the rows that may matter (draft i's, and the
// target's up to the position after the last draft) once, a CTA 32 KB of a row,
// and leaves the largest logit and the sum of each such segment: no loop, the
// whole segment is in registers between the two passes over it. race_kernel, a
// number of CTAs a sequence, joins the segments of the sequence's rows, looks at
// every draft (each CTA for itself) and runs the race over its part of the one row
// that is sampled from; the CTAs' winners meet in one 64-bit maximum.
//
// 64 sequences with up to four drafts of 100003 BF16 tokens take 32 us, 19 of them the
// statistics (92 MB, 4.8 TB/s, 64% of the issue slots in longer runs), 13 the race (45
// MB; some 5 of it are its start, the chain of loads by which a CTA learns which row
// is sampled from, and the meeting of the winners). 128 sequences with four drafts of
// 131072: 81 us (437 MB). One sequence: 7.4 us of latency, and 24 of the host's. One
// token sampled by each of 128 sequences, without drafts: 30 us (101 MB; the logits are
// read by both kernels).
//
// Sums are kept without the maximum's own term, r = s - 1, and log s = log1p(r):
// the log probability of an almost certain token is not lost beside the 1.
#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVectors = 4;       // 32-byte vectors a thread holds of its segment
constexpr int kRaceCtas = 4;      // of an SM
constexpr int kMaxDrafts = 31;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  const void* target;       // [B][S + 1][V]
  const void* draft;        // [B][S][V], or null
  int64_t target_ld, draft_ld, noise_ld;
  const int32_t* draft_tokens;  // [B][S]
  const float* uniforms;        // [B][S]
  const float* noise;           // [B][V]
  int64_t V;
  int S;
  float inv_t, k2;          // 1 / T, log2(e) / T
  int target_segs, draft_segs;
  float2* target_part;      // [B][S + 1][target_segs] {largest logit, sum without one maximum}
  float2* draft_part;       // [B][S][draft_segs]
  unsigned long long* best; // [B] the race so far, zeroed by stats_kernel
  uint32_t* arrived;        // [B] CTAs that have run their part, likewise
  int ctas;                 // of a sequence in race_kernel
  int32_t* tokens;          // [B][S + 1]
  float* logprobs;          // [B][S + 1], or null
  int32_t* accepted;        // [B]
  int32_t* status;
};

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// 2^x, within 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <typename T> constexpr int kPerVec = 32 / static_cast<int>(sizeof(T));
template <typename T> inline int segments(int64_t V) {
  constexpr int64_t per = static_cast<int64_t>(kThreads) * kVectors * kPerVec<T>;
  return static_cast<int>((V + per - 1) / per);
}

struct Vec { uint32_t w[8]; };
__device__ __forceinline__ Vec load_vec(const void* p) {
  Vec v;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                 "=r"(v.w[7]) : "l"(p) : "memory");
  return v;
}
template <typename T> __device__ __forceinline__ void values(const Vec& v, float (&x)[kPerVec<T>]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v.w[i]);
  } else {
    unpack_bf16x16(v.w, x);
  }
}

// The largest of a thread's logits, NaN if there is one.
template <typename T> __device__ __forceinline__ float max_of(const Vec (&v)[kVectors]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max_nan(m, __uint_as_float(v[i].w[j]));
    return m;
  } else {
    uint32_t m = v[0].w[0];
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(v[i].w[j]));
    return max_nan(bf16lo(m), bf16hi(m));
  }
}

// A set of logits: the largest, and the sum of 2^((x - m) k) over the others. No
// logit above -inf: m = -inf. NaN and +inf stay in m.
__device__ __forceinline__ float2 join(float2 a, float2 b, float k) {
  const float m = max_nan(a.x, b.x);
  if (!(fabsf(m) < INFINITY)) return make_float2(m, 0.0f);
  const float ca = ex2((a.x - m) * k), cb = ex2((b.x - m) * k);   // -inf: 0
  float r = a.x == m && b.x == m ? 1.0f : 0.0f;   // one maximum of the two counts
  r += a.x == m ? a.y : ca * (a.y + 1.0f);
  r += b.x == m ? b.y : cb * (b.y + 1.0f);
  return make_float2(m, r);
}
// One segment of one row: its largest logit, then the sum over the others. Only the
// warps that hold the largest look at every element for it; the rest add two
// elements an instruction.
template <typename T>
__device__ __forceinline__ void segment(const T* row, int64_t V, int seg, int segs, float k, float2* out) {
  __shared__ float s_max[kWarps], s_sum[kWarps];
  constexpr int kPer = kPerVec<T>;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  // the row as a head up to a 32-byte boundary, vectors, and a tail
  int head = static_cast<int>(((32 - (reinterpret_cast<uintptr_t>(row) & 31)) & 31) / sizeof(T));
  if (head > V) head = static_cast<int>(V);
  const int64_t nv = (V - head) / kPer;
  const int tail = static_cast<int>(V - head - nv * kPer);
  const int64_t v0 = static_cast<int64_t>(seg) * kThreads * kVectors + tid;
  Vec v[kVectors];
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    if (v0 + i * kThreads < nv) {
      v[i] = load_vec(row + head + (v0 + i * kThreads) * kPer);
    } else {   // logits of -inf
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i].w[j] = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
    }
  }
  float xh = -INFINITY, xt = -INFINITY;
  if (seg == 0 && tid < head) xh = value(row[tid]);
  if (seg == segs - 1 && tid < tail) xt = value(row[V - tail + tid]);
  const float mine = max_nan(max_nan(xh, xt), max_of<T>(v));
  float m = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_max[wid] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = max_nan(m, s_max[w]);
  if (!(fabsf(m) < INFINITY)) {   // no logit, or no probabilities
    if (tid == 0) *out = make_float2(m, 0.0f);
    return;
  }
  float r;
  // |m| k at or above 2^24 (a temperature near 0, rows of the type's lowest value): the
  // difference first, too. What the product below loses is up to 2^-24 of it, and
  // would be no factor that FP32 holds.
  const float mk = -(m * k);
  if (__any_sync(0xffffffffu, mine == m) || !(fabsf(mk) < 0x1p24f)) {
    float n = 0.0f;
    r = 0.0f;
    auto add = [&](float x) {
      if (x == m) n += 1.0f;
      else r += ex2((x - m) * k);
    };
    add(xh);
    add(xt);
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      float x[kPer];
      values<T>(v[i], x);
#pragma unroll
      for (int j = 0; j < kPer; ++j) add(x[j]);
    }
    // the lanes' counts, less the one maximum that is left out
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      r += __shfl_xor_sync(0xffffffffu, r, o);
      n += __shfl_xor_sync(0xffffffffu, n, o);
    }
    bool first = s_max[wid] == m;
    for (int w = 0; w < wid; ++w) first &= s_max[w] != m;
    r += first ? n - 1.0f : n;
  } else {
    // x k - m k in one operation: what the product m k lost, at most 1/2, is a factor of
    // every term
    const float lost = fmaf(m, k, mk);
    uint64_t acc = pair(ex2(fmaf(xh, k, mk)), ex2(fmaf(xt, k, mk)));
    const uint64_t minus = pair(mk, mk), k2 = pair(k, k);
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      float x[kPer];
      values<T>(v[i], x);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        float a, b;
        unpair(fma2(pair(x[j], x[j + 1]), k2, minus), a, b);
        acc = add2(acc, pair(ex2(a), ex2(b)));
      }
    }
    float a, b;
    unpair(acc, a, b);
    r = (a + b) * ex2(-lost);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  }
  if (lane == 0) s_sum[wid] = r;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) r += s_sum[w];
    *out = make_float2(m, r);
  }
}

template <typename T, typename D>
__global__ void __launch_bounds__(kThreads) stats_kernel(const Params p, int64_t B) {
  pdl_wait();
  pdl_trigger();
  const int64_t target_units = B * (p.S + 1) * p.target_segs;
  int64_t u = blockIdx.x;
  if (u < target_units) {
    const int64_t row = div_nonneg(u, p.target_segs);
    const int seg = static_cast<int>(u - row * p.target_segs);
    const int64_t b = div_nonneg(row, p.S + 1);
    const int i = static_cast<int>(row - b * (p.S + 1));
    if (i == 0 && seg == 0 && threadIdx.x == 0) {
      p.best[b] = 0;
      p.arrived[b] = 0;
    }
    if (i > 0) {   // a position behind a missing draft is not reached
      const int x = p.draft_tokens[b * p.S + i - 1];
      if (x < 0 || x >= p.V) return;
    }
    segment<T>(static_cast<const T*>(p.target) + row * p.target_ld, p.V, seg, p.target_segs, p.k2,
               p.target_part + u);
  } else {
    u -= target_units;
    const int64_t row = div_nonneg(u, p.draft_segs);
    const int x = p.draft_tokens[row];
    if (x < 0 || x >= p.V) return;
    segment<D>(static_cast<const D*>(p.draft) + row * p.draft_ld, p.V,
               static_cast<int>(u - row * p.draft_segs), p.draft_segs, p.k2, p.draft_part + u);
  }
}

// A row's probabilities: p(x) = 2^((x - m) k - shift).
struct Row {
  float m, log_s;
  __device__ __forceinline__ bool usable() const { return fabsf(m) < INFINITY && fabsf(log_s) < INFINITY; }
  __device__ __forceinline__ float p(float x, float k, float shift) const { return ex2(fmaf(x - m, k, -shift)); }
  __device__ __forceinline__ float p(float x, float k) const { return p(x, k, log_s * kLog2e); }
};
// A row's first 32 segments, one a lane of a warp, and the row that all of them make.
__device__ __forceinline__ float2 first_part(const float2* part, int segs) {
  const int lane = threadIdx.x & 31;
  return lane < segs ? part[lane] : make_float2(-INFINITY, 0.0f);
}
__device__ __forceinline__ Row row_of(float2 v, const float2* part, int segs, float k) {
  for (int s = 32 + (threadIdx.x & 31); s < segs; s += 32) v = join(v, part[s], k);
  float m = v.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool top = v.x == m;
  float r = top ? v.y : ex2((v.x - m) * k) * (v.y + 1.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  r += static_cast<float>(__popc(__ballot_sync(0xffffffffu, top)) - 1);   // one maximum is left out
  return {m, log1pf(r)};   // m is not finite: not usable, whatever r is
}

// The race: the largest weight / variate, the lower index where they are equal. No
// weight above 0: v stays 0.
struct Lead {
  float v = 0.0f;
  int32_t j = 0;
  // Weight (0 or more) times the variate's reciprocal, within 2 units; offered in
  // rising order. Negative variates and NaN make a quotient that leads nothing, and so
  // does a weight of 0 with any variate. The sum takes -0 to 0.
  __device__ __forceinline__ void offer(float weight, float e, int32_t at) {
    float q;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(e + 0.0f));
    q *= weight;
    if (q > v) {
      v = q;
      j = at;
    }
  }
  __device__ __forceinline__ unsigned long long key() const {
    return v > 0.0f ? (static_cast<unsigned long long>(__float_as_uint(v)) << 32) |
                          (0xFFFFFFFFu - static_cast<uint32_t>(j))
                    : 0ull;
  }
};
__device__ __forceinline__ unsigned long long warp_larger(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u > v ? u : v;
  }
  return v;
}

constexpr int kAhead = 8;   // elements of a thread in flight
constexpr int kRound = kThreads * kAhead;

// Elements [j0, j1) of the race. WITH_Q: less the draft's probabilities; otherwise
// token `without` has none. Some 20 instructions an element; whole rounds carry no
// checks (with them, 60).
template <bool WITH_Q, typename T, typename D>
__device__ __forceinline__ Lead race(const T* xt, const D* xd, const float* noise, Row rt, Row rd, float k,
                                     int32_t without, int32_t j0, int32_t j1) {
  Lead lead;
  const float st = rt.log_s * kLog2e, sd = rd.log_s * kLog2e;
  auto weight = [&](T a, D b, int32_t j) {
    float w = rt.p(value(a), k, st);
    if (WITH_Q) w = fmaxf(w - rd.p(value(b), k, sd), 0.0f);   // below 0 a negative variate would make it win
    else if (j == without) w = 0.0f;
    return w;
  };
  auto round = [&](int32_t j, bool whole) {
    const T* pa = xt + j;
    const D* pb = xd + j;
    const float* pe = noise + j;
    T a[kAhead];
    D b[kAhead];
    float e[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (whole || j + i * kThreads < j1) {
        e[i] = pe[i * kThreads];
        a[i] = pa[i * kThreads];
        if (WITH_Q) b[i] = pb[i * kThreads];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (whole || j + i * kThreads < j1)
        lead.offer(weight(a[i], b[i], j + i * kThreads), e[i], j + i * kThreads);
  };
  int32_t j = j0;
  for (; j1 - j >= kRound; j += kRound) round(j + threadIdx.x, true);
  if (j < j1) round(j + threadIdx.x, false);
  return lead;
}

template <typename T, typename D>
__global__ void __launch_bounds__(kThreads, kRaceCtas) race_kernel(const Params p) {
  __shared__ Row s_target[kMaxDrafts + 1], s_draft[kMaxDrafts + 1];
  __shared__ uint8_t s_given[kMaxDrafts + 1], s_stands[kMaxDrafts + 1];
  __shared__ unsigned long long s_best[kWarps];
  __shared__ int s_last;
  const int64_t b = div_nonneg(blockIdx.x, p.ctas);
  const int rank = static_cast<int>(blockIdx.x - b * p.ctas);
  // whole rounds a CTA, but for the last
  const int32_t rounds = static_cast<int32_t>((p.V + kRound - 1) / kRound);
  const int32_t j0 = static_cast<int32_t>(static_cast<int64_t>(rounds) * rank / p.ctas) * kRound;
  const int32_t j1 = min(static_cast<int32_t>(p.V),
                         static_cast<int32_t>(static_cast<int64_t>(rounds) * (rank + 1) / p.ctas) * kRound);
  const float* noise = p.noise + b * p.noise_ld;
  // the variates that this CTA will need, into L2 while the statistics are finished
  // and the drafts looked at
  for (int32_t j = j0 + 32 * static_cast<int32_t>(threadIdx.x); j < j1; j += 32 * kThreads)
    asm volatile("prefetch.global.L2 [%0];" :: "l"(noise + j));
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const T* target = static_cast<const T*>(p.target) + b * (p.S + 1) * p.target_ld;
  const D* draft = p.draft ? static_cast<const D*>(p.draft) + b * p.S * p.draft_ld : nullptr;
  const int32_t* drafts = p.draft_tokens + b * p.S;
  for (int i = wid; i <= p.S; i += kWarps) {   // a warp a position
    const int before = i > 0 ? drafts[i - 1] : 0, x = i < p.S ? drafts[i] : -1;
    // asked for together; where the row is not reached they were not written, and are not used
    const float2* target_part = p.target_part + (b * (p.S + 1) + i) * p.target_segs;
    const float2* draft_part = p.draft_part + (b * p.S + i) * p.draft_segs;
    const bool with_draft = draft && i < p.S;
    const float2 vt = first_part(target_part, p.target_segs);
    const float2 vd = first_part(draft_part, with_draft ? p.draft_segs : 0);
    const bool reached = before >= 0 && before < p.V, given = x >= 0 && x < p.V;
    float xt = 0.0f, xd = 0.0f, u = 0.0f;
    if (given) {
      xt = value(target[i * p.target_ld + x]);
      if (draft) xd = value(draft[i * p.draft_ld + x]);
      u = p.uniforms[b * p.S + i];
    }
    const Row rt = row_of(vt, target_part, p.target_segs, p.k2);
    Row rd = {0.0f, 0.0f};
    if (with_draft) rd = row_of(vd, draft_part, p.draft_segs, p.k2);
    if (lane == 0) {
      bool stands = false;
      if (reached && given && rt.usable() && rd.usable()) {
        const float qx = draft ? rd.p(xd, p.k2) : 1.0f;
        stands = u * qx < rt.p(xt, p.k2);
      }
      s_target[i] = rt;
      s_draft[i] = rd;
      s_given[i] = given;
      s_stands[i] = stands;
    }
  }
  __syncthreads();
  int n = 0;   // drafts that stand
  while (n < p.S && s_stands[n]) ++n;
  const bool falls = n < p.S && s_given[n];   // draft n is there and does not
  const Row rt = s_target[n], rd = s_draft[n];
  const bool usable = rt.usable() && (!falls || rd.usable());
  const T* xt = target + n * p.target_ld;
  unsigned long long best = 0;
  if (usable) {
    Lead lead;
    if (falls && draft)
      lead = race<true>(xt, draft + n * p.draft_ld, noise, rt, rd, p.k2, -1, j0, j1);
    else
      lead = race<false>(xt, xt, noise, rt, rt, p.k2, falls ? drafts[n] : -1, j0, j1);
    best = warp_larger(lead.key());
  }
  if (lane == 0) s_best[wid] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) best = s_best[w] > best ? s_best[w] : best;
    if (best) atomicMax(p.best + b, best);
    __threadfence();
    s_last = atomicAdd(p.arrived + b, 1u) == static_cast<uint32_t>(p.ctas) - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  best = *reinterpret_cast<volatile unsigned long long*>(p.best + b);
  if (usable && best == 0) {   // q is as large as p everywhere but for roundings: p itself
    best = warp_larger(race<false>(xt, xt, noise, rt, rt, p.k2, -1, 0, static_cast<int32_t>(p.V)).key());
    if (lane == 0) s_best[wid] = best;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) best = s_best[w] > best ? s_best[w] : best;
  }
  if (wid != 0) return;
  const int32_t next = best ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
  if (lane == 0) {
    p.accepted[b] = n;
    int given = 0;   // what ends the drafts may be a token out of range
    while (given < p.S && s_given[given]) ++given;
    if (given < p.S && drafts[given] >= 0) set_status(p.status, MINITE_ERR_BAD_TOKEN);
  }
  if (lane <= p.S) {
    const int32_t x = lane < n ? drafts[lane] : lane == n ? next : -1;
    p.tokens[b * (p.S + 1) + lane] = x;
    if (p.logprobs) {
      float lp = 0.0f;
      if (x >= 0) lp = (value(target[lane * p.target_ld + x]) - s_target[lane].m) * p.inv_t - s_target[lane].log_s;
      else if (lane == n) lp = __int_as_float(0x7FC00000);   // nothing to sample from
      p.logprobs[b * (p.S + 1) + lane] = lp;
    }
  }
}

template <typename T, typename D>
cudaError_t launch(Params& p, int64_t B, cudaStream_t s) {
  const int64_t units = B * ((p.S + 1) * static_cast<int64_t>(p.target_segs) + static_cast<int64_t>(p.S) * p.draft_segs);
  if (units > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaError_t e = launch_pdl(stats_kernel<T, D>, dim3(static_cast<unsigned>(units)), dim3(kThreads), 0, s, p, B);
  if (e != cudaSuccess) return e;
  // CTAs of a sequence: one round of its threads' loads each where sequences are
  // few, otherwise as many as are resident at once (the look at the drafts costs every
  // CTA some 2 us). The quotient is rounded down: 256, 304, 305, 400, 608, 609, 1000
  // sequences with two drafts of 32768 BF16 take 32.4, 35.8, 42.1, 50.0, 66.5, 70.2, 106
  // us, 126, 118, 138, 125, 109, 115, 106 ns a sequence.
  int64_t ctas = (p.V + kRound - 1) / kRound;
  const int64_t resident = kRaceCtas * static_cast<int64_t>(num_sms());
  const int64_t fill = resident / B > 1 ? resident / B : 1;
  if (ctas > fill) ctas = fill;
  p.ctas = static_cast<int>(ctas);
  return launch_pdl(race_kernel<T, D>, dim3(static_cast<unsigned>(B * ctas)), dim3(kThreads), 0, s, p);
}

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
// Segments are counted for FP32 rows, which have the most.
inline size_t target_bytes(int64_t B, int64_t S, int64_t V) {
  return align256(static_cast<size_t>(B) * (S + 1) * segments<float>(V) * sizeof(float2));
}
inline size_t draft_bytes(int64_t B, int64_t S, int64_t V) {
  return align256(static_cast<size_t>(B) * S * segments<float>(V) * sizeof(float2));
}

}  // namespace verify

size_t verify_workspace_bytes(int64_t B, int64_t S, int64_t V) {
  using namespace verify;
  return target_bytes(B, S, V) + draft_bytes(B, S, V) + align256(static_cast<size_t>(B) * 12);
}

}  // namespace minite

using namespace minite;

extern "C" int minite_verify_drafts(const void* target, int target_dtype, int64_t target_stride, const void* draft,
                                    int draft_dtype, int64_t draft_stride, const int32_t* draft_tokens,
                                    const float* uniforms, const float* noise, int64_t noise_stride, int64_t B,
                                    int32_t S, int64_t V, float temperature, int32_t* tokens, int32_t* accepted,
                                    float* logprobs, void* workspace, size_t ws_bytes, int32_t* status,
                                    minite_stream_t stream) {
  using namespace verify;
  const bool tf = target_dtype == MINITE_OUT_FP32, df = draft_dtype == MINITE_OUT_FP32;
  const float k2 = static_cast<float>(1.4426950408889634 / static_cast<double>(temperature));   // one rounding
  if ((!tf && target_dtype != MINITE_OUT_BF16) || (draft && !df && draft_dtype != MINITE_OUT_BF16) ||
      !(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(k2))
    return MINITE_ERR_INVALID_ARG;
  if (B < 0 || S < 0 || S > kMaxDrafts || V < 1 || V > (int64_t(1) << 30) || B > (int64_t(1) << 31) ||
      B * (S + 1) * V > (int64_t(1) << 42) || B * (2 * S + 1) > (int64_t(1) << 24) || target_stride < V ||
      (draft && draft_stride < V) || noise_stride < V)
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return MINITE_OK;
  if (!target || !noise || !tokens || !accepted || !workspace || (S > 0 && (!draft_tokens || !uniforms)) ||
      !aligned(target, tf ? 4 : 2) || !aligned(draft, df ? 4 : 2) || !aligned(draft_tokens, 4) ||
      !aligned(uniforms, 4) || !aligned(noise, 4) || !aligned(tokens, 4) || !aligned(accepted, 4) ||
      !aligned(logprobs, 4) || !aligned(workspace, 256) || !aligned(status, 4) ||
      ws_bytes < verify_workspace_bytes(B, S, V))
    return MINITE_ERR_INVALID_ARG;
  if (S == 0) draft = nullptr;
  Params p = {};
  char* ws = static_cast<char*>(workspace);
  p.target_part = reinterpret_cast<float2*>(ws);
  ws += target_bytes(B, S, V);
  p.draft_part = reinterpret_cast<float2*>(ws);
  ws += draft_bytes(B, S, V);
  p.best = reinterpret_cast<unsigned long long*>(ws);
  p.arrived = reinterpret_cast<uint32_t*>(p.best + B);
  p.target = target;
  p.draft = draft;
  p.target_ld = target_stride;
  p.draft_ld = draft_stride;
  p.noise_ld = noise_stride;
  p.draft_tokens = draft_tokens;
  p.uniforms = uniforms;
  p.noise = noise;
  p.V = V;
  p.S = S;
  p.inv_t = 1.0f / temperature;
  p.k2 = k2;
  p.target_segs = tf ? segments<float>(V) : segments<uint16_t>(V);
  p.draft_segs = !draft ? 0 : df ? segments<float>(V) : segments<uint16_t>(V);
  p.tokens = tokens;
  p.logprobs = logprobs;
  p.accepted = accepted;
  p.status = status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (tf) e = df ? launch<float, float>(p, B, s) : launch<float, uint16_t>(p, B, s);
  else e = df ? launch<uint16_t, float>(p, B, s) : launch<uint16_t, uint16_t>(p, B, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}
