// minite_token_logprobs / minite_token_logprobs_backward: the log probability
// of a given token of each row of logits, the row's entropy and its top
// alternatives, and the gradient of the first two.
//
// With y = x / T over a row's V logits, M = max y, s = sum exp(y - M) and
// t = sum (y - M) exp(y - M):
//   log p_j = y_j - M - log s,  logprob = log p_i,  H = log s - t / s
//   dx_j = (1/T) (g_lp ([j = i] - p_j) - g_H p_j (log p_j + H))
// M (as a logit) and log s are kept apart for the backward: their sum would
// lose log s beside a large M.
// M, s and t come from one pass: a running maximum, with s and t moved to the
// new one when it grows (s <- c s, t <- c (t + d s) for a shift d, c = exp d).
//
// The top alternatives cost the streaming loop nothing. Every thread's running
// maximum is the largest of the values it saw, so the k-th largest of these
// maxima is a lower bound of the row's k-th largest logit, and only threads
// whose maximum reaches it can hold one of the top k (about k of them): a warp
// then reads those threads' elements again, from L2, and keeps its k best in
// its lanes. Equal logits rank by the lower index.
#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace logprobs {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e+38f;

struct Params {
  const void* logits;
  int64_t ld;
  int64_t V;
  const void* targets;      // int32 or int64 [N], or null
  int targets64;
  float inv_t;
  float* logprob;
  float* entropy;
  float2* stats;            // [N] {largest logit, log s}, or null
  int k;
  int32_t* alt_ids;
  float* alt_lp;
  int32_t* status;
};

template <typename T> struct Elem;
template <> struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float value(float x) { return x; }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
};
template <> struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float value(uint16_t x) {
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) { unpack_bf16x8(u, x); }
};

// A row as an unaligned head, 16-byte vectors and a tail.
template <typename T>
struct Row {
  const T* x;
  int64_t V;
  int head, tail;
  int64_t nv;
  __device__ __forceinline__ Row(const T* row, int64_t V_) : x(row), V(V_) {
    const uintptr_t off = (16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15;
    head = static_cast<int>(off / sizeof(T));
    if (head > V) head = static_cast<int>(V);
    nv = (V - head) / Elem<T>::kVec;
    tail = static_cast<int>(V - head - nv * Elem<T>::kVec);
  }
  __device__ __forceinline__ uint4 vec(int64_t i) const {
    return __ldg(reinterpret_cast<const uint4*>(x + head) + i);
  }
  __device__ __forceinline__ int64_t tail0() const { return head + nv * Elem<T>::kVec; }
};

// Running (maximum, sum, weighted sum) of a set of logits; `k` turns a
// difference of logits into a power of two.
struct Stat {
  float m = kLowest, s = 0.0f, t = 0.0f;
  __device__ __forceinline__ void raise(float nm, float k) {
    const float d = m - nm;
    const float c = exp2f(d * k);
    t = c > 0.0f ? c * (t + d * s) : 0.0f;   // d * s may be infinite where c is 0
    s = c * s;
    m = nm;
  }
  __device__ __forceinline__ void add(float x, float k) {
    const float d = x - m;
    const float e = exp2f(d * k);
    s += e;
    t += fmaxf(d, -1e30f) * e;   // a masked logit (-inf) adds 0, not -inf * 0
  }
  __device__ __forceinline__ void merge(const Stat& o, float k) {
    Stat a = o;
    if (a.m > m) raise(a.m, k);
    else if (a.m < m) a.raise(m, k);
    s += a.s;
    t += a.t;
  }
};

__device__ __forceinline__ Stat shfl_xor(const Stat& a, int o) {
  Stat r;
  r.m = __shfl_xor_sync(0xffffffffu, a.m, o);
  r.s = __shfl_xor_sync(0xffffffffu, a.s, o);
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

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const Params p) {
  constexpr int VEC = Elem<T>::kVec;
  __shared__ float s_m[kThreads];
  __shared__ Stat s_stat[kWarps];
  __shared__ uint32_t s_thr;
  __shared__ uint64_t s_list[kWarps][32];
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x;
  int64_t target = -1;
  if (p.targets) {
    target = p.targets64 ? static_cast<const int64_t*>(p.targets)[row]
                         : static_cast<const int32_t*>(p.targets)[row];
    if (target < 0) {   // a row without a token to score: nothing is read
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
  const Row<T> r(static_cast<const T*>(p.logits) + row * p.ld, p.V);
  const float k2 = p.inv_t * kLog2e;
  Stat st;
  if (tid < r.head) {
    const float x = Elem<T>::value(r.x[tid]);
    if (x > st.m) st.raise(x, k2);
    st.add(x, k2);
  }
  if (tid < r.tail) {
    const float x = Elem<T>::value(r.x[r.tail0() + tid]);
    if (x > st.m) st.raise(x, k2);
    st.add(x, k2);
  }
  for (int64_t i = tid; i < r.nv; i += kThreads) {
    float x[VEC];
    Elem<T>::unpack(r.vec(i), x);
    float vm = x[0];
#pragma unroll
    for (int j = 1; j < VEC; ++j) vm = fmaxf(vm, x[j]);
    if (vm > st.m) st.raise(vm, k2);
#pragma unroll
    for (int j = 0; j < VEC; ++j) st.add(x[j], k2);
  }
  const float mine_max = st.m;
  s_m[tid] = mine_max;
  if (tid == 0) s_thr = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) st.merge(shfl_xor(st, o), k2);
  if (lane == 0) s_stat[warp] = st;
  __syncthreads();
  st = s_stat[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) st.merge(s_stat[w], k2);
  const float inf = __int_as_float(0x7F800000);
  const float log_s = logf(st.s);
  const bool none = st.s == 0.0f;   // every logit is -inf
  if (tid == 0) {
    if (p.targets) {
      float lp;
      if (target >= p.V) {
        set_status(p.status, MINITE_ERR_BAD_TOKEN);
        lp = __int_as_float(0x7FC00000);
      } else {
        lp = none ? -inf : (Elem<T>::value(r.x[target]) - st.m) * p.inv_t - log_s;
      }
      p.logprob[row] = lp;
    }
    if (p.entropy) p.entropy[row] = none ? 0.0f : log_s - (st.t / st.s) * p.inv_t;
    if (p.stats) p.stats[row] = make_float2(none ? -inf : st.m, none ? 0.0f : log_s);
  }
  if (p.k == 0) return;
  // threshold: the largest thread maximum that at least k maxima reach
  int reach = 0;
  for (int j = 0; j < kThreads; ++j) reach += s_m[j] >= mine_max ? 1 : 0;
  if (reach >= p.k) atomicMax(&s_thr, static_cast<uint32_t>(rank_key(mine_max, 0) >> 32));
  __syncthreads();
  float thr = key_value(static_cast<uint64_t>(s_thr) << 32);
  if (thr <= kLowest) thr = -inf;   // a thread without elements has this maximum too
  uint64_t list = 0;
  for (int j = warp; j < kThreads; j += kWarps) {
    if (!(s_m[j] >= thr)) continue;
    float x = -inf;
    int64_t at = 0;
    if (lane == 0 && j < r.head) x = Elem<T>::value(r.x[at = j]);
    if (lane == 1 && j < r.tail) x = Elem<T>::value(r.x[at = r.tail0() + j]);
    list_offer(list, p.k, x, at, thr);
    for (int64_t i0 = j; i0 < r.nv; i0 += 32 * kThreads) {
      const int64_t i = i0 + static_cast<int64_t>(lane) * kThreads;
      float v[VEC];
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[q] = -inf;
      if (i < r.nv) Elem<T>::unpack(r.vec(i), v);
#pragma unroll
      for (int q = 0; q < VEC; ++q) list_offer(list, p.k, v[q], r.head + i * VEC + q, thr);
    }
  }
  s_list[warp][lane] = list;
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < kWarps; ++w)
    for (int l = 0; l < p.k; ++l) {
      const uint64_t cand = s_list[w][l];
      if (cand <= __shfl_sync(0xffffffffu, list, p.k - 1)) break;   // the lists are sorted
      list_insert(list, cand);
    }
  if (lane < p.k) {
    const bool ok = list != 0 && st.s == st.s;   // a NaN or +inf logit: no ranking
    p.alt_ids[row * p.k + lane] = ok ? key_index(list) : -1;
    p.alt_lp[row * p.k + lane] =
        st.s != st.s ? st.s : (ok ? (key_value(list) - st.m) * p.inv_t - log_s : -inf);
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
  constexpr int VEC = Elem<T>::kVec;
  pdl_wait();
  const int64_t row = blockIdx.y;
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
  auto grad = [&](float v, int64_t j) {
    const float lp = fmaf(v - st.x, p.inv_t, -st.y);
    const float q = exp2f(lp * kLog2e);
    float g = -q * fmaf(ge, fmaxf(lp, -1e30f) + h, gl);
    if (j == target) g += gl;
    return zero ? 0.0f : g * p.inv_t;
  };
  const uintptr_t ax = reinterpret_cast<uintptr_t>(x + c0) & 15, ad = reinterpret_cast<uintptr_t>(d + c0) & 15;
  int64_t a = c0, b = c0;
  if (ax == ad) {   // 16-byte vectors over the part where both rows are aligned
    a = c0 + static_cast<int64_t>(((16 - ax) & 15) / sizeof(T));
    if (a > c1) a = c1;
    b = a + (c1 - a) / VEC * VEC;
  }
  for (int64_t i = a + static_cast<int64_t>(threadIdx.x) * VEC; i < b; i += kThreads * VEC) {
    float v[VEC];
    if (!zero) Elem<T>::unpack(*reinterpret_cast<const uint4*>(x + i), v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = zero ? 0.0f : grad(v[j], i + j);
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint4*>(d + i) =
          make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                     pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
    else
      *reinterpret_cast<float4*>(d + i) = make_float4(v[0], v[1], v[2], v[3]);
  }
  const int64_t rest = (a - c0) + (c1 - b);
  for (int64_t i = threadIdx.x; i < rest; i += kThreads) {
    const int64_t j = i < a - c0 ? c0 + i : b + (i - (a - c0));
    const float g = zero ? 0.0f : grad(Elem<T>::value(x[j]), j);
    if constexpr (sizeof(T) == 2) d[j] = static_cast<T>(pack_bf16x2_rn(g, 0.0f));
    else d[j] = g;
  }
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
      !aligned(stats, 8) || !aligned(alt_ids, 4) || !aligned(alt_logprobs, 4))
    return MINITE_ERR_INVALID_ARG;
  Params p = {};
  p.logits = logits;
  p.ld = row_stride;
  p.V = V;
  p.targets = targets;
  p.targets64 = targets_int64;
  p.inv_t = 1.0f / temperature;
  p.logprob = logprob;
  p.entropy = entropy;
  p.stats = reinterpret_cast<float2*>(stats);
  p.k = k;
  p.alt_ids = alt_ids;
  p.alt_lp = alt_logprobs;
  p.status = status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(N));
  const cudaError_t e = dtype == MINITE_OUT_FP32
                            ? launch_pdl(logprobs_kernel<float>, grid, dim3(kThreads), 0, s, p)
                            : launch_pdl(logprobs_kernel<uint16_t>, grid, dim3(kThreads), 0, s, p);
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
      !aligned(grad_entropy, 4))
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
