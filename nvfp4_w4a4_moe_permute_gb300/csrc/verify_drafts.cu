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
// The rows' maxima and sums come from the log probabilities' kernel, which
// streams target and draft rows once. Here a cluster of CTAs per sequence looks
// at every draft (each CTA for itself), then runs the race over its parts of
// the one row that is sampled from.
#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  const void* target;       // [B][S + 1][V]
  const void* draft;        // [B][S][V], or null
  int64_t target_ld, draft_ld, noise_ld;
  const float2* target_stats;   // [B][S + 1] {largest logit, log of the sum}
  const float2* draft_stats;    // [B][S]
  const int32_t* draft_tokens;  // [B][S]
  const float* uniforms;        // [B][S]
  const float* noise;           // [B][V]
  int64_t V;
  int S;
  float inv_t, k2;
  int32_t* tokens;          // [B][S + 1]
  float* logprobs;          // [B][S + 1], or null
  int32_t* accepted;        // [B]
  int32_t* status;
};

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// Whether a row has probabilities: neither NaN, nor +inf, nor a logit above -inf missing.
__device__ __forceinline__ bool usable(float2 st) { return fabsf(st.x) < INFINITY && fabsf(st.y) < INFINITY; }

struct Row {
  float m, shift, k2;   // largest logit, log2 of the sum, log2(e) / T
  __device__ __forceinline__ Row(float2 st, float k) : m(st.x), shift(st.y * kLog2e), k2(k) {}
  __device__ __forceinline__ float p(float x) const { return exp2f(fmaf(x - m, k2, -shift)); }
};

// A place in the race: larger weight / variate first, then the lower index. 0: no weight.
__device__ __forceinline__ uint64_t place(float weight, float e, int64_t j) {
  if (!(weight > 0.0f)) return 0;
  const float v = e > 0.0f ? __fdiv_rn(weight, e) : INFINITY;
  return (static_cast<uint64_t>(__float_as_uint(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t warp_larger(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = larger(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T, typename D>
__global__ void __launch_bounds__(kThreads) verify_kernel(const Params p, int cluster) {
  __shared__ int s_n, s_falls;
  __shared__ uint64_t s_best[kWarps][2];
  __shared__ uint32_t s_all[kMaxCluster][4];   // every CTA's best, in the cluster's first CTA
  cluster_arrive();   // every CTA runs before one writes to another's shared memory
  pdl_wait();
  const int64_t b = blockIdx.x / cluster;
  const int rank = blockIdx.x % cluster;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const T* target = static_cast<const T*>(p.target) + b * (p.S + 1) * p.target_ld;
  const D* draft = p.draft ? static_cast<const D*>(p.draft) + b * p.S * p.draft_ld : nullptr;
  const float2* tst = p.target_stats + b * (p.S + 1);
  const float2* dst = p.draft_stats + b * p.S;
  const int32_t* drafts = p.draft_tokens + b * p.S;
  if (wid == 0) {   // lane i looks at draft i
    int x = -1;
    bool stands = false;
    if (lane < p.S) {
      x = drafts[lane];
      if (x >= p.V) {
        if (rank == 0) set_status(p.status, MINITE_ERR_BAD_TOKEN);
        x = -1;
      }
      if (x >= 0 && usable(tst[lane]) && (!draft || usable(dst[lane]))) {
        const float px = Row(tst[lane], p.k2).p(value(target[lane * p.target_ld + x]));
        const float qx = draft ? Row(dst[lane], p.k2).p(value(draft[lane * p.draft_ld + x])) : 1.0f;
        stands = p.uniforms[b * p.S + lane] * qx < px;
      }
    }
    const uint32_t none = ~__ballot_sync(0xffffffffu, x >= 0), out = ~__ballot_sync(0xffffffffu, stands);
    const int given = none ? __ffs(none) - 1 : 32, n = out ? __ffs(out) - 1 : 32;   // S <= 31: never 32
    if (lane == 0) {
      s_n = min(n, given);
      s_falls = n < given;
    }
  }
  __syncthreads();
  const int n = s_n;
  const bool falls = s_falls;
  const Row rt(tst[n], p.k2);
  const bool ok = usable(tst[n]) && (!falls || !draft || usable(dst[n]));
  uint64_t best = 0, best_p = 0;   // of what is left of p without q, and of p itself
  if (ok) {
    const T* xt = target + n * p.target_ld;
    const float* e = p.noise + b * p.noise_ld;
    const int64_t j0 = p.V * rank / cluster, j1 = p.V * (rank + 1) / cluster;
    const int64_t drafted = falls && !draft ? drafts[n] : -1;
    const bool with_q = falls && draft;
    const Row rd(with_q ? dst[n] : make_float2(0.0f, 0.0f), p.k2);
    const D* xd = with_q ? draft + n * p.draft_ld : nullptr;
    for (int64_t j = j0 + threadIdx.x; j < j1; j += kThreads) {
      const float w = rt.p(value(xt[j])), v = e[j];
      best_p = larger(best_p, place(w, v, j));
      float r = w;
      if (with_q) r = w - rd.p(value(xd[j]));
      else if (j == drafted) r = 0.0f;
      best = larger(best, place(r, v, j));
    }
  }
  best = warp_larger(best);
  best_p = warp_larger(best_p);
  cluster_wait();
  if (lane == 0) {
    s_best[wid][0] = best;
    s_best[wid][1] = best_p;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) {
      best = larger(best, s_best[w][0]);
      best_p = larger(best_p, s_best[w][1]);
    }
    const uint32_t at = mapa_shared(smem_u32(&s_all[rank][0]), 0);
    st_shared_cluster(at, static_cast<uint32_t>(best));
    st_shared_cluster(at + 4, static_cast<uint32_t>(best >> 32));
    st_shared_cluster(at + 8, static_cast<uint32_t>(best_p));
    st_shared_cluster(at + 12, static_cast<uint32_t>(best_p >> 32));
  }
  cluster_sync_all();
  if (rank != 0 || wid != 0) return;
  best = best_p = 0;
  if (lane < cluster) {
    best = s_all[lane][0] | static_cast<uint64_t>(s_all[lane][1]) << 32;
    best_p = s_all[lane][2] | static_cast<uint64_t>(s_all[lane][3]) << 32;
  }
  best = warp_larger(best);
  best_p = warp_larger(best_p);
  // q may be as large as p everywhere but for roundings: p itself then
  const uint64_t key = best ? best : best_p;
  const int32_t next = key ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key)) : -1;
  if (lane == 0) p.accepted[b] = n;
  if (lane <= p.S) {
    const int32_t x = lane < n ? drafts[lane] : lane == n ? next : -1;
    p.tokens[b * (p.S + 1) + lane] = x;
    if (p.logprobs) {
      float lp = 0.0f;
      if (x >= 0) lp = (value(target[lane * p.target_ld + x]) - tst[lane].x) * p.inv_t - tst[lane].y;
      else if (lane == n) lp = __int_as_float(0x7FC00000);   // nothing to sample from
      p.logprobs[b * (p.S + 1) + lane] = lp;
    }
  }
}

template <typename T, typename D>
cudaError_t launch(const Params& p, int64_t B, cudaStream_t s) {
  // enough CTAs a sequence to fill the SMs, with 2048 tokens each at least
  int cluster = 1;
  while (cluster < kMaxCluster && p.V >= 4096 * cluster && B * cluster < 4 * num_sms()) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, D>, p, cluster);
}

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace verify

size_t verify_workspace_bytes(int64_t B, int64_t S) {
  using verify::align256;
  return align256(static_cast<size_t>(B) * (S + 1) * 8) + align256(static_cast<size_t>(B) * S * 8) +
         align256(static_cast<size_t>(B) * S * 4);
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
  if ((!tf && target_dtype != MINITE_OUT_BF16) || (draft && !df && draft_dtype != MINITE_OUT_BF16) ||
      !(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.0f / temperature))
    return MINITE_ERR_INVALID_ARG;
  if (B < 0 || S < 0 || S > 31 || B > (int64_t(1) << 24) || V < 1 || V > 0x7FFFFFFF || target_stride < V ||
      (draft && draft_stride < V) || noise_stride < V)
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (B == 0) return MINITE_OK;
  if (!target || !noise || !tokens || !accepted || !workspace || (S > 0 && (!draft_tokens || !uniforms)) ||
      !aligned(target, tf ? 4 : 2) || !aligned(draft, df ? 4 : 2) || !aligned(draft_tokens, 4) ||
      !aligned(uniforms, 4) || !aligned(noise, 4) || !aligned(tokens, 4) || !aligned(accepted, 4) ||
      !aligned(logprobs, 4) || !aligned(workspace, 256) || !aligned(status, 4) ||
      ws_bytes < verify_workspace_bytes(B, S))
    return MINITE_ERR_INVALID_ARG;
  if (S == 0) draft = nullptr;
  char* ws = static_cast<char*>(workspace);
  float* tst = reinterpret_cast<float*>(ws);
  ws += align256(static_cast<size_t>(B) * (S + 1) * 8);
  float* dst = reinterpret_cast<float*>(ws);
  ws += align256(static_cast<size_t>(B) * S * 8);
  int rc = minite_token_logprobs(target, target_dtype, B * (S + 1), V, target_stride, nullptr, 0, temperature,
                                 nullptr, nullptr, tst, 0, nullptr, nullptr, nullptr, stream);
  if (rc != MINITE_OK) return rc;
  if (draft) {   // rows without a draft are not read
    rc = minite_token_logprobs(draft, draft_dtype, B * S, V, draft_stride, draft_tokens, 0, temperature,
                               reinterpret_cast<float*>(ws), nullptr, dst, 0, nullptr, nullptr, nullptr, stream);
    if (rc != MINITE_OK) return rc;
  }
  Params p = {};
  p.target = target;
  p.draft = draft;
  p.target_ld = target_stride;
  p.draft_ld = draft_stride;
  p.noise_ld = noise_stride;
  p.target_stats = reinterpret_cast<const float2*>(tst);
  p.draft_stats = reinterpret_cast<const float2*>(dst);
  p.draft_tokens = draft_tokens;
  p.uniforms = uniforms;
  p.noise = noise;
  p.V = V;
  p.S = S;
  p.inv_t = 1.0f / temperature;
  p.k2 = p.inv_t * kLog2e;
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
