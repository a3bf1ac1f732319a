// minite_grad_norm and minite_clip_grads: the global norm of many gradients, the
// clipping factor, and gradients times that factor.
//
//   norm = sqrt(sum over all tensors of g^2)   or   max |g|
//   factor = min(1, max_norm / (norm + 1e-6))
//
// A thread adds the squares of 128 bytes of elements in FP32 and their sum to a
// double; everything after that is in 64 bits and in a fixed order. Where the squares
// leave the range in which FP32 adds them without loss, they are added again,
// scaled by a power of two that brings their largest to a harmless size: the norm
// is right for every finite gradient, FP32 denormals and 3e38 among them.
//
// Bound by HBM: 604M FP32 gradients 330 us (7.3 TB/s), 250M BF16 ones 79 us (6.3
// TB/s; a third of its issue slots are busy, and a second chunk in flight is all that
// the registers hold), 400M FP32 ones clipped into BF16 600 us (4.0 GB, the gradients
// read twice: the factor is known only when all have been seen). Asynchronous copies
// through shared memory, four or six chunks ahead, took 343 and 355, 95 and 106 us.
#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace gradnorm {

constexpr int kThreads = 256;
constexpr int kVectors = 4;       // 32-byte vectors of a thread in a chunk
constexpr int kBlocksPerSm = 2;
constexpr int64_t kChunkBytes = static_cast<int64_t>(kThreads) * kVectors * 32;
constexpr int kMaxBlocks = 1024;  // partial sums of a launch

struct Tensor {
  const void* g;
  void* out;
  int64_t n;
};

// The tensors of a launch: chunks chunk0[i] .. chunk0[i + 1] belong to tensor i.
template <int CAP> struct Batch {
  Tensor t[CAP];
  int32_t chunk0[CAP + 1];
  uint8_t fp32[CAP];       // bit 0: the gradient, bit 1: its destination
  int32_t count;
};

// A tensor's chunks start at the 32-byte boundary at or before its first element,
// `lead` elements before it, so that all vectors but the first and last are whole
// and aligned, wherever the tensor starts.
template <typename T> constexpr int kPer = 32 / static_cast<int>(sizeof(T));
__host__ __device__ __forceinline__ int lead_of(const void* p, int size) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 31) / size);
}

__device__ __forceinline__ float narrow(float x, float) { return x; }
__device__ __forceinline__ uint16_t narrow(float x, uint16_t) {
  return static_cast<uint16_t>(pack_bf16x2_rn(x, 0.0f));
}

struct Vec { uint32_t w[8]; };
template <typename T> __device__ __forceinline__ void values(const Vec& u, float (&v)[kPer<T>]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u.w[i]);
  } else {
    unpack_bf16x16(u.w, v);
  }
}
// Elements [at, at + kPer) of p[0 .. n); those outside are 0.
template <typename T> __device__ __forceinline__ Vec load_vec(const T* p, int64_t at, int64_t n) {
  Vec u;
  if (at >= 0 && at + kPer<T> <= n) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(u.w[0]), "=r"(u.w[1]), "=r"(u.w[2]), "=r"(u.w[3]), "=r"(u.w[4]), "=r"(u.w[5]), "=r"(u.w[6]),
                   "=r"(u.w[7]) : "l"(p + at) : "memory");
    return u;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u.w[i] = 0;
  if (at < n && at + kPer<T> > 0) {
#pragma unroll
    for (int i = 0; i < kPer<T>; ++i) {
      if (at + i < 0 || at + i >= n) continue;
      if constexpr (sizeof(T) == 4) u.w[i] = __float_as_uint(p[at + i]);
      else u.w[i / 2] |= static_cast<uint32_t>(p[at + i]) << (16 * (i & 1));
    }
  }
  return u;
}
// A thread's vectors of chunk `index` of a tensor.
template <typename T>
__device__ __forceinline__ void load_chunk(const Tensor& t, int64_t index, Vec (&u)[kVectors]) {
  const T* p = static_cast<const T*>(t.g);
  const int64_t first = index * (kChunkBytes / static_cast<int64_t>(sizeof(T))) - lead_of(p, sizeof(T));
#pragma unroll
  for (int i = 0; i < kVectors; ++i)
    u[i] = load_vec(p, first + (i * kThreads + static_cast<int>(threadIdx.x)) * kPer<T>, t.n);
}

// N values to elements [at, at + N) of o[0 .. n): wide where gradient and destination lie
// alike modulo their vectors, otherwise an element a store. 400M FP32 gradients in 291
// tensors into BF16 take 595 us at boundaries of 256 elements, 998 packed without gaps.
template <typename T, int N>
__device__ __forceinline__ void store_values(T* o, int64_t at, int64_t n, const float (&v)[N]) {
  constexpr int kBytes = N * static_cast<int>(sizeof(T)) < 32 ? N * static_cast<int>(sizeof(T)) : 32;
  if (at >= 0 && at + N <= n && (reinterpret_cast<uintptr_t>(o + at) & (kBytes - 1)) == 0) {
    constexpr int kWords = N * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = pack_bf16x2_rn(v[2 * i], v[2 * i + 1]);
    }
    if constexpr (kBytes == 16) {
      st_global_v4(o + at, w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 8; ++i)
        st_global_v8(reinterpret_cast<char*>(o + at) + 32 * i, w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3],
                     w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at + i >= 0 && at + i < n) o[at + i] = narrow(v[i], T());
}

// |v| as an integer: ordered as the values are, NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The sum of the squares of a thread's vectors of a chunk.
template <typename T> __device__ __forceinline__ double squares(const Vec (&u)[kVectors]) {
  uint64_t s[2] = {};
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    float v[kPer<T>];
    values<T>(u[i], v);
#pragma unroll
    for (int j = 0; j < kPer<T>; j += 2) {
      const uint64_t x = pair(v[j], v[j + 1]);
      s[(j >> 1) & 1] = fma2(x, x, s[(j >> 1) & 1]);
    }
  }
  float a, b;
  unpair(add2(s[0], s[1]), a, b);
  const float sum = a + b;
  // below 2^-90 squares may have been lost under FP32's smallest value, above
  // 2^126 their sum may have left its range
  if (sum >= 0x1p-90f && sum < 0x1p126f) return static_cast<double>(sum);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    float v[kPer<T>];
    values<T>(u[i], v);
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) m = max(m, magnitude(v[j]));
  }
  if (m == 0) return 0.0;
  const bool large = m >= 0x3F800000u;             // 1
  const float up = large ? 0x1p-70f : 0x1p100f;
  float r = 0.0f;
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    float v[kPer<T>];
    values<T>(u[i], v);
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) {
      const float x = v[j] * up;
      r = fmaf(x, x, r);
    }
  }
  return static_cast<double>(r) * (large ? 0x1p140 : 0x1p-200);
}
template <typename T> __device__ __forceinline__ uint32_t largest(const Vec (&u)[kVectors]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    float v[kPer<T>];
    values<T>(u[i], v);
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) m = max(m, magnitude(v[j]));
  }
  return m;
}

// A chunk's tensor: the last one that starts at or before it.
template <int CAP> __device__ __forceinline__ int tensor_of(const Batch<CAP>& b, int64_t chunk) {
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.chunk0[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// The sum, or the largest, over a block, in a fixed order (thread 0's result).
template <bool MAX> __device__ __forceinline__ double join(double a, double b) {
  if constexpr (MAX) return (a >= b || a != a) ? a : b;   // NaN stays
  else return a + b;
}
template <bool MAX> __device__ __forceinline__ double block_join(double v) {
  __shared__ double s[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join<MAX>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < kThreads / 32; ++w) v = join<MAX>(v, s[w]);
  return v;
}

// What the tensors of a launch are: the loops of one type need not ask then. FP32 and
// the maximum spill nothing; the 2-norm of BF16 spills 96 bytes at its 128 registers,
// the mixed one 108.
enum Kind { kAllBf16, kAllFp32, kMixed };
template <Kind KIND> __device__ __forceinline__ bool is_fp32(uint8_t flags) {
  return KIND == kAllFp32 || (KIND == kMixed && (flags & 1));
}

// This block's part of the norm: of chunks first, first + step, ... (thread 0's
// result). One chunk is on its way while another is added.
template <int CAP, bool MAX, Kind KIND>
__device__ __forceinline__ double part_of(const Batch<CAP>& b, int64_t first, int64_t step) {
  const int64_t chunks = b.chunk0[b.count];
  double acc = 0.0;
  uint32_t most = 0;
  auto load = [&](int64_t c, Vec (&u)[kVectors]) {   // returns whether it is FP32
    if (c >= chunks) return false;
    const int i = tensor_of(b, c);
    const bool fp32 = is_fp32<KIND>(b.fp32[i]);
    if (fp32) load_chunk<float>(b.t[i], c - b.chunk0[i], u);
    else load_chunk<uint16_t>(b.t[i], c - b.chunk0[i], u);
    return fp32;
  };
  auto add = [&](int64_t c, bool fp32, const Vec (&u)[kVectors]) {
    if (c >= chunks) return;
    fp32 = KIND == kAllFp32 || (KIND == kMixed && fp32);
    if constexpr (MAX) most = max(most, fp32 ? largest<float>(u) : largest<uint16_t>(u));
    else acc += fp32 ? squares<float>(u) : squares<uint16_t>(u);
  };
  Vec u[kVectors], v[kVectors];
  bool fu = load(first, u);
  for (int64_t c = first; c < chunks; c += 2 * step) {
    const bool fv = load(c + step, v);
    add(c, fu, u);
    fu = load(c + 2 * step, u);
    add(c + step, fv, v);
  }
  if constexpr (MAX) acc = static_cast<double>(__uint_as_float(most));
  return block_join<MAX>(acc);
}

// Norm and factor from the joined sum.
template <bool MAX>
__device__ __forceinline__ void write_norm(double total, double max_norm, float* norm, float* factor) {
  const double r = MAX ? total : sqrt(total);
  // without a limit 1, whatever the norm: infinity over infinity is none of its business
  const double f = isinf(max_norm) && r == r ? 1.0 : max_norm / (r + 1e-6);
  if (norm) *norm = static_cast<float>(r);
  if (factor) *factor = f > 1.0 ? 1.0f : static_cast<float>(f);   // NaN stays
}

template <int CAP, bool MAX, Kind KIND>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) norm_kernel(const __grid_constant__ Batch<CAP> b,
                                                                      double* partial) {
  pdl_wait();
  pdl_trigger();
  const double part = part_of<CAP, MAX, KIND>(b, blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) partial[blockIdx.x] = part;
}

// Few elements: one cluster of CTAs, whose parts meet in the first one's shared
// memory, in place of a second launch and a workspace. 300001 BF16 elements take 5.2
// us on the device, 5.0 by the two launches, but a call 18 to 20 us instead of 28: the
// host's time is what bounds it.
constexpr int kCluster = 8;
template <int CAP, bool MAX>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1) small_norm_kernel(
    const __grid_constant__ Batch<CAP> b, double max_norm, float* norm, float* factor) {
  __shared__ uint2 s_part[kCluster];
  cluster_arrive();   // every CTA runs before one writes to another's shared memory
  pdl_wait();
  const double part = part_of<CAP, MAX, kMixed>(b, blockIdx.x, kCluster);
  cluster_wait();
  if (threadIdx.x == 0) {
    const uint32_t at = mapa_shared(smem_u32(&s_part[blockIdx.x]), 0);
    st_shared_cluster(at, static_cast<uint32_t>(__double2loint(part)));
    st_shared_cluster(at + 4, static_cast<uint32_t>(__double2hiint(part)));
  }
  cluster_sync_all();
  if (blockIdx.x != 0 || threadIdx.x != 0) return;
  double total = 0.0;
  for (int r = 0; r < kCluster; ++r)
    total = join<MAX>(total, __hiloint2double(static_cast<int>(s_part[r].y), static_cast<int>(s_part[r].x)));
  write_norm<MAX>(total, max_norm, norm, factor);
}

template <bool MAX>
__global__ void __launch_bounds__(kThreads) finish_kernel(const double* partial, int n, double max_norm, float* norm,
                                                          float* factor) {
  pdl_wait();
  pdl_trigger();
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v = join<MAX>(v, partial[i]);
  const double total = block_join<MAX>(v);
  if (threadIdx.x == 0) write_norm<MAX>(total, max_norm, norm, factor);
}

template <typename G, typename O>
__device__ __forceinline__ void scale_chunk(const Tensor& t, int64_t index, float f) {
  Vec u[kVectors];
  load_chunk<G>(t, index, u);
  const int64_t first = index * (kChunkBytes / static_cast<int64_t>(sizeof(G))) - lead_of(t.g, sizeof(G));
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    float v[kPer<G>];
    values<G>(u[i], v);
#pragma unroll
    for (int j = 0; j < kPer<G>; ++j) v[j] *= f;
    store_values(static_cast<O*>(t.out), first + (i * kThreads + static_cast<int>(threadIdx.x)) * kPer<G>, t.n, v);
  }
}

// in_place: every destination is its gradient, and a factor of 1 changes nothing.
// The last chunks first: the norm has left them in L2.
constexpr int kClipBlocksPerSm = 3;
template <int CAP>
__global__ void __launch_bounds__(kThreads, kClipBlocksPerSm) clip_kernel(const __grid_constant__ Batch<CAP> b,
                                                                          const float* factor,
                                                                          bool in_place) {
  pdl_wait();
  const float f = *factor;
  if (in_place && f == 1.0f) return;
  const int64_t chunks = b.chunk0[b.count];
  for (int64_t r = blockIdx.x; r < chunks; r += gridDim.x) {
    const int64_t c = chunks - 1 - r;
    const int i = tensor_of(b, c);
    const Tensor& t = b.t[i];
    const int64_t index = c - b.chunk0[i];
    switch (b.fp32[i]) {
      case 0: scale_chunk<uint16_t, uint16_t>(t, index, f); break;
      case 1: scale_chunk<float, uint16_t>(t, index, f); break;
      case 2: scale_chunk<uint16_t, float>(t, index, f); break;
      default: scale_chunk<float, float>(t, index, f); break;
    }
  }
}

constexpr int kSmall = 128, kLarge = 1000;   // tensors of a launch
constexpr int64_t kFewElements = 1 << 19;
// Up to 96 chunks: the sizes' sum and their number decide.
inline bool few(int64_t n_tensors, int64_t elements) { return n_tensors <= 32 && elements <= kFewElements; }

inline int grid_of(int64_t chunks, int per_sm) {
  int64_t cap = static_cast<int64_t>(num_sms()) * per_sm;
  if (cap > kMaxBlocks) cap = kMaxBlocks;
  return static_cast<int>(chunks < cap ? chunks : cap);
}

// As many tensors as a launch takes into a batch; the next one's index.
template <int CAP>
int64_t fill(Batch<CAP>& b, const minite_grad_tensor* t, int64_t i, int64_t n) {
  int64_t chunks = 0;   // below 2^31: check() bounds the elements of all tensors
  b.count = 0;
  for (; i < n && b.count < CAP; ++i) {
    if (t[i].n == 0) continue;
    const int size = t[i].grad_dtype == MINITE_OUT_FP32 ? 4 : 2;
    const int64_t c = ((t[i].n + lead_of(t[i].grad, size)) * size + kChunkBytes - 1) / kChunkBytes;
    b.t[b.count] = {t[i].grad, t[i].out, t[i].n};
    b.fp32[b.count] = static_cast<uint8_t>((t[i].grad_dtype == MINITE_OUT_FP32 ? 1 : 0) |
                                           (t[i].out_dtype == MINITE_OUT_FP32 ? 2 : 0));
    b.chunk0[b.count++] = static_cast<int32_t>(chunks);
    chunks += c;
  }
  b.chunk0[b.count] = static_cast<int32_t>(chunks);
  return i;
}

// `launch` for the tensors in batches of up to CAP.
template <int CAP, typename Launch>
cudaError_t in_batches(const minite_grad_tensor* t, int64_t n, int per_sm, Launch launch) {
  static_assert(sizeof(Batch<kSmall>) <= 4096 && sizeof(Batch<kLarge>) + 64 <= 32764, "parameters");
  Batch<CAP> b;
  for (int64_t i = 0; i < n;) {
    i = fill(b, t, i, n);
    if (b.count == 0) break;
    const cudaError_t e = launch(b, grid_of(b.chunk0[b.count], per_sm));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int64_t launches_of(int64_t n) { return n <= kSmall ? 1 : (n + kLarge - 1) / kLarge; }

template <int CAP, bool MAX, Kind KIND>
cudaError_t norm_of(const minite_grad_tensor* t, int64_t n, double max_norm, float* norm, float* factor,
                    double* partial, cudaStream_t s) {
  int parts = 0;
  const cudaError_t e = in_batches<CAP>(t, n, kBlocksPerSm, [&](const Batch<CAP>& b, int grid) {
    const cudaError_t r = launch_pdl(norm_kernel<CAP, MAX, KIND>, dim3(grid), dim3(kThreads), 0, s, b, partial + parts);
    parts += grid;
    return r;
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(finish_kernel<MAX>, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(partial), parts,
                    max_norm, norm, factor);
}
template <int CAP, bool MAX>
cudaError_t norm_as(const minite_grad_tensor* t, int64_t n, double max_norm, float* norm, float* factor,
                    double* partial, cudaStream_t s) {
  int64_t fp32 = 0;
  for (int64_t i = 0; i < n; ++i) fp32 += t[i].grad_dtype == MINITE_OUT_FP32;
  if (fp32 == n) return norm_of<CAP, MAX, kAllFp32>(t, n, max_norm, norm, factor, partial, s);
  if (fp32 == 0) return norm_of<CAP, MAX, kAllBf16>(t, n, max_norm, norm, factor, partial, s);
  return norm_of<CAP, MAX, kMixed>(t, n, max_norm, norm, factor, partial, s);
}

template <bool MAX>
cudaError_t few_as(const minite_grad_tensor* t, int64_t n, double max_norm, float* norm, float* factor,
                   cudaStream_t s) {
  Batch<32> b;
  fill(b, t, 0, n);
  return launch_pdl(small_norm_kernel<32, MAX>, dim3(kCluster), dim3(kThreads), 0, s, b, max_norm, norm, factor);
}

template <int CAP>
cudaError_t clip_as(const minite_grad_tensor* t, int64_t n, const float* factor, bool in_place, cudaStream_t s) {
  return in_batches<CAP>(t, n, kClipBlocksPerSm, [&](const Batch<CAP>& b, int grid) {
    return launch_pdl(clip_kernel<CAP>, dim3(grid), dim3(kThreads), 0, s, b, factor, in_place);
  });
}

bool dtype_ok(int d) { return d == MINITE_OUT_BF16 || d == MINITE_OUT_FP32; }

int check(const minite_grad_tensor* t, int64_t n, bool out) {
  if (n < 0 || (n > 0 && !t)) return MINITE_ERR_INVALID_ARG;
  if (n > (int64_t(1) << 24)) return MINITE_ERR_UNSUPPORTED_SHAPE;
  int64_t elements = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (t[i].n < 0 || t[i].n >= (int64_t(1) << 42)) return MINITE_ERR_UNSUPPORTED_SHAPE;
    elements += t[i].n;
    if (elements >= (int64_t(1) << 42)) return MINITE_ERR_UNSUPPORTED_SHAPE;
    if (!dtype_ok(t[i].grad_dtype) || (out && !dtype_ok(t[i].out_dtype))) return MINITE_ERR_INVALID_ARG;
    if (t[i].n == 0) continue;
    if (!t[i].grad || !aligned(t[i].grad, t[i].grad_dtype == MINITE_OUT_FP32 ? 4 : 2)) return MINITE_ERR_INVALID_ARG;
    if (out && (!t[i].out || !aligned(t[i].out, t[i].out_dtype == MINITE_OUT_FP32 ? 4 : 2) ||
                (t[i].out == t[i].grad && t[i].out_dtype != t[i].grad_dtype)))
      return MINITE_ERR_INVALID_ARG;
  }
  return MINITE_OK;
}

}  // namespace gradnorm

size_t grad_norm_workspace_bytes(int64_t n_tensors, int64_t elements) {
  if (gradnorm::few(n_tensors, elements)) return 0;
  return static_cast<size_t>(gradnorm::launches_of(n_tensors)) * gradnorm::kMaxBlocks * sizeof(double);
}

}  // namespace minite

using namespace minite;

extern "C" int minite_grad_norm(const minite_grad_tensor* tensors, int64_t n_tensors, int order, double max_norm,
                                float* norm, float* factor, void* workspace, size_t ws_bytes,
                                minite_stream_t stream) {
  using namespace gradnorm;
  const int rc = check(tensors, n_tensors, false);
  if (rc != MINITE_OK) return rc;
  int64_t elements = 0;
  for (int64_t i = 0; i < n_tensors && elements <= kFewElements; ++i) elements += tensors[i].n;
  const size_t need = grad_norm_workspace_bytes(n_tensors, elements);
  if ((order != MINITE_NORM_2 && order != MINITE_NORM_MAX) || !(max_norm >= 0.0) || (!norm && !factor) ||
      !aligned(norm, 4) || !aligned(factor, 4) ||
      (need > 0 && (!workspace || !aligned(workspace, 8) || ws_bytes < need)))
    return MINITE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* p = static_cast<double*>(workspace);
  cudaError_t e;
  if (need == 0)
    e = order == MINITE_NORM_2 ? few_as<false>(tensors, n_tensors, max_norm, norm, factor, s)
                               : few_as<true>(tensors, n_tensors, max_norm, norm, factor, s);
  else if (n_tensors <= kSmall)
    e = order == MINITE_NORM_2 ? norm_as<kSmall, false>(tensors, n_tensors, max_norm, norm, factor, p, s)
                               : norm_as<kSmall, true>(tensors, n_tensors, max_norm, norm, factor, p, s);
  else
    e = order == MINITE_NORM_2 ? norm_as<kLarge, false>(tensors, n_tensors, max_norm, norm, factor, p, s)
                               : norm_as<kLarge, true>(tensors, n_tensors, max_norm, norm, factor, p, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

extern "C" int minite_clip_grads(const minite_grad_tensor* tensors, int64_t n_tensors, const float* factor,
                                 minite_stream_t stream) {
  using namespace gradnorm;
  const int rc = check(tensors, n_tensors, true);
  if (rc != MINITE_OK) return rc;
  if (!factor || !aligned(factor, 4)) return MINITE_ERR_INVALID_ARG;
  bool in_place = true, any = false;
  for (int64_t i = 0; i < n_tensors; ++i) {
    any |= tensors[i].n > 0;
    in_place &= tensors[i].n == 0 || tensors[i].out == tensors[i].grad;
  }
  if (!any) return MINITE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = n_tensors <= kSmall ? clip_as<kSmall>(tensors, n_tensors, factor, in_place, s)
                                            : clip_as<kLarge>(tensors, n_tensors, factor, in_place, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}
