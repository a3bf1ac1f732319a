// minite_adamw_step: one AdamW step over many tensors in one launch, with
// FP32 states or 8-bit ones (E4M3 codes, one FP32 scale per 256 elements).
//
// Per element, with g the gradient times the optional device-side factor:
//   m <- b1 m + (1 - b1) g          v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit states: a block of 256 consecutive elements of a tensor keeps
// s_m = max(max|m| * FP32(1/448), 2^-126) and the codes E4M3(m / s_m); for the second
// moment the codes hold sqrt(v) (E4M3 spans 2^18, so v itself spans 2^36
// within a block) with s_v likewise. A sqrt(v) above zero never rounds to the
// zero code: it takes the smallest one instead, since a v of 0 beside an m
// that is not would divide the step by eps alone.
//
// Every operation is one IEEE float operation in the order written above (no
// contraction), so that the codes do not depend on how a compiler fuses them.
#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace adamw {

constexpr int kBlock = 256;      // elements per 8-bit scale
constexpr int kThreads = 256;
constexpr int kChunk = 4096;     // elements per CTA
constexpr float kInvMax = 1.0f / 448.0f;  // rounded to FP32
constexpr float kTiny = 1.17549435e-38f;  // 2^-126

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  int64_t n;
};

struct Hyper {
  float b1, c1, b2, c2;      // beta1, 1 - beta1, beta2, 1 - beta2
  float keep, rate, isq, eps;  // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  const float* scale;        // device factor of the gradients, or null
};

template <int CAP>
struct Batch {
  Hyper h;
  int count;
  int32_t chunk0[CAP];       // chunks of the tensors before this one
  Tensor t[CAP];
};

__device__ __forceinline__ void update(float& p, float g, float& m, float& v, float& r,
                                       const Hyper& h) {
  m = __fadd_rn(__fmul_rn(m, h.b1), __fmul_rn(g, h.c1));
  v = __fadd_rn(__fmul_rn(v, h.b2), __fmul_rn(__fmul_rn(g, g), h.c2));
  r = __fsqrt_rn(v);
  const float u = __fdiv_rn(m, __fadd_rn(__fmul_rn(r, h.isq), h.eps));
  p = __fsub_rn(__fmul_rn(p, h.keep), __fmul_rn(u, h.rate));
}

// Eight consecutive elements from index i of a tensor of n; `vec` when all
// eight exist and the address is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* a, int64_t i, int64_t n, bool vec, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    if (vec) {
      const float4 u = *reinterpret_cast<const float4*>(a + i);
      const float4 w = *reinterpret_cast<const float4*>(a + i + 4);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
      x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = i + j < n ? static_cast<float>(a[i + j]) : 0.0f;
    }
  } else {
    if (vec) {
      unpack_bf16x8(*reinterpret_cast<const uint4*>(a + i), x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = i + j < n ? __uint_as_float(static_cast<uint32_t>(a[i + j]) << 16) : 0.0f;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* a, int64_t i, int64_t n, bool vec, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    if (vec) {
      *reinterpret_cast<float4*>(a + i) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(a + i + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < n) a[i + j] = static_cast<T>(x[j]);
    }
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2_rn(x[2 * j], x[2 * j + 1]);
    if (vec) {
      *reinterpret_cast<uint4*>(a + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < n) a[i + j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// E4M3 code of a value scaled into [-448, 448]; NaN keeps its code (0x7F).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t o;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(o) : "f"(lo), "f"(hi));
  return o;
}
__device__ __forceinline__ void e4m3x2_values(uint32_t c, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(h));
}

__device__ __forceinline__ void load_codes(const uint8_t* a, int64_t i, int64_t n, bool vec,
                                           float (&x)[8]) {
  uint32_t w[2] = {0, 0};
  if (vec) {
    const uint2 u = *reinterpret_cast<const uint2*>(a + i);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) w[j >> 2] |= static_cast<uint32_t>(a[i + j]) << (8 * (j & 3));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) e4m3x2_values((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu, x[2 * j], x[2 * j + 1]);
}

__device__ __forceinline__ void store_codes(uint8_t* a, int64_t i, int64_t n, bool vec,
                                            const float (&x)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    w[j] = e4m3x2(x[4 * j], x[4 * j + 1]) | (e4m3x2(x[4 * j + 2], x[4 * j + 3]) << 16);
  if (vec) {
    *reinterpret_cast<uint2*>(a + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) a[i + j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
  }
}

// Scale of a block whose largest magnitude is the warp's: the bits of
// non-negative floats order as integers, NaN above all, so that a block with
// a NaN gets a NaN scale.
__device__ __forceinline__ float warp_block_scale(float amax) {
  const float a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  const float s = __fmul_rn(a, kInvMax);
  return s < kTiny ? kTiny : s;
}

__device__ __forceinline__ float abs_max_nan(const float (&x)[8]) {
  uint32_t b = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) b = max(b, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  return __uint_as_float(b);
}

template <typename P, typename G, bool EIGHT, int CAP>
__global__ void __launch_bounds__(kThreads)
adamw_kernel(const __grid_constant__ Batch<CAP> b) {
  pdl_wait();
  int lo = 0, hi = b.count;
  const int chunk = static_cast<int>(blockIdx.x);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.chunk0[mid] <= chunk) lo = mid; else hi = mid;
  }
  const Tensor& t = b.t[lo];
  const Hyper& h = b.h;
  const int64_t base = static_cast<int64_t>(chunk - b.chunk0[lo]) * kChunk;
  const int64_t n = t.n;
  P* p = static_cast<P*>(t.p);
  const G* g = static_cast<const G*>(t.g);
  const bool wide = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(g) |
                      reinterpret_cast<uintptr_t>(t.copy)) & 15) == 0;
  const float gs = h.scale ? __ldg(h.scale) : 1.0f;
#pragma unroll 1
  for (int64_t i = base + 8 * threadIdx.x; i < base + kChunk; i += 8 * kThreads) {
    // a warp's 256 elements are one block of the states
    if (i - 8 * (threadIdx.x & 31) >= n) break;
    const bool full = i + 8 <= n;
    const bool vec = full && wide;
    float x[8], d[8], m[8], v[8], r[8];
    load8(p, i, n, vec, x);
    load8(g, i, n, vec, d);
    if constexpr (EIGHT) {
      const int64_t blk = i / kBlock;
      const float sm = t.ms[blk], sv = t.vs[blk];
      load_codes(static_cast<uint8_t*>(t.m), i, n, full, m);
      load_codes(static_cast<uint8_t*>(t.v), i, n, full, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = __fmul_rn(m[j], sm);
        v[j] = __fmul_rn(v[j], sv);
        v[j] = __fmul_rn(v[j], v[j]);
      }
    } else {
      load8(static_cast<float*>(t.m), i, n, full, m);
      load8(static_cast<float*>(t.v), i, n, full, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) update(x[j], __fmul_rn(d[j], gs), m[j], v[j], r[j], h);
    store8(p, i, n, vec, x);
    if (t.copy) store8(t.copy, i, n, vec, x);
    if constexpr (EIGHT) {
      const int64_t blk = i / kBlock;
      const float sm = warp_block_scale(abs_max_nan(m));
      const float sv = warp_block_scale(abs_max_nan(r));
      const float im = __fdiv_rn(1.0f, sm), iv = __fdiv_rn(1.0f, sv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = __fmul_rn(m[j], im);
        const float q = __fmul_rn(r[j], iv);
        r[j] = r[j] > 0.0f && q < 0.001953125f ? 0.001953125f : q;
      }
      store_codes(static_cast<uint8_t*>(t.m), i, n, full, m);
      store_codes(static_cast<uint8_t*>(t.v), i, n, full, r);
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {
        t.ms[blk] = sm;
        t.vs[blk] = sv;
      }
    } else {
      store8(static_cast<float*>(t.m), i, n, full, m);
      store8(static_cast<float*>(t.v), i, n, full, v);
    }
  }
}

template <typename P, typename G, bool EIGHT, int CAP>
cudaError_t launch_batch(const minite_adamw_tensor* t, int64_t count, const Hyper& h,
                         cudaStream_t s) {
  Batch<CAP> b;
  b.h = h;
  b.count = 0;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    Tensor& d = b.t[b.count];
    b.chunk0[b.count++] = static_cast<int32_t>(chunks);
    d.p = t[i].param;
    d.g = t[i].grad;
    d.m = t[i].exp_avg;
    d.v = t[i].exp_avg_sq;
    d.ms = t[i].exp_avg_scale;
    d.vs = t[i].exp_avg_sq_scale;
    d.copy = static_cast<uint16_t*>(t[i].param_bf16);
    d.n = t[i].n;
    chunks += (t[i].n + kChunk - 1) / kChunk;
  }
  if (chunks == 0) return cudaSuccess;
  return launch_pdl(adamw_kernel<P, G, EIGHT, CAP>, dim3(static_cast<unsigned>(chunks)),
                    dim3(kThreads), 0, s, b);
}

template <typename P, typename G, bool EIGHT>
int step(const minite_adamw_tensor* t, int64_t n, const Hyper& h, cudaStream_t s) {
  // kernel parameters carry the tensors' pointers (4 KB or 32 KB of them)
  constexpr int kSmall = 48, kLarge = 440;
  static_assert(sizeof(Batch<kSmall>) <= 4096 && sizeof(Batch<kLarge>) <= 32764, "parameters");
  int64_t i = 0;
  while (i < n) {
    const int cap = n - i <= kSmall ? kSmall : kLarge;
    int64_t c = 0, chunks = 0;  // as many tensors as fit the parameters and the grid
    while (i + c < n && c < cap) {
      chunks += (t[i + c].n + kChunk - 1) / kChunk;
      if (c > 0 && chunks > 0x7FFFFFFF) break;
      ++c;
    }
    const cudaError_t e = cap == kSmall ? launch_batch<P, G, EIGHT, kSmall>(t + i, c, h, s)
                                        : launch_batch<P, G, EIGHT, kLarge>(t + i, c, h, s);
    if (e != cudaSuccess) return MINITE_ERR_CUDA;
    i += c;
  }
  return MINITE_OK;
}

}  // namespace adamw
}  // namespace minite

using namespace minite;

extern "C" int minite_adamw_step(const minite_adamw_tensor* tensors, int64_t n_tensors,
                                 int param_dtype, int grad_dtype, int state_bits, double lr,
                                 double beta1, double beta2, double eps, double weight_decay,
                                 int64_t step, const float* grad_scale, minite_stream_t stream) {
  using namespace adamw;
  if ((n_tensors > 0 && !tensors) || n_tensors < 0 || step < 1) return MINITE_ERR_INVALID_ARG;
  if ((param_dtype != MINITE_OUT_BF16 && param_dtype != MINITE_OUT_FP32) ||
      (grad_dtype != MINITE_OUT_BF16 && grad_dtype != MINITE_OUT_FP32) ||
      (state_bits != 8 && state_bits != 32))
    return MINITE_ERR_INVALID_ARG;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) ||
      !std::isfinite(lr) || !std::isfinite(eps) || !std::isfinite(weight_decay))
    return MINITE_ERR_INVALID_ARG;
  const bool eight = state_bits == 8;
  const uintptr_t pa = param_dtype == MINITE_OUT_FP32 ? 4 : 2;
  const uintptr_t ga = grad_dtype == MINITE_OUT_FP32 ? 4 : 2;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const minite_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n >= (int64_t(1) << 42)) return MINITE_ERR_UNSUPPORTED_SHAPE;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq ||
        (eight && (!t.exp_avg_scale || !t.exp_avg_sq_scale)))
      return MINITE_ERR_INVALID_ARG;
    if (!aligned(t.param, pa) || !aligned(t.grad, ga) || !aligned(t.param_bf16, 2) ||
        !aligned(t.exp_avg, eight ? 8 : 16) || !aligned(t.exp_avg_sq, eight ? 8 : 16) ||
        (eight && (!aligned(t.exp_avg_scale, 4) || !aligned(t.exp_avg_sq_scale, 4))))
      return MINITE_ERR_INVALID_ARG;
  }
  if (grad_scale && !aligned(grad_scale, 4)) return MINITE_ERR_INVALID_ARG;
  const double bc1 = 1.0 - std::pow(beta1, static_cast<double>(step));
  const double bc2 = 1.0 - std::pow(beta2, static_cast<double>(step));
  Hyper h;
  h.b1 = static_cast<float>(beta1);
  h.c1 = static_cast<float>(1.0 - beta1);
  h.b2 = static_cast<float>(beta2);
  h.c2 = static_cast<float>(1.0 - beta2);
  h.keep = static_cast<float>(1.0 - lr * weight_decay);
  h.rate = static_cast<float>(lr / bc1);
  h.isq = static_cast<float>(1.0 / std::sqrt(bc2));
  h.eps = static_cast<float>(eps);
  h.scale = grad_scale;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool pf = param_dtype == MINITE_OUT_FP32, gf = grad_dtype == MINITE_OUT_FP32;
  if (eight) {
    if (pf && gf) return adamw::step<float, float, true>(tensors, n_tensors, h, s);
    if (pf) return adamw::step<float, uint16_t, true>(tensors, n_tensors, h, s);
    if (gf) return adamw::step<uint16_t, float, true>(tensors, n_tensors, h, s);
    return adamw::step<uint16_t, uint16_t, true>(tensors, n_tensors, h, s);
  }
  if (pf && gf) return adamw::step<float, float, false>(tensors, n_tensors, h, s);
  if (pf) return adamw::step<float, uint16_t, false>(tensors, n_tensors, h, s);
  if (gf) return adamw::step<uint16_t, float, false>(tensors, n_tensors, h, s);
  return adamw::step<uint16_t, uint16_t, false>(tensors, n_tensors, h, s);
}
