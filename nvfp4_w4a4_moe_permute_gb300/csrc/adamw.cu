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
// Codes round to nearest where one step, together with the change of the block's
// scale, moves a moment far enough: beta1 <= 0.9, beta2 <= 0.95. A larger beta takes
// a moment down by much less than half a code's distance (3 to 6%) a step, and
// rounding to nearest would give the old code back for ever: with beta2 0.99 and gradients that fall to a hundredth, sqrt(v) stayed
// 87 to 137 times too large (5th and 95th percentile over elements, 2000 steps),
// with beta1 0.95 and gradients that stop, parameters moved 22 times too far. Such
// a moment's code is drawn from its two neighbours so that it is right on average,
// by a hash of step and element, hence repeatable: 0.79 to 1.30 times, and as far
// as with 32 bits. At the limits nearest is the closer one: 0.88 to 1.15 at beta2
// 0.95, drawn 0.85 to 1.21.
//
// Every operation is rounded to nearest on its own in the order written above
// (no contraction), so that the codes do not depend on how a compiler fuses
// them. Where the moments lie in the usual range, two elements go through the
// packed FP32 instructions with a root and a quotient of their own; the rest
// (zeros among them) takes the IEEE ones.
//
// Bound by HBM. FP32 states (28 bytes an element with a BF16 copy): plain 16-byte
// loads, 604M elements in 2.41 ms, 7.0 TB/s. 8-bit states (10 bytes an element
// with BF16 parameters and gradients, 50 instructions): asynchronous copies three
// reads ahead, the scales of 64 blocks read and written at once; 400M elements
// in 0.65 ms, 6.2 TB/s (1.11 ms with plain loads and IEEE roots and quotients), in
// 0.87 ms where the second moment's codes are drawn (72 instructions, issue slots
// 78% busy), 1.04 where both are.
// Up to 440 tensors' pointers travel as kernel parameters (48 in a small set),
// so that a step is one launch and nothing is copied to the device first.
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace adamw {

constexpr int kBlock = 256;      // elements per 8-bit scale
constexpr int kThreads = 256;
// Elements per CTA. The 8-bit states' CTAs run longer to fill their pipeline less often.
__host__ __device__ constexpr int64_t chunk_elements(bool eight) { return eight ? 16384 : 4096; }
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
  float minus_zero;          // -0
  uint32_t key;              // of the step's draws
  bool draw_m, draw_v;       // 8-bit states: which moment's codes are drawn
  const float* scale;        // device factor of the gradients, or null
};

template <int CAP>
struct Batch {
  Hyper h;
  int count;
  int32_t chunk0[CAP];       // chunks of the tensors before this one
  Tensor t[CAP];
};

// Finaliser of SplitMix64 (Steele, Lea and Flood, 2014).
__host__ __device__ inline uint64_t split_mix(uint64_t x) {
  uint64_t z = x + 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

__device__ __forceinline__ uint64_t twice(float x) { return pair(x, x); }

// A product that no sum after it is contracted with: packed products and sums
// are, in spite of their rounding modifiers, unless the product has an addend
// that the compiler does not know (nz, -0: the product rounded once).
struct Product {
  uint64_t nz;
  __device__ __forceinline__ uint64_t operator()(uint64_t a, uint64_t b) const { return fma2(a, b, nz); }
};

// sqrt(v) of two floats in [2^-100, 2^100], correctly rounded: the remainder of
// v y, y the hardware's approximate 1 / sqrt(v), corrects it (Markstein, 1990;
// equal to the IEEE root for every significand, counted on the device).
__device__ __forceinline__ uint64_t sqrt2_rn(uint64_t v) {
  float a, b, ya, yb;
  unpair(v, a, b);
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(ya) : "f"(a));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(yb) : "f"(b));
  const uint64_t y = pair(ya, yb), r = mul2(v, y);
  return fma2(fma2(mul2(r, twice(-1.0f)), r, v), mul2(y, twice(0.5f)), r);
}

// m / d of two floats, rounded to nearest in the same way from 1 / d after a
// Newton step: equal to the IEEE quotient in 2^30 pairs drawn on the device and
// their negatives, 2^-100 <= |m| < 2^60, 2^-51 <= d < 2^65, where the quotient is a
// normal number. Below, its last place may be another one.
__device__ __forceinline__ uint64_t div2_rn(uint64_t m, uint64_t d) {
  float a, b, ya, yb;
  unpair(d, a, b);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ya) : "f"(a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(yb) : "f"(b));
  const uint64_t y0 = pair(ya, yb), nd = mul2(d, twice(-1.0f));
  const uint64_t y = fma2(fma2(nd, y0, twice(1.0f)), y0, y0);
  const uint64_t q = mul2(m, y);
  return fma2(fma2(nd, q, m), y, q);
}

// The larger magnitude, with some sign; NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float d;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];   // BF16: one, FP32: two (codes below: half of one)
  __device__ __forceinline__ void load(const T* a) {   // 16-byte aligned
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T) / 2); ++j) w[j] = reinterpret_cast<const uint4*>(a)[j];
  }
  __device__ __forceinline__ void load(const T* a, int64_t left) {   // any alignment, `left` exist
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (sizeof(T) == 4) {
        u[j] = j < left ? __float_as_uint(a[j]) : 0u;
      } else {
        const uint32_t x = j < left ? static_cast<uint32_t>(a[j]) : 0u;
        u[j >> 1] = (j & 1) ? u[j >> 1] | (x << 16) : x;
      }
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (sizeof(T) == 4) {
      x[0] = __uint_as_float(w[0].x); x[1] = __uint_as_float(w[0].y);
      x[2] = __uint_as_float(w[0].z); x[3] = __uint_as_float(w[0].w);
      x[4] = __uint_as_float(w[1].x); x[5] = __uint_as_float(w[1].y);
      x[6] = __uint_as_float(w[1].z); x[7] = __uint_as_float(w[1].w);
    } else {
      unpack_bf16x8(w[0], x);
    }
  }
};

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

// Eight E4M3 codes.
template <>
struct Raw8<uint8_t> {
  uint2 w;
  __device__ __forceinline__ void load(const uint8_t* a) { w = *reinterpret_cast<const uint2*>(a); }
  __device__ __forceinline__ void load(const uint8_t* a, int64_t left) {
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) u[j >> 2] |= static_cast<uint32_t>(a[j]) << (8 * (j & 3));
    w = make_uint2(u[0], u[1]);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t c = j < 2 ? w.x : w.y;
      e4m3x2_values((c >> (16 * (j & 1))) & 0xFFFFu, x[2 * j], x[2 * j + 1]);
    }
  }
};

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

// One of the two E4M3 values around x, drawn by the upper 20 bits of `bits` so that
// it is right on average: they are added to the part of x's fraction that the
// format has no room for, and what is left of that part is cut off. Below 2^-6 the
// values lie 2^-9 apart, as they do from there to 2^-5: x is moved there and back.
__device__ __forceinline__ float drawn(float x, uint32_t bits) {
  const float to = fabsf(x) < 0.015625f ? copysignf(0.015625f, x) : 0.0f;
  return __uint_as_float((__float_as_uint(x + to) + (bits >> 12)) & 0xFFF00000u) - to;
}
// Mixed bits, the upper ones of use: multiplications by odd numbers (bits of the
// roots of 2 and 3) and shifts, so that every bit of x reaches them.
__device__ __forceinline__ uint32_t mixed(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  return (x ^ (x >> 15)) * 0xBB67AE85u;
}

// Scale of a block whose largest magnitude is a, NaN if a is not finite: with an
// infinite one the block's other moments would read back as infinite too and its
// parameters stand still without a sign of it.
__device__ __forceinline__ float block_scale_of(float a) {
  const float s = __fadd_rn(__fmul_rn(a, kInvMax), __fsub_rn(a, a));
  return s < kTiny ? kTiny : s;
}
// The warp's largest non-negative float: their bits order as integers, NaN
// above all, so that a block with a NaN gets a NaN scale.
__device__ __forceinline__ float warp_max_nan(float a) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}

// What a thread reads for its eight elements.
template <typename P, typename G, bool EIGHT>
struct Input {
  using S = std::conditional_t<EIGHT, uint8_t, float>;
  Raw8<P> p;
  Raw8<G> g;
  Raw8<S> m, v;
  // `wide`: parameters and gradients are 16-byte aligned; `full`: all eight exist
  __device__ __forceinline__ void load(const Tensor& t, int64_t i, bool full, bool wide) {
    const P* tp = static_cast<const P*>(t.p) + i;
    const G* tg = static_cast<const G*>(t.g) + i;
    const S* tm = static_cast<const S*>(t.m) + i;
    const S* tv = static_cast<const S*>(t.v) + i;
    if (full && wide) {
      p.load(tp);
      g.load(tg);
    } else {
      p.load(tp, t.n - i);
      g.load(tg, t.n - i);
    }
    if (full) {
      m.load(tm);
      v.load(tv);
    } else {
      m.load(tm, t.n - i);
      v.load(tv, t.n - i);
    }
  }
};

// The same by asynchronous copies to slots of shared memory that only this
// thread uses (so that no barrier is needed), kDepth reads ahead. The 8-bit
// states need it: their step has 50 instructions an element for 10 bytes, and
// with loads into registers a warp waited 40% of its time for them.
constexpr int kDepth = 3;
template <typename T>
struct Slots {
  static constexpr int kWords = sizeof(T) == 1 ? 1 : sizeof(T) / 2;
  using Word = std::conditional_t<sizeof(T) == 1, uint2, uint4>;
  Word w[kWords][kThreads];
  __device__ __forceinline__ void fetch(const T* a) {
#pragma unroll
    for (int j = 0; j < kWords; ++j)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                   :: "r"(smem_u32(&w[j][threadIdx.x])), "l"(reinterpret_cast<const Word*>(a) + j),
                      "n"(sizeof(Word)) : "memory");
  }
  __device__ __forceinline__ void take(Raw8<T>& r) const {
#pragma unroll
    for (int j = 0; j < kWords; ++j) reinterpret_cast<Word*>(&r)[j] = w[j][threadIdx.x];
  }
};
template <typename P, typename G>
struct Stage {
  Slots<P> p;
  Slots<G> g;
  Slots<uint8_t> m, v;
  __device__ __forceinline__ void fetch(const Tensor& t, int64_t i) {
    p.fetch(static_cast<const P*>(t.p) + i);
    g.fetch(static_cast<const G*>(t.g) + i);
    m.fetch(static_cast<const uint8_t*>(t.m) + i);
    v.fetch(static_cast<const uint8_t*>(t.v) + i);
  }
  __device__ __forceinline__ void take(Input<P, G, true>& in) const {
    p.take(in.p);
    g.take(in.g);
    m.take(in.m);
    v.take(in.v);
  }
};

template <typename P, typename G, bool EIGHT, bool DRAW, int CAP>
__global__ void __launch_bounds__(kThreads)
adamw_kernel(const __grid_constant__ Batch<CAP> b) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Stage<P, G>* stages = reinterpret_cast<Stage<P, G>*>(smem_raw);   // kDepth of them, 8-bit states only
  pdl_wait();
  int lo = 0, hi = b.count;
  const int chunk = static_cast<int>(blockIdx.x);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.chunk0[mid] <= chunk) lo = mid; else hi = mid;
  }
  const Tensor t = b.t[lo];
  const Hyper h = b.h;
  const int64_t n = t.n;
  constexpr int64_t kPart = chunk_elements(EIGHT);
  const int64_t base = static_cast<int64_t>(chunk - b.chunk0[lo]) * kPart;
  const int64_t end = base + kPart < n ? base + kPart : n;
  P* p = static_cast<P*>(t.p);
  const bool wide = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(t.g) |
                      reinterpret_cast<uintptr_t>(t.copy)) & 15) == 0;
  const Product mul = {twice(h.minus_zero)};
  const int lane8 = 8 * (threadIdx.x & 31);
  constexpr int64_t kStep = 8 * kThreads;
  // a read of less than eight elements, or of unaligned ones, waits for its turn
  auto ask = [&](int64_t i, int stage) {
    if (wide && i + 8 <= end) stages[stage].fetch(t, i);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t i = base + 8 * threadIdx.x;
  int stage = 0;
  if constexpr (EIGHT) {
#pragma unroll
    for (int j = 0; j < kDepth; ++j) ask(i + j * kStep, j);
  }
  // The chunk's scales are read at once and written at once: a word a block,
  // read and written by its warp, cost a third of the kernel's time.
  constexpr int kBlocks = static_cast<int>(kPart) / kBlock;
  __shared__ float s_scale[2][EIGHT ? kBlocks : 1];
  const int my_blk = threadIdx.x % kBlocks;
  const int my_side = threadIdx.x / kBlocks;   // 0: the first moment's, 1: the second's
  const bool my_scale = EIGHT && my_side < 2 && base + static_cast<int64_t>(my_blk) * kBlock < end;
  float* const scales = (my_side == 0 ? t.ms : t.vs) + base / kBlock + my_blk;
  if constexpr (EIGHT) {
    if (my_scale) s_scale[my_side][my_blk] = *scales;
    __syncthreads();
  }
  const float gs = h.scale ? __ldg(h.scale) : 1.0f;
  // a warp's 256 elements are one block of the states
#pragma unroll 1
  for (; i - lane8 < end; i += kStep) {
    const bool full = i + 8 <= n;
    const bool vec = full && wide;
    Input<P, G, EIGHT> in;
    const int blk = static_cast<int>((i - base) / kBlock);
    float old_sm = 0.0f, old_sv = 0.0f;
    if constexpr (EIGHT) {
      asm volatile("cp.async.wait_group %0;" :: "n"(kDepth - 1) : "memory");
      old_sm = s_scale[0][blk];
      old_sv = s_scale[1][blk];
      if (vec) stages[stage].take(in);
      else in.load(t, i, full, wide);
    } else {
      in.load(t, i, full, wide);
    }
    float x[8], d[8], m[8], v[8];
    in.p.get(x);
    in.g.get(d);
    in.m.get(m);
    in.v.get(v);
    uint64_t m2[4], v2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m2[j] = pair(m[2 * j], m[2 * j + 1]);
      v2[j] = pair(v[2 * j], v[2 * j + 1]);
      if constexpr (EIGHT) {
        m2[j] = mul(m2[j], twice(old_sm));
        v2[j] = mul(v2[j], twice(old_sv));
        v2[j] = mul(v2[j], v2[j]);
      }
    }
    // the moments, and their range over this thread's elements
    float m_max = 0.0f, v_max = 0.0f, v_min = kFltMax;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t gj = mul(pair(d[2 * j], d[2 * j + 1]), twice(gs));
      m2[j] = add2(mul(m2[j], twice(h.b1)), mul(gj, twice(h.c1)));
      v2[j] = add2(mul(v2[j], twice(h.b2)), mul(mul(gj, gj), twice(h.c2)));
      unpair(m2[j], m[2 * j], m[2 * j + 1]);
      unpair(v2[j], v[2 * j], v[2 * j + 1]);
      m_max = max_abs_nan(m_max, max_abs_nan(m[2 * j], m[2 * j + 1]));
      v_max = max_abs_nan(v_max, max_abs_nan(v[2 * j], v[2 * j + 1]));
      v_min = fminf(v_min, fminf(v[2 * j], v[2 * j + 1]));
    }
    m_max = fabsf(m_max);
    v_max = fabsf(v_max);
    float sm = 0.0f, sv = 0.0f, im = 0.0f, iv = 0.0f;   // the block's new scales and their inverses
    if constexpr (EIGHT) {
      sm = block_scale_of(warp_max_nan(m_max));
      sv = block_scale_of(__fsqrt_rn(warp_max_nan(v_max)));   // the root is monotone
      im = __fdiv_rn(1.0f, sm);
      iv = __fdiv_rn(1.0f, sv);
    }
    constexpr float kSmallest = 0.001953125f;   // 2^-9, the smallest E4M3 value above zero
    float r[8];
    if (v_min >= 7.888609e-31f && v_max <= 1.2676506e30f && m_max <= 1.1529215e18f) {
      // 2^-100 <= v <= 2^100, |m| <= 2^60: two elements at a time
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t rj = sqrt2_rn(v2[j]);
        const uint64_t u = div2_rn(m2[j], add2(mul(rj, twice(h.isq)), twice(h.eps)));
        const uint64_t xj = add2(mul(pair(x[2 * j], x[2 * j + 1]), twice(h.keep)), mul(u, twice(-h.rate)));
        unpair(xj, x[2 * j], x[2 * j + 1]);
        if constexpr (EIGHT) {
          unpair(mul(m2[j], twice(im)), m[2 * j], m[2 * j + 1]);
          unpair(mul(rj, twice(iv)), r[2 * j], r[2 * j + 1]);
          r[2 * j] = fmaxf(r[2 * j], kSmallest);
          r[2 * j + 1] = fmaxf(r[2 * j + 1], kSmallest);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = __fsqrt_rn(v[j]);
        const float u = __fdiv_rn(m[j], __fadd_rn(__fmul_rn(r[j], h.isq), h.eps));
        x[j] = __fsub_rn(__fmul_rn(x[j], h.keep), __fmul_rn(u, h.rate));
        if constexpr (EIGHT) {
          m[j] = __fmul_rn(m[j], im);
          const float q = __fmul_rn(r[j], iv);
          r[j] = r[j] > 0.0f && q < kSmallest ? kSmallest : q;
        }
      }
    }
    if constexpr (DRAW) {
      const uint32_t first = static_cast<uint32_t>(i) + static_cast<uint32_t>(i >> 32) * 0x3C6EF373u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t bits = mixed((first + j) * 0x9E3779B1u + h.key);
        if (h.draw_m) m[j] = drawn(m[j], bits * 0xA54FF53Bu);
        if (h.draw_v) r[j] = r[j] > 0.0f ? fmaxf(drawn(r[j], bits), kSmallest) : r[j];
      }
    }
    if constexpr (EIGHT) {
      // everything that the slot held has been worked on
      ask(i + kDepth * kStep, stage);
      stage = stage + 1 == kDepth ? 0 : stage + 1;
    }
    store8(p, i, n, vec, x);
    if (t.copy) store8(t.copy, i, n, vec, x);
    if constexpr (EIGHT) {
      store_codes(static_cast<uint8_t*>(t.m), i, n, full, m);
      store_codes(static_cast<uint8_t*>(t.v), i, n, full, r);
      __syncwarp();   // every lane has read the old scales
      if ((threadIdx.x & 31) == 0) {
        s_scale[0][blk] = sm;
        s_scale[1][blk] = sv;
      }
    } else {
      store8(static_cast<float*>(t.m), i, n, full, m);
      store8(static_cast<float*>(t.v), i, n, full, v);
    }
  }
  if constexpr (EIGHT) {
    __syncthreads();
    if (my_scale) *scales = s_scale[my_side][my_blk];
  }
}

template <typename P, typename G, bool EIGHT, bool DRAW, int CAP>
cudaError_t launch_batch(const minite_adamw_tensor* t, int64_t count, const Hyper& h,
                         cudaStream_t s) {
  constexpr int64_t kChunk = chunk_elements(EIGHT);
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
  constexpr size_t kSmem = EIGHT ? kDepth * sizeof(Stage<P, G>) : 0;
  if constexpr (kSmem + 1024 > 48 * 1024) {   // with the static part
    static std::atomic<uint64_t> devices{0};
    const cudaError_t attr_err = allow_smem(devices, adamw_kernel<P, G, EIGHT, DRAW, CAP>, kSmem);
    if (attr_err != cudaSuccess) return attr_err;
  }
  return launch_pdl(adamw_kernel<P, G, EIGHT, DRAW, CAP>, dim3(static_cast<unsigned>(chunks)),
                    dim3(kThreads), kSmem, s, b);
}

template <typename P, typename G, bool EIGHT, bool DRAW>
int step_as(const minite_adamw_tensor* t, int64_t n, const Hyper& h, cudaStream_t s) {
  // kernel parameters carry the tensors' pointers (4 KB or 32 KB of them)
  constexpr int kSmall = 48, kLarge = 440;
  constexpr int64_t kChunk = chunk_elements(EIGHT);
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
    const cudaError_t e = cap == kSmall ? launch_batch<P, G, EIGHT, DRAW, kSmall>(t + i, c, h, s)
                                        : launch_batch<P, G, EIGHT, DRAW, kLarge>(t + i, c, h, s);
    if (e != cudaSuccess) return MINITE_ERR_CUDA;
    i += c;
  }
  return MINITE_OK;
}

template <typename P, typename G, bool EIGHT>
int step(const minite_adamw_tensor* t, int64_t n, const Hyper& h, cudaStream_t s) {
  if constexpr (EIGHT) {
    if (h.draw_m || h.draw_v) return step_as<P, G, true, true>(t, n, h, s);
  }
  return step_as<P, G, EIGHT, false>(t, n, h, s);
}

// Roots of every significand at even and odd exponents, and quotients of 2^30
// hashed pairs and their negatives, that differ from the IEEE ones.
__global__ void math_test_kernel(unsigned long long* mismatches) {
  unsigned long long roots = 0, quotients = 0;
  const uint32_t stride = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
  for (uint32_t i = first; i < (1u << 24); i += stride) {
    const float v = __uint_as_float(0x3F800000u + i);   // [1, 4)
    float a, b;
    unpair(sqrt2_rn(pair(v, v * 0x1p-98f)), a, b);
    roots += (a != __fsqrt_rn(v)) + (b != __fsqrt_rn(v * 0x1p-98f));
    unpair(sqrt2_rn(pair(v * 0x1p96f, v * 0x1p-40f)), a, b);
    roots += (a != __fsqrt_rn(v * 0x1p96f)) + (b != __fsqrt_rn(v * 0x1p-40f));
  }
  for (uint32_t i = first; i < (1u << 30); i += stride) {
    const uint64_t z = split_mix(i);
    // m in +-[2^-100, 2^60), d in [2^-51, 2^65)
    const uint32_t me = 27 + static_cast<uint32_t>((z >> 23) % 160), de = 76 + static_cast<uint32_t>((z >> 55) % 116);
    const float m = __uint_as_float(static_cast<uint32_t>(z & 0x807FFFFFu) | (me << 23));
    const float d = __uint_as_float(static_cast<uint32_t>((z >> 32) & 0x7FFFFFu) | (de << 23));
    float a, b;
    unpair(div2_rn(pair(m, -m), pair(d, d)), a, b);
    const float q = __fdiv_rn(m, d);
    if (fabsf(q) >= kTiny) quotients += (a != q) + (b != -q);
  }
  if (roots) atomicAdd(mismatches, roots);
  if (quotients) atomicAdd(mismatches + 1, quotients);
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
  h.minus_zero = -0.0f;
  h.key = static_cast<uint32_t>(split_mix(static_cast<uint64_t>(step)));
  h.draw_m = beta1 > 0.9;
  h.draw_v = beta2 > 0.95;
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

extern "C" int minite_test_adamw_math(unsigned long long* mismatches, minite_stream_t stream) {
  if (!mismatches) return MINITE_ERR_INVALID_ARG;
  adamw::math_test_kernel<<<4 * num_sms(), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(mismatches);
  return cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}
