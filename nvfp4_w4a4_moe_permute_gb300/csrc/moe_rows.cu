// minite_moe_permute_rows, minite_moe_spread_rows, minite_moe_combine_rows and
// minite_moe_combine_rows_backward: rows in BF16 or FP32 into expert order and
// back, the routing weight applied on the way back, and the gradients.
//
//   permute   rows[d(t, j)] = x[t],              d = stable rank by (expert, token, slot)
//   its gradient                                 dx[t] = sum_j drows[d(t, j)]
//   combine   y[t] = sum_j w[t, j] rows[d(t, j)]
//   its gradient   drows[d(t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], rows[d(t, j)]>
//
// All of it is driven by tokens: a warp holds a piece of token t's row in
// registers and visits the k rows of its slots, so x, dy and y are moved once
// and every permuted row once. Sums are FP32, in slot order; a dot product is
// summed piece by piece in column order, the same for every grid.
//
// Bound by HBM.
#include <initializer_list>

#include "common.cuh"
#include "host_util.h"

namespace minite {

size_t routing_workspace_bytes(int64_t T, int E, int k);
void launch_routing(const int32_t* ids, int64_t T, int k, int E, void* workspace,
                    int32_t* expert_offsets, const int32_t** table, const int32_t** rank, int* ct,
                    int* nchunks, int32_t* status, cudaStream_t s);

namespace rows {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlots = 8;   // rows of a token in flight at once

// B bytes, one access of a lane. Loads are volatile and clobber memory, so that
// they stay behind pdl_wait().
template <int B> struct Word;
template <> struct Word<32> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const char* p) {
    asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                   "=r"(w[7]) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void store(char* p) const {
    st_global_v8(p, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  }
};
template <> struct Word<16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const char* p) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
  __device__ __forceinline__ void store(char* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Word<4> {
  uint32_t w[1];
  __device__ __forceinline__ void load(const char* p) { w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<uint32_t*>(p) = w[0]; }
};
template <> struct Word<2> {
  uint32_t w[1];
  __device__ __forceinline__ void load(const char* p) { w[0] = __ldcs(reinterpret_cast<const uint16_t*>(p)); }
  __device__ __forceinline__ void store(char* p) const {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
  }
};

// The values of a word of elements of type T (float, or uint16_t for BF16).
template <typename T, int B> struct Values {
  static constexpr int kN = B / static_cast<int>(sizeof(T));
  static __device__ __forceinline__ void get(const Word<B>& u, float (&v)[kN]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = __uint_as_float(u.w[i]);
    } else if constexpr (kN == 1) {
      v[0] = bf16lo(u.w[0]);
    } else {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        v[2 * i] = bf16lo(u.w[i]);
        v[2 * i + 1] = bf16hi(u.w[i]);
      }
    }
  }
  static __device__ __forceinline__ void put(Word<B>& u, const float (&v)[kN]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i) u.w[i] = __float_as_uint(v[i]);
    } else if constexpr (kN == 1) {
      u.w[0] = pack_bf16x2_rn(v[0], 0.0f);
    } else {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) u.w[i] = pack_bf16x2_rn(v[2 * i], v[2 * i + 1]);
    }
  }
};

struct Matrix {
  char* p;
  int64_t ld;   // bytes from row to row
};

// Every pair's row: from ids and what launch_routing left, or from dest_row.
struct Routing {
  const int32_t* ids;       // or null: dest_row is given
  const int32_t* offsets;
  const int32_t* table;
  const int32_t* rank;
  int ct, nchunks, E;
  int32_t* dest_row;
  int32_t* perm_src;
};

// x's rows to the rows of their slots. A unit is a token and U words a lane of
// its row; lane j < k holds slot j's row.
template <int B, int U>
__global__ void __launch_bounds__(kThreads) copy_kernel(Matrix x, int64_t T, int64_t words, int k,
                                                        Routing r, Matrix out, int64_t M, int32_t* status) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t parts = (words + 32 * U - 1) / (32 * U);
  const int64_t units = T * parts;
  for (int64_t u = warp; u < units; u += nwarps) {
    const int64_t t = div_nonneg(u, parts);
    const int64_t part = u - t * parts;
    const int64_t w0 = part * (32 * U) + lane;
    Word<B> v[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (w0 + 32 * i < words) v[i].load(x.p + t * x.ld + (w0 + 32 * i) * B);
    int dest = -1;
    if (lane < k) {
      if (r.ids) {
        const int e = r.ids[t * k + lane];
        if (e >= 0 && e < r.E)
          dest = r.offsets[e] + r.table[static_cast<int64_t>(e) * r.nchunks + t / r.ct] + r.rank[t * k + lane];
        if (part == 0) {
          r.dest_row[t * k + lane] = dest;
          if (dest >= 0) r.perm_src[dest] = static_cast<int32_t>(t);
        }
      } else {
        dest = r.dest_row[t * k + lane];
        if (dest >= M) {
          set_status(status, MINITE_ERR_BAD_ROUTING);
          dest = -1;
        }
      }
    }
    for (int j = 0; j < k; ++j) {
      const int d = __shfl_sync(0xffffffffu, dest, j);
      if (d < 0) continue;
      char* row = out.p + d * out.ld;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (w0 + 32 * i < words) v[i].store(row + (w0 + 32 * i) * B);
    }
  }
  if (r.ids)   // rows that no pair has
    for (int64_t i = r.offsets[r.E] + blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; i < M;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      r.perm_src[i] = -1;
}

// y[t] = sum over slots of weight * row, U words of 32 lanes a unit.
template <typename T, int B, int U>
__global__ void __launch_bounds__(kThreads, 2) combine_kernel(Matrix rows, const int32_t* __restrict__ dest_row,
                                                              const float* __restrict__ weights, int64_t T_,
                                                              int64_t M, int64_t words, int k, Matrix y,
                                                              int32_t* status) {
  using V = Values<T, B>;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t parts = (words + 32 * U - 1) / (32 * U);
  const int64_t units = T_ * parts;
  int next = -1;
  float next_w = 1.0f;
  auto ask = [&](int64_t u) {
    const int64_t t = div_nonneg(u, parts);
    if (lane < k) {
      next = dest_row[t * k + lane];
      if (weights) next_w = weights[t * k + lane];
    }
  };
  if (warp < units) ask(warp);
  for (int64_t u = warp; u < units; u += nwarps) {
    const int64_t t = div_nonneg(u, parts);
    const int64_t w0 = (u - t * parts) * (32 * U) + lane;
    int mine = next;
    const float my_w = next_w;
    if (u + nwarps < units) ask(u + nwarps);
    if (mine >= M) {
      set_status(status, MINITE_ERR_BAD_ROUTING);
      mine = -1;
    }
    float acc[U][V::kN];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int c = 0; c < V::kN; ++c) acc[i][c] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += kSlots) {
      Word<B> v[kSlots][U];
#pragma unroll
      for (int jj = 0; jj < kSlots; ++jj) {
        const int d = __shfl_sync(0xffffffffu, mine, (j0 + jj) & 31);
        const char* row = rows.p + d * rows.ld;
        if (j0 + jj < k && d >= 0) {
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (w0 + 32 * i < words) v[jj][i].load(row + (w0 + 32 * i) * B);
        }
      }
#pragma unroll
      for (int jj = 0; jj < kSlots; ++jj) {
        const int d = __shfl_sync(0xffffffffu, mine, (j0 + jj) & 31);
        const float w = __shfl_sync(0xffffffffu, my_w, (j0 + jj) & 31);
        if (j0 + jj < k && d >= 0) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            float f[V::kN];
            V::get(v[jj][i], f);
#pragma unroll
            for (int c = 0; c < V::kN; ++c) acc[i][c] = fmaf(w, f[c], acc[i][c]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (w0 + 32 * i < words) {
        Word<B> o;
        V::put(o, acc[i]);
        o.store(y.p + t * y.ld + (w0 + 32 * i) * B);
      }
  }
}

// Eight values a lane to their sums over the warp: lane l returns the sum of
// value l / 4.
__device__ __forceinline__ float warp_sum8(float (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 4; s > 0; s >>= 1) {
    const bool up = lane & (4 * s);
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float give = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * s);
    }
  }
  float r = v[0];
  r += __shfl_xor_sync(0xffffffffu, r, 2);
  r += __shfl_xor_sync(0xffffffffu, r, 1);
  return r;
}

// drows[d] = weight * dy[t] and, with DOT, dweights = <dy[t], rows[d]>. `group`
// warps of a CTA (a power of two) share a token, taking its pieces in turn; a
// piece's dot products are summed over the warp, then over the pieces in order,
// so that the sums do not depend on `group`. drows may be rows: every piece is
// read by the warp that writes it, before it does.
template <typename T, int B, int U, bool DOT>
__global__ void __launch_bounds__(kThreads, 2) combine_backward_kernel(
    Matrix dy, Matrix rows, const int32_t* __restrict__ dest_row, const float* __restrict__ weights,
    int64_t T_, int64_t M, int64_t words, int k, int group, Matrix drows, float* __restrict__ dweights,
    int32_t* status) {
  using V = Values<T, B>;
  extern __shared__ float s_part[];   // [kWarps / group][parts][kSlots], with group > 1
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int per_cta = kWarps / group;
  const int member = wid % group, team = wid / group;
  const int parts = static_cast<int>((words + 32 * U - 1) / (32 * U));
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_cta;
  // every warp of a CTA makes the same number of turns, for the barriers
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * per_cta; t0 < T_; t0 += step) {
    const int64_t t = t0 + team;
    const bool live = t < T_;
    int mine = -1;
    float my_w = 0.0f;
    if (live && lane < k) {
      mine = dest_row[t * k + lane];
      my_w = weights[t * k + lane];
      if (mine >= M) {
        set_status(status, MINITE_ERR_BAD_ROUTING);
        mine = -1;
      }
    }
    for (int j0 = 0; j0 < k; j0 += kSlots) {
      float sum = 0.0f;
      if (live) {
        for (int part = member; part < parts; part += group) {
          const int64_t w0 = static_cast<int64_t>(part) * (32 * U) + lane;
          float d[U][V::kN];
          Word<B> v[kSlots][U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            Word<B> u = {};
            if (w0 + 32 * i < words) u.load(dy.p + t * dy.ld + (w0 + 32 * i) * B);
            V::get(u, d[i]);
          }
          if constexpr (DOT) {
#pragma unroll
            for (int jj = 0; jj < kSlots; ++jj) {
              const int to = __shfl_sync(0xffffffffu, mine, (j0 + jj) & 31);
              const char* row = rows.p + to * rows.ld;
#pragma unroll
              for (int i = 0; i < U; ++i) {
                v[jj][i] = {};
                if (j0 + jj < k && to >= 0 && w0 + 32 * i < words) v[jj][i].load(row + (w0 + 32 * i) * B);
              }
            }
          }
          float dot[kSlots];
#pragma unroll
          for (int jj = 0; jj < kSlots; ++jj) {
            const int to = __shfl_sync(0xffffffffu, mine, (j0 + jj) & 31);
            const float w = __shfl_sync(0xffffffffu, my_w, (j0 + jj) & 31);
            dot[jj] = 0.0f;
            if (j0 + jj < k && to >= 0) {
              char* row = drows.p + to * drows.ld;
#pragma unroll
              for (int i = 0; i < U; ++i) {
                float f[V::kN];
                if constexpr (DOT) {
                  V::get(v[jj][i], f);
#pragma unroll
                  for (int c = 0; c < V::kN; ++c) dot[jj] = fmaf(d[i][c], f[c], dot[jj]);
                }
#pragma unroll
                for (int c = 0; c < V::kN; ++c) f[c] = w * d[i][c];
                Word<B> o;
                V::put(o, f);
                if (w0 + 32 * i < words) o.store(row + (w0 + 32 * i) * B);
              }
            }
          }
          if constexpr (DOT) {
            const float s = warp_sum8(dot);
            if (group == 1) sum += s;
            else if ((lane & 3) == 0) s_part[(team * parts + part) * kSlots + (lane >> 2)] = s;
          }
        }
      }
      if constexpr (DOT) {
        if (group > 1) {
          __syncthreads();
          if (live && member == 0 && (lane & 3) == 0)
            for (int part = 0; part < parts; ++part) sum += s_part[(team * parts + part) * kSlots + (lane >> 2)];
          __syncthreads();
        }
        if (live && member == 0 && (lane & 3) == 0 && j0 + (lane >> 2) < k)
          dweights[t * k + j0 + (lane >> 2)] = sum;
      }
    }
  }
}

inline bool dtype_ok(int d) { return d == MINITE_OUT_BF16 || d == MINITE_OUT_FP32; }
inline int64_t size_of(int d) { return d == MINITE_OUT_FP32 ? 4 : 2; }

// The widest access that every row of these matrices allows, in bytes.
inline int width(int64_t row_bytes, std::initializer_list<Matrix> ms) {
  uintptr_t bits = static_cast<uintptr_t>(row_bytes);
  for (const Matrix& m : ms) bits |= reinterpret_cast<uintptr_t>(m.p) | static_cast<uintptr_t>(m.ld);
  for (int b : {32, 16, 4}) if (bits % b == 0) return b;
  return 2;
}

inline unsigned blocks_for(int64_t warps, int per_sm) {
  const int64_t b = (warps + kWarps - 1) / kWarps, cap = static_cast<int64_t>(num_sms()) * per_sm;
  return static_cast<unsigned>(b < 1 ? 1 : b < cap ? b : cap);
}

template <int B, int U>
cudaError_t copy_as(const Matrix& x, int64_t T, int64_t row_bytes, int k, const Routing& r, const Matrix& out,
                    int64_t M, int32_t* status, cudaStream_t s) {
  const int64_t words = row_bytes / B, parts = (words + 32 * U - 1) / (32 * U);
  return launch_pdl(copy_kernel<B, U>, dim3(blocks_for(T * parts, 6)), dim3(kThreads), 0, s, x, T, words, k, r,
                    out, M, status);
}
cudaError_t copy(const Matrix& x, int64_t T, int64_t row_bytes, int k, const Routing& r, const Matrix& out,
                 int64_t M, int32_t* status, cudaStream_t s) {
  switch (width(row_bytes, {x, out})) {
    case 32: return copy_as<32, 4>(x, T, row_bytes, k, r, out, M, status, s);
    case 16: return copy_as<16, 4>(x, T, row_bytes, k, r, out, M, status, s);
    case 4: return copy_as<4, 8>(x, T, row_bytes, k, r, out, M, status, s);
    default: return copy_as<2, 8>(x, T, row_bytes, k, r, out, M, status, s);
  }
}

template <typename T, int B, int U>
cudaError_t combine_as(const Matrix& rows, const int32_t* dest_row, const float* weights, int64_t T_, int64_t M,
                       int64_t H, int k, const Matrix& y, int32_t* status, cudaStream_t s) {
  const int64_t words = H * static_cast<int64_t>(sizeof(T)) / B, parts = (words + 32 * U - 1) / (32 * U);
  return launch_pdl(combine_kernel<T, B, U>, dim3(blocks_for(T_ * parts, 2)), dim3(kThreads), 0, s, rows, dest_row,
                    weights, T_, M, words, k, y, status);
}
template <typename T>
cudaError_t combine(const Matrix& rows, const int32_t* dest_row, const float* weights, int64_t T_, int64_t M,
                    int64_t H, int k, const Matrix& y, int32_t* status, cudaStream_t s) {
  switch (width(H * static_cast<int64_t>(sizeof(T)), {rows, y})) {
    case 32: return combine_as<T, 32, 1>(rows, dest_row, weights, T_, M, H, k, y, status, s);
    case 16: return combine_as<T, 16, 1>(rows, dest_row, weights, T_, M, H, k, y, status, s);
    default: return combine_as<T, sizeof(T), 8>(rows, dest_row, weights, T_, M, H, k, y, status, s);
  }
}

template <typename T, int B, int U, bool DOT>
cudaError_t backward_as(const Matrix& dy, const Matrix& rows, const int32_t* dest_row, const float* weights,
                        int64_t T_, int64_t M, int64_t H, int k, const Matrix& drows, float* dweights,
                        int32_t* status, cudaStream_t s) {
  const int64_t words = H * static_cast<int64_t>(sizeof(T)) / B, parts = (words + 32 * U - 1) / (32 * U);
  int group = 1;   // warps a token, so that few tokens still fill the SMs
  if (parts <= 256)   // their sums take 32 KB of shared memory at most
    while (group < kWarps && group < parts && T_ * group < 16 * static_cast<int64_t>(num_sms())) group *= 2;
  const size_t smem = group > 1 ? static_cast<size_t>(kWarps / group) * parts * kSlots * sizeof(float) : 0;
  return launch_pdl(combine_backward_kernel<T, B, U, DOT>, dim3(blocks_for(T_ * group, 2)), dim3(kThreads), smem, s,
                    dy, rows, dest_row, weights, T_, M, words, k, group, drows, dweights, status);
}
template <typename T, bool DOT>
cudaError_t backward(const Matrix& dy, const Matrix& rows, const int32_t* dest_row, const float* weights, int64_t T_,
                     int64_t M, int64_t H, int k, const Matrix& drows, float* dweights, int32_t* status,
                     cudaStream_t s) {
  const int64_t row_bytes = H * static_cast<int64_t>(sizeof(T));
  switch (DOT ? width(row_bytes, {dy, rows, drows}) : width(row_bytes, {dy, drows})) {
    case 32: return backward_as<T, 32, 1, DOT>(dy, rows, dest_row, weights, T_, M, H, k, drows, dweights, status, s);
    case 16: return backward_as<T, 16, 1, DOT>(dy, rows, dest_row, weights, T_, M, H, k, drows, dweights, status, s);
    default:
      return backward_as<T, sizeof(T), 8, DOT>(dy, rows, dest_row, weights, T_, M, H, k, drows, dweights, status, s);
  }
}

// The shape rules that all four entry points share.
inline int check(int dtype, int64_t T, int64_t M, int64_t H, int32_t k, std::initializer_list<int64_t> strides) {
  if (!dtype_ok(dtype)) return MINITE_ERR_INVALID_ARG;
  if (T < 0 || M < 0 || H < 1 || H >= (int64_t(1) << 30) || k < 1 || k > 32 || T >= (int64_t(1) << 31) ||
      T * k >= (int64_t(1) << 31) || M >= (int64_t(1) << 31))
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  for (int64_t s : strides)
    if (s < H || s >= (int64_t(1) << 31)) return MINITE_ERR_UNSUPPORTED_SHAPE;
  return MINITE_OK;
}
inline Matrix matrix(const void* p, int dtype, int64_t stride) {
  return {const_cast<char*>(static_cast<const char*>(p)), stride * size_of(dtype)};
}

}  // namespace rows
}  // namespace minite

using namespace minite;

extern "C" int minite_moe_permute_rows(const void* x, int dtype, int64_t x_stride, const int32_t* topk_ids,
                                       int64_t T, int64_t H, int32_t E, int32_t k, void* rows_out,
                                       int64_t rows_stride, int32_t* expert_offsets, int32_t* perm_src,
                                       int32_t* dest_row, void* workspace, size_t ws_bytes, int32_t* status,
                                       minite_stream_t stream) {
  using namespace rows;
  const int rc = check(dtype, T, 0, H, k, {x_stride, rows_stride});
  if (rc != MINITE_OK) return rc;
  if (E < 1 || E > 1024) return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (!expert_offsets || !aligned(expert_offsets, 4) || !aligned(status, 4)) return MINITE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(expert_offsets, 0, (static_cast<size_t>(E) + 1) * 4, s) == cudaSuccess ? MINITE_OK
                                                                                                  : MINITE_ERR_CUDA;
  const uintptr_t a = static_cast<uintptr_t>(size_of(dtype));
  if (!x || !topk_ids || !rows_out || !perm_src || !dest_row || !workspace || !aligned(x, a) ||
      !aligned(rows_out, a) || !aligned(topk_ids, 4) || !aligned(perm_src, 4) || !aligned(dest_row, 4) ||
      !aligned(workspace, 256) || ws_bytes < routing_workspace_bytes(T, E, k))
    return MINITE_ERR_INVALID_ARG;
  Routing r = {};
  r.ids = topk_ids;
  r.offsets = expert_offsets;
  r.E = E;
  r.dest_row = dest_row;
  r.perm_src = perm_src;
  launch_routing(topk_ids, T, k, E, workspace, expert_offsets, &r.table, &r.rank, &r.ct, &r.nchunks, status, s);
  const cudaError_t e = copy(matrix(x, dtype, x_stride), T, H * size_of(dtype), k, r,
                             matrix(rows_out, dtype, rows_stride), T * k, status, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

extern "C" int minite_moe_spread_rows(const void* x, int dtype, int64_t x_stride, const int32_t* dest_row, int64_t T,
                                      int64_t M, int64_t H, int32_t k, void* rows_out, int64_t rows_stride,
                                      int32_t* status, minite_stream_t stream) {
  using namespace rows;
  const int rc = check(dtype, T, M, H, k, {x_stride, rows_stride});
  if (rc != MINITE_OK) return rc;
  if (T == 0 || M == 0) return MINITE_OK;
  const uintptr_t a = static_cast<uintptr_t>(size_of(dtype));
  if (!x || !dest_row || !rows_out || !aligned(x, a) || !aligned(rows_out, a) || !aligned(dest_row, 4) ||
      !aligned(status, 4))
    return MINITE_ERR_INVALID_ARG;
  Routing r = {};
  r.dest_row = const_cast<int32_t*>(dest_row);
  const cudaError_t e = copy(matrix(x, dtype, x_stride), T, H * size_of(dtype), k, r,
                             matrix(rows_out, dtype, rows_stride), M, status,
                             reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

extern "C" int minite_moe_combine_rows(const void* rows_in, int dtype, int64_t rows_stride, const int32_t* dest_row,
                                       const float* weights, int64_t T, int64_t M, int64_t H, int32_t k, void* y,
                                       int64_t y_stride, int32_t* status, minite_stream_t stream) {
  using namespace rows;
  const int rc = check(dtype, T, M, H, k, {rows_stride, y_stride});
  if (rc != MINITE_OK) return rc;
  if (T == 0) return MINITE_OK;
  const uintptr_t a = static_cast<uintptr_t>(size_of(dtype));
  if ((!rows_in && M > 0) || !dest_row || !y || !aligned(rows_in, a) || !aligned(y, a) || !aligned(dest_row, 4) ||
      !aligned(weights, 4) || !aligned(status, 4))
    return MINITE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Matrix r = matrix(rows_in, dtype, rows_stride), o = matrix(y, dtype, y_stride);
  const cudaError_t e = dtype == MINITE_OUT_FP32 ? combine<float>(r, dest_row, weights, T, M, H, k, o, status, s)
                                                 : combine<uint16_t>(r, dest_row, weights, T, M, H, k, o, status, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

extern "C" int minite_moe_combine_rows_backward(const void* dy, int dtype, int64_t dy_stride, const void* rows_in,
                                                int64_t rows_stride, const int32_t* dest_row, const float* weights,
                                                int64_t T, int64_t M, int64_t H, int32_t k, void* drows,
                                                int64_t drows_stride, float* dweights, int32_t* status,
                                                minite_stream_t stream) {
  using namespace rows;
  const int rc = check(dtype, T, M, H, k, {dy_stride, rows_in ? rows_stride : H, drows_stride});
  if (rc != MINITE_OK) return rc;
  if ((rows_in == nullptr) != (dweights == nullptr)) return MINITE_ERR_INVALID_ARG;
  if (rows_in == drows && rows_stride != drows_stride) return MINITE_ERR_INVALID_ARG;
  if (T == 0) return MINITE_OK;
  const uintptr_t a = static_cast<uintptr_t>(size_of(dtype));
  if (!dy || !dest_row || !weights || (!drows && M > 0) || !aligned(dy, a) || !aligned(rows_in, a) ||
      !aligned(drows, a) || !aligned(dest_row, 4) || !aligned(weights, 4) || !aligned(dweights, 4) ||
      !aligned(status, 4))
    return MINITE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Matrix d = matrix(dy, dtype, dy_stride), r = matrix(rows_in, dtype, rows_in ? rows_stride : 0),
               o = matrix(drows, dtype, drows_stride);
  cudaError_t e;
  if (dtype == MINITE_OUT_FP32)
    e = rows_in ? backward<float, true>(d, r, dest_row, weights, T, M, H, k, o, dweights, status, s)
                : backward<float, false>(d, r, dest_row, weights, T, M, H, k, o, nullptr, status, s);
  else
    e = rows_in ? backward<uint16_t, true>(d, r, dest_row, weights, T, M, H, k, o, dweights, status, s)
                : backward<uint16_t, false>(d, r, dest_row, weights, T, M, H, k, o, nullptr, status, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}
