// minite_moe_permute_rows, minite_moe_spread_rows, minite_moe_combine_rows and
// minite_moe_combine_rows_backward: rows in BF16 or FP32 into expert order and
// back, the routing weight applied on the way back, and the gradients.
//
//   permute   rows[d(t, j)] = x[t],              d = stable rank by (expert, token, slot)
//   its gradient                                 dx[t] = sum_j drows[d(t, j)]
//   combine   y[t] = sum_j w[t, j] rows[d(t, j)]
//   its gradient   drows[d(t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], rows[d(t, j)]>
//
// All of it is driven by tokens: a warp holds a piece of token t's row and visits
// the k rows of its slots, so x, dy and y are moved once and every permuted row once.
// Sums are FP32, in slot order; a dot product is summed in an order that follows from
// the row's size and alignment alone.
//
// Bound by HBM, reads at up to 7.3 TB/s and writes at 6.4. BF16 rows of 2048 columns,
// top-8 of 128 experts, a pass among others (in brackets what the bytes take at the
// measured copy rate): 32768 tokens permuted 199 us (181), combined 180 (181); a
// micro-batch of 4096 permuted 25.8 (22.6), summed back 24.0 (22.6), weighted gradient
// 48.8 (42.7). What a micro-batch permuted has above its writes (21) is the sort, 5 us.
// One token takes 3.5 us.
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
// Rows of a token in flight at once, whatever k is: with fewer slots less is on its way.
// 32768 BF16 tokens of 2048 combined over 1, 2, 4, 8 slots take 91, 103, 124, 180 us (40,
// 60, 100, 180 at the copy rate), their gradient 108, 133, 190, 355 (60, 100, 180, 341).
constexpr int kSlots = 8;

// B bytes, one access of a lane (32 bytes were 4% slower in the copies, more in the
// sums).
template <int B> struct Word;
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
// its row; lane j < k holds slot j's row. Each warp writes 2 KB of a row at a time
// (words of 16 bytes; the copies of 32768 tokens take 190 us, 1.07 GB of stores
// alone 168).
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

// Permutations of up to kClusterPairs slots in one launch: every CTA has a range of
// tokens, and finds out by itself how many slots of each expert come before them and
// in all. It counts by atomics in shared memory (10 cycles each 32 ids): up to
// kDirectPairs slots all ids, above that a CL-th of them, what the CTAs of a cluster
// have counted being added up from one another's shared memory. A thread has one slot
// of the range; those of the warps in front are a row of 16 bytes for each expert.
// With rows of 32 bytes, top-8 of 128 experts, on the device: 1024 tokens 4.1 us, 2048
// 5.5, 4096 in clusters 7.4 and 8192 9.9; by ranking, scan kernel and copies 4096 take
// 11.0, and the host 9 us more a call. In 76 clusters of 2 they take 7.5 and 11.5; of
// clusters of 8 only 15 are resident, too few for 8192.
// Rows are written faster by somewhat fewer SMs than there are: rows of 4 KB, 4096
// tokens, in 104 CTAs 28.0 us, 112 26.8, 120 and 124 26.0, 136 27.8, 144 27.6; rows of
// 14 KB, 5000 tokens, 110, 110, 109, 118, 114. Rows of 32 bytes take 0.9 us less in 144.
constexpr int64_t kDirectPairs = 16384;
constexpr int64_t kClusterPairs = 65536;
constexpr int kRangeCluster = 4;
constexpr int kRangeSms = 80;   // CTAs in clusters, of 100 SMs (95 would be resident)
constexpr int kRangeThreads = 512;
constexpr int kRangeWarps = kRangeThreads / 32;

// Sum of v over the threads in front of this one, and over all.
__device__ __forceinline__ int scan_before(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += u;
  }
  if (lane == 31) s_warp[wid] = in;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kRangeWarps; ++w) {
    const int x = s_warp[w];
    if (w < wid) before += x;
    all += x;
  }
  *total = all;
  return before + in - v;
}

template <int B, int U, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kRangeThreads, 1) range_kernel(
    Matrix x, int64_t T, int64_t words, int k, int E, const int32_t* ids, int32_t* offsets, int32_t* perm_src,
    int32_t* dest_row, Matrix out, int32_t* status) {
  extern __shared__ __align__(16) int32_t sm[];
  __shared__ int s_warp[kRangeWarps];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int member = static_cast<int>(blockIdx.x) % CL;
  const int per = static_cast<int>((T + gridDim.x - 1) / gridDim.x);
  const int t0 = min(static_cast<int>(T), static_cast<int>(blockIdx.x) * per), t1 = min(static_cast<int>(T), t0 + per);
  const int p0 = t0 * k, own = (t1 - t0) * k, pairs = static_cast<int>(T) * k;
  // the cluster's first slot, and the slots that this CTA counts
  const int first = min(static_cast<int>(T), (static_cast<int>(blockIdx.x) - member) * per) * k;
  const int share = (pairs + 4 * CL - 1) / (4 * CL) * 4;
  const int lo = min(pairs, member * share), hi = min(pairs, lo + share);
  int32_t* s_before = sm;            // [E] counted slots before the cluster's first
  int32_t* s_after = sm + E;         // [E] the others
  int32_t* s_own = sm + 2 * E;       // [E] slots of the range
  int32_t* s_first = sm + 3 * E;     // [E] row of the range's first slot
  // [E][kRangeWarps] the slots of each warp's 32 of the range, a byte each; [per * k] rows
  uint8_t* s_warps = reinterpret_cast<uint8_t*>(sm + 4 * E);
  int32_t* s_dest = sm + 8 * E;
  for (int e = tid; e < 3 * E; e += kRangeThreads) sm[e] = 0;
  for (int e = tid; e < E; e += kRangeThreads) reinterpret_cast<uint4*>(s_warps)[e] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  pdl_wait();
  // units of this CTA: a token and U words a lane
  const int parts = static_cast<int>((words + 32 * U - 1) / (32 * U));
  const int units = (t1 - t0) * parts;
  auto fetch = [&](int u, Word<B> (&v)[U]) {
    if (u >= units) return;
    const int t = u / parts;
    const int64_t w0 = static_cast<int64_t>(u - t * parts) * (32 * U) + lane;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (w0 + 32 * i < words) v[i].load(x.p + (t0 + t) * x.ld + (w0 + 32 * i) * B);
  };
  Word<B> va[U], vb[U];
  fetch(wid, va);
  bool bad = false;
  auto count = [&](int p, int e) {
    bad |= e >= E;
    if (e >= 0 && e < E) atomicAdd((p < first ? s_before : s_after) + e, 1);
  };
  if ((reinterpret_cast<uintptr_t>(ids) & 15) == 0) {
    const int4* ids4 = reinterpret_cast<const int4*>(ids);
    for (int q = lo / 4 + tid; q < hi / 4; q += kRangeThreads) {
      const int4 a = ids4[q];
      count(4 * q, a.x);
      count(4 * q + 1, a.y);
      count(4 * q + 2, a.z);
      count(4 * q + 3, a.w);
    }
    for (int p = max(lo, hi & ~3) + tid; p < hi; p += kRangeThreads) count(p, ids[p]);
  } else {
    for (int p = lo + tid; p < hi; p += kRangeThreads) count(p, ids[p]);
  }
  // slot tid of the range, which has no more than threads
  const int id = tid < own ? ids[p0 + tid] : -1;
  const int my_e = id >= 0 && id < E ? id : E;
  const uint32_t same = same_id_lanes(my_e, E);
  const int in_warp = __popc(same & ((1u << lane) - 1u));
  if (my_e < E && in_warp == 0) {
    s_warps[my_e * kRangeWarps + wid] = static_cast<uint8_t>(__popc(same));
    if (CL > 1) atomicAdd(s_own + my_e, __popc(same));
  }
  if (bad && blockIdx.x < CL) set_status(status, MINITE_ERR_BAD_ROUTING);
  if constexpr (CL > 1) cluster_sync_all(); else __syncthreads();
  int used = 0;
  for (int base = 0; base < E; base += kRangeThreads) {
    const int e = base + tid;
    int before = 0, after = 0, others = 0;   // others: of the cluster's ranges in front
    if (e < E) {
      if constexpr (CL > 1) {
#pragma unroll
        for (int m = 0; m < CL; ++m) {
          const uint32_t at = mapa_shared(smem_u32(sm + e), m);
          before += static_cast<int>(ld_shared_cluster(at));
          after += static_cast<int>(ld_shared_cluster(at + 4 * E));
          const int n = static_cast<int>(ld_shared_cluster(at + 8 * E));
          if (m < member) others += n;
        }
      } else {
        before = s_before[e];
        after = s_after[e];
      }
    }
    int total;
    const int at = used + scan_before(before + after, s_warp, &total);
    if (e < E) {
      s_first[e] = at + before + others;
      if (blockIdx.x == 0) offsets[e] = at;
    }
    used += total;
    __syncthreads();
  }
  if constexpr (CL > 1) cluster_arrive();   // nobody leaves while its counts are read
  if (blockIdx.x == 0 && tid == 0) offsets[E] = used;
  if (tid < own) {
    int dest = -1;
    if (my_e < E) {   // after the slots of the warps in front
      dest = s_first[my_e] + in_warp;
      const uint4 c = reinterpret_cast<const uint4*>(s_warps)[my_e];
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = min(max(wid - 4 * i, 0), 4);   // of these four bytes
        dest += __dp4a(w[i], n == 4 ? 0x01010101u : 0x01010101u & ((1u << (8 * n)) - 1u), 0u);
      }
      perm_src[dest] = t0 + tid / k;
    }
    s_dest[tid] = dest;
    dest_row[p0 + tid] = dest;
  }
  __syncthreads();
  auto spread = [&](int u, const Word<B> (&v)[U]) {
    if (u >= units) return;
    const int t = u / parts;
    const int64_t w0 = static_cast<int64_t>(u - t * parts) * (32 * U) + lane;
    for (int j = 0; j < k; ++j) {
      const int d = s_dest[t * k + j];
      if (d < 0) continue;
      char* row = out.p + d * out.ld;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (w0 + 32 * i < words) v[i].store(row + (w0 + 32 * i) * B);
    }
  };
  for (int u = wid; u < units; u += 2 * kRangeWarps) {
    fetch(u + kRangeWarps, vb);
    spread(u, va);
    fetch(u + 2 * kRangeWarps, va);
    spread(u + kRangeWarps, vb);
  }
  for (int i = used + blockIdx.x * kRangeThreads + tid; i < pairs; i += gridDim.x * kRangeThreads) perm_src[i] = -1;
  if constexpr (CL > 1) {
    __syncwarp();
    cluster_wait();
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

// y[t] = sum over slots of weight * row. A unit is a token and U words a lane of its
// row, in eight slots at once: 64 registers of loads, two CTAs an SM. Rows of whole
// 16-byte words take two of them a lane, 1 KB of each row a warp (32768 tokens of 8
// slots 179 us; one word of 32 bytes 215, four of 8 bytes 180, two of 8 bytes, with
// more CTAs, 254 to 319; asynchronous copies through shared memory, four steps
// ahead, 189). Others take eight of 4 or of 2 bytes.
template <typename T, int B, int U>
__global__ void __launch_bounds__(kThreads, 2) combine_kernel(
    Matrix rows, const int32_t* dest_row, const float* weights, int64_t T_, int64_t M, int64_t words, int k, Matrix y,
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

// drows[d] = weight * dy[t] and, with DOT, dweights = <dy[t], rows[d]>. `team` warps of
// a CTA share a token: member m takes pieces m, m + team, ... of its row, a piece being
// U words of 32 lanes, in eight slots at once. A member's dot products stay in its
// lanes until its last piece and then wait in shared memory for the other members';
// every kHeld items (a token and eight slots) all are added, in the members' order.
// team follows from the row's size alone, so the sums do not depend on the other
// tokens. drows may be rows: a piece is read by the warp that writes it, before it does.
constexpr int kHeld = 16;
template <typename T, int B, int U, bool DOT>
__global__ void __launch_bounds__(kThreads, 2) combine_backward_kernel(
    Matrix dy, Matrix rows, const int32_t* dest_row, const float* weights, int64_t T_, int64_t M, int64_t words, int k,
    int team, Matrix drows, float* dweights, int32_t* status) {
  using V = Values<T, B>;
  __shared__ float s_dot[kHeld][kWarps][kSlots];
  pdl_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int teams = kWarps / team, mine = wid / team, member = wid % team;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * teams;   // the CTA's first token
  const int64_t stride = static_cast<int64_t>(gridDim.x) * teams;
  const int64_t turns = first < T_ ? (T_ - first - 1) / stride + 1 : 0;   // the same for every team
  const int groups = (k + kSlots - 1) / kSlots;
  const int parts = static_cast<int>((words + 32 * U - 1) / (32 * U));
  int next = -1;
  float next_w = 0.0f;
  auto ask = [&](int64_t turn) {
    const int64_t t = first + mine + turn * stride;
    next = -1;
    if (turn < turns && t < T_ && lane < k) {
      next = dest_row[t * k + lane];
      next_w = weights[t * k + lane];
    }
  };
  ask(0);
  int held = 0;
  int64_t item0 = 0;   // the first item that is held
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t t = first + mine + turn * stride;
    int dest = next;
    const float my_w = next_w;
    ask(turn + 1);
    if (dest >= M) {
      set_status(status, MINITE_ERR_BAD_ROUTING);
      dest = -1;
    }
    for (int g = 0; g < groups; ++g) {
      const int j0 = g * kSlots;
      float dot[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) dot[j] = 0.0f;
      for (int part = t < T_ ? member : parts; part < parts; part += team) {
        const int64_t w0 = static_cast<int64_t>(part) * (32 * U) + lane;
        // every word is used under the condition under which it is loaded: one that
        // was set to 0 first made each load wait for the one before it (95 us in
        // place of 24 for 12000 tokens of 201 columns)
        Word<B> d[U], v[kSlots][U];
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (w0 + 32 * i < words) d[i].load(dy.p + t * dy.ld + (w0 + 32 * i) * B);
        if constexpr (DOT) {
#pragma unroll
          for (int jj = 0; jj < kSlots; ++jj) {
            const int to = __shfl_sync(0xffffffffu, dest, (j0 + jj) & 31);
            const char* row = rows.p + to * rows.ld;
            if (j0 + jj < k && to >= 0) {
#pragma unroll
              for (int i = 0; i < U; ++i)
                if (w0 + 32 * i < words) v[jj][i].load(row + (w0 + 32 * i) * B);
            }
          }
        }
#pragma unroll
        for (int jj = 0; jj < kSlots; ++jj) {
          const int to = __shfl_sync(0xffffffffu, dest, (j0 + jj) & 31);
          const float w = __shfl_sync(0xffffffffu, my_w, (j0 + jj) & 31);
          if (j0 + jj < k && to >= 0) {
            char* row = drows.p + to * drows.ld;
#pragma unroll
            for (int i = 0; i < U; ++i)
              if (w0 + 32 * i < words) {
                float x[V::kN], f[V::kN];
                V::get(d[i], x);
                if constexpr (DOT) {
                  V::get(v[jj][i], f);
#pragma unroll
                  for (int c = 0; c < V::kN; ++c) dot[jj] = fmaf(x[c], f[c], dot[jj]);
                }
#pragma unroll
                for (int c = 0; c < V::kN; ++c) f[c] = w * x[c];
                Word<B> o;
                V::put(o, f);
                o.store(row + (w0 + 32 * i) * B);
              }
          }
        }
      }
      if constexpr (DOT) {
        const float sum = warp_sum8(dot);
        if ((lane & 3) == 0) s_dot[held][wid][lane >> 2] = sum;
        if (++held == kHeld || (turn + 1 == turns && g + 1 == groups)) {
          __syncthreads();
          for (int x = threadIdx.x; x < held * teams * kSlots; x += kThreads) {
            const int j = x % kSlots, q = x / kSlots % teams, h = x / (kSlots * teams);
            const int64_t at = div_nonneg(item0 + h, groups), token = first + q + at * stride;
            const int slot = static_cast<int>(item0 + h - at * groups) * kSlots + j;
            if (token < T_ && slot < k) {
              float sum_of = 0.0f;
              for (int m = 0; m < team; ++m) sum_of += s_dot[h][q * team + m][j];
              dweights[token * k + slot] = sum_of;
            }
          }
          __syncthreads();
          item0 += held;
          held = 0;
        }
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
  for (int b : {16, 4}) if (bits % b == 0) return b;
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

struct Sorted {   // what a permutation writes besides the rows
  int32_t* offsets;
  int32_t* perm_src;
  int32_t* dest_row;
};
template <int B, int U, int CL>
cudaError_t range_as(const Matrix& x, int64_t T, int64_t row_bytes, int k, int E, const int32_t* ids, const Sorted& o,
                     const Matrix& out, int32_t* status, cudaStream_t s) {
  const int64_t tokens = kRangeThreads / k;   // a range has no more: a thread a slot
  const int64_t many = CL == 1 ? num_sms() : num_sms() * kRangeSms / 100 / CL * CL;
  int64_t grid = T < many ? T : many;
  if (grid * tokens < T) grid = (T + tokens - 1) / tokens;
  grid = (grid + CL - 1) / CL * CL;
  const size_t smem = (8 * static_cast<size_t>(E) + static_cast<size_t>((T + grid - 1) / grid) * k) * sizeof(int32_t);
  return launch_pdl(range_kernel<B, U, CL>, dim3(static_cast<unsigned>(grid)), dim3(kRangeThreads), smem, s, x, T,
                    row_bytes / B, k, E, ids, o.offsets, o.perm_src, o.dest_row, out, status);
}
template <int CL>
cudaError_t range(const Matrix& x, int64_t T, int64_t row_bytes, int k, int E, const int32_t* ids, const Sorted& o,
                  const Matrix& out, int32_t* status, cudaStream_t s) {
  switch (width(row_bytes, {x, out})) {
    case 16: return range_as<16, 8, CL>(x, T, row_bytes, k, E, ids, o, out, status, s);
    case 4: return range_as<4, 8, CL>(x, T, row_bytes, k, E, ids, o, out, status, s);
    default: return range_as<2, 8, CL>(x, T, row_bytes, k, E, ids, o, out, status, s);
  }
}

cudaError_t copy(const Matrix& x, int64_t T, int64_t row_bytes, int k, const Routing& r, const Matrix& out,
                 int64_t M, int32_t* status, cudaStream_t s) {
  switch (width(row_bytes, {x, out})) {
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
  const int w = width(H * static_cast<int64_t>(sizeof(T)), {rows, y});
  if (w == 16) return combine_as<T, 16, 2>(rows, dest_row, weights, T_, M, H, k, y, status, s);
  if constexpr (sizeof(T) == 2)
    if (w == 2) return combine_as<T, 2, 8>(rows, dest_row, weights, T_, M, H, k, y, status, s);
  return combine_as<T, 4, 8>(rows, dest_row, weights, T_, M, H, k, y, status, s);
}

template <typename T, int B, int U, bool DOT>
cudaError_t backward_as(const Matrix& dy, const Matrix& rows, const int32_t* dest_row, const float* weights,
                        int64_t T_, int64_t M, int64_t H, int k, const Matrix& drows, float* dweights,
                        int32_t* status, cudaStream_t s) {
  const int64_t words = H * static_cast<int64_t>(sizeof(T)) / B, parts = (words + 32 * U - 1) / (32 * U);
  int team = 1;
  while (team < kWarps && team < parts) team *= 2;
  return launch_pdl(combine_backward_kernel<T, B, U, DOT>, dim3(blocks_for(T_ * team, 2)), dim3(kThreads), 0, s, dy,
                    rows, dest_row, weights, T_, M, words, k, team, drows, dweights, status);
}
template <typename T, bool DOT>
cudaError_t backward(const Matrix& dy, const Matrix& rows, const int32_t* dest_row, const float* weights, int64_t T_,
                     int64_t M, int64_t H, int k, const Matrix& drows, float* dweights, int32_t* status,
                     cudaStream_t s) {
  const int64_t row_bytes = H * static_cast<int64_t>(sizeof(T));
  const int w = DOT ? width(row_bytes, {dy, rows, drows}) : width(row_bytes, {dy, drows});
  if (w == 16) return backward_as<T, 16, 2, DOT>(dy, rows, dest_row, weights, T_, M, H, k, drows, dweights, status, s);
  if constexpr (sizeof(T) == 2)
    if (w == 2) return backward_as<T, 2, 8, DOT>(dy, rows, dest_row, weights, T_, M, H, k, drows, dweights, status, s);
  return backward_as<T, 4, 8, DOT>(dy, rows, dest_row, weights, T_, M, H, k, drows, dweights, status, s);
}

// The shape rules that all four entry points share.
inline int check(int dtype, int64_t T, int64_t M, int64_t H, int32_t k, std::initializer_list<int64_t> strides) {
  if (!dtype_ok(dtype)) return MINITE_ERR_INVALID_ARG;
  if (T < 0 || M < 0 || H < 1 || H > (int64_t(1) << 24) || k < 1 || k > 32 || T >= (int64_t(1) << 31) ||
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

// 0: minite_moe_permute_rows takes one launch and needs none.
size_t permute_rows_workspace_bytes(int64_t T, int E, int k) {
  return T * k <= rows::kClusterPairs ? 0 : routing_workspace_bytes(T, E, k);
}

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
  const size_t need = permute_rows_workspace_bytes(T, E, k);
  if (!x || !topk_ids || !rows_out || !perm_src || !dest_row || !aligned(x, a) || !aligned(rows_out, a) ||
      !aligned(topk_ids, 4) || !aligned(perm_src, 4) || !aligned(dest_row, 4) ||
      (need > 0 && (!workspace || !aligned(workspace, 256) || ws_bytes < need)))
    return MINITE_ERR_INVALID_ARG;
  const Matrix from = matrix(x, dtype, x_stride), to = matrix(rows_out, dtype, rows_stride);
  const int64_t row_bytes = H * size_of(dtype);
  const Sorted o = {expert_offsets, perm_src, dest_row};
  cudaError_t e;
  if (T * k <= kDirectPairs) {
    e = range<1>(from, T, row_bytes, k, E, topk_ids, o, to, status, s);
  } else if (need == 0) {
    e = range<kRangeCluster>(from, T, row_bytes, k, E, topk_ids, o, to, status, s);
  } else {
    Routing r = {};
    r.ids = topk_ids;
    r.offsets = expert_offsets;
    r.E = E;
    r.dest_row = dest_row;
    r.perm_src = perm_src;
    launch_routing(topk_ids, T, k, E, workspace, expert_offsets, &r.table, &r.rank, &r.ct, &r.nchunks, status, s);
    e = copy(from, T, row_bytes, k, r, to, T * k, status, s);
  }
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

extern "C" int minite_moe_spread_rows(const void* x, int dtype, int64_t x_stride, const int32_t* dest_row, int64_t T,
                                      int64_t M, int64_t H, int32_t k, void* rows_out, int64_t rows_stride,
                                      int32_t* status, minite_stream_t stream) {
  using namespace rows;
  const int rc = check(dtype, T, M, H, k, {x_stride, rows_stride});
  if (rc != MINITE_OK) return rc;
  if (T == 0 || (M == 0 && !status)) return MINITE_OK;   // without rows: only to report those that are named
  const uintptr_t a = static_cast<uintptr_t>(size_of(dtype));
  if (!x || !dest_row || (!rows_out && M > 0) || !aligned(x, a) || !aligned(rows_out, a) || !aligned(dest_row, 4) ||
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
  if (T == 0) return MINITE_OK;
  const bool dot = dweights != nullptr;
  if ((rows_in && !dot) || (dot && !rows_in && M > 0)) return MINITE_ERR_INVALID_ARG;
  if (rows_in && rows_in == drows && rows_stride != drows_stride) return MINITE_ERR_INVALID_ARG;
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
    e = dot ? backward<float, true>(d, r, dest_row, weights, T, M, H, k, o, dweights, status, s)
            : backward<float, false>(d, r, dest_row, weights, T, M, H, k, o, nullptr, status, s);
  else
    e = dot ? backward<uint16_t, true>(d, r, dest_row, weights, T, M, H, k, o, dweights, status, s)
            : backward<uint16_t, false>(d, r, dest_row, weights, T, M, H, k, o, nullptr, status, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}
