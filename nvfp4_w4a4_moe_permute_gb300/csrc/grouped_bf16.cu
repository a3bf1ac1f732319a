// minite_grouped_gemm_bf16 / minite_grouped_wgrad_bf16: BF16 matrix products
// grouped by expert over ragged row ranges, FP32 sums on the tensor cores.
//
//   forward   out[m, n] = sum_k a[m, k] w[e][n, k]     w [E, N, K]
//   dgrad     out[m, n] = sum_k a[m, k] w[e][k, n]     w [E, K, N], read as stored
//   wgrad     out[e][i, j] (+)= sum_m a[m, i] b[m, j]  m over expert e's rows
//
// e is the expert of row m, from device-side offsets; one persistent launch
// covers all experts.
//
// Design (sm_103a):
//  * The output is computed transposed: the matrix instruction's M is the
//    output's contiguous dimension (features: rows of the weight, or the second
//    operand's columns of a weight gradient) and its N the output's rows
//    (tokens, or the first operand's columns). N may be any multiple of 32 up
//    to 256, so a ragged expert costs its rows rounded up to 32 instead of to a
//    tile, one token costs 32, and the tile's width is chosen per launch. A
//    TMEM lane then holds one feature and a warp writes 32 neighbouring
//    features of a row, without a transposition.
//  * The two CTAs of a cluster work on one 256 (features) x N tile with
//    tcgen05.mma.cta_group::2: each loads 128 features and half the rows, K
//    consumed 64 values (128 bytes) a stage, and holds 128 x N sums in TMEM,
//    twice, so that a tile's epilogue runs under the next one's products. Every
//    copy is a CTA's own: no load is multicast, so that no call can make one
//    read memory of another GPU.
//    8 experts of 8192 rows, 2048 x 1536, take 226 to 232 us (1827 to 1778
//    TFLOP/s, 95 to 92% of the measured burst rate), with FP32 results 271.
//  * Large experts (bound by the tensor cores and L2) and small ones (bound by
//    DRAM) are interleaved, so that all are busy: 65536 rows in Zipf shares, 2048
//    x 1536, 315 to 327 us (floors: tensor 214, HBM 191). 128 experts of 256 rows,
//    1536 x 2048: 165 to 168 us, 95 to 93% of the copy rate; of 16 rows 129 to 131.
//  * Operands come by TMA with the 128-byte swizzle, K-major (rows of 64 K
//    values) or, where memory has the other dimension contiguous (dgrad's
//    weight, both operands of the weight gradient), MN-major: boxes of 64 such
//    values x 64 K rows. No operand is transposed in memory.
//  * Ragged ends: rows past an expert's last one are read and not stored. A K
//    tail reads zeros (the weight's tensor map is three-dimensional, so it
//    never reaches into the next expert). The weight gradient's K range ends
//    inside a 64-row box that already holds the next expert's rows: only the
//    K = 16 steps that hold rows are issued, and the rows of the last step past
//    the end are zeroed in shared memory in both operands (a NaN there would
//    survive a product with zero). For such a stage the odd CTA's copies count
//    on its own barrier; its second warp zeroes and reports to the even CTA.
//  * FP32 outputs: the tensor cores' FP32 sums lose up to 2^-22 of the running
//    sum at every K = 16 step, always towards zero. Sums longer than
//    kChunkBlocks blocks are therefore split: each chunk is summed in TMEM and
//    the chunks are added in FP32 registers (round to nearest) by the
//    epilogue warps. BF16 outputs are split after 16384
//    values, where 2^-12 beside their last rounding of 2^-8 may be lost (sums of
//    65536 values of one sign lost 3.3e-4, of 2^25 more than that rounding).
//    Weight gradients in FP32 leave by bulk copies that store or add in L2:
//    589 to 606 us for 128 experts of 256 rows, 1536 x 2048, added (floor 517).
//  * Fixed K order, no split over CTAs: results do not depend on the launch.
//  * Every mbarrier wait is bounded; on expiry the CTA records
//    MINITE_ERR_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "host_util.h"

namespace minite {
namespace gbf16 {

constexpr int BF = 256;                           // features of a tile, 128 for each CTA
constexpr int MAX_N = 256;                        // rows of a tile at most
constexpr int BK = 64;                            // K values per stage (128 bytes)
constexpr int MAX_STAGES = 8;
constexpr int A_BYTES = 128 * 128;                // this CTA's 128 features
constexpr int B_BYTES = (MAX_N / 2) * 128;        // this CTA's half of the rows
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX_BYTES = 64 * 128;               // MN-major box: 64 values x 64 K rows
constexpr int kTokenBoxes = 4;                    // K-major boxes of 16, 32, 64 and 128 tokens
constexpr int NUM_EPI_WARPS = 16;                 // four per TMEM lane quarter, 64 columns each
constexpr int EPI_WARP0 = 2;
constexpr int ODD_WARP = EPI_WARP0 + NUM_EPI_WARPS;   // the second producer
constexpr int NUM_THREADS = (ODD_WARP + 1) * 32;
constexpr int EPI_COLS = MAX_N / (NUM_EPI_WARPS / 4);
constexpr int OUT_ROWS = 16;                      // FP32 weight gradients: rows of a staged box
constexpr int OUT_BOX_BYTES = OUT_ROWS * 512;      // 128 features
constexpr int OUT_BYTES = NUM_EPI_WARPS / 4 * OUT_BOX_BYTES;
constexpr int kChunkBlocks = 4;                   // FP32 outputs: K blocks summed in TMEM at a time
constexpr int kChunkBlocksBf16 = 256;             // BF16 outputs
constexpr size_t kMaxSmem = 232448;

enum Mode { FORWARD = 0, DGRAD = 1, WGRAD = 2 };

struct Smem {
  uint64_t full[MAX_STAGES];        // even CTA: all copies to both CTAs have landed
  uint64_t empty[MAX_STAGES];       // the products of the stage are done
  uint64_t tail_full[MAX_STAGES];   // odd CTA: its copies of a stage with rows to zero
  uint64_t tail_ready[MAX_STAGES];  // even CTA: the odd CTA has zeroed them
  uint64_t acc_full[2];
  uint64_t acc_empty[2];            // even CTA: both CTAs' epilogues
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int total_tiles;
  int pad_;
};

// The first units of a cluster's list as every role of its CTAs needs them,
// looked up by all threads at once: a look-up takes a warp about 1000 cycles,
// and the ring would wait for it at every unit's start.
constexpr int kListed = 64;
struct ListedTile {
  int row0;
  uint16_t rows, f, e, pad;
};

struct Params {
  const int32_t* offsets;
  void* out;
  int64_t ldo;
  int32_t* status;
  int64_t M;       // rows of the activations
  int F;           // features: columns of the output
  int K;           // forward, dgrad: length of the sums; wgrad: output rows of an expert
  int E;
  int units;       // wgrad: length of the list of work
  int max_n;       // rows of a tile at most, a multiple of 32
  int a_two, b_two;  // the maps of two boxes of features (wgrad: of output rows) serve
  int stages;
  int chunk;       // K blocks summed in TMEM before the epilogue takes them
  int accumulate;  // FP32 output: added to what it holds
  uint64_t budget_ns;
};

// Boxes of every size that a stage can need: a stage is two to four copies a CTA.
struct Maps {
  CUtensorMap a1, a2;           // 64 and 128 features
  CUtensorMap b[kTokenBoxes];   // tokens; wgrad: b[0], b[1] are 64 and 128 output rows
  CUtensorMap out;              // wgrad in FP32
};

struct Tile {
  int e, f0;
  int row0;        // forward, dgrad: first token; wgrad: first of the rows summed over
  int i0;          // wgrad: first output row within the expert
  int64_t orow0;   // first output row
  int rows;        // output rows of the tile
  int n;           // rows the matrix instruction covers: `rows` rounded up to 32
  int len;         // length of the sums
};

// The list of work, one tile a unit.
struct Work {
  const int32_t* off;      // [E+1]
  const int32_t* large;    // [E+1] tiles of the larger experts before e
  const int32_t* small;    // [E+1] tiles of the experts of at most max_n rows before e
  const uint16_t* size;    // [E] rows of a larger expert's tiles
  const ListedTile* list;  // [kListed]
  int f_tiles;
};

__device__ __forceinline__ int expert_of(const int32_t* prefix, int E, int u) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// Unit t of the list.
template <int MODE>
__device__ __forceinline__ Tile decode(int t, const Work& w, const Params& p) {
  Tile r;
  const uint32_t f_tiles = w.f_tiles;
  if constexpr (MODE == WGRAD) {
    const int it = t / w.f_tiles, i_tiles = (p.K + p.max_n - 1) / p.max_n;
    r.e = it / i_tiles;
    r.f0 = (t - it * w.f_tiles) * BF;
    r.i0 = (it - r.e * i_tiles) * p.max_n;
    r.row0 = w.off[r.e];
    r.orow0 = static_cast<int64_t>(r.e) * p.K + r.i0;
    r.rows = min(p.max_n, p.K - r.i0);
    r.len = w.off[r.e + 1] - w.off[r.e];
  } else {
    // the larger experts' units spread evenly over the list
    const uint64_t L = static_cast<uint32_t>(w.large[p.E]), all = L + static_cast<uint32_t>(w.small[p.E]);
    const uint64_t tl = static_cast<uint32_t>(t) * L;
    int before;
    uint32_t rest;   // of t L / all: the next one is large if the quotient grows
    if ((tl >> 32) == 0) {
      before = static_cast<int>(static_cast<uint32_t>(tl) / static_cast<uint32_t>(all));
      rest = static_cast<uint32_t>(tl) - static_cast<uint32_t>(before) * static_cast<uint32_t>(all);
    } else {
      before = static_cast<int>(tl / all);
      rest = static_cast<uint32_t>(tl - before * all);
    }
    int at = 0, size = p.max_n;
    if (rest + L >= all) {
      r.e = expert_of(w.large, p.E, before);
      const uint32_t u = before - w.large[r.e], row_tile = u / f_tiles;
      size = w.size[r.e];
      r.f0 = static_cast<int>(u - row_tile * f_tiles) * BF;
      at = static_cast<int>(row_tile) * size;
    } else {
      const int u = t - before;
      r.e = expert_of(w.small, p.E, u);
      r.f0 = (u - w.small[r.e]) * BF;
    }
    r.i0 = 0;
    r.row0 = w.off[r.e] + at;
    r.orow0 = r.row0;
    r.rows = max(0, min(size, w.off[r.e + 1] - r.row0));
    r.len = p.K;
  }
  r.n = max(32, (r.rows + 31) & ~31);
  return r;
}

// Instruction descriptor of kind::f16 without its N: FP32 accumulator (bit 4),
// A and B BF16 (bits 7, 10), MN-major A / B at bits 15 / 16, N >> 3 at bit 17,
// M >> 4 at bit 24.
template <int MODE>
constexpr uint32_t idesc_base() {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((MODE != FORWARD ? 1u : 0u) << 15) |
         ((MODE == WGRAD ? 1u : 0u) << 16) | (static_cast<uint32_t>(BF >> 4) << 24);
}

// Unit t, the i-th of this cluster.
template <int MODE>
__device__ __forceinline__ Tile unit(int t, int i, const Work& w, const Params& p) {
  if (MODE == WGRAD || i >= kListed) return decode<MODE>(t, w, p);
  const ListedTile l = w.list[i];
  Tile r;
  r.e = l.e;
  r.f0 = l.f * BF;
  r.row0 = l.row0;
  r.i0 = 0;
  r.orow0 = l.row0;
  r.rows = l.rows;
  r.n = max(32, (r.rows + 31) & ~31);
  r.len = p.K;
  return r;
}

__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// TMA loads into this CTA, counted on an mbarrier of either CTA of the pair.
template <int D>
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t mbar, int x, int y,
                                              int z = 0, int w = 0) {
  const uint32_t d = smem_u32(dst);
  const uint64_t m = reinterpret_cast<uint64_t>(map);
#define MINITE_TMA(dim, coords)                                                                   \
  asm volatile("cp.async.bulk.tensor." dim ".cta_group::2.shared::cluster.global.tile"             \
               ".mbarrier::complete_tx::bytes [%0], [%1, " coords "], [%2];"                       \
               :: "r"(d), "l"(m), "r"(mbar), "r"(x), "r"(y), "r"(z), "r"(w) : "memory")
  if constexpr (D == 2) MINITE_TMA("2d", "{%3, %4}");
  else if constexpr (D == 3) MINITE_TMA("3d", "{%3, %4, %5}");
  else MINITE_TMA("4d", "{%3, %4, %5, %6}");
#undef MINITE_TMA
}

// Arrival and wait that order shared-memory writes between the two CTAs.
__device__ __forceinline__ void mbar_arrive_remote_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint64_t budget_ns,
                                                  volatile int* abort) {
  const uint64_t start = globaltimer();
  for (;;) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    if (ok) return true;
    if (*abort || globaltimer() - start > budget_ns) return false;
  }
}

// Warp: 16 / 8 consecutive FP32 columns of this warp's 32 TMEM lanes, the 16 to
// r[first ...].
template <int N>
__device__ __forceinline__ void tmem_ld_cols16(uint32_t taddr, float (&r)[N], int first = 0) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[first]), "=f"(r[first + 1]), "=f"(r[first + 2]), "=f"(r[first + 3]), "=f"(r[first + 4]),
        "=f"(r[first + 5]), "=f"(r[first + 6]), "=f"(r[first + 7]), "=f"(r[first + 8]),
        "=f"(r[first + 9]), "=f"(r[first + 10]), "=f"(r[first + 11]), "=f"(r[first + 12]),
        "=f"(r[first + 13]), "=f"(r[first + 14]), "=f"(r[first + 15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_cols8(uint32_t taddr, float (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7])
      : "r"(taddr)
      : "memory");
}

// 16 rows of the lane's feature, v[first ...], `out` at the first, `rows` of them in the
// output. Even lanes take the even rows of both lanes' features and odd lanes
// the odd rows, so that a lane writes four bytes and the warp 64 of each of
// two rows.
template <int N>
__device__ __forceinline__ void store_16rows(uint16_t* out, int64_t ldo, int rows, bool ok,
                                             const float (&v)[N], int first = 0) {
  const int odd = threadIdx.x & 1;
  uint16_t* o = out + (odd ? ldo - 1 : 0);
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float a = v[first + j], b = v[first + j + 1];
    const float other = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
    const uint32_t w = odd ? pack_bf16x2_rn(other, b) : pack_bf16x2_rn(a, other);
    if (ok && j + odd < rows) *reinterpret_cast<uint32_t*>(o) = w;
    o += 2 * ldo;
  }
}
// 64 rows in FP32, a warp 128 bytes of each.
__device__ __forceinline__ void store_64rows(float* out, int64_t ldo, int rows, bool ok,
                                             const float (&v)[64]) {
#pragma unroll
  for (int j = 0; j < 64; ++j) {
    if (ok && j < rows) *out = v[j];
    out += ldo;
  }
}

// A box of OUT_ROWS rows x 128 features in shared memory to (or, with `add`, added
// to) the FP32 output [experts, rows, features]; what lies outside is left out.
// The sum is made in L2, one rounding to nearest an element, so that no SM
// waits for what the output holds.
__device__ __forceinline__ void tma_out_3d(const CUtensorMap* map, const void* src, bool add, int x, int y,
                                           int z) {
  const uint64_t m = reinterpret_cast<uint64_t>(map);
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group"
                 " [%0, {%2, %3, %4}], [%1];"
                 :: "l"(m), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z) : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 :: "l"(m), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z) : "memory");
}

// SPLIT: sums may have several chunks, always so with FP32 outputs. With BF16 ones
// the kernel without costs less where tiles are short (weight gradients of 128
// experts of 256 rows, 1536 x 2048: 187 us, split 197), so the host takes it
// if no sum can be longer than a chunk.
template <int MODE, bool F32, bool SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
grouped_bf16_kernel(const __grid_constant__ Maps maps, const Params p) {
  constexpr bool A_MN = MODE != FORWARD, B_MN = MODE == WGRAD;
  constexpr bool TMA_OUT = MODE == WGRAD && F32;
  // barriers and tables, then (1024-byte aligned) the stages and the staged output
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>(smem_raw);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem_raw + sizeof(Smem));   // [E+1] each
  int32_t* s_large = s_off + (p.E + 1);
  int32_t* s_small = s_large + (p.E + 1);
  ListedTile* s_list = reinterpret_cast<ListedTile*>(s_small + (p.E + 1));
  uint16_t* s_size = reinterpret_cast<uint16_t*>(s_list + (MODE == WGRAD ? 0 : kListed));   // [E]
  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(s_size + p.E) + 1023) & ~uintptr_t(1023));
  uint8_t* out_stage = stages + p.stages * STAGE_BYTES;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(num_clusters_x());
  const Work work = {s_off, s_large, s_small, s_size, s_list, (p.F + BF - 1) / BF};
  constexpr uint16_t kBoth = 0x3;

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.a1);
    tma_prefetch_desc(&maps.a2);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
      mbar_init(&S.tail_full[s], 1);
      mbar_init(&S.tail_ready[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.acc_full[b], 1);
      mbar_init(&S.acc_empty[b], 2 * NUM_EPI_WARPS);
    }
    mbar_init(&S.drain, 1);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(&S.tmem_base, 2 * MAX_N);
  pdl_wait();
  if (warp == 2) {
    int n_large = 0, n_small = 0;
    bool bad = false;
    if (lane == 0) {
      s_large[0] = 0;
      s_small[0] = 0;
    }
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      int large = 0, small = 0;
      if (e < p.E) {
        const int o0 = __ldg(p.offsets + e), o1 = __ldg(p.offsets + e + 1);
        s_off[e + 1] = o1;
        if (e == 0) s_off[0] = o0;
        if (o1 < o0 || (e == 0 && o0 != 0) || (e == p.E - 1 && o1 > p.M)) bad = true;
        const int cnt = o1 - o0;
        if (cnt > p.max_n) {
          // row tiles of about equal size
          const int tiles = (cnt + p.max_n - 1) / p.max_n;
          large = tiles * work.f_tiles;
          s_size[e] = static_cast<uint16_t>(((cnt + tiles - 1) / tiles + 31) & ~31);
        } else if (cnt > 0) small = work.f_tiles;
      }
      int il = large, is = small;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int tl = __shfl_up_sync(0xffffffffu, il, o), ts = __shfl_up_sync(0xffffffffu, is, o);
        if (lane >= o) {
          il += tl;
          is += ts;
        }
      }
      if (e < p.E) {
        s_large[e + 1] = n_large + il;
        s_small[e + 1] = n_small + is;
      }
      n_large += __shfl_sync(0xffffffffu, il, 31);
      n_small += __shfl_sync(0xffffffffu, is, 31);
    }
    // what the launch counted on: the stages start on a 1024-byte boundary within the allocation
    uint32_t have;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(have));
    if (out_stage + (TMA_OUT ? OUT_BYTES : 0) > smem_raw + have) bad = true;
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      S.total_tiles = bad ? 0 : MODE == WGRAD ? p.units : n_large + n_small;
      if (bad && blockIdx.x == 0) set_status(p.status, MINITE_ERR_INVALID_ARG);
    }
  }
  if (MODE != WGRAD) {
    __syncthreads();
    const int t = cid + static_cast<int>(threadIdx.x) * ncl;
    if (threadIdx.x < kListed && t < S.total_tiles) {
      const Tile tl = decode<MODE>(t, work, p);
      s_list[threadIdx.x] = {tl.row0, static_cast<uint16_t>(tl.rows), static_cast<uint16_t>(tl.f0 / BF),
                             static_cast<uint16_t>(tl.e), 0};
    }
  }
  // both CTAs' barriers exist and TMEM is allocated before any cross-CTA traffic
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();

  const uint32_t tmem = S.tmem_base;
  const int total = S.total_tiles;
  volatile int* abort_flag = &S.abort_flag;
  const uint64_t budget = p.budget_ns;
  constexpr uint64_t kDrainBudget = 200000000ull;
  auto fail = [&]() {
    for (int c = 0; c < 2; ++c)
      st_shared_cluster(mapa_shared(smem_u32(&S.abort_flag), c), 1u);
    set_status(p.status, MINITE_ERR_TIMEOUT);
  };
  // the stage whose rows [left, 16 steps) belong to the next expert
  auto zero_tail = [&](int stage, int left, int boxes) {
    const int steps = (left + 15) / 16;
    const int n16 = (16 * steps - left) * 8;   // 16-byte words per box
    uint8_t* base = stages + stage * STAGE_BYTES + left * 128;
    for (int i = lane; i < n16 * boxes; i += 32)
      *reinterpret_cast<uint4*>(base + (i / n16) * BOX_BYTES + (i % n16) * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp == 0 || warp == ODD_WARP) {
    // ------------------------------------------------------------ producers of every other K block
    const int which = warp == 0 ? 0 : 1;
    // The whole warp runs the loop and one elected lane issues, so that a
    // copy's operands are warp-uniform. Even so each copy costs its warp about
    // 180 cycles and a block as much again for its barriers, 520 in all where
    // the tensor cores take 512; so two warps take the blocks in turn.
    const uint32_t leader_full0 = mapa_shared(smem_u32(&S.full[0]), 0);
    uint32_t armed_mask = 0, armed_parity = 0;
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = cid, i = 0; t < total && ok; t += ncl, ++i) {
      const Tile tl = unit<MODE>(t, i, work, p);
      const int kt_n = (tl.len + BK - 1) / BK;
      const int half = tl.n / 2;
      const int f0 = tl.f0 + 128 * static_cast<int>(rank);
      // Half of the tile's rows come in a main box and, if need be, a second one.
      // Boxes hold 2^i 16 rows (wgrad: 64), the main one at least half of them: rows
      // that nobody needs cost traffic from L2.
      int box, box2;   // index of the main box and of the second, -1 if there is none
      if constexpr (B_MN) {
        box = 0;
        box2 = half > 64 ? 0 : -1;
      } else {
        box = 27 - __clz(half);
        box2 = half > 16 << box ? 28 - __clz((half - (16 << box) - 1) | 15) : -1;
      }
      const int main_rows = (B_MN ? 64 : 16) << box;
      const int b0 = (B_MN ? tl.i0 : tl.row0) + half * static_cast<int>(rank);
      const uint32_t bytes =
          A_BYTES + 128 * (main_rows + (box2 >= 0 ? (B_MN ? 64 : 16) << box2 : 0));
      const bool b_two = B_MN && box2 >= 0 && p.b_two && b0 % 64 == 0;
      for (int kt = 0; kt < kt_n; ++kt, turn ^= 1) {
        if (turn != which) {   // the other warp's
          armed_mask &= ~(1u << stage);
          if (++stage == p.stages) { stage = 0; phase ^= 1u; }
          continue;
        }
        // the block before this warp's last one has been consumed by then, so
        // that the barrier cannot be a whole turn of the ring behind
        if (!__all_sync(0xffffffffu, mbar_wait(&S.empty[stage], phase ^ 1u, budget, abort_flag))) {
          ok = false;
          break;
        }
        uint8_t* sA = stages + stage * STAGE_BYTES;
        uint8_t* sB = sA + A_BYTES;
        const int left = tl.len - kt * BK;
        const bool tail = MODE == WGRAD && left < BK && left % 16 != 0;
        const uint32_t bar = rank != 0 && tail ? smem_u32(&S.tail_full[stage]) : leader_full0 + 8u * stage;
        const int k0 = MODE == WGRAD ? tl.row0 + kt * BK : kt * BK;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&S.full[stage], tail ? bytes : 2 * bytes);
          else if (tail) mbar_arrive_expect_tx(&S.tail_full[stage], bytes);
          if constexpr (MODE == FORWARD) {
            tma_load_pair<3>(sA, &maps.a2, bar, k0, f0, tl.e);
          } else if (p.a_two) {
            if constexpr (MODE == DGRAD) tma_load_pair<4>(sA, &maps.a2, bar, 0, k0, f0 / 64, tl.e);
            else tma_load_pair<3>(sA, &maps.a2, bar, 0, k0, f0 / 64);
          } else {   // features that do not come in whole boxes
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if constexpr (MODE == DGRAD)
                tma_load_pair<3>(sA + j * BOX_BYTES, &maps.a1, bar, f0 + 64 * j, k0, tl.e);
              else tma_load_pair<2>(sA + j * BOX_BYTES, &maps.a1, bar, f0 + 64 * j, k0);
            }
          }
          const uint32_t at2 = main_rows * 128;
          if constexpr (B_MN) {
            if (b_two) {
              tma_load_pair<3>(sB, &maps.b[1], bar, 0, k0, b0 / 64);
            } else {
              tma_load_pair<2>(sB, &maps.b[0], bar, b0, k0);
              if (box2 >= 0) tma_load_pair<2>(sB + at2, &maps.b[0], bar, b0 + 64, k0);
            }
          } else {
            tma_load_pair<2>(sB, &maps.b[box], bar, k0, b0);
            if (box2 >= 0) tma_load_pair<2>(sB + at2, &maps.b[box2], bar, k0, b0 + main_rows);
          }
        }
        __syncwarp();
        armed_mask |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && lane == 0) fail();
    // No copy may be in flight when a CTA exits: each stage's last ones are waited
    // for by the warp that issued them. After a wait that ran out the two warps
    // stop at different blocks, and a stage may hold one CTA's copies alone: each
    // producer then gives its own time to land before it comes to the last barrier.
    volatile int no_abort = 0;
    if (rank == 0) {
      for (int s = 0; s < p.stages; ++s)
        if (armed_mask & (1u << s))
          mbar_wait(&S.full[s], (armed_parity >> s) & 1u, kDrainBudget, &no_abort);
    }
    if (*abort_flag) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 100000ull) {}
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    // The whole warp runs the loop (uniform values, barrier waits); one
    // elected lane issues.
    // K-major: rows of 128 bytes, 8-row groups 1024 bytes apart, a K step is 32
    // bytes. MN-major: 64-value boxes BOX_BYTES apart (leading offset), 8-row K
    // groups 1024 bytes apart (stride offset), a K step is 16 rows of 128 bytes.
    const uint64_t adesc0 = smem_desc(smem_u32(stages), A_MN ? BOX_BYTES : 16, 1024, kLayoutSwizzle128B);
    const uint64_t bdesc0 =
        smem_desc(smem_u32(stages + A_BYTES), B_MN ? BOX_BYTES : 16, 1024, kLayoutSwizzle128B);
    constexpr uint64_t a_step = A_MN ? 128 : 2, b_step = B_MN ? 128 : 2;
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0, tail_parity = 0;
    bool ok = true, issued = false;
    for (int t = cid, i = 0; t < total && ok; t += ncl, ++i) {
      const Tile tl = unit<MODE>(t, i, work, p);
      const uint32_t idesc = idesc_base<MODE>() | (static_cast<uint32_t>(tl.n >> 3) << 17);
      int in_chunk = 0;
      for (int left = tl.len; left > 0; left -= BK) {
        bool w_ok = true;
        if (in_chunk == 0) w_ok = mbar_wait(&S.acc_empty[buf], acc_phase ^ 1u, budget, abort_flag);
        w_ok = w_ok && mbar_wait(&S.full[stage], phase, budget, abort_flag);
        if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
        const int ks = left >= BK ? BK / 16 : (left + 15) / 16;
        if (MODE == WGRAD && left < BK && left % 16 != 0) {
          zero_tail(stage, left, 2 + (tl.n / 2 + 63) / 64);
          w_ok = mbar_wait_cluster(&S.tail_ready[stage], (tail_parity >> stage) & 1u, budget, abort_flag);
          tail_parity ^= 1u << stage;
          if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
        }
        tc_fence_after();
        const uint64_t soff = static_cast<uint64_t>(stage * STAGE_BYTES) >> 4;
        const uint32_t acc = tmem + buf * MAX_N;
        const bool last = in_chunk == p.chunk - 1 || left <= BK;
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < BK / 16; ++s)
            if (s < ks)
              mma_bf16_pair(acc, adesc0 + soff + a_step * s, bdesc0 + soff + b_step * s, idesc,
                            (in_chunk | s) != 0);
          tc_commit_pair_mc(&S.empty[stage], kBoth);
          if (last) tc_commit_pair_mc(&S.acc_full[buf], kBoth);
        }
        __syncwarp();
        issued = true;
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        ++in_chunk;
        if (last) {
          in_chunk = 0;
          buf ^= 1;
          if (buf == 0) acc_phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) fail();
    if (issued) {
      // all MMAs complete before TMEM is freed
      if (elect_one()) tc_commit_pair_mc(&S.drain, 0x1);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(&S.drain, 0, kDrainBudget, &no_abort);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ tail rows of the odd CTA
    if constexpr (MODE == WGRAD) {
      const uint32_t leader_ready0 = mapa_shared(smem_u32(&S.tail_ready[0]), 0);
      int stage = 0;
      uint32_t tail_parity = 0;
      bool ok = true;
      for (int t = cid, i = 0; t < total && ok; t += ncl, ++i) {
        const Tile tl = unit<MODE>(t, i, work, p);
        const int kt_n = (tl.len + BK - 1) / BK;
        if (kt_n == 0) continue;
        stage = (stage + kt_n - 1) % p.stages;   // the sum's last stage
        const int left = tl.len - (kt_n - 1) * BK;
        if (left < BK && left % 16 != 0) {
          // over in time for the whole sum: a budget for each 1024 blocks (they take
          // 0.3 ms or more). Where the pipeline stands still another role's wait for
          // one block runs out first and raises the abort flag.
          const uint64_t all = budget < (uint64_t(1) << 40) ? budget * (1 + kt_n / 1024) : budget;
          const bool w_ok = mbar_wait(&S.tail_full[stage], (tail_parity >> stage) & 1u, all, abort_flag);
          if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
          tail_parity ^= 1u << stage;
          zero_tail(stage, left, 2 + (tl.n / 2 + 63) / 64);
          if (lane == 0) mbar_arrive_remote_release(leader_ready0 + 8u * stage);
        }
        stage = (stage + 1) % p.stages;
      }
      if (!ok && lane == 0) fail();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t leader_acc_empty0 = mapa_shared(smem_u32(&S.acc_empty[0]), 0);
    const int quarter = warp & 3;
    const int c0 = ((warp - EPI_WARP0) >> 2) * EPI_COLS;   // this warp's rows of a tile
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = cid, i = 0; t < total && ok; t += ncl, ++i) {
      const Tile tl = unit<MODE>(t, i, work, p);
      const int chunks = ((tl.len + BK - 1) / BK + p.chunk - 1) / p.chunk;
      if (chunks == 0 && p.accumulate) continue;
      const int rows = tl.rows - c0;
      const int f = tl.f0 + 128 * static_cast<int>(rank) + quarter * 32 + lane;
      const bool f_ok = f < p.F;
      const int64_t at = (tl.orow0 + c0) * p.ldo + f;
      if (TMA_OUT && p.accumulate && f - lane < p.F) {
        // what the sums will be added to, to L2 while the products run: the
        // additions there took 613 us instead of 580 when each had to fetch its line
        const float* o = static_cast<const float*>(p.out) + at - lane;
        for (int r = lane; r < EPI_COLS && r < rows; r += 32)
          asm volatile("prefetch.global.L2 [%0];" :: "l"(o + r * p.ldo));
      }
      const uint32_t tb0 = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c0;
      auto wait_acc = [&]() {
        if (!mbar_wait(&S.acc_full[buf], acc_phase, budget, abort_flag)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        return ok;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(&S.acc_empty[buf]);
          else mbar_arrive_remote(leader_acc_empty0 + 8u * buf);
        }
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1u;
      };
      if constexpr (SPLIT) {
        float acc[EPI_COLS];
#pragma unroll
        for (int j = 0; j < EPI_COLS; ++j) acc[j] = 0.0f;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          if (!wait_acc()) break;
          const uint32_t tb = tb0 + buf * MAX_N;
          if (!F32 && c == 0) {   // often the only one (FP32 results of short sums lost 6% by it)
#pragma unroll
            for (int g = 0; g < EPI_COLS; g += 16)
              if (g < rows) tmem_ld_cols16(tb + g, acc, g);
          } else {
#pragma unroll
            for (int g = 0; g < EPI_COLS; g += 8)
              if (g < rows) {
                float r[8];
                tmem_ld_cols8(tb + g, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[g + j] += r[j];
              }
          }
          release();
        }
        // The four warps that meet at a named barrier below, which has no bound, go
        // on or leave together: one alone may have given up. All four come here
        // once a tile, since every wait above is bounded.
        const uint32_t bar_id = 1 + c0 / EPI_COLS;
        if constexpr (TMA_OUT) ok = bar_all_named(bar_id, 128, ok);
        if (!ok) break;
        if constexpr (TMA_OUT) {
          // the four warps of the same rows stage 128 features together: a copy
          // out costs about as much as one in
          uint8_t* box = out_stage + (c0 / EPI_COLS) * OUT_BOX_BYTES;
          const int x = tl.f0 + 128 * static_cast<int>(rank), y = tl.i0 + c0;
          if (x < p.F) {
#pragma unroll
            for (int g = 0; g < EPI_COLS; g += OUT_ROWS)
              if (g < rows) {
                if (quarter == 0 && lane == 0) bulk_wait_group_read0();   // the box before has been read
                bar_sync_named(bar_id, 128);
#pragma unroll
                for (int j = 0; j < OUT_ROWS; ++j)
                  *reinterpret_cast<float*>(box + j * 512 + quarter * 128 + lane * 4) = acc[g + j];
                fence_proxy_async_smem();
                bar_sync_named(bar_id, 128);
                if (quarter == 0 && lane == 0) {
                  tma_out_3d(&maps.out, box, p.accumulate != 0, x, y + g, tl.e);
                  bulk_commit_group();
                }
              }
          }
        } else if constexpr (F32) {
          store_64rows(static_cast<float*>(p.out) + at, p.ldo, rows, f_ok, acc);
        } else {
          uint16_t* out = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
          for (int g = 0; g < EPI_COLS; g += 16)
            if (g < rows) store_16rows(out + g * p.ldo, p.ldo, rows - g, f_ok, acc, g);
        }
      } else {
        // one chunk, or none: an expert without rows
        uint16_t* out = static_cast<uint16_t*>(p.out) + at;
        if (chunks == 0) {
          const float zero[16] = {};
          for (int g = 0; g < EPI_COLS && g < rows; g += 16)
            store_16rows(out + g * p.ldo, p.ldo, rows - g, f_ok, zero);
          continue;
        }
        if (!wait_acc()) break;
        const uint32_t tb = tb0 + buf * MAX_N;
#pragma unroll
        for (int g = 0; g < EPI_COLS; g += 16) {
          float r[16];
          if (g < rows) tmem_ld_cols16(tb + g, r);
          if (g == EPI_COLS - 16) release();
          if (g < rows) store_16rows(out + g * p.ldo, p.ldo, rows - g, f_ok, r);
        }
      }
    }
    if (TMA_OUT && lane == 0) bulk_wait_group0();
    if (!ok && lane == 0) fail();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * MAX_N);
}

namespace {

// BF16 tensor, 128-byte swizzle, zeros outside: dimensions innermost first,
// strides in elements of all but the innermost, a box of 64 x box1 x box2.
bool make_map(CUtensorMap* m, const void* base, int dims, const cuuint64_t (&d)[4],
              const cuuint64_t (&ld)[3], uint32_t box1, uint32_t box2 = 1) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t strides[3] = {ld[0] * 2, ld[1] * 2, ld[2] * 2};
  cuuint32_t box[4] = {64, box1, box2, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, const_cast<void*>(base), d, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows x columns (row stride ld) as 64 x 64 boxes: `one` box, and `two` boxes
// side by side where the columns are whole boxes (else *two_ok is 0).
bool make_column_maps(CUtensorMap* one, CUtensorMap* two, int* two_ok, const void* base, cuuint64_t rows,
                      cuuint64_t cols, cuuint64_t ld) {
  *two_ok = cols % 64 == 0;
  return make_map(one, base, 2, {cols, rows}, {ld}, 64) &&
         (!*two_ok || make_map(two, base, 3, {64, rows, cols / 64}, {ld, 64}, 64, 2));
}

// The FP32 output of a weight gradient, boxes of 128 features x OUT_ROWS rows.
bool make_out_map(CUtensorMap* m, void* out, cuuint64_t E, cuuint64_t rows, cuuint64_t cols) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, E}, strides[2] = {cols * 4, rows * cols * 4};
  const cuuint32_t box[3] = {128, OUT_ROWS, 1}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, out, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool F32, bool SPLIT>
int launch_as(const Maps& maps, Params& p, cudaStream_t s) {
  static std::atomic<uint64_t> devices{0};
  const cudaError_t attr_err = allow_smem(devices, grouped_bf16_kernel<MODE, F32, SPLIT>, kMaxSmem);
  if (attr_err != cudaSuccess) return MINITE_ERR_CUDA;
  p.chunk = F32 ? kChunkBlocks : kChunkBlocksBf16;
  p.budget_ns = wait_budget_ns();
  // barriers, offsets, list and sizes in front of the stages
  const size_t head = (sizeof(Smem) + 3 * (static_cast<size_t>(p.E) + 1) * sizeof(int32_t) +
                       (MODE == WGRAD ? 0 : kListed * sizeof(ListedTile)) + p.E * sizeof(uint16_t) + 1023) /
                      1024 * 1024;
  const size_t rest = head + (MODE == WGRAD && F32 ? OUT_BYTES : 0);
  p.stages = static_cast<int>((kMaxSmem - rest) / STAGE_BYTES);
  if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
  const size_t smem = rest + static_cast<size_t>(p.stages) * STAGE_BYTES;
  int clusters = resident_pairs<10 + 4 * MODE + 2 * F32 + SPLIT>(grouped_bf16_kernel<MODE, F32, SPLIT>, NUM_THREADS, smem);
  if (clusters <= 0) return MINITE_ERR_CUDA;
  const int64_t f_tiles = (p.F + BF - 1) / BF;
  // tiles of n rows (forward and dgrad: if all experts had as many rows)
  auto units = [&](int64_t n) -> int64_t {
    if (MODE == WGRAD) return p.E * ((p.K + n - 1) / n) * f_tiles;
    const int64_t experts = p.E < p.M ? p.E : p.M;
    const int64_t rows = (p.M + experts - 1) / experts;
    return experts * ((rows + n - 1) / n) * f_tiles;
  };
  // tiles of 256 rows, narrower ones where those would leave most pairs idle
  p.max_n = MAX_N;
  while (p.max_n > 64 && units(p.max_n) * 2 <= clusters) p.max_n /= 2;
  // at most (forward and dgrad): every expert's last tile may be nearly empty
  const int64_t most =
      MODE == WGRAD ? units(p.max_n) : (p.M / p.max_n + (p.E < p.M ? p.E : p.M)) * f_tiles;
  if (most >= (int64_t(1) << 30)) return MINITE_ERR_UNSUPPORTED_SHAPE;
  p.units = static_cast<int>(most);
  if (most < clusters) clusters = static_cast<int>(most);
  if (launch_pair_pdl(grouped_bf16_kernel<MODE, F32, SPLIT>, clusters, NUM_THREADS, smem, s, maps, p) !=
      cudaSuccess)
    return MINITE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

template <int MODE>
int launch(const Maps& maps, Params& p, int out_dtype, cudaStream_t s) {
  if (out_dtype == MINITE_OUT_FP32) return launch_as<MODE, true, true>(maps, p, s);
  // the longest sum that there can be
  const int64_t longest = MODE == WGRAD ? p.M : p.K;
  return longest > kChunkBlocksBf16 * BK ? launch_as<MODE, false, true>(maps, p, s)
                                         : launch_as<MODE, false, false>(maps, p, s);
}

constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxRows = int64_t(1) << 30;        // row indexes of padded tiles stay within 32 bits
constexpr int64_t kMaxWeight = int64_t(1) << 38;      // elements of one expert: strides of tensor maps
                                                      // are below 2^40 bytes

}  // namespace
}  // namespace gbf16
}  // namespace minite

using namespace minite;

extern "C" int minite_grouped_gemm_bf16(const void* a, int64_t a_stride, const void* w,
                                        int w_layout, const int32_t* expert_offsets,
                                        int64_t M_total, int64_t N, int64_t K, int32_t E, void* out,
                                        int64_t out_stride, int out_dtype, int32_t* status,
                                        minite_stream_t stream) {
  using namespace gbf16;
  if (out_dtype != MINITE_OUT_BF16 && out_dtype != MINITE_OUT_FP32) return MINITE_ERR_INVALID_ARG;
  if (w_layout != MINITE_W_NK && w_layout != MINITE_W_KN) return MINITE_ERR_INVALID_ARG;
  if (M_total < 0 || M_total >= kMaxRows || N < 8 || N % 8 != 0 || N > kMaxDim ||
      K < 8 || K % 8 != 0 || K > kMaxDim || N * K >= kMaxWeight || E < 1 || E > 1024 || a_stride < K || a_stride % 8 != 0 ||
      out_stride < N || out_stride % 8 != 0 || a_stride > (int64_t(1) << 32) ||
      out_stride > (int64_t(1) << 32))
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (M_total == 0) return MINITE_OK;
  if (!a || !w || !expert_offsets || !out) return MINITE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(expert_offsets, 4) ||
      !aligned(status, 4))
    return MINITE_ERR_INVALID_ARG;
  const bool nk = w_layout == MINITE_W_NK;
  Maps maps = {};
  Params p = {};
  const cuuint64_t un = N, uk = K, ue = E, um = M_total, us = a_stride;
  bool ok = true;
  if (nk) {
    ok = make_map(&maps.a2, w, 3, {uk, un, ue}, {uk, un * uk}, 128);
  } else {
    p.a_two = N % 64 == 0;   // else a box of two could reach past the last row's end
    ok = make_map(&maps.a1, w, 3, {un, uk, ue}, {un, un * uk}, 64) &&
         (!p.a_two || make_map(&maps.a2, w, 4, {64, uk, un / 64, ue}, {un, 64, un * uk}, 64, 2));
  }
  for (int i = 0; i < kTokenBoxes; ++i)
    ok = ok && make_map(&maps.b[i], a, 2, {uk, um}, {us}, 16u << i);
  if (!ok) return MINITE_ERR_CUDA;
  p.offsets = expert_offsets;
  p.out = out;
  p.ldo = out_stride;
  p.status = status;
  p.M = M_total;
  p.F = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.E = E;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return nk ? launch<FORWARD>(maps, p, out_dtype, s) : launch<DGRAD>(maps, p, out_dtype, s);
}

extern "C" int minite_grouped_wgrad_bf16(const void* a, int64_t a_stride, const void* b,
                                         int64_t b_stride, const int32_t* expert_offsets,
                                         int64_t M_total, int64_t Na, int64_t Nb, int32_t E,
                                         void* out, int out_dtype, int accumulate, int32_t* status,
                                         minite_stream_t stream) {
  using namespace gbf16;
  if (out_dtype != MINITE_OUT_BF16 && out_dtype != MINITE_OUT_FP32) return MINITE_ERR_INVALID_ARG;
  if (accumulate && out_dtype != MINITE_OUT_FP32) return MINITE_ERR_INVALID_ARG;
  if (M_total < 0 || M_total >= kMaxRows || Na < 8 || Na % 8 != 0 || Na > kMaxDim ||
      Nb < 8 || Nb % 8 != 0 || Nb > kMaxDim || Na * Nb >= kMaxWeight || E < 1 || E > 1024 || a_stride < Na ||
      a_stride % 8 != 0 || b_stride < Nb || b_stride % 8 != 0 || a_stride > (int64_t(1) << 32) ||
      b_stride > (int64_t(1) << 32))
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (!expert_offsets || !out || (M_total > 0 && (!a || !b))) return MINITE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16) || !aligned(expert_offsets, 4) ||
      !aligned(status, 4))
    return MINITE_ERR_INVALID_ARG;
  Maps maps = {};   // without rows no copy is issued
  Params p = {};
  if (M_total > 0 && (!make_column_maps(&maps.a1, &maps.a2, &p.a_two, b, M_total, Nb, b_stride) ||
                      !make_column_maps(&maps.b[0], &maps.b[1], &p.b_two, a, M_total, Na, a_stride)))
    return MINITE_ERR_CUDA;
  if (out_dtype == MINITE_OUT_FP32 && !make_out_map(&maps.out, out, E, Na, Nb)) return MINITE_ERR_CUDA;
  p.offsets = expert_offsets;
  p.out = out;
  p.ldo = Nb;
  p.status = status;
  p.M = M_total;
  p.F = static_cast<int>(Nb);
  p.K = static_cast<int>(Na);
  p.E = E;
  p.accumulate = accumulate ? 1 : 0;
  return launch<WGRAD>(maps, p, out_dtype, reinterpret_cast<cudaStream_t>(stream));
}
