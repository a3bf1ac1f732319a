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
//  * Two CTAs on the SMs of a cluster work on one 256 (features) x N tile with
//    tcgen05.mma.cta_group::2: each loads 128 features and half the rows, K
//    consumed 64 values (128 bytes) a stage, and holds 128 x N sums in TMEM,
//    twice, so that a tile's epilogue runs under the next one's products.
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
//  * FP32 outputs: the tensor cores' FP32 sums lose about 2^-24 of the running
//    sum at every K = 16 step, always towards zero. Sums longer than
//    kChunkBlocks blocks are therefore split: each chunk is summed in TMEM and
//    the chunks are added in FP32 registers (round to nearest) by the
//    epilogue warps. For BF16 outputs the final rounding hides that loss.
//  * Fixed K order, no split over CTAs: results do not depend on the launch.
//  * Every mbarrier wait is bounded; on expiry the CTA records
//    MINITE_ERR_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

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
constexpr int ROW_BOX = 32;                       // rows of a K-major box of tokens
constexpr int NUM_EPI_WARPS = 16;                 // four per TMEM lane quarter, 64 columns each
constexpr int EPI_WARP0 = 2;
constexpr int NUM_THREADS = (EPI_WARP0 + NUM_EPI_WARPS) * 32;
constexpr int EPI_COLS = MAX_N / (NUM_EPI_WARPS / 4);
constexpr int kChunkBlocks = 4;                   // FP32 outputs: K blocks summed in TMEM at a time
constexpr size_t kMaxSmem = 232448;
constexpr uint16_t kBoth = 0x3;

enum Mode { FORWARD = 0, DGRAD = 1, WGRAD = 2 };

struct Smem {
  uint64_t full[MAX_STAGES];        // even CTA: both CTAs' copies have landed
  uint64_t empty[MAX_STAGES];
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

struct Params {
  const int32_t* offsets;
  void* out;
  int64_t ldo;
  int32_t* status;
  int64_t M;       // rows of the activations
  int F;           // features: columns of the output
  int K;           // forward, dgrad: length of the sums; wgrad: output rows of an expert
  int E;
  int max_n;       // rows of a tile at most, a multiple of 32
  int stages;
  int chunk;       // K blocks summed in TMEM before the epilogue takes them
  int accumulate;  // FP32 output: added to what it holds
  uint64_t budget_ns;
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

template <int MODE>
__device__ __forceinline__ Tile decode(int t, int f_tiles, const int32_t* prefix,
                                       const int32_t* off, const Params& p) {
  Tile r;
  const int bt = t / f_tiles;
  r.f0 = (t - bt * f_tiles) * BF;
  if constexpr (MODE == WGRAD) {
    const int per = (p.K + p.max_n - 1) / p.max_n;
    r.e = bt / per;
    r.i0 = (bt - r.e * per) * p.max_n;
    r.row0 = off[r.e];
    r.orow0 = static_cast<int64_t>(r.e) * p.K + r.i0;
    r.rows = min(p.max_n, p.K - r.i0);
    r.len = off[r.e + 1] - off[r.e];
  } else {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= bt) lo = mid; else hi = mid;
    }
    r.e = lo;
    // an expert's tiles have about the same number of rows
    const int cnt = off[lo + 1] - off[lo], tiles = prefix[lo + 1] - prefix[lo];
    const int size = ((cnt + tiles - 1) / tiles + 31) & ~31;
    const int at = (bt - prefix[lo]) * size;
    r.i0 = 0;
    r.row0 = off[lo] + at;
    r.orow0 = r.row0;
    r.rows = min(size, cnt - at);
    r.len = p.K;
  }
  r.n = (r.rows + 31) & ~31;
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

__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// 3-D TMA load whose completion is counted on an mbarrier of either CTA.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const void* desc, uint32_t mbar_cluster,
                                                 int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(desc)), "r"(mbar_cluster), "r"(x),
         "r"(y), "r"(z)
      : "memory");
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

// Warp: 16 / 8 consecutive FP32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7])
      : "r"(taddr)
      : "memory");
}

// 16 rows of the lane's feature, `out` at the first, `rows` of them in the
// output. Even lanes take the even rows of both lanes' features and odd lanes
// the odd rows, so that a lane writes four bytes and the warp 64 of each of
// two rows.
__device__ __forceinline__ void store_16rows(uint16_t* out, int64_t ldo, int rows, bool ok,
                                             const float (&v)[16]) {
  const int odd = threadIdx.x & 1;
  uint16_t* o = out + (odd ? ldo - 1 : 0);
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
    const uint32_t w = odd ? pack_bf16x2_rn(other, v[j + 1]) : pack_bf16x2_rn(v[j], other);
    if (ok && j + odd < rows) *reinterpret_cast<uint32_t*>(o) = w;
    o += 2 * ldo;
  }
}
// 64 rows in FP32, a warp 128 bytes of each; with `add` to what is there.
__device__ __forceinline__ void store_64rows(float* out, int64_t ldo, int rows, bool ok, bool add,
                                             const float (&v)[64]) {
#pragma unroll
  for (int g = 0; g < 64; g += 8) {
    if (g < rows && ok) {
      if (add) {   // eight loads in flight
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = g + j < rows ? out[j * ldo] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (g + j < rows) out[j * ldo] = v[g + j] + w[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (g + j < rows) out[j * ldo] = v[g + j];
      }
    }
    out += 8 * ldo;
  }
}

template <int MODE, bool F32>
__global__ void __launch_bounds__(NUM_THREADS, 1)
grouped_bf16_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_b, const Params p) {
  constexpr bool A_MN = MODE != FORWARD, B_MN = MODE == WGRAD;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Smem& S = *reinterpret_cast<Smem*>(stages + p.stages * STAGE_BYTES);
  int32_t* s_off = reinterpret_cast<int32_t*>(&S + 1);   // [E+1]
  int32_t* s_prefix = s_off + (p.E + 1);                 // [E+1] row tiles of the experts before
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cid = static_cast<int>(cluster_id_x());
  const int ncl = static_cast<int>(num_clusters_x());
  const int f_tiles = (p.F + BF - 1) / BF;

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_b);
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
    int carry = 0;
    bool bad = false;
    if (lane == 0) s_prefix[0] = 0;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      int cnt = 0;
      if (e < p.E) {
        const int o0 = __ldg(p.offsets + e), o1 = __ldg(p.offsets + e + 1);
        s_off[e + 1] = o1;
        if (e == 0) s_off[0] = o0;
        if (o1 < o0 || (e == 0 && o0 != 0) || (e == p.E - 1 && o1 > p.M)) bad = true;
        cnt = o1 > o0 ? (o1 - o0 + p.max_n - 1) / p.max_n : 0;
      }
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (e < p.E) s_prefix[e + 1] = carry + incl;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    bad = __any_sync(0xffffffffu, bad);
    if (MODE == WGRAD) carry = p.E * ((p.K + p.max_n - 1) / p.max_n);
    if (lane == 0) {
      S.total_tiles = bad ? 0 : carry * f_tiles;
      if (bad && blockIdx.x == 0) set_status(p.status, MINITE_ERR_INVALID_ARG);
    }
  }
  // both CTAs' barriers exist and TMEM is allocated before any cross-CTA traffic
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();

  const uint32_t tmem = S.tmem_base;
  const int total = S.total_tiles;
  volatile int* abort_flag = &S.abort_flag;
  const uint32_t peer_abort = mapa_shared(smem_u32(&S.abort_flag), rank ^ 1u);
  const uint64_t budget = p.budget_ns;
  constexpr uint64_t kDrainBudget = 200000000ull;
  auto fail = [&]() {
    *abort_flag = 1;
    st_shared_cluster(peer_abort, 1u);
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

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t leader_full0 = mapa_shared(smem_u32(&S.full[0]), 0);
      uint32_t armed_mask = 0, armed_parity = 0;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl) {
        const Tile tl = decode<MODE>(t, f_tiles, s_prefix, s_off, p);
        const int kt_n = (tl.len + BK - 1) / BK;
        const int half = tl.n / 2;
        const int f0 = tl.f0 + 128 * static_cast<int>(rank);
        const int b0 = (B_MN ? tl.i0 : tl.row0) + half * static_cast<int>(rank);
        const int b_boxes = B_MN ? (half + 63) / 64 : (half + ROW_BOX - 1) / ROW_BOX;
        const uint32_t bytes = A_BYTES + b_boxes * (B_MN ? BOX_BYTES : ROW_BOX * 128);
        for (int kt = 0; kt < kt_n; ++kt) {
          if (!mbar_wait(&S.empty[stage], phase ^ 1u, budget, abort_flag)) { ok = false; break; }
          uint8_t* sA = stages + stage * STAGE_BYTES;
          uint8_t* sB = sA + A_BYTES;
          const int left = tl.len - kt * BK;
          const bool tail = MODE == WGRAD && left < BK && left % 16 != 0;
          uint32_t bar = leader_full0 + 8u * stage;
          if (rank == 0) {
            mbar_arrive_expect_tx(&S.full[stage], tail ? bytes : 2 * bytes);
          } else if (tail) {
            mbar_arrive_expect_tx(&S.tail_full[stage], bytes);
            bar = smem_u32(&S.tail_full[stage]);
          }
          const int k0 = MODE == WGRAD ? tl.row0 + kt * BK : kt * BK;
          if constexpr (MODE == FORWARD) {
            tma_load_3d_pair(sA, &tmap_a, bar, k0, f0, tl.e);
          } else if constexpr (MODE == DGRAD) {
            tma_load_3d_pair(sA, &tmap_a, bar, f0, k0, tl.e);
            tma_load_3d_pair(sA + BOX_BYTES, &tmap_a, bar, f0 + 64, k0, tl.e);
          } else {
            tma_load_2d_pair(sA, &tmap_a, bar, f0, k0);
            tma_load_2d_pair(sA + BOX_BYTES, &tmap_a, bar, f0 + 64, k0);
          }
          for (int b = 0; b < b_boxes; ++b) {
            if constexpr (B_MN) tma_load_2d_pair(sB + b * BOX_BYTES, &tmap_b, bar, b0 + 64 * b, k0);
            else tma_load_2d_pair(sB + b * ROW_BOX * 128, &tmap_b, bar, k0, b0 + ROW_BOX * b);
          }
          armed_mask |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) fail();
      volatile int no_abort = 0;
      if (rank == 0) {
        // every armed stage's copies must have landed before exit
        for (int s = 0; s < p.stages; ++s)
          if (armed_mask & (1u << s))
            mbar_wait(&S.full[s], (armed_parity >> s) & 1u, kDrainBudget, &no_abort);
      } else if (!ok) {
        // this CTA's copies count on the other CTA's barriers: give any copy
        // still in flight time to land before the CTA can exit
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 100000ull) {}
      }
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
    for (int t = cid; t < total && ok; t += ncl) {
      const Tile tl = decode<MODE>(t, f_tiles, s_prefix, s_off, p);
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
      for (int t = cid; t < total && ok; t += ncl) {
        const Tile tl = decode<MODE>(t, f_tiles, s_prefix, s_off, p);
        const int kt_n = (tl.len + BK - 1) / BK;
        if (kt_n == 0) continue;
        stage = (stage + kt_n - 1) % p.stages;   // the sum's last stage
        const int left = tl.len - (kt_n - 1) * BK;
        if (left < BK && left % 16 != 0) {
          const bool w_ok = mbar_wait(&S.tail_full[stage], (tail_parity >> stage) & 1u, budget, abort_flag);
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
    for (int t = cid; t < total && ok; t += ncl) {
      const Tile tl = decode<MODE>(t, f_tiles, s_prefix, s_off, p);
      const int chunks = ((tl.len + BK - 1) / BK + p.chunk - 1) / p.chunk;
      if (chunks == 0 && p.accumulate) continue;
      const int rows = tl.rows - c0;
      const int f = tl.f0 + 128 * static_cast<int>(rank) + quarter * 32 + lane;
      const bool f_ok = f < p.F;
      const int64_t at = (tl.orow0 + c0) * p.ldo + f;
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
      if constexpr (F32) {
        float acc[EPI_COLS];
#pragma unroll
        for (int j = 0; j < EPI_COLS; ++j) acc[j] = 0.0f;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          if (!wait_acc()) break;
          const uint32_t tb = tb0 + buf * MAX_N;
#pragma unroll
          for (int g = 0; g < EPI_COLS; g += 8)
            if (g < rows) {
              float r[8];
              tmem_ld_cols(tb + g, r);
#pragma unroll
              for (int j = 0; j < 8; ++j) acc[g + j] += r[j];
            }
          release();
        }
        if (!ok) break;
        store_64rows(static_cast<float*>(p.out) + at, p.ldo, rows, f_ok, p.accumulate, acc);
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
          if (g < rows) tmem_ld_cols(tb + g, r);
          if (g == EPI_COLS - 16) release();
          if (g < rows) store_16rows(out + g * p.ldo, p.ldo, rows - g, f_ok, r);
        }
      }
    }
    if (!ok && lane == 0) fail();
  }

  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 2 * MAX_N);
}

namespace {

// BF16 tensor of up to three dimensions (innermost first, strides in elements
// of the outer two), 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* m, const void* base, uint64_t d0, uint64_t d1, uint64_t ld1, uint64_t d2,
              uint64_t ld2, uint32_t box1) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {ld1 * 2, ld2 * 2};
  cuuint32_t box[3] = {64, box1, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d2 ? 3 : 2, const_cast<void*>(base), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool F32>
int launch_as(const CUtensorMap& ta, const CUtensorMap& tb, Params& p, cudaStream_t s) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(grouped_bf16_kernel<MODE, F32>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kMaxSmem));
  });
  if (attr_err != cudaSuccess) return MINITE_ERR_CUDA;
  p.chunk = F32 ? kChunkBlocks : 1 << 30;
  p.budget_ns = wait_budget_ns();
  const size_t rest = 1024 + sizeof(Smem) + 2 * (static_cast<size_t>(p.E) + 1) * sizeof(int32_t);
  p.stages = static_cast<int>((kMaxSmem - rest) / STAGE_BYTES);
  if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
  const size_t smem = rest + static_cast<size_t>(p.stages) * STAGE_BYTES;
  int pairs = resident_pairs<10 + 2 * MODE + F32>(grouped_bf16_kernel<MODE, F32>, NUM_THREADS, smem);
  if (pairs <= 0) return MINITE_ERR_CUDA;
  const int64_t f_tiles = (p.F + BF - 1) / BF;
  // tiles of 256 rows, narrower ones where those would leave most pairs idle
  p.max_n = MAX_N;
  auto row_tiles = [&](int n) {
    return MODE == WGRAD ? p.E * ((static_cast<int64_t>(p.K) + n - 1) / n) : (p.M + n - 1) / n;
  };
  while (p.max_n > 64 && row_tiles(p.max_n) * f_tiles * 2 <= pairs) p.max_n /= 2;
  const int64_t most = (MODE == WGRAD ? row_tiles(p.max_n) : p.M / p.max_n + (p.E < p.M ? p.E : p.M)) * f_tiles;
  if (most > 0x7FFFFFFF) return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (most < pairs) pairs = static_cast<int>(most);
  if (launch_pair_pdl(grouped_bf16_kernel<MODE, F32>, pairs, NUM_THREADS, smem, s, ta, tb, p) != cudaSuccess)
    return MINITE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
}

template <int MODE>
int launch(const CUtensorMap& ta, const CUtensorMap& tb, Params& p, int out_dtype, cudaStream_t s) {
  return out_dtype == MINITE_OUT_FP32 ? launch_as<MODE, true>(ta, tb, p, s)
                                      : launch_as<MODE, false>(ta, tb, p, s);
}

constexpr int64_t kMaxDim = int64_t(1) << 20;

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
  if (M_total < 0 || M_total >= (int64_t(1) << 31) - MAX_N || N < 8 || N % 8 != 0 || N > kMaxDim ||
      K < 8 || K % 8 != 0 || K > kMaxDim || E < 1 || E > 1024 || a_stride < K || a_stride % 8 != 0 ||
      out_stride < N || out_stride % 8 != 0 || a_stride > (int64_t(1) << 32) ||
      out_stride > (int64_t(1) << 32))
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (M_total == 0) return MINITE_OK;
  if (!a || !w || !expert_offsets || !out) return MINITE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(expert_offsets, 4))
    return MINITE_ERR_INVALID_ARG;
  CUtensorMap ta, tb;
  const bool nk = w_layout == MINITE_W_NK;
  if (nk ? !make_map(&ta, w, K, N, K, E, N * K, 128) : !make_map(&ta, w, N, K, N, E, N * K, 64))
    return MINITE_ERR_CUDA;
  if (!make_map(&tb, a, K, M_total, a_stride, 0, 0, ROW_BOX)) return MINITE_ERR_CUDA;
  Params p = {};
  p.offsets = expert_offsets;
  p.out = out;
  p.ldo = out_stride;
  p.status = status;
  p.M = M_total;
  p.F = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.E = E;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return nk ? launch<FORWARD>(ta, tb, p, out_dtype, s) : launch<DGRAD>(ta, tb, p, out_dtype, s);
}

extern "C" int minite_grouped_wgrad_bf16(const void* a, int64_t a_stride, const void* b,
                                         int64_t b_stride, const int32_t* expert_offsets,
                                         int64_t M_total, int64_t Na, int64_t Nb, int32_t E,
                                         void* out, int out_dtype, int accumulate, int32_t* status,
                                         minite_stream_t stream) {
  using namespace gbf16;
  if (out_dtype != MINITE_OUT_BF16 && out_dtype != MINITE_OUT_FP32) return MINITE_ERR_INVALID_ARG;
  if (accumulate && out_dtype != MINITE_OUT_FP32) return MINITE_ERR_INVALID_ARG;
  if (M_total < 0 || M_total >= (int64_t(1) << 31) - MAX_N || Na < 8 || Na % 8 != 0 || Na > kMaxDim ||
      Nb < 8 || Nb % 8 != 0 || Nb > kMaxDim || E < 1 || E > 1024 || a_stride < Na ||
      a_stride % 8 != 0 || b_stride < Nb || b_stride % 8 != 0 || a_stride > (int64_t(1) << 32) ||
      b_stride > (int64_t(1) << 32))
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (!expert_offsets || !out || (M_total > 0 && (!a || !b))) return MINITE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16) || !aligned(expert_offsets, 4))
    return MINITE_ERR_INVALID_ARG;
  CUtensorMap ta = {}, tb = {};   // without rows no copy is issued
  if (M_total > 0 && (!make_map(&ta, b, Nb, M_total, b_stride, 0, 0, 64) ||
                      !make_map(&tb, a, Na, M_total, a_stride, 0, 0, 64)))
    return MINITE_ERR_CUDA;
  Params p = {};
  p.offsets = expert_offsets;
  p.out = out;
  p.ldo = Nb;
  p.status = status;
  p.M = M_total;
  p.F = static_cast<int>(Nb);
  p.K = static_cast<int>(Na);
  p.E = E;
  p.accumulate = accumulate ? 1 : 0;
  return launch<WGRAD>(ta, tb, p, out_dtype, reinterpret_cast<cudaStream_t>(stream));
}
