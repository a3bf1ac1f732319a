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
//  * Output tile 128 x 256, K consumed 64 values (128 bytes) per pipeline
//    stage, four tcgen05.mma kind::f16 (K = 16) per stage, two accumulators of
//    256 TMEM columns so that one tile's epilogue runs under the next's MMAs.
//  * Operands come by TMA with the 128-byte swizzle, either K-major (rows of
//    64 K values) or, where memory has the other dimension contiguous (dgrad's
//    weight, both operands of the weight gradient), MN-major: boxes of 64 such
//    values x 64 K rows. No operand is transposed in memory.
//  * Ragged ends: output rows past an expert's last row are computed from the
//    next expert's rows and not stored. A K tail reads zeros (the tensor maps
//    are three-dimensional, so it never reaches into the next expert). The
//    weight gradient's K range ends inside a 64-row box that already holds
//    the next expert's rows: only the K = 16 steps that hold rows are issued,
//    and the rows of the last step past the end are zeroed in shared memory
//    in both operands (a NaN there would survive a product with zero).
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

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 64;                            // K values per stage (128 bytes)
constexpr int MAX_STAGES = 8;
constexpr int A_BYTES = BM * 128;
constexpr int B_BYTES = BN * 128;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX_BYTES = 64 * 128;               // MN-major box: 64 values x 64 K rows
constexpr int NUM_EPI_WARPS = 16;                 // four per TMEM lane quarter, 64 columns each
constexpr int EPI_WARP0 = 2;
constexpr int NUM_THREADS = (EPI_WARP0 + NUM_EPI_WARPS) * 32;
constexpr int EPI_COLS = BN / (NUM_EPI_WARPS / 4);
constexpr int OUT_WARP_BYTES = 2048;              // staging: 32 rows x 64 bytes per epilogue warp
constexpr int OUT_BYTES = NUM_EPI_WARPS * OUT_WARP_BYTES;
constexpr int kChunkBlocks = 4;                   // FP32 outputs: K blocks summed in TMEM at a time
constexpr size_t kMaxSmem = 232448;

enum Mode { FORWARD = 0, DGRAD = 1, WGRAD = 2 };

struct Smem {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
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
  int N;           // output columns
  int K;           // forward, dgrad: length of the sums; wgrad: output rows of an expert
  int E;
  int stages;
  int chunk;       // K blocks summed in TMEM before the epilogue takes them
  int out_fp32;
  int accumulate;
  uint64_t budget_ns;
};

struct Tile {
  int e, n0;
  int row0;        // first activation row (wgrad: first row of the sums)
  int64_t orow0;   // first output row
  int rows;        // output rows of the tile
  int len;         // length of the sums
};

template <int MODE>
__device__ __forceinline__ Tile decode(int t, int n_tiles, const int32_t* prefix,
                                       const int32_t* off, const Params& p) {
  Tile r;
  const int mt = t / n_tiles;
  r.n0 = (t - mt * n_tiles) * BN;
  if constexpr (MODE == WGRAD) {
    const int per = (p.K + BM - 1) / BM;
    r.e = mt / per;
    const int i0 = (mt - r.e * per) * BM;
    r.row0 = off[r.e];
    r.orow0 = static_cast<int64_t>(r.e) * p.K + i0;
    r.rows = min(BM, p.K - i0);
    r.len = off[r.e + 1] - off[r.e];
  } else {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= mt) lo = mid; else hi = mid;
    }
    r.e = lo;
    r.row0 = off[lo] + (mt - prefix[lo]) * BM;
    r.orow0 = r.row0;
    r.rows = min(BM, off[lo + 1] - r.row0);
    r.len = p.K;
  }
  return r;
}

// Instruction descriptor of kind::f16: FP32 accumulator (bit 4), A and B BF16
// (bits 7, 10), MN-major A / B at bits 15 / 16, N >> 3 at bit 17, M >> 4 at 24.
template <int MODE>
constexpr uint32_t make_idesc() {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((MODE == WGRAD ? 1u : 0u) << 15) |
         ((MODE != FORWARD ? 1u : 0u) << 16) | (static_cast<uint32_t>(BN >> 3) << 17) |
         (static_cast<uint32_t>(BM >> 4) << 24);
}

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// Warp: 16 consecutive FP32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, float (&r)[16]) {
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

// One warp's 32 rows x 64 columns (lane L holds row L) to global memory,
// through a staging buffer of 32 rows x 64 bytes so that four lanes write 64
// consecutive bytes of a row. Chunk c of row r sits at chunk c ^ (r >> 1 & 3):
// eight consecutive lanes then touch all 32 banks on both sides. `rows` of the
// warp's rows exist, columns below N are written (N a multiple of 8).
__device__ __forceinline__ void store_tile(const Params& p, uint8_t* stage, int64_t row0, int rows,
                                           int n0, const float (&acc)[EPI_COLS]) {
  const int lane = threadIdx.x & 31;
  const int rd_row = lane >> 2, rd_chunk = lane & 3;
  uint8_t* wr = stage + lane * 64;
  const int swz = (lane >> 1) & 3;
  if (!p.out_fp32) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int o = 32 * g + 8 * c;
        *reinterpret_cast<uint4*>(wr + ((c ^ swz) << 4)) =
            make_uint4(pack_bf16x2_rn(acc[o], acc[o + 1]), pack_bf16x2_rn(acc[o + 2], acc[o + 3]),
                       pack_bf16x2_rn(acc[o + 4], acc[o + 5]), pack_bf16x2_rn(acc[o + 6], acc[o + 7]));
      }
      __syncwarp();
      const int col = n0 + 32 * g + 8 * rd_chunk;
      uint16_t* out = static_cast<uint16_t*>(p.out) + (row0 + rd_row) * p.ldo + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + rd_row;
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 64 + ((rd_chunk ^ ((r >> 1) & 3)) << 4));
        if (r < rows && col < p.N) *reinterpret_cast<uint4*>(out + 8 * i * p.ldo) = v;
      }
    }
  } else {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int o = 16 * g + 4 * c;
        *reinterpret_cast<float4*>(wr + ((c ^ swz) << 4)) =
            make_float4(acc[o], acc[o + 1], acc[o + 2], acc[o + 3]);
      }
      __syncwarp();
      const int col = n0 + 16 * g + 4 * rd_chunk;
      float* out = static_cast<float*>(p.out) + (row0 + rd_row) * p.ldo + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + rd_row;
        float4 v = *reinterpret_cast<const float4*>(stage + r * 64 + ((rd_chunk ^ ((r >> 1) & 3)) << 4));
        if (r < rows && col < p.N) {
          float4* o = reinterpret_cast<float4*>(out + 8 * i * p.ldo);
          if (p.accumulate) {
            const float4 w = *o;
            v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
          }
          *o = v;
        }
      }
    }
  }
}

template <int MODE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
grouped_bf16_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_b, const Params p) {
  constexpr bool A_MN = MODE == WGRAD, B_MN = MODE != FORWARD;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_stage = stages + p.stages * STAGE_BYTES;
  Smem& S = *reinterpret_cast<Smem*>(out_stage + OUT_BYTES);
  int32_t* s_off = reinterpret_cast<int32_t*>(&S + 1);   // [E+1]
  int32_t* s_prefix = s_off + (p.E + 1);                 // [E+1] row tiles of the experts before
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_tiles = (p.N + BN - 1) / BN;

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmap_a);
    tma_prefetch_desc(&tmap_b);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&S.acc_full[b], 1);
      mbar_init(&S.acc_empty[b], NUM_EPI_WARPS);
    }
    mbar_init(&S.drain, 1);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&S.tmem_base, 2 * BN);
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
        cnt = o1 > o0 ? (o1 - o0 + BM - 1) / BM : 0;
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
    if (MODE == WGRAD) carry = p.E * ((p.K + BM - 1) / BM);
    if (lane == 0) {
      S.total_tiles = bad ? 0 : carry * n_tiles;
      if (bad && blockIdx.x == 0) set_status(p.status, MINITE_ERR_INVALID_ARG);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = S.tmem_base;
  const int total = S.total_tiles;
  volatile int* abort_flag = &S.abort_flag;
  const uint64_t budget = p.budget_ns;
  constexpr uint64_t kDrainBudget = 200000000ull;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t armed_mask = 0, armed_parity = 0;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Tile tl = decode<MODE>(t, n_tiles, s_prefix, s_off, p);
        const int kt_n = (tl.len + BK - 1) / BK;
        for (int kt = 0; kt < kt_n; ++kt) {
          if (!mbar_wait(&S.empty[stage], phase ^ 1u, budget, abort_flag)) { ok = false; break; }
          uint8_t* sA = stages + stage * STAGE_BYTES;
          uint8_t* sB = sA + A_BYTES;
          mbar_arrive_expect_tx(&S.full[stage], STAGE_BYTES);
          if constexpr (A_MN) {
            const int i0 = static_cast<int>(tl.orow0 - static_cast<int64_t>(tl.e) * p.K);
#pragma unroll
            for (int b = 0; b < BM / 64; ++b)
              tma_load_2d(sA + b * BOX_BYTES, &tmap_a, &S.full[stage], i0 + 64 * b, tl.row0 + kt * BK);
#pragma unroll
            for (int b = 0; b < BN / 64; ++b)
              tma_load_2d(sB + b * BOX_BYTES, &tmap_b, &S.full[stage], tl.n0 + 64 * b, tl.row0 + kt * BK);
          } else {
            tma_load_2d(sA, &tmap_a, &S.full[stage], kt * BK, tl.row0);
            if constexpr (B_MN) {
#pragma unroll
              for (int b = 0; b < BN / 64; ++b)
                tma_load_3d(sB + b * BOX_BYTES, &tmap_b, &S.full[stage], tl.n0 + 64 * b, kt * BK, tl.e);
            } else {
              tma_load_3d(sB, &tmap_b, &S.full[stage], kt * BK, tl.n0, tl.e);
            }
          }
          armed_mask |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        set_status(p.status, MINITE_ERR_TIMEOUT);
      }
      volatile int no_abort = 0;   // every armed stage's copies must have landed before exit
      for (int s = 0; s < p.stages; ++s)
        if (armed_mask & (1u << s))
          mbar_wait(&S.full[s], (armed_parity >> s) & 1u, kDrainBudget, &no_abort);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop (uniform values, barrier waits); one
    // elected lane issues.
    constexpr uint32_t idesc = make_idesc<MODE>();
    // K-major: rows of 128 bytes, 8-row groups 1024 bytes apart, a K step is 32
    // bytes. MN-major: 64-value boxes BOX_BYTES apart (leading offset), 8-row K
    // groups 1024 bytes apart (stride offset), a K step is 16 rows of 128 bytes.
    const uint64_t adesc0 = smem_desc(smem_u32(stages), A_MN ? BOX_BYTES : 16, 1024, kLayoutSwizzle128B);
    const uint64_t bdesc0 =
        smem_desc(smem_u32(stages + A_BYTES), B_MN ? BOX_BYTES : 16, 1024, kLayoutSwizzle128B);
    constexpr uint64_t a_step = A_MN ? 128 : 2, b_step = B_MN ? 128 : 2;
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued = false;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile tl = decode<MODE>(t, n_tiles, s_prefix, s_off, p);
      const int kt_n = (tl.len + BK - 1) / BK;
      for (int kt = 0; kt < kt_n; ++kt) {
        const int in_chunk = kt % p.chunk;
        bool w_ok = true;
        if (in_chunk == 0) w_ok = mbar_wait(&S.acc_empty[buf], acc_phase ^ 1u, budget, abort_flag);
        w_ok = w_ok && mbar_wait(&S.full[stage], phase, budget, abort_flag);
        if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
        const int left = tl.len - kt * BK;
        const int ks = left >= BK ? BK / 16 : (left + 15) / 16;
        if (MODE == WGRAD && left < 16 * ks) {
          // rows [left, 16 ks) of the stage belong to the next expert
          const int n16 = (16 * ks - left) * 8;   // 16-byte words per box
          uint8_t* base = stages + stage * STAGE_BYTES + left * 128;
          for (int i = lane; i < n16 * (STAGE_BYTES / BOX_BYTES); i += 32)
            *reinterpret_cast<uint4*>(base + (i / n16) * BOX_BYTES + (i % n16) * 16) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        const uint64_t soff = static_cast<uint64_t>(stage * STAGE_BYTES) >> 4;
        const uint32_t acc = tmem + buf * BN;
        const bool last = in_chunk == p.chunk - 1 || kt == kt_n - 1;
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < BK / 16; ++s)
            if (s < ks)
              mma_bf16(acc, adesc0 + soff + a_step * s, bdesc0 + soff + b_step * s, idesc,
                       (in_chunk | s) != 0);
          tc_commit(&S.empty[stage]);
          if (last) tc_commit(&S.acc_full[buf]);
        }
        __syncwarp();
        issued = true;
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        if (last) {
          buf ^= 1;
          if (buf == 0) acc_phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      set_status(p.status, MINITE_ERR_TIMEOUT);
    }
    if (issued) {
      // all MMAs complete before TMEM is freed
      if (elect_one()) {
        tc_commit(&S.drain);
        volatile int no_abort = 0;
        mbar_wait(&S.drain, 0, kDrainBudget, &no_abort);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int cb = (warp - EPI_WARP0) >> 2;
    uint8_t* stage = out_stage + (warp - EPI_WARP0) * OUT_WARP_BYTES;
    int buf = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile tl = decode<MODE>(t, n_tiles, s_prefix, s_off, p);
      const int chunks = ((tl.len + BK - 1) / BK + p.chunk - 1) / p.chunk;
      if (chunks == 0 && p.accumulate) continue;
      float acc[EPI_COLS];
#pragma unroll
      for (int j = 0; j < EPI_COLS; ++j) acc[j] = 0.0f;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        if (!mbar_wait(&S.acc_full[buf], acc_phase, budget, abort_flag)) ok = false;
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tb = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * BN + cb * EPI_COLS;
#pragma unroll
        for (int g = 0; g < EPI_COLS / 16; ++g) {
          float r[16];
          tmem_ld_16cols(tb + 16 * g, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[16 * g + j] += r[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.acc_empty[buf]);
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1u;
      }
      if (!ok) break;
      const int n0 = tl.n0 + cb * EPI_COLS;
      const int rows = tl.rows - quarter * 32;
      if (n0 < p.N && rows > 0) store_tile(p, stage, tl.orow0 + quarter * 32, rows, n0, acc);
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      set_status(p.status, MINITE_ERR_TIMEOUT);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * BN);
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

template <int MODE>
int launch(const CUtensorMap& ta, const CUtensorMap& tb, Params& p, int64_t max_tiles,
           cudaStream_t s) {
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(grouped_bf16_kernel<MODE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kMaxSmem));
  });
  if (attr_err != cudaSuccess) return MINITE_ERR_CUDA;
  const size_t rest = 1024 + OUT_BYTES + sizeof(Smem) + 2 * (static_cast<size_t>(p.E) + 1) * sizeof(int32_t);
  p.stages = static_cast<int>((kMaxSmem - rest) / STAGE_BYTES);
  if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
  if (max_tiles > 0x7FFFFFFF) return MINITE_ERR_UNSUPPORTED_SHAPE;
  int grid = num_sms();
  if (max_tiles < grid) grid = static_cast<int>(max_tiles);
  if (launch_pdl(grouped_bf16_kernel<MODE>, dim3(grid), dim3(NUM_THREADS),
                 rest + static_cast<size_t>(p.stages) * STAGE_BYTES, s, ta, tb, p) != cudaSuccess)
    return MINITE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MINITE_OK : MINITE_ERR_CUDA;
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
  if (M_total < 0 || M_total >= (int64_t(1) << 31) - BM || N < 8 || N % 8 != 0 || N > kMaxDim ||
      K < 8 || K % 8 != 0 || K > kMaxDim || E < 1 || E > 1024 || a_stride < K || a_stride % 8 != 0 ||
      out_stride < N || out_stride % 8 != 0 || a_stride > (int64_t(1) << 32) ||
      out_stride > (int64_t(1) << 32))
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (M_total == 0) return MINITE_OK;
  if (!a || !w || !expert_offsets || !out) return MINITE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(expert_offsets, 4))
    return MINITE_ERR_INVALID_ARG;
  CUtensorMap ta, tb;
  if (!make_map(&ta, a, K, M_total, a_stride, 0, 0, BM)) return MINITE_ERR_CUDA;
  const bool nk = w_layout == MINITE_W_NK;
  if (nk ? !make_map(&tb, w, K, N, K, E, N * K, BN) : !make_map(&tb, w, N, K, N, E, N * K, 64))
    return MINITE_ERR_CUDA;
  Params p = {};
  p.offsets = expert_offsets;
  p.out = out;
  p.ldo = out_stride;
  p.status = status;
  p.M = M_total;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.E = E;
  p.out_fp32 = out_dtype == MINITE_OUT_FP32;
  p.chunk = p.out_fp32 ? kChunkBlocks : 1 << 30;
  p.budget_ns = wait_budget_ns();
  const int64_t tiles = (M_total / BM + (E < M_total ? E : M_total)) * ((N + BN - 1) / BN);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return nk ? launch<FORWARD>(ta, tb, p, tiles, s) : launch<DGRAD>(ta, tb, p, tiles, s);
}

extern "C" int minite_grouped_wgrad_bf16(const void* a, int64_t a_stride, const void* b,
                                         int64_t b_stride, const int32_t* expert_offsets,
                                         int64_t M_total, int64_t Na, int64_t Nb, int32_t E,
                                         void* out, int out_dtype, int accumulate, int32_t* status,
                                         minite_stream_t stream) {
  using namespace gbf16;
  if (out_dtype != MINITE_OUT_BF16 && out_dtype != MINITE_OUT_FP32) return MINITE_ERR_INVALID_ARG;
  if (accumulate && out_dtype != MINITE_OUT_FP32) return MINITE_ERR_INVALID_ARG;
  if (M_total < 0 || M_total >= (int64_t(1) << 31) - BM || Na < 8 || Na % 8 != 0 || Na > kMaxDim ||
      Nb < 8 || Nb % 8 != 0 || Nb > kMaxDim || E < 1 || E > 1024 || a_stride < Na ||
      a_stride % 8 != 0 || b_stride < Nb || b_stride % 8 != 0 || a_stride > (int64_t(1) << 32) ||
      b_stride > (int64_t(1) << 32))
    return MINITE_ERR_UNSUPPORTED_SHAPE;
  if (!expert_offsets || !out || (M_total > 0 && (!a || !b))) return MINITE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16) || !aligned(expert_offsets, 4))
    return MINITE_ERR_INVALID_ARG;
  CUtensorMap ta = {}, tb = {};   // without rows no copy is issued
  if (M_total > 0 && (!make_map(&ta, a, Na, M_total, a_stride, 0, 0, 64) ||
                      !make_map(&tb, b, Nb, M_total, b_stride, 0, 0, 64)))
    return MINITE_ERR_CUDA;
  Params p = {};
  p.offsets = expert_offsets;
  p.out = out;
  p.ldo = Nb;
  p.status = status;
  p.M = M_total;
  p.N = static_cast<int>(Nb);
  p.K = static_cast<int>(Na);
  p.E = E;
  p.out_fp32 = out_dtype == MINITE_OUT_FP32;
  p.accumulate = accumulate ? 1 : 0;
  p.chunk = p.out_fp32 ? kChunkBlocks : 1 << 30;
  p.budget_ns = wait_budget_ns();
  const int64_t tiles = int64_t(E) * ((Na + BM - 1) / BM) * ((Nb + BN - 1) / BN);
  return launch<WGRAD>(ta, tb, p, tiles, reinterpret_cast<cudaStream_t>(stream));
}
