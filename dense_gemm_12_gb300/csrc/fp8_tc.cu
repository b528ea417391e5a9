// fp8_tc.cu -- products of two fp8 (E4M3) matrices with block scales, dense or
// grouped by expert, on the 5th-generation tensor cores:
//
//     D[i][j] = alpha * sum_b sa[b][i] sb[b][j'] sum_{k in block b} A[i][k] B[j][k]
//               + beta * D[i][j]
//
// A is M x K and B is N x K (both contiguous along k); block b is 128 values
// of k; sb has one scale per row of B (j' = j) or per 128 rows (j' = j / 128).
//
// The scales change along k, so the tensor core cannot sum across blocks: its
// accumulator holds one block's product at a time, and CUDA cores add it,
// scaled, to sums in registers:
//   * warp 0       TMA producer: 128 x 128 of A and 256 x 128 of B per k-block
//                  into a 4-stage ring (one 128-byte swizzle atom of fp8 wide)
//   * warp 1       TMEM and MMAs (M = 128, N = 256, K = 32; four per block),
//                  into two TMEM accumulators of 256 columns in turn
//   * warp 2       the block's scales into a ring of their own (cp.async: any
//                  address), on the operands' barrier
//   * warps 4..11  sums: 32 rows x 128 columns per warp, one row per thread,
//                  128 fp32 sums in registers, updated with packed FMAs
// Registers move from the first warpgroup to the other two (setmaxnreg) to
// hold the sums.
//
// What bounds it.  The sum warps.  A block's MMAs take 512 cycles at the tensor
// core's rate, and a block takes 730 to 750.  By clock readings in the roles'
// loops (which add 100 cycles to a block), the issuer finds its operands there
// and waits 200 to 300 cycles for an accumulator, while the sum warps find every
// block done when they come to it: of their 840 cycles then, 190 go to the
// barrier's answer, 380 to 400 to three TMEM loads and the additions up to the
// accumulator's release, 250 to the last additions and the way round the loop.
// Scales and barriers lie in shared memory, which is busy with operands (48 KB
// written and 48 KB read per block) and answers late.  So the visits are few:
// one barrier for operands and scales, one commit per block that both frees the
// stage and announces the accumulator, no copies of loaded registers.
// A tile's end costs 3400 cycles more (64 KB of bf16 leave in 2850, 128 KB of
// fp32 in 5900), in which the MMAs run two blocks ahead at most.  Measured
// 394-423 us at 8192^3 (2.6-2.8 PFLOP/s, the clock at the power limit), 61 us at
// 4096^3 (2.2; 68 us into fp32).  CTA pairs, which halve the operands' traffic,
// came to the same: it is not the operands that are waited for, and each block's
// accumulator then travels through two CTAs' barriers.  Scales for each row of B
// cost a second product per element and all scales in all threads: 980 cycles to
// the release instead of 400, 1330 a block, 92 us at 4096^3 (98 when the next
// two were tried).  Reading the accumulator with four threads to a row, each
// with a quarter of the scales, took 102 us, and the two halves of the columns
// half a block apart 100 us.
//
// Few tiles: the CTAs of a cluster split a tile's k-blocks and add their sums
// through distributed shared memory, in k order.  Rows of A beyond a group's
// end (or M) only reach rows of the accumulator that nobody reads.
#include <cstddef>

#include "groups.cuh"
#include "ops.cuh"

namespace g12 {
namespace {

constexpr int BM = 128, BN = 256, BK = kFp8Block;
constexpr int STAGES = 4;
constexpr int kStageBytesA = BM * BK;
constexpr int kStageBytes = kStageBytesA + BN * BK;  // 48 KB
constexpr int kRingBytes = STAGES * kStageBytes;
// Slots of the scales' ring.  A block's scales are loaded with its operands
// (one barrier for both), that is once the MMAs of the block STAGES before it
// are done; those followed the release of the accumulator two further back, by
// which time every sum warp had read that block's scales.
constexpr int SSLOTS = STAGES + 2;
constexpr int kScaleFloats = BM + BN;
constexpr int kThreads = 384;
constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kWarpCols = BN / 2;  // columns of one sum warp
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdesc = idesc_e4m3_f32(BM, BN);
// 384 threads launch with 168 registers each; 40 + 2 x 232 = 3 x 168.
constexpr int kFewRegs = 40, kManyRegs = 232;
// k-blocks of B that a CTA of a split tile asks L2 for early.
constexpr int kEarlyBlocks = 4;
// A warp's output staging: 32 rows x 64 bytes.
constexpr int kOutBytes = 32 * 64;

struct Fp8Args {
  int M, N;
  int num_kb;           // k-blocks; 0: D <- beta * D
  int groups;
  const int32_t* offsets;  // nullptr: one group of M rows
  float alpha, beta;
  const float* sa;      // [k-block][row of A]
  int64_t ld_sa;
  const float* sb;      // [group][k-block][row, or row block, of B]
  int64_t ld_sb, stride_sb;
  void* D;
  int64_t ldd;
  int d_type;
  int d_vec;            // rows of D can be written in 16-byte pieces
  int tile_rows;        // rows of A per tile: 16, 32, 64 or 128
  int band;             // row tiles per band of the schedule
  int cluster;          // > 1: CTAs that split one tile's k-blocks
  uint32_t* err;
};

struct __align__(16) Tail {
  float scales[SSLOTS][kScaleFloats];
  uint64_t full[STAGES];
  uint64_t done[STAGES];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  GroupTable groups;
};

constexpr size_t kSmemBytes = 1024 + kRingBytes + kSumWarps * kOutBytes + sizeof(Tail);
static_assert(kSmemBytes <= 227 * 1024, "fp8 kernel shared memory");
static_assert(BM * BN * 4 <= kRingBytes, "a cluster's sums fit in the ring");

// Sums of two columns plus their accumulator values, scaled.  Volatile, and
// taking the values as they were loaded: so nothing of it moves above the
// (volatile) wait for the loads, and no register is copied to tie the loads to
// it -- the copies cost as many instructions as the additions.
__device__ __forceinline__ uint64_t add_pair(uint64_t sum, uint32_t lo, uint32_t hi, uint64_t s) {
  uint64_t r;
  asm volatile(
      "{\n\t.reg .b64 v;\n\t"
      "mov.b64 v, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, v, %3, %4;\n\t}"
      : "=l"(r)
      : "r"(lo), "r"(hi), "l"(s), "l"(sum));
  return r;
}
// The same with a second scale per column.
__device__ __forceinline__ uint64_t add_pair(uint64_t sum, uint32_t lo, uint32_t hi, uint64_t s,
                                             float c0, float c1) {
  uint64_t r;
  asm volatile(
      "{\n\t.reg .b64 v, c;\n\t"
      "mov.b64 v, {%1, %2};\n\t"
      "mov.b64 c, {%5, %6};\n\t"
      "mul.rn.f32x2 v, v, %3;\n\t"
      "fma.rn.f32x2 %0, v, c, %4;\n\t}"
      : "=l"(r)
      : "r"(lo), "r"(hi), "l"(s), "l"(sum), "f"(c0), "f"(c1));
  return r;
}

// Adds C columns of one block's accumulator (r) to the sums.
template <bool ROWS, int C>
__device__ __forceinline__ void add_scaled(uint64_t* acc, const uint32_t (&r)[C], uint64_t s,
                                           uint32_t sb) {
#pragma unroll
  for (int i = 0; i < C / 2; i += 2) {
    if (ROWS) {
      const float4 c = ld_shared_v4(sb + 8 * i);
      acc[i] = add_pair(acc[i], r[2 * i], r[2 * i + 1], s, c.x, c.y);
      acc[i + 1] = add_pair(acc[i + 1], r[2 * i + 2], r[2 * i + 3], s, c.z, c.w);
    } else {
      acc[i] = add_pair(acc[i], r[2 * i], r[2 * i + 1], s);
      acc[i + 1] = add_pair(acc[i + 1], r[2 * i + 2], r[2 * i + 3], s);
    }
  }
}

// D of four consecutive columns from `col` on, given their sums.
__device__ __forceinline__ void store4(const Fp8Args& p, int64_t row, int col, float4 s) {
  const float a = p.num_kb > 0 ? p.alpha : 0.0f;
  float v[4] = {a * s.x, a * s.y, a * s.z, a * s.w};
  const int64_t at = row * p.ldd + col;
  const bool whole = col + 4 <= p.N && p.d_vec;
  if (p.beta != 0.0f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < p.N) v[i] = fmaf(p.beta, load1(p.D, p.d_type, at + i), v[i]);
  }
  if (p.d_type == GEMM_OUT_F32) {
    float* d = static_cast<float*>(p.D) + at;
    if (whole) {
      *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
  } else if (whole) {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.D) + at) =
        make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < p.N) store1(p.D, p.d_type, at + i, v[i]);
}

// write_sums where nothing is clipped and D is only written: 64 bytes of each
// row at a time, addresses advanced by constants.
template <bool BF16>
__device__ __forceinline__ void write_whole(const Fp8Args& p, uint8_t* stage, const uint64_t* acc,
                                            int64_t row_base, int col_base) {
  constexpr int kElem = BF16 ? 2 : 4, kPairs = BF16 ? 16 : 8;
  const int lane = threadIdx.x & 31;
  const int swz = (lane >> 1) & 3;
  uint4* mine = reinterpret_cast<uint4*>(stage + lane * 64);
  const int rl = lane >> 2, pc = lane & 3;
  const float a = p.num_kb > 0 ? p.alpha : 0.0f;
  uint8_t* d = static_cast<uint8_t*>(p.D) + ((row_base + rl) * p.ldd + col_base) * kElem + pc * 16;
  const int64_t step = 8 * p.ldd * kElem;
  const uint4* theirs = reinterpret_cast<const uint4*>(stage + rl * 64) + (pc ^ ((rl >> 1) & 3));
#pragma unroll
  for (int c = 0; c < kWarpCols * kElem / 64; ++c) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < kPairs / 4; ++i) {
        const float2 f = f32x2_parts(acc[c * kPairs + q * (kPairs / 4) + i]);
        if (BF16) {
          w[i] = pack_bf16(a * f.x, a * f.y);
        } else {
          w[2 * i] = __float_as_uint(a * f.x);
          w[2 * i + 1] = __float_as_uint(a * f.y);
        }
      }
      mine[q ^ swz] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    uint4 w[4];  // rows rl, rl + 8, ...: 8 rows on, the swizzle is the same
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = theirs[i * 8 * 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(d + i * step + c * 64) = w[i];
    __syncwarp();
  }
}

// This warp's 32 rows x 128 columns of sums to D.  A thread holds one row, so
// its values are turned around in the warp's 2 KB of shared memory -- 64-byte
// rows whose 16-byte pieces are XOR-swizzled, so that neither side conflicts
// on banks -- and leave with four lanes to a row: 32 columns of bf16 at a
// time, or 16 sums in fp32 where D is fp32 or read as well (beta != 0).
__device__ __forceinline__ void write_sums(const Fp8Args& p, uint8_t* stage, const uint64_t* acc,
                                           int64_t row_base, int rows, int col_base) {
  if (rows == 32 && col_base + kWarpCols <= p.N && p.d_vec && p.beta == 0.0f) {
    if (p.d_type == GEMM_OUT_BF16)
      write_whole<true>(p, stage, acc, row_base, col_base);
    else
      write_whole<false>(p, stage, acc, row_base, col_base);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int swz = (lane >> 1) & 3;
  uint4* mine = reinterpret_cast<uint4*>(stage + lane * 64);
  const int rl = lane >> 2, pc = lane & 3;
  if (p.d_type == GEMM_OUT_BF16 && p.beta == 0.0f) {
    const float a = p.num_kb > 0 ? p.alpha : 0.0f;
#pragma unroll
    for (int c = 0; c < kWarpCols / 32; ++c) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = f32x2_parts(acc[c * 16 + q * 4 + i]);
          w[i] = pack_bf16(a * f.x, a * f.y);
        }
        mine[q ^ swz] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + rl;
        const uint4 w = reinterpret_cast<const uint4*>(stage + r * 64)[pc ^ ((r >> 1) & 3)];
        const int col = col_base + c * 32 + pc * 8;
        if (r >= rows || col >= p.N) continue;
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + (row_base + r) * p.ldd + col;
        if (p.d_vec && col + 8 <= p.N) {
          *reinterpret_cast<uint4*>(d) = w;
        } else {
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j < p.N)
              reinterpret_cast<uint16_t*>(d)[j] = static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)));
        }
      }
      __syncwarp();
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < kWarpCols / 16; ++c) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = f32x2_parts(acc[c * 8 + q * 2]), g = f32x2_parts(acc[c * 8 + q * 2 + 1]);
      mine[q ^ swz] = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(g.x),
                                 __float_as_uint(g.y));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + rl;
      const float4 s = reinterpret_cast<const float4*>(stage + r * 64)[pc ^ ((r >> 1) & 3)];
      const int col = col_base + c * 16 + pc * 4;
      if (r < rows && col < p.N) store4(p, row_base + r, col, s);
    }
    __syncwarp();
  }
}

// ROWS: sb has a scale per row of B (else per 128 rows).  CLUSTER: one tile
// per cluster of p.cluster CTAs, its k-blocks split among them.  Every thread
// of a CTA reaches the cluster barriers, also after a bounded wait ran out.
template <bool ROWS, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_kernel(const __grid_constant__ Fp8Args p, const __grid_constant__ CUtensorMap tmA,
               const __grid_constant__ CUtensorMap tmB) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem<1024>(smem_raw);
  uint8_t* out_stage = smem + kRingBytes;
  Tail* tail = reinterpret_cast<Tail*>(out_stage + kSumWarps * kOutBytes);
  // 32-bit shared addresses of what the loops below touch
  const uint32_t tail_at = smem_u32(tail);
  const uint32_t abort_flag = tail_at + offsetof(Tail, abort_flag);
  const uint32_t full_at = tail_at + offsetof(Tail, full), done_at = tail_at + offsetof(Tail, done);
  const uint32_t tmem_empty_at = tail_at + offsetof(Tail, tmem_empty);
  const uint32_t scales_at = tail_at + offsetof(Tail, scales);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1 + 32);  // the producer, and the scale warp's lanes
      mbar_init(&tail->done[s], 1);
    }
    for (int b = 0; b < 2; ++b) mbar_init(&tail->tmem_empty[b], kSumWarps);
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tail->tmem_base, kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  if (CLUSTER && warp == 0 && lane == 0) {
    // One tile per cluster, so the CTA's part of B is known: its first blocks
    // may come to L2 while the previous kernel ends (nothing is read from
    // them before the wait below).
    const int parts = p.cluster, part = static_cast<int>(cluster_cta_rank());
    const int tn = (static_cast<int>(blockIdx.x) / parts) / ((p.M + p.tile_rows - 1) / p.tile_rows);
    const int kb = part * p.num_kb / parts, end = (part + 1) * p.num_kb / parts;
    for (int i = 0; i < kEarlyBlocks && kb + i < end; ++i)
      tma_prefetch_l2_3d(&tmB, (kb + i) * BK, tn * BN, 0);
  }
  // Everything above reads no global memory and may overlap the previous
  // kernel's last CTAs; every global access below follows its completion.
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  if (warp == 3) build_groups(tail->groups, p.offsets, p.groups, p.M, p.tile_rows);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = tail->tmem_base;
  const GroupTable& groups = tail->groups;
  const int tiles_n = (p.N + BN - 1) / BN;
  const int tiles = groups.tile[p.groups] * tiles_n;
  const int split = CLUSTER ? p.cluster : 1;  // CTAs per tile
  const int part = CLUSTER ? static_cast<int>(cluster_cta_rank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / split;
  const int stride = CLUSTER ? tiles : static_cast<int>(gridDim.x);  // CLUSTER: one tile
  const int kb0 = CLUSTER ? part * p.num_kb / split : 0;  // num_kb <= 2^24, part <= 8
  const int kb1 = CLUSTER ? (part + 1) * p.num_kb / split : p.num_kb;

  if (warp < 4) {
    regs_give_back<kFewRegs>();
    if (warp == 0) {
      // ------------------------------------------------------ TMA producer
      if (lane == 0) {
        uint32_t it = 0;
        int g = 0;
        bool ok = true;
        const uint32_t bytes = static_cast<uint32_t>((p.tile_rows + BN) * BK);
        for (int t = first; t < tiles && ok; t += stride) {
          const GroupTile w = group_tile(groups, t, tiles_n, p.band, p.tile_rows, g);
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const uint32_t s = it % STAGES, round = it / STAGES;
            if (!mbar_wait_at(done_at + 8 * s, (round & 1u) ^ 1u, abort_flag, p.err)) {
              ok = false;
              break;
            }
            uint8_t* sa = smem + s * kStageBytes;
            mbar_arrive_expect_tx(&tail->full[s], bytes);
            tma_load_2d(sa, &tmA, kb * BK, w.row0, &tail->full[s]);
            tma_load_3d(sa + kStageBytesA, &tmB, kb * BK, w.tn * BN, w.group, &tail->full[s]);
          }
        }
        if (!ok) {
          for (uint32_t j = it > STAGES ? it - STAGES : 0u; j < it; ++j)
            mbar_drain_wait(&tail->full[j % STAGES], (j / STAGES) & 1u);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      uint32_t it = 0;
      bool ok = true, issued = false;
      // K-major: 8-row groups 1024 B apart.  A stage, and 32 B for each step of
      // 32 of k, only move the address field: the descriptors are sums.
      const uint64_t da0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t db0 = smem_desc_sw128(smem_u32(smem) + kStageBytesA, 16, 1024);
      for (int t = first; t < tiles && ok; t += stride) {
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const uint32_t s = it % STAGES, b = it & 1u;
          const bool got =
              mbar_wait_at(full_at + 8 * s, (it / STAGES) & 1u, abort_flag, p.err) &&
              mbar_wait_at(tmem_empty_at + 8 * b, ((it >> 1) & 1u) ^ 1u, abort_flag, p.err);
          if (__any_sync(0xffffffffu, !got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t step = static_cast<uint64_t>(s * (kStageBytes >> 4));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              tc_mma_f8(tmem_base + b * BN, da0 + step + kk * 2, db0 + step + kk * 2, kIdesc,
                        kk != 0 ? 1u : 0u);
            tc_commit(&tail->done[s]);
          }
          __syncwarp();
          issued = true;
        }
      }
      if (!ok && issued) {
        if (elect_one()) tc_commit(&tail->drain);
        __syncwarp();
        mbar_drain_wait(&tail->drain, 0);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ scales
      uint32_t it = 0;
      int g = 0;
      bool ok = true;
      const int nb = (p.N + kFp8Block - 1) / kFp8Block;
      for (int t = first; t < tiles && ok; t += stride) {
        const GroupTile w = group_tile(groups, t, tiles_n, p.band, p.tile_rows, g);
        const int col0 = ROWS ? w.tn * BN : w.tn * 2;        // first scale of B,
        const int cols = min(ROWS ? BN : 2, (ROWS ? p.N : nb) - col0);  // and how many
        const float* sa = p.sa + kb0 * p.ld_sa + w.row0;
        const float* sb = p.sb + w.group * p.stride_sb + kb0 * p.ld_sb + col0;
        for (int kb = kb0; kb < kb1; ++kb, ++it, sa += p.ld_sa, sb += p.ld_sb) {
          const uint32_t s = it % STAGES;
          const bool got =
              mbar_wait_at(done_at + 8 * s, ((it / STAGES) & 1u) ^ 1u, abort_flag, p.err);
          if (__any_sync(0xffffffffu, !got)) {
            ok = false;
            break;
          }
          const uint32_t dst = scales_at + it % SSLOTS * (kScaleFloats * 4);
#pragma unroll 1
          for (int i = lane; i < BM; i += 32)
            cp_async_4_at(dst + 4 * i, i < w.rows ? sa + i : p.sa, i < w.rows ? 4u : 0u);
#pragma unroll 1
          for (int i = lane; i < (ROWS ? BN : 2); i += 32)
            cp_async_4_at(dst + 4 * (BM + i), i < cols ? sb + i : p.sb, i < cols ? 4u : 0u);
          cp_async_mbar_arrive_noinc(&tail->full[s]);
        }
      }
      cp_async_wait_all();
    }
    if (CLUSTER) {  // with the sum warps' two barriers
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ---------------------------------------------------------------- sums
    regs_take<kManyRegs>();
    const int quarter = warp & 3;         // TMEM lanes this warp may access
    const int half = (warp - 4) >> 2;     // which 128 columns
    const int row = quarter * 32 + lane;
    uint8_t* stage = out_stage + (warp - 4) * kOutBytes;
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                               static_cast<uint32_t>(half * kWarpCols);
    uint32_t it = 0, slot = 0;  // slot: it % SSLOTS
    int g = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += stride) {
      // where the sums go; kept in the warp's staging area, since the loop below
      // needs the registers
      bool live;
      {
        const GroupTile w = group_tile(groups, t, tiles_n, p.band, p.tile_rows, g);
        const int rows = min(w.rows - quarter * 32, 32), col_base = w.tn * BN + half * kWarpCols;
        live = rows > 0 && col_base < p.N;
        if (!CLUSTER && lane == 0)
          *reinterpret_cast<int4*>(stage) = make_int4(w.row0 + quarter * 32, rows, col_base, 0);
        __syncwarp();
      }
      uint64_t acc[kWarpCols / 2];
#pragma unroll
      for (int i = 0; i < kWarpCols / 2; ++i) acc[i] = 0ull;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t b = it & 1u;
        // Lanes that had to poll may have left the wait apart, and where it runs
        // out with different answers: the vote brings the warp together for the
        // loads below, or out of the loop.
        ok = __all_sync(0xffffffffu, mbar_wait_at(done_at + 8 * (it % STAGES), (it / STAGES) & 1u,
                                                  abort_flag, p.err));
        if (!ok) break;
        const uint32_t sc = scales_at + slot * (kScaleFloats * 4);
        if (++slot == SSLOTS) slot = 0;
        tc_fence_after_sync();
        // Warps without rows or columns of the tile add too: a branch around this
        // costs more (3000 x 5000 x 1999, a scale per row of B: 56 us against 54).
        const uint32_t taddr = lane_base + b * BN;
        // 32 and 16 columns in turn, two loads on their way at a time: 128
        // sums and 48 values fit the registers, and what the accumulator's
        // release waits for is three loads' latency.
        uint32_t ra[32], rb[16];
        tmem_ld_32x32b_x32(taddr, ra);
        tmem_ld_32x32b_x16(taddr + 32, rb);
        // this thread's row's scale, and (ROWS: those of) the columns
        float f1 = ld_shared_f32(sc + 4 * row);
        if (!ROWS) f1 *= ld_shared_f32(sc + 4 * (BM + half));
        const uint32_t sb = sc + 4 * (BM + half * kWarpCols);
        const uint64_t f = f32x2(f1, f1);
        tc_wait_ld();
        add_scaled<ROWS>(acc, ra, f, sb);
        tmem_ld_32x32b_x32(taddr + 48, ra);
        add_scaled<ROWS>(acc + 16, rb, f, sb + 128);
        tmem_ld_32x32b_x16(taddr + 80, rb);
        tc_wait_ld();
        add_scaled<ROWS>(acc + 24, ra, f, sb + 192);
        tmem_ld_32x32b_x32(taddr + 96, ra);
        add_scaled<ROWS>(acc + 40, rb, f, sb + 320);
        tc_wait_ld();
        // The accumulator has been read, and by rows the scales are used up:
        // the MMAs of the block after next may overwrite it while its last
        // columns are added.
        if (ROWS) add_scaled<ROWS>(acc + 48, ra, f, sb + 384);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(tmem_empty_at + 8 * b);
        if (!ROWS) add_scaled<ROWS>(acc + 48, ra, f, sb + 384);
      }
      if (CLUSTER) {
        // This CTA's k-blocks are done, and with them every use of the ring:
        // its sums go there, 1 KB per row, 16-byte pieces swizzled by row.
        if (live) {
          float4* out = reinterpret_cast<float4*>(smem) + row * (BN / 4);
#pragma unroll
          for (int i = 0; i < kWarpCols / 4; ++i) {
            const float2 x = f32x2_parts(acc[2 * i]), y = f32x2_parts(acc[2 * i + 1]);
            out[(half * (kWarpCols / 4) + i) ^ (row & 7)] = make_float4(x.x, x.y, y.x, y.y);
          }
        }
        break;
      }
      const int4 w = ld_shared_i4(smem_u32(stage));
      __syncwarp();
      if (ok && live) write_sums(p, stage, acc, w.x, w.y, w.z);
    }
    if (CLUSTER) {
      __syncwarp();
      cluster_sync();  // every part's sums are in its shared memory
      // after a wait ran out the sums are not complete; the error word says so
      if (first < tiles && !ld_shared_volatile(abort_flag)) {
        g = 0;
        const GroupTile w = group_tile(groups, first, tiles_n, p.band, p.tile_rows, g);
        const int c0 = part * (BN / 4) / split, c1 = (part + 1) * (BN / 4) / split;
        const int width = c1 - c0;
        // 8, 16 or 32 threads to a row's pieces of this CTA; the rows of a thread
        // are a multiple of 8 apart, so their swizzle is the same.
        const int lanes = width <= 8 ? 8 : (width <= 16 ? 16 : 32);
        const int tid = static_cast<int>(threadIdx.x) - 128;
        const int c = c0 + (tid & (lanes - 1)), step = kSumThreads / lanes;
        const int r0 = tid / lanes, col = w.tn * BN + c * 4;
        const uint32_t at = smem_u32(smem) + static_cast<uint32_t>((c ^ (r0 & 7)) * 16);
        if (c < c1 && col < p.N) {
          // (Four rows at a time took longer: 9.9 us against 8.5 for four CTAs'
          // parts of 128 x 4096 x 1024.)
          for (int r = r0; r < w.rows; r += step) {
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int src = 0; src < split; ++src) {
              const float4 v =
                  ld_shared_cluster_v4(mapa_shared(at + r * (BN * 4), static_cast<uint32_t>(src)));
              sum.x += v.x;
              sum.y += v.y;
              sum.z += v.z;
              sum.w += v.w;
            }
            store4(p, w.row0 + r, col, sum);
          }
        }
      }
      __syncwarp();
      cluster_sync();  // no CTA leaves while another may still read its shared memory
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem_base, kTmemCols);
}

// Clusters of S CTAs that can be resident at once on the current device; 0 if
// unknown.
int max_clusters(int S) {
  static std::atomic<int> cache[64][9];
  int dev = 0;
  if (S < 2 || S > 8 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int known = cache[dev][S].load(std::memory_order_relaxed);
  if (known != 0) return known;
  int n = 0;
  if (ops_allow_smem<fp8_kernel<false, true>>(kSmemBytes) == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(S));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, fp8_kernel<false, true>, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  if (n > 0) cache[dev][S].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs that split each tile's k-blocks, when all tiles fit in one round: the
// S whose longest share of k-blocks plus the cost of adding S sums is least.
// In k-block times (0.4 us, 0.75 with a scale per row of B); exchanging and
// adding the sums costs 6 or 4 of them (128 x 4096 x 1024 in four parts 8.5 us
// against 8.0 whole, 512 x 2048 x 2048 10.3 against 11.1; with a scale per row
// 1000^3 10.3 against 13.2).
int choose_split(int64_t tiles, int num_kb, int num_sms, bool by_rows) {
  int best = 1;
  double cost = num_kb;
  for (int s = 2; s <= 8 && s <= num_kb; ++s) {
    if (tiles * s > num_sms || tiles > max_clusters(s)) continue;
    const double c = (num_kb + s - 1) / s + (by_rows ? 4.0 : 6.0);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

struct Operand {
  const void* p;
  int64_t rows, cols, ld;   // of each matrix
  int64_t count, stride;    // matrices
};

// Row pitch in a tensor map.  A single row has none of its own: any will do.
int64_t map_pitch(const Operand& o) { return o.rows == 1 ? (o.cols + 15) / 16 * 16 : o.ld; }

bool tma_describes(const Operand& o) {
  return !ops_misaligned(o.p, 16) && map_pitch(o) % 16 == 0 &&
         (o.count == 1 || o.stride % 16 == 0);
}

// Bytes of the copies that TMA can describe (rows padded to 16 bytes).
__global__ void stage_bytes_kernel(const uint8_t* src, int64_t ld, int64_t stride, uint8_t* dst,
                                   int64_t ld2, int64_t rows, int64_t cols, int64_t count) {
  grid_dependency_wait();
  const int64_t pieces = ld2 / 16;
  const int64_t total = count * rows * pieces;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t line = i / pieces, c = (i - line * pieces) * 16;
    const int64_t m = line / rows, r = line - m * rows;
    const uint8_t* s = src + m * stride + r * ld + c;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c + j < cols) w[j >> 2] |= static_cast<uint32_t>(s[j]) << (8 * (j & 3));
    *reinterpret_cast<uint4*>(dst + line * ld2 + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

cudaError_t stage(Operand& o, uint8_t* dst, int num_sms, cudaStream_t s) {
  const int64_t ld2 = (o.cols + 15) / 16 * 16;
  const int64_t total = o.count * o.rows * (ld2 / 16);
  const int64_t want = (total + 255) / 256, fit = static_cast<int64_t>(num_sms) * 8;
  const uint8_t* src = static_cast<const uint8_t*>(o.p);
  const int64_t ld = o.ld, stride = o.stride, rows = o.rows, cols = o.cols, count = o.count;
  const cudaError_t e = ops_launch<stage_bytes_kernel>(
      dim3(static_cast<unsigned>(want < fit ? want : fit)), 256, 0, 1, s, src, ld, stride, dst, ld2,
      rows, cols, count);
  o.p = dst;
  o.ld = ld2;
  o.stride = o.rows * ld2;
  return e;
}

int64_t staged_bytes(const Operand& o) {
  return (o.count * o.rows * ((o.cols + 15) / 16 * 16) + 255) / 256 * 256;
}

template <bool CLUSTER>
gemm_status_t launch(bool by_rows, int64_t ctas, int cluster, const Fp8Args& a,
                     const CUtensorMap& tmA, const CUtensorMap& tmB, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ctas));
  return abi_from_cuda(
      by_rows ? ops_launch<fp8_kernel<true, CLUSTER>>(grid, kThreads, kSmemBytes, cluster, s, a, tmA, tmB)
              : ops_launch<fp8_kernel<false, CLUSTER>>(grid, kThreads, kSmemBytes, cluster, s, a, tmA,
                                                    tmB));
}

gemm_status_t run(int64_t G, const int32_t* offsets, int64_t M, int64_t N, int64_t K, float alpha,
                  const void* A, int64_t lda, const float* sa, int64_t ld_sa, const void* B,
                  int64_t ldb, int64_t stride_b, const float* sb, int64_t ld_sb, int64_t stride_sb,
                  int b_block, float beta, void* D, int64_t ldd, int d_type, bool grouped,
                  void* stream) {
  const int d_bytes = float_type_bytes(d_type);
  if (M < 0 || N < 0 || K < 0 || M > kOpsMaxTiled || N > kOpsMaxTiled || K > kOpsMaxDim ||
      d_bytes == 0 || (b_block != GEMM_BLOCK_ROWS && b_block != GEMM_BLOCK_TILES))
    return GEMM_ERR_INVALID_VALUE;
  if (G < 0) return GEMM_ERR_INVALID_VALUE;
  if (M == 0 || N == 0 || G == 0) return GEMM_OK;
  const int64_t nsb = b_block == GEMM_BLOCK_TILES ? (N + 127) / 128 : N;
  const bool product = K > 0 && alpha != 0.0f;
  if (D == nullptr || ldd < N || ldd > kOpsMaxDim || ops_misaligned(D, d_bytes))
    return GEMM_ERR_INVALID_VALUE;
  if (grouped && (offsets == nullptr || ops_misaligned(offsets, 4))) return GEMM_ERR_INVALID_VALUE;
  if (product) {
    if (A == nullptr || B == nullptr || sa == nullptr || sb == nullptr || lda < K || ldb < K ||
        ld_sa < M || ld_sb < nsb || lda > kOpsMaxDim || ldb > kOpsMaxDim || ld_sa > kOpsMaxDim ||
        ld_sb > kOpsMaxDim || ops_misaligned(sa, 4) || ops_misaligned(sb, 4))
      return GEMM_ERR_INVALID_VALUE;
    const int64_t kb = (K + kFp8Block - 1) / kFp8Block;
    if (grouped && G > 1 && (stride_b < (N - 1) * ldb + K || stride_sb < (kb - 1) * ld_sb + nsb))
      return GEMM_ERR_INVALID_VALUE;
  }
  if (G > kMaxGroups) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  Fp8Args a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.num_kb = product ? static_cast<int>((K + BK - 1) / BK) : 0;
  a.groups = static_cast<int>(G);
  a.offsets = grouped ? offsets : nullptr;
  a.alpha = alpha;
  a.beta = beta;
  a.sa = sa;
  a.ld_sa = ld_sa;
  a.sb = sb;
  a.ld_sb = ld_sb;
  a.stride_sb = stride_sb;
  a.D = D;
  a.ldd = ldd;
  a.d_type = d_type;
  a.d_vec = !ops_misaligned(D, 16) && (M == 1 || ldd % (16 / d_bytes) == 0);
  a.err = err;
  a.band = 8;
  a.tile_rows = M >= BM ? BM : (M > 32 ? (M > 64 ? BM : 64) : (M > 16 ? 32 : 16));

  std::unique_lock<std::mutex> lock;
  CUtensorMap tmA{}, tmB{};
  if (product) {
    Operand oa{A, M, K, lda, 1, 0}, ob{B, N, K, ldb, G, stride_b};
    const int64_t need_a = tma_describes(oa) ? 0 : staged_bytes(oa);
    const int64_t need_b = tma_describes(ob) ? 0 : staged_bytes(ob);
    if (need_a + need_b > 0) {
      uint8_t* buf = nullptr;
      st = abi_stage(s, need_a + need_b, lock, &buf);
      if (st != GEMM_OK) return st;
      cudaError_t e = need_a > 0 ? stage(oa, buf, sms, s) : cudaSuccess;
      if (e == cudaSuccess && need_b > 0) e = stage(ob, buf + need_a, sms, s);
      if (e != cudaSuccess) return abi_from_cuda(e);
    }
    const int64_t da[2] = {K, M}, ta[1] = {map_pitch(oa)};
    const uint32_t ba[2] = {BK, static_cast<uint32_t>(a.tile_rows)};
    // one matrix: any stride describes it
    const int64_t db[3] = {K, N, G}, tb[2] = {map_pitch(ob),
                                              G > 1 ? ob.stride : map_pitch(ob) * N};
    const uint32_t bb[3] = {BK, BN, 1};
    if (!abi_encode_tiled(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, oa.p, da, ta, ba) ||
        !abi_encode_tiled(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, ob.p, db, tb, bb))
      return GEMM_ERR_LAUNCH;
  }
  const int64_t tiles_n = (N + BN - 1) / BN;
  // at most this many tiles: every group may end in a partial row tile
  const int64_t row_tiles = (M + a.tile_rows - 1) / a.tile_rows + (grouped ? (G < M ? G : M) : 0);
  const int64_t tiles = row_tiles * tiles_n;
  if (tiles + sms > kOpsMaxDim) return GEMM_ERR_UNSUPPORTED;
  const bool by_rows = b_block == GEMM_BLOCK_ROWS;
  a.cluster = grouped ? 1 : choose_split(tiles, a.num_kb, sms, by_rows);
  if (a.cluster > 1) return launch<true>(by_rows, tiles * a.cluster, a.cluster, a, tmA, tmB, s);
  return launch<false>(by_rows, tiles < sms ? tiles : sms, 1, a, tmA, tmB, s);
}

}  // namespace
}  // namespace g12

extern "C" {

gemm_status_t gemm_fp8gemm(int64_t M, int64_t N, int64_t K, float alpha, const void* A, int64_t lda,
                           const float* a_scales, int64_t ld_as, const void* B, int64_t ldb,
                           const float* b_scales, int64_t ld_bs, int b_block, float beta, void* D,
                           int64_t ldd, int d_type, void* stream) {
  return g12::run(1, nullptr, M, N, K, alpha, A, lda, a_scales, ld_as, B, ldb, 0, b_scales, ld_bs, 0,
                  b_block, beta, D, ldd, d_type, false, stream);
}

gemm_status_t gemm_fp8gemm_grouped(int64_t G, const int32_t* offsets, int64_t M, int64_t N,
                                   int64_t K, float alpha, const void* A, int64_t lda,
                                   const float* a_scales, int64_t ld_as, const void* B, int64_t ldb,
                                   int64_t stride_b, const float* b_scales, int64_t ld_bs,
                                   int64_t stride_bs, int b_block, float beta, void* D, int64_t ldd,
                                   int d_type, void* stream) {
  return g12::run(G, offsets, M, N, K, alpha, A, lda, a_scales, ld_as, B, ldb, stride_b, b_scales,
                  ld_bs, stride_bs, b_block, beta, D, ldd, d_type, true, stream);
}

}  // extern "C"
