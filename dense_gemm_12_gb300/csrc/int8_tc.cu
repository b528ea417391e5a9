// int8_tc.cu -- products of two int8 matrices with a scale for each row of both
// (each token and each output channel), on the 5th-generation tensor cores:
//
//     D[i][j] = alpha sa[i] sb[j] sum_k A[i][k] B[j][k] + bias[j] + beta D[i][j]
//
// A is M x K and B is N x K, both contiguous along k.  The sum is exact.
//
// This GPU's tensor cores have no 8-bit integer kind (tcgen05.mma kind::i8 does
// not exist for sm_103a), so the values are widened to fp16 on their way:
// whole numbers up to 2048 are fp16 values, products of two int8 at most 2^14,
// and 1024 of them add up to at most 2^24, below which fp32 holds every whole
// number.  So an accumulator is exact over 1024 of k, and its sums are carried
// on as 32-bit integers.
//
// The operands are swapped, D^T = B A^T: the MMA's rows are B's (the weights,
// from TMEM) and its columns A's (the tokens, from shared memory).  A tile is
// 256 weights by 16 to 128 tokens, so a decoding step's few tokens cost no
// rows of an MMA, and a finished value of one token lies in one register of
// every thread, 32 neighbouring channels to a warp: rows of D leave without
// being turned around.
//   * warp 0       TMA producer: 256 x 128 of B and up to 128 x 128 of A per
//                  k-block, as int8, into a ring
//   * warp 1       TMEM and MMAs (M = 128, K = 16): two halves of the weights
//   * warps 4..19  widening, 128 values of k at a time: a thread takes half of
//                  a weight row into its TMEM lane (tcgen05.st: shared memory
//                  is not written or read again for it) and its share of the
//                  tokens into shared memory; two buffers of each.  Then, every
//                  8 k-blocks, the accumulator's values of 32 weights and half
//                  of the tokens per warp to integer sums in registers, and at
//                  a tile's end to D.
// Registers move from the first warpgroup to the other four for the sums.
//
// Few tiles: the CTAs of a cluster split a tile's k-blocks and add their sums
// through distributed shared memory.  Many tiles: int8_wide.cu, if the stream's
// buffer can hold both operands widened.
//
// Measured: 16 x 12288 x 4096 13.5 us (96 CTAs take 6.1 TB/s of weights -- more
// buffers and half of the MMAs change little -- between a start and an end of
// 5.7 us together), 16 x 38912 x 4096 29.2 (HBM: 6.8 TB/s
// between them), 64 x 12288 x 4096 17.1, 128 x 4096 x 4096 12.9 (tiles of 64),
// 128 x 12288 x 4096 23.6.
#include <cstddef>

#include "int8.cuh"

namespace g12 {
namespace {

constexpr int WN = 256;        // weights per tile, two halves of 128
constexpr int BK = 128;        // of k per block
constexpr int kMaxTokens = 128;
constexpr int kChunk = 8;      // k-blocks that an accumulator sums exactly
constexpr int kMaxStages = 5;
constexpr int kRawW = WN * BK;  // a stage's bytes of weights
constexpr int kPool = 208 * 1024;  // the ring and the widened tokens
constexpr int kThreads = 640;
constexpr int kWorkThreads = 512;
constexpr int kWorkWarps = kWorkThreads / 32;
constexpr uint32_t kTmemCols = 512;
// TMEM columns: sums of the two halves, then two buffers of widened weights
constexpr uint32_t kSumCols = 128, kWideAt = 256, kWideCols = 128, kWideHalf = 64;
// 64 tokens: half of the warps widen a block, the others the next one (64 x
// 12288 x 4096 18.3 us against 19.1, 64 x 20000 x 2048 14.7 against 15.5; with 32
// tokens 14.7 against 14.5, with 128 the MMAs are slower than the warps).
constexpr bool in_turn(int tm) { return tm == 64; }
// 640 threads launch with 96 registers each; 64 + 4 x 104 = 5 x 96.
constexpr int kFewRegs = 64, kManyRegs = 104;
// k-blocks of B that a CTA of a split tile asks L2 for early.
constexpr int kEarlyBlocks = 4;

constexpr int stage_bytes(int tm) { return kRawW + tm * BK; }
constexpr int wide_bytes(int tm) { return tm * BK * 2; }  // one buffer of widened tokens
constexpr int stages(int tm) {
  const int n = (kPool - 2 * wide_bytes(tm)) / stage_bytes(tm);
  return n < kMaxStages ? n : kMaxStages;
}

struct __align__(16) Tail {
  float scales[kWorkWarps][kMaxTokens / 2];  // of the tokens of a warp's sums
  uint64_t full[kMaxStages];   // raw operands are there
  uint64_t empty[kMaxStages];  // ... have been read
  uint64_t wide_full[2];       // widened operands are there
  uint64_t wide_empty[2];      // ... have been used
  uint64_t sum_full;           // an accumulator is finished
  uint64_t sum_empty;          // ... has been read
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int4 order;  // tiles, column tiles, row tiles, tiles to step: for the working
               // warps, which have no registers to keep them in
};

constexpr size_t kSmemBytes = 1024 + kPool + sizeof(Tail);
static_assert(kSmemBytes <= 227 * 1024, "int8 kernel shared memory");
static_assert(stages(16) >= 2 && stages(kMaxTokens) >= 2, "stages");
static_assert(kMaxTokens * WN * 4 <= kPool, "a cluster's sums fit in the ring");

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Tile t of the order: bands of 8 column tiles, row tile by row tile within a
// band (neighbouring CTAs share weights and tokens in L2).
struct Tile {
  int tn, tm;
};
__device__ __forceinline__ Tile tile_of(int t, int tiles_n, int tiles_m) {
  const int per_band = 8 * tiles_m;
  const int b = t / per_band;
  const int wide = min(tiles_n - b * 8, 8);
  const int in = t - b * per_band;
  Tile r;
  r.tm = in / wide;
  r.tn = b * 8 + in - r.tm * wide;
  return r;
}

template <int TM, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
    int8_kernel(const __grid_constant__ Int8Args p, const __grid_constant__ CUtensorMap tmA,
                const __grid_constant__ CUtensorMap tmB) {
  constexpr int STAGES = stages(TM), kStageBytes = stage_bytes(TM), kWideBytes = wide_bytes(TM);
  constexpr uint32_t kIdesc = idesc_f16_f32(128, TM);
  constexpr bool TURN = in_turn(TM);
  constexpr int kBlockWarps = TURN ? kWorkWarps / 2 : kWorkWarps;  // that widen a block
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem<1024>(smem_raw);
  uint8_t* wide = smem + STAGES * kStageBytes;  // multiples of 1024
  Tail* tail = reinterpret_cast<Tail*>(smem + kPool);
  const uint32_t tail_at = smem_u32(tail);
  const uint32_t abort_flag = tail_at + offsetof(Tail, abort_flag);
  const uint32_t full_at = tail_at + offsetof(Tail, full), empty_at = tail_at + offsetof(Tail, empty);
  const uint32_t wide_full_at = tail_at + offsetof(Tail, wide_full);
  const uint32_t wide_empty_at = tail_at + offsetof(Tail, wide_empty);
  const uint32_t sum_full_at = tail_at + offsetof(Tail, sum_full);
  const uint32_t sum_empty_at = tail_at + offsetof(Tail, sum_empty);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], kBlockWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail->wide_full[b], kBlockWarps);
      mbar_init(&tail->wide_empty[b], 1);
    }
    mbar_init(&tail->sum_full, 1);
    mbar_init(&tail->sum_empty, kWorkWarps);
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    const int cols = (p.N + WN - 1) / WN, rows = (p.M + TM - 1) / TM;
    tail->order = make_int4(cols * rows, cols, rows, static_cast<int>(gridDim.x));
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tail->tmem_base, kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  const int tiles_n = (p.N + WN - 1) / WN, tiles_m = (p.M + TM - 1) / TM;
  const int tiles = tiles_n * tiles_m;
  const int split = CLUSTER ? p.cluster : 1;  // CTAs per tile
  const int part = CLUSTER ? static_cast<int>(cluster_cta_rank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / split;
  const int stride = static_cast<int>(gridDim.x);
  const int kb0 = CLUSTER ? part * p.num_kb / split : 0;  // num_kb <= 2^10
  const int kb1 = CLUSTER ? (part + 1) * p.num_kb / split : p.num_kb;
  if (CLUSTER && warp == 0 && lane == 0) {
    // The CTA's part of B may come to L2 while the previous kernel ends
    // (nothing is read from it before the wait below).
    const Tile w = tile_of(first, tiles_n, tiles_m);
    for (int i = 0; i < kEarlyBlocks && kb0 + i < kb1; ++i)
      tma_prefetch_l2_2d(&tmB, (kb0 + i) * BK, w.tn * WN);
  }
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = tail->tmem_base;

  if (warp < 4) {
    regs_give_back<kFewRegs>();
    if (warp == 0) {
      // ------------------------------------------------------ TMA producer
      if (lane == 0) {
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += stride) {
          const Tile w = tile_of(t, tiles_n, tiles_m);
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const uint32_t s = it % STAGES, round = it / STAGES;
            if (!mbar_wait_at(empty_at + 8 * s, (round & 1u) ^ 1u, abort_flag, p.err)) {
              ok = false;
              break;
            }
            uint8_t* to = smem + s * kStageBytes;
            mbar_arrive_expect_tx(&tail->full[s], kStageBytes);
            tma_load_2d(to, &tmB, kb * BK, w.tn * WN, &tail->full[s]);
            tma_load_2d(to + kRawW, &tmA, kb * BK, w.tm * TM, &tail->full[s]);
          }
          if (CLUSTER) break;  // one tile
        }
        if (!ok) {
          for (uint32_t j = it > STAGES ? it - STAGES : 0u; j < it; ++j)
            mbar_drain_wait(&tail->full[j % STAGES], (j / STAGES) & 1u);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      uint32_t it = 0, chunk = 0;
      bool ok = true, issued = false;
      // K-major, 64 of k to a row of 128 bytes: 8-row groups 1024 bytes apart
      const uint64_t db0 = smem_desc_sw128(smem_u32(wide), 16, 1024);
      for (int t = first; t < tiles && ok; t += stride) {
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const uint32_t b = it & 1u;
          const int in_chunk = (kb - kb0) % kChunk;
          bool got = mbar_wait_at(wide_full_at + 8 * b, (it >> 1) & 1u, abort_flag, p.err);
          if (in_chunk == 0)
            got = got && mbar_wait_at(sum_empty_at, (chunk & 1u) ^ 1u, abort_flag, p.err);
          if (__any_sync(0xffffffffu, !got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const bool last = in_chunk == kChunk - 1 || kb + 1 == kb1;
          if (elect_one()) {
            const uint32_t at = tmem_base + kWideAt + b * kWideCols;
            const uint64_t db = db0 + b * (kWideBytes >> 4);
#pragma unroll 1
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                tc_mma_f16_ta(tmem_base + half * kSumCols, at + half * kWideHalf + kk * 8,
                              db + (kk >> 2) * (TM * 128 >> 4) + (kk & 3) * 2, kIdesc,
                              in_chunk != 0 || kk != 0 ? 1u : 0u);
            tc_commit(&tail->wide_empty[b]);
            if (last) tc_commit(&tail->sum_full);
          }
          __syncwarp();
          issued = true;
          if (last) ++chunk;
        }
        if (CLUSTER) break;
      }
      if (!ok && issued) {
        if (elect_one()) tc_commit(&tail->drain);
        __syncwarp();
        mbar_drain_wait(&tail->drain, 0);
      }
      __syncwarp();
    }
    if (CLUSTER) {  // with the working warps' two barriers
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    // -------------------------------------------------- widening and sums
    regs_take<kManyRegs>();
    const int tid = static_cast<int>(threadIdx.x) - 128;
    const int quarter = warp & 3;             // TMEM lanes this warp may access
    const int half = ((warp - 4) >> 2) & 1;   // which 128 weights
    const int side = (warp - 4) >> 3;         // which half of the tokens' sums, and
    const int part_k = TURN ? 0 : side;       // ... of a block's k, or every other block
    const int wrow = half * 128 + quarter * 32 + lane;
    constexpr int kMySums = TM / 2;
    constexpr int kStep = kMySums == 16 || kMySums == 32 ? 16 : 8;  // sums per TMEM load
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t sums_at = tmem_base + lanes + static_cast<uint32_t>(half) * kSumCols + side * kMySums;
    const uint32_t wide_at = tmem_base + lanes + kWideAt + static_cast<uint32_t>(half) * kWideHalf + part_k * 32;
    const uint32_t raw = smem_u32(smem), wide_smem = smem_u32(wide);
    const uint32_t raw_w = raw + static_cast<uint32_t>(wrow) * BK;
    const uint32_t turn = static_cast<uint32_t>((part_k * 4) ^ (wrow & 7)) * 16;
    constexpr int kRounds = TURN ? 4 : 2;  // of 32 of k
    constexpr int kPieces = TM * 8;  // 16-byte pieces of a block's tokens
    constexpr int kBlockThreads = kBlockWarps * 32;
    constexpr int kMine = (kPieces + kBlockThreads - 1) / kBlockThreads;
    const uint32_t token = static_cast<uint32_t>(tid & (TM - 1));
    const int piece0 = (tid & (kBlockThreads - 1)) / TM;
    const uint32_t raw_x = raw + kRawW + token * BK, turn_x = (token & 7) * 16;
    uint32_t it = 0, chunk = 0;
    uint32_t sum[kMySums];

    // Widens k-block `it`; false if a wait ran out.
    auto convert = [&]() -> bool {
      const uint32_t s = it % STAGES, b = it & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait_at(full_at + 8 * s, (it / STAGES) & 1u, abort_flag, p.err)))
        return false;
      const uint32_t from = s * kStageBytes;
      // 16-byte pieces, swizzled by their row: this side's four of the weight
      // row, then the tokens'
      uint4 w[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) w[c] = ld_shared_u4(raw_w + from + (turn ^ (c * 16)));
      if (!__all_sync(0xffffffffu,
                      mbar_wait_at(wide_empty_at + 8 * b, ((it >> 1) & 1u) ^ 1u, abort_flag, p.err)))
        return false;
      tc_fence_after_sync();
#pragma unroll
      for (int h = 0; h < kRounds; ++h) {
        uint32_t r[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 v = w[c];
          widen4(v.x, r[c * 8], r[c * 8 + 1]);
          widen4(v.y, r[c * 8 + 2], r[c * 8 + 3]);
          widen4(v.z, r[c * 8 + 4], r[c * 8 + 5]);
          widen4(v.w, r[c * 8 + 6], r[c * 8 + 7]);
        }
        if (h + 1 < kRounds) {
#pragma unroll
          for (int c = 0; c < 2; ++c) w[c] = ld_shared_u4(raw_w + from + (turn ^ (c * 16 + (h + 1) * 32)));
        }
        tmem_st_32x32b_x16(wide_at + b * kWideCols + h * 16, r);
      }
      // Neighbouring threads take neighbouring tokens and the same piece, so that
      // reads and writes of eight lanes fall in different banks.
      const uint32_t to = wide_smem + b * kWideBytes;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int c = piece0 + i * (kBlockThreads / TM);
        if (kPieces < kBlockThreads && c >= 8) continue;
        const uint4 x = ld_shared_u4(raw_x + from + (static_cast<uint32_t>(c * 16) ^ turn_x));
        uint32_t v[8];
        widen4(x.x, v[0], v[1]);
        widen4(x.y, v[2], v[3]);
        widen4(x.z, v[4], v[5]);
        widen4(x.w, v[6], v[7]);
        // two pieces of the first or the other 64 of k
        const uint32_t at = to + (c >= 4 ? TM * 128 : 0) + token * 128;
        const uint32_t first = static_cast<uint32_t>((c & 3) * 32) ^ turn_x;
        st_shared_u4(at + first, v[0], v[1], v[2], v[3]);
        st_shared_u4(at + (first ^ 16), v[4], v[5], v[6], v[7]);
      }
      tc_wait_st();
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_at(empty_at + 8 * s);
        mbar_arrive_at(wide_full_at + 8 * b);
      }
      ++it;
      return true;
    };
    // Adds the finished accumulator to the sums.
    auto take = [&]() -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait_at(sum_full_at, chunk & 1u, abort_flag, p.err))) return false;
      tc_fence_after_sync();
#pragma unroll
      for (int j = 0; j < kMySums; j += kStep) {
        uint32_t r[kStep];
        if constexpr (kStep == 8)
          tmem_ld_32x32b_x8(sums_at + j, r);
        else
          tmem_ld_32x32b_x16(sums_at + j, r);
        tmem_wait_ld(r);
        if (by_unit(j)) {
#pragma unroll
          for (int i = 0; i < kStep; ++i) sum[j + i] += static_cast<uint32_t>(__float2int_rn(__uint_as_float(r[i])));
        } else {
#pragma unroll
          for (int i = 0; i < kStep; i += 2) add_whole(sum[j + i], sum[j + i + 1], r[i], r[i + 1]);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(sum_empty_at);
      ++chunk;
      return true;
    };

    // This CTA's blocks of a tile.  A warp's first block of a chunk is ready
    // before it takes the last chunk.
    auto sums = [&]() -> bool {
      const uint32_t start = 0u - kWholeOff * static_cast<uint32_t>((kb1 - kb0 + kChunk - 1) / kChunk);
#pragma unroll
      for (int i = 0; i < kMySums; ++i) sum[i] = by_unit(i / kStep * kStep) ? 0u : start;
      int left = (kb1 - kb0 + kChunk - 1) / kChunk;  // chunks to take
      for (int kb = kb0; kb < kb1; ++kb) {
        if (TURN && (it & 1u) != static_cast<uint32_t>(side)) {
          ++it;
          continue;
        }
        if (!convert()) return false;
        if (kb - kb0 >= kChunk && (kb - kb0) % kChunk < (TURN ? 2 : 1)) {
          if (!take()) return false;
          if (TURN) --left;
        }
      }
      if constexpr (TURN) {  // (the last chunk may have had no block for this warp)
        for (; left > 0; --left)
          if (!take()) return false;
        return true;
      }
      return kb1 == kb0 || take();
    };

    const uint32_t my_scales = tail_at + offsetof(Tail, scales) +
                               static_cast<uint32_t>(warp - 4) * sizeof(tail->scales[0]);
    const uint32_t order_at = tail_at + offsetof(Tail, order);
    for (int t = first; !CLUSTER && t < ld_shared_i4(order_at).x; t += ld_shared_i4(order_at).w) {
      if (p.num_kb > 0) {
        const int4 o = ld_shared_i4(order_at);
        fetch_scales<kMySums>(p, my_scales, tile_of(t, o.y, o.z).tm * TM + side * kMySums);
      }
      if (!sums()) break;
      cp_async_wait_all();
      __syncwarp();
      const int4 o = ld_shared_i4(order_at);
      const Tile w = tile_of(t, o.y, o.z);
      write_channel<kMySums>(p, sum, my_scales, w.tn * WN + wrow, w.tm * TM + side * kMySums);
      __syncwarp();  // the scales have been read
    }
    if (CLUSTER) {
      sums();
      // This CTA's k-blocks are done, and with them every use of the ring: its
      // sums go there, a token's 256 values to a row.
      uint32_t* out = reinterpret_cast<uint32_t*>(smem) + side * kMySums * WN + wrow;
#pragma unroll
      for (int j = 0; j < kMySums; ++j) out[j * WN] = sum[j];
      __syncwarp();
      const Tile w = tile_of(first, tiles_n, tiles_m);
      // four channels of every eighth token to a thread
      const int n = w.tn * WN + (tid & 63) * 4, row0 = w.tm * TM;
      const int in = first < tiles ? min(p.N - n, 4) : 0;  // channels
      float cs[4], bias[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = i < in ? p.alpha * p.sb[n + i] : 0.0f;
        bias[i] = i < in && p.bias != nullptr ? p.bias[n + i] : 0.0f;
      }
      cluster_sync();  // every part's sums are in its shared memory
      // after a wait ran out the sums are not complete; the error word says so
      if (in > 0 && !ld_shared_volatile(abort_flag)) {
        const int j1 = min((part + 1) * TM / split, p.M - row0);
        const uint32_t mine = smem_u32(smem) + static_cast<uint32_t>(tid & 63) * 16;
        // Other CTAs' values are on their way for a microsecond: those of two
        // tokens and four parts at once.
        for (int j0 = part * TM / split + (tid >> 6); j0 < j1; j0 += 16) {
          const bool two = j0 + 8 < j1;
          const float sa[2] = {p.sa[row0 + j0], two ? p.sa[row0 + j0 + 8] : 0.0f};
          uint32_t total[2][4] = {};
          for (int src = 0; src < split; src += 4) {
            float4 v[4][2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t from = mapa_shared(mine, static_cast<uint32_t>(min(src + q, split - 1)));
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                v[q][u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (src + q < split && (u == 0 || two))
                  v[q][u] = ld_shared_cluster_v4(from + static_cast<uint32_t>(j0 + 8 * u) * (WN * 4));
              }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                total[u][0] += __float_as_uint(v[q][u].x);
                total[u][1] += __float_as_uint(v[q][u].y);
                total[u][2] += __float_as_uint(v[q][u].z);
                total[u][3] += __float_as_uint(v[q][u].w);
              }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (u == 1 && !two) continue;
            float d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = value(p, total[u][i], cs[i], sa[u], bias[i]);
            const int64_t at = (row0 + j0 + 8 * u) * p.ldd + n;
            if (p.d_pair && in == 4) {
              uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.D) + at);
              to[0] = pack_bf16(d[0], d[1]);
              to[1] = pack_bf16(d[2], d[3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < in) finish(p, at + i, d[i]);
            }
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
  if (ops_allow_smem<int8_kernel<kMaxTokens, true>>(kSmemBytes) == cudaSuccess) {
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
    if (cudaOccupancyMaxActiveClusters(&n, int8_kernel<kMaxTokens, true>, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  if (n > 0) cache[dev][S].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs that split each tile's k-blocks, when all tiles fit in one round: the S
// whose longest share of k-blocks plus the cost of adding S sums is least.
int choose_split(int64_t tiles, int num_kb, int num_sms) {
  int best = 1;
  double cost = num_kb;
  for (int s = 2; s <= 8 && s <= num_kb; ++s) {
    if (tiles * s > num_sms || tiles > max_clusters(s)) continue;
    const double c = (num_kb + s - 1) / s + 4.0;
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

// A call's tiles of tm tokens, the CTAs that share each, and its time in
// microseconds by what was measured: a tile's start and end, its k-blocks, and
// the parts' sums.
struct Plan {
  int tm, split;
  int64_t tiles;
  double us;
};
Plan plan_for(int tm, int64_t M, int64_t N, int num_kb, int num_sms) {
  Plan p;
  p.tm = tm;
  p.tiles = ((N + WN - 1) / WN) * ((M + tm - 1) / tm);
  p.split = choose_split(p.tiles, num_kb, num_sms);
  const int64_t rounds = (p.tiles * p.split + num_sms - 1) / num_sms;
  const int share = (num_kb + p.split - 1) / p.split;
  p.us = static_cast<double>(rounds) * (tm > 64 ? 0.96 * share + 5.5 : 0.65 * share + 4.4) +
         (p.split == 1 ? 0.0 : (tm > 64 ? 4.0 : 2.7));
  return p;
}
// 128 tokens to a tile widen each weight for the most of them; 64, where that
// makes tiles for more CTAs (us, 64 / 128: 128 x 4096 x 4096 12.9 / 16.5, 512 x
// 1024 x 4096 12.9 / 16.5, 256 x 4096 x 1024 9.5 / 12.2, 512 x 4096 x 4096 25.4 /
// 24.0, 768 x 4096 x 4096 48.6 / 35.9).
Plan choose_plan(int64_t M, int64_t N, int num_kb, int num_sms) {
  if (M <= 64) return plan_for(M > 32 ? 64 : (M > 16 ? 32 : 16), M, N, num_kb, num_sms);
  const Plan a = plan_for(64, M, N, num_kb, num_sms), b = plan_for(128, M, N, num_kb, num_sms);
  return a.us < b.us ? a : b;
}

template <int TM>
cudaError_t launch(int64_t tiles, int num_sms, const Int8Args& a, const CUtensorMap& tmA,
                   const CUtensorMap& tmB, cudaStream_t s) {
  if (a.cluster > 1)
    return ops_launch<int8_kernel<TM, true>>(dim3(static_cast<unsigned>(tiles * a.cluster)), kThreads,
                                             kSmemBytes, a.cluster, s, a, tmA, tmB);
  return ops_launch<int8_kernel<TM, false>>(dim3(static_cast<unsigned>(tiles < num_sms ? tiles : num_sms)),
                                            kThreads, kSmemBytes, 1, s, a, tmA, tmB);
}

// Largest K whose sums fit 32 bits: K * 2^14 < 2^31.
constexpr int64_t kMaxK = (int64_t{1} << 17) - 1;

}  // namespace
}  // namespace g12

using namespace g12;

extern "C" gemm_status_t gemm_int8gemm(int64_t M, int64_t N, int64_t K, float alpha, const int8_t* A,
                                       int64_t lda, const float* a_scales, const int8_t* B, int64_t ldb,
                                       const float* b_scales, const float* bias, float beta, void* D,
                                       int64_t ldd, int d_type, void* stream) {
  const int d_bytes = float_type_bytes(d_type);
  if (M < 0 || N < 0 || K < 0 || M > kOpsMaxTiled || N > kOpsMaxTiled || K > kOpsMaxDim || d_bytes == 0)
    return GEMM_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) return GEMM_OK;
  const bool product = K > 0 && alpha != 0.0f;
  if (D == nullptr || ldd < N || ldd > kOpsMaxDim || ops_misaligned(D, d_bytes) ||
      (bias != nullptr && ops_misaligned(bias, 4)))
    return GEMM_ERR_INVALID_VALUE;
  if (product && (A == nullptr || B == nullptr || a_scales == nullptr || b_scales == nullptr || lda < K ||
                  ldb < K || lda > kOpsMaxDim || ldb > kOpsMaxDim || ops_misaligned(a_scales, 4) ||
                  ops_misaligned(b_scales, 4)))
    return GEMM_ERR_INVALID_VALUE;
  if (product && K > kMaxK) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Int8Args a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.num_kb = product ? static_cast<int>((K + BK - 1) / BK) : 0;
  a.alpha = alpha;
  a.beta = beta;
  a.sa = a_scales;
  a.sb = b_scales;
  a.bias = bias;
  a.D = D;
  a.ldd = ldd;
  a.d_type = d_type;
  a.d_pair = d_type == GEMM_OUT_BF16 && beta == 0.0f && !ops_misaligned(D, 4) && (M == 1 || ldd % 2 == 0);
  a.err = err;
  const Plan plan = choose_plan(M, N, a.num_kb, sms);
  if (plan.tiles + sms > kOpsMaxDim) return GEMM_ERR_UNSUPPORTED;
  a.cluster = plan.split;
  std::unique_lock<std::mutex> lock;
  if (product && M > 64 && int8_wide_pays(M, N, K, plan.us)) {
    // without the memory (inside a capture, say) the way below: the same sums
    uint8_t* buf = nullptr;
    st = abi_stage(s, int8_wide_bytes(M, N, K), lock, &buf);
    if (st == GEMM_OK) return int8_wide(a, K, A, lda, B, ldb, buf, sms, s);
    if (st != GEMM_ERR_NO_MEMORY) return st;
    lock = std::unique_lock<std::mutex>();
  }
  CUtensorMap tmA{}, tmB{};
  if (product) {
    ByteOperand oa{A, M, K, lda, 1, 0}, ob{B, N, K, ldb, 1, 0};
    const int64_t need_a = byte_tma_ok(oa) ? 0 : byte_staged(oa);
    const int64_t need_b = byte_tma_ok(ob) ? 0 : byte_staged(ob);
    if (need_a + need_b > 0) {
      uint8_t* buf = nullptr;
      st = abi_stage(s, need_a + need_b, lock, &buf);
      if (st != GEMM_OK) return st;
      cudaError_t e = need_a > 0 ? byte_stage(oa, buf, sms, s) : cudaSuccess;
      if (e == cudaSuccess && need_b > 0) e = byte_stage(ob, buf + need_a, sms, s);
      if (e != cudaSuccess) return abi_from_cuda(e);
    }
    const int64_t da[2] = {K, M}, ta[1] = {byte_pitch(oa)};
    const int64_t db[2] = {K, N}, tb[1] = {byte_pitch(ob)};
    const uint32_t ba[2] = {BK, static_cast<uint32_t>(plan.tm)}, bb[2] = {BK, WN};
    if (!abi_encode_tiled(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, oa.p, da, ta, ba) ||
        !abi_encode_tiled(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, ob.p, db, tb, bb))
      return GEMM_ERR_LAUNCH;
  }
  switch (plan.tm) {
    case 16: return abi_from_cuda(launch<16>(plan.tiles, sms, a, tmA, tmB, s));
    case 32: return abi_from_cuda(launch<32>(plan.tiles, sms, a, tmA, tmB, s));
    case 64: return abi_from_cuda(launch<64>(plan.tiles, sms, a, tmA, tmB, s));
    default: return abi_from_cuda(launch<128>(plan.tiles, sms, a, tmA, tmB, s));
  }
}
