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
// through distributed shared memory.
#include <cstddef>

#include "ops.cuh"

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
// 640 threads launch with 96 registers each; 64 + 4 x 104 = 5 x 96.
constexpr int kFewRegs = 64, kManyRegs = 104;
// k-blocks of B that a CTA of a split tile asks L2 for early.
constexpr int kEarlyBlocks = 4;

// kSplit: the CTAs of a cluster split a tile's k-blocks.  kWide: the tokens come
// in fp16, widened by a kernel of their own; TMA writes them where the MMAs read
// them.
enum Mode : int { kSingle = 0, kSplit = 1, kWide = 2 };

constexpr int wide_bytes(int tm) { return tm * BK * 2; }  // a block's tokens, widened
// Buffers of them: the threads' two, or a ring as deep as the weights'.
constexpr int wide_buffers(int mode) { return mode == kWide ? 3 : 2; }
constexpr int stage_bytes(int tm, int mode) { return kRawW + (mode == kWide ? 0 : tm * BK); }
constexpr int stages(int tm, int mode) {
  const int n = (kPool - wide_buffers(mode) * wide_bytes(tm)) / stage_bytes(tm, mode);
  const int most = mode == kWide ? 3 : kMaxStages;
  return n < most ? n : most;
}

struct Int8Args {
  int M, N;
  int num_kb;          // k-blocks; 0: D <- bias + beta * D
  float alpha, beta;
  const float* sa;
  const float* sb;
  const float* bias;   // or nullptr
  void* D;
  int64_t ldd;
  int d_type;
  int d_pair;          // bf16, beta == 0: two channels can be written at once
  int cluster;         // > 1: CTAs that split one tile's k-blocks
  uint32_t* err;
};

struct __align__(16) Tail {
  float scales[kWorkWarps][kMaxTokens / 2];  // of the tokens of a warp's sums
  uint64_t full[kMaxStages];   // raw operands are there
  uint64_t empty[kMaxStages];  // ... have been read
  uint64_t wide_full[2];       // widened operands are there
  uint64_t wide_empty[2];      // ... have been used
  uint64_t x_full[3];          // kWide: tokens are there
  uint64_t x_empty[3];         // ... have been used
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
static_assert(stages(16, kSingle) >= 2 && stages(kMaxTokens, kSingle) >= 2 && stages(kMaxTokens, kWide) == 3,
              "stages");
static_assert(kMaxTokens * WN * 4 <= kPool, "a cluster's sums fit in the ring");

// Four int8 -> four fp16: with the sign bit turned over, a byte is its value +
// 128, and as the low byte of 0x6400 it is the fp16 number 1024 + that.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Adds two whole numbers of at most 2^24, as fp32, to 32-bit integers, each with
// kWholeOff on top.  Adding kRound leaves f rounded to a multiple of 2^13, which
// its last bits then count; what is left, less than 2^13, is counted by the last
// bits of its sum with 1.5 * 2^23 (the constants are chosen so that the second
// and third sums are exact).  The conversion instruction, 16 a cycle, would take
// as long as two k-blocks' MMAs for a tile's accumulator.
constexpr float kRound = 103079215104.0f;               // 1.5 * 2^36
constexpr float kRoundLeft = 103079215104.0f + 12582912.0f;  // and 1.5 * 2^23
constexpr uint32_t kWholeOff = 0x51c00000u * 8192u + 0x4b400000u;  // their bits, as added below
__device__ __forceinline__ void add_whole(uint32_t& a, uint32_t& b, uint32_t f, uint32_t g) {
  uint32_t t0, t1, u0, u1;
  asm("{\n\t.reg .b64 f, c, d, m, t, u;\n\t"
      "mov.b64 f, {%4, %5};\n\t"
      "mov.b64 c, {%6, %6};\n\t"
      "mov.b64 d, {%7, %7};\n\t"
      "mov.b64 m, {%8, %8};\n\t"
      "add.rn.f32x2 t, f, c;\n\t"
      "fma.rn.f32x2 u, t, m, d;\n\t"
      "add.rn.f32x2 u, u, f;\n\t"
      "mov.b64 {%0, %1}, t;\n\t"
      "mov.b64 {%2, %3}, u;\n\t}"
      : "=r"(t0), "=r"(t1), "=r"(u0), "=r"(u1)
      : "r"(f), "r"(g), "f"(kRound), "f"(kRoundLeft), "f"(-1.0f));
  a += (t0 << 13) + u0;
  b += (t1 << 13) + u1;
}
// Which group of sums goes through the conversion instruction all the same: a
// quarter, as long as the others take on the other units.
__host__ __device__ constexpr bool by_unit(int j) { return j >= 48; }

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

// A value of D without beta's part, given its integer sum.  cs: alpha times the
// channel's scale.
__device__ __forceinline__ float value(const Int8Args& p, uint32_t sum, float cs, float sa, float bias) {
  return p.num_kb > 0 ? fmaf(static_cast<float>(static_cast<int>(sum)) * sa, cs, bias) : bias;
}
__device__ __forceinline__ void finish(const Int8Args& p, int64_t at, float v) {
  if (p.beta != 0.0f) v = fmaf(p.beta, load1(p.D, p.d_type, at), v);
  store1(p.D, p.d_type, at, v);
}

template <int TM, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    int8_kernel(const __grid_constant__ Int8Args p, const __grid_constant__ CUtensorMap tmA,
                const __grid_constant__ CUtensorMap tmB) {
  constexpr bool CLUSTER = MODE == kSplit, WIDE = MODE == kWide;
  constexpr int STAGES = stages(TM, MODE), kStageBytes = stage_bytes(TM, MODE), kWideBytes = wide_bytes(TM);
  constexpr int kXBuffers = wide_buffers(MODE);
  constexpr uint32_t kIdesc = idesc_f16_f32(128, TM);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem<1024>(smem_raw);
  uint8_t* wide = smem + STAGES * kStageBytes;  // multiples of 1024
  Tail* tail = reinterpret_cast<Tail*>(smem + kPool);
  const uint32_t tail_at = smem_u32(tail);
  const uint32_t abort_flag = tail_at + offsetof(Tail, abort_flag);
  const uint32_t full_at = tail_at + offsetof(Tail, full), empty_at = tail_at + offsetof(Tail, empty);
  const uint32_t wide_full_at = tail_at + offsetof(Tail, wide_full);
  const uint32_t wide_empty_at = tail_at + offsetof(Tail, wide_empty);
  const uint32_t x_full_at = tail_at + offsetof(Tail, x_full), x_empty_at = tail_at + offsetof(Tail, x_empty);
  const uint32_t sum_full_at = tail_at + offsetof(Tail, sum_full);
  const uint32_t sum_empty_at = tail_at + offsetof(Tail, sum_empty);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], kWorkWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail->wide_full[b], kWorkWarps);
      mbar_init(&tail->wide_empty[b], 1);
    }
    for (int b = 0; WIDE && b < kXBuffers; ++b) {
      mbar_init(&tail->x_full[b], 1);
      mbar_init(&tail->x_empty[b], 1);
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
            if (!WIDE) {
              tma_load_2d(to + kRawW, &tmA, kb * BK, w.tm * TM, &tail->full[s]);
              continue;
            }
            const uint32_t x = it % kXBuffers;
            if (!mbar_wait_at(x_empty_at + 8 * x, ((it / kXBuffers) & 1u) ^ 1u, abort_flag, p.err)) {
              ok = false;
              ++it;  // the weights are on their way
              break;
            }
            mbar_arrive_expect_tx(&tail->x_full[x], kWideBytes);
#pragma unroll
            for (int half = 0; half < 2; ++half)
              tma_load_2d(wide + x * kWideBytes + half * (TM * 128), &tmA, kb * BK + half * 64, w.tm * TM,
                          &tail->x_full[x]);
          }
          if (CLUSTER) break;  // one tile
        }
        if (!ok) {
          for (uint32_t j = it > STAGES ? it - STAGES : 0u; j < it; ++j)
            mbar_drain_wait(&tail->full[j % STAGES], (j / STAGES) & 1u);
          // (of the last block perhaps only the weights: that wait runs out)
          for (uint32_t j = it > kXBuffers ? it - kXBuffers : 0u; WIDE && j < it; ++j)
            mbar_drain_wait(&tail->x_full[j % kXBuffers], (j / kXBuffers) & 1u);
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
          const uint32_t x = WIDE ? it % kXBuffers : b;  // buffer of tokens
          if (WIDE) got = got && mbar_wait_at(x_full_at + 8 * x, (it / kXBuffers) & 1u, abort_flag, p.err);
          if (__any_sync(0xffffffffu, !got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const bool last = in_chunk == kChunk - 1 || kb + 1 == kb1;
          if (elect_one()) {
            const uint32_t at = tmem_base + kWideAt + b * kWideCols;
            const uint64_t db = db0 + x * (kWideBytes >> 4);
#pragma unroll 1
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                tc_mma_f16_ta(tmem_base + half * kSumCols, at + half * kWideHalf + kk * 8,
                              db + (kk >> 2) * (TM * 128 >> 4) + (kk & 3) * 2, kIdesc,
                              in_chunk != 0 || kk != 0 ? 1u : 0u);
            tc_commit(&tail->wide_empty[b]);
            if (WIDE) tc_commit(&tail->x_empty[x]);
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
    const int side = (warp - 4) >> 3;         // which half of a block's k, and of the tokens' sums
    const int wrow = half * 128 + quarter * 32 + lane;
    constexpr int kMySums = TM / 2;
    constexpr int kStep = kMySums == 16 || kMySums == 32 ? 16 : 8;  // sums per TMEM load
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t sums_at = tmem_base + lanes + static_cast<uint32_t>(half) * kSumCols + side * kMySums;
    const uint32_t wide_at = tmem_base + lanes + kWideAt + static_cast<uint32_t>(half) * kWideHalf + side * 32;
    const uint32_t raw_w = smem_u32(smem) + static_cast<uint32_t>(wrow) * BK;
    const uint32_t turn = static_cast<uint32_t>((side * 4) ^ (wrow & 7)) * 16;
    constexpr int kPieces = TM * 8;  // 16-byte pieces of a block's tokens
    constexpr int kMine = (kPieces + kWorkThreads - 1) / kWorkThreads;
    static_assert(kMine <= 2, "a thread's second piece lies in the other 64 of k");
    const uint32_t token = static_cast<uint32_t>(tid & (TM - 1));
    const int piece = tid / TM;  // the first; the second is piece + 4
    const bool has_piece = kPieces >= kWorkThreads || piece < 8;
    // where it lies, and the first of its two widened pieces (the other: ^ 16)
    const uint32_t x_from = smem_u32(smem) + kRawW + token * BK +
                            (static_cast<uint32_t>(piece * 16) ^ ((token & 7) * 16));
    const uint32_t x_to = smem_u32(wide) + (piece >= 4 ? TM * 128 : 0) + token * 128 +
                          (static_cast<uint32_t>((piece & 3) * 32) ^ ((token & 7) * 16));
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
      for (int h = 0; h < 2; ++h) {
        uint32_t r[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 v = w[c];
          widen4(v.x, r[c * 8], r[c * 8 + 1]);
          widen4(v.y, r[c * 8 + 2], r[c * 8 + 3]);
          widen4(v.z, r[c * 8 + 4], r[c * 8 + 5]);
          widen4(v.w, r[c * 8 + 6], r[c * 8 + 7]);
        }
        if (h == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c) w[c] = ld_shared_u4(raw_w + from + (turn ^ (c * 16 + 32)));
        }
        tmem_st_32x32b_x16(wide_at + b * kWideCols + h * 16, r);
      }
      // Neighbouring threads take neighbouring tokens and the same piece, so that
      // reads and writes of eight lanes fall in different banks.
      // Neighbouring threads take neighbouring tokens and the same piece, so that
      // reads and writes of eight lanes fall in different banks.
      if (!WIDE && has_piece) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const uint4 x = ld_shared_u4((x_from ^ (i * 64)) + from);
          uint32_t v[8];
          widen4(x.x, v[0], v[1]);
          widen4(x.y, v[2], v[3]);
          widen4(x.z, v[4], v[5]);
          widen4(x.w, v[6], v[7]);
          const uint32_t to = x_to + b * kWideBytes + i * (TM * 128);
          st_shared_u4(to, v[0], v[1], v[2], v[3]);
          st_shared_u4(to ^ 16, v[4], v[5], v[6], v[7]);
        }
      }
      tc_wait_st();
      if (!WIDE) fence_proxy_async_smem();
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

    // This CTA's blocks of a tile.  The first block of a chunk is ready before
    // the last chunk is taken.
    auto sums = [&]() -> bool {
      const uint32_t start = 0u - kWholeOff * static_cast<uint32_t>((kb1 - kb0 + kChunk - 1) / kChunk);
#pragma unroll
      for (int i = 0; i < kMySums; ++i) sum[i] = by_unit(i / kStep * kStep) ? 0u : start;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!convert()) return false;
        if (kb > kb0 && (kb - kb0) % kChunk == 0 && !take()) return false;
      }
      return kb1 == kb0 || take();
    };

    const uint32_t my_scales = tail_at + offsetof(Tail, scales) +
                               static_cast<uint32_t>(warp - 4) * sizeof(tail->scales[0]);
    const uint32_t order_at = tail_at + offsetof(Tail, order);
    for (int t = first; !CLUSTER && t < ld_shared_i4(order_at).x; t += ld_shared_i4(order_at).w) {
      if (p.num_kb > 0) {
        const int4 o = ld_shared_i4(order_at);
        const int row0 = tile_of(t, o.y, o.z).tm * TM + side * kMySums;
        for (int j = lane; j < kMySums; j += 32)
          cp_async_4_at(my_scales + 4 * j, row0 + j < p.M ? p.sa + row0 + j : p.sa,
                        row0 + j < p.M ? 4u : 0u);
      }
      if (!sums()) break;
      cp_async_wait_all();
      __syncwarp();
      const int4 o = ld_shared_i4(order_at);
      const Tile w = tile_of(t, o.y, o.z);
      const int n = w.tn * WN + wrow, row0 = w.tm * TM + side * kMySums;
      const int rows = min(p.M - row0, kMySums);  // below 1: none
      const bool in = n < p.N;
      const float cs = in && p.num_kb > 0 ? p.alpha * p.sb[n] : 0.0f;
      const float bias = in && p.bias != nullptr ? p.bias[n] : 0.0f;
      const int64_t at = row0 * p.ldd + n;
      if (p.d_pair && w.tn * WN + WN <= p.N && rows == kMySums) {
        // Two tokens' values of a channel become two channels' of a token: even
        // lanes take the first token's, odd ones the second's.
        const bool odd = lane & 1;
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + at + (odd ? p.ldd - 1 : 0);
#pragma unroll
        for (int j = 0; j < kMySums; j += 4) {
          const float4 sa = ld_shared_v4(my_scales + 4 * j);
          const float v0 = value(p, sum[j], cs, sa.x, bias), v1 = value(p, sum[j + 1], cs, sa.y, bias);
          const float v2 = value(p, sum[j + 2], cs, sa.z, bias), v3 = value(p, sum[j + 3], cs, sa.w, bias);
          const float x = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
          const float y = __shfl_xor_sync(0xffffffffu, odd ? v2 : v3, 1);
          *reinterpret_cast<uint32_t*>(d) = odd ? pack_bf16(x, v1) : pack_bf16(v0, x);
          d += 2 * p.ldd;
          *reinterpret_cast<uint32_t*>(d) = odd ? pack_bf16(y, v3) : pack_bf16(v2, y);
          d += 2 * p.ldd;
        }
      } else if (in) {
#pragma unroll
        for (int j = 0; j < kMySums; j += 4) {
          const float4 sa = ld_shared_v4(my_scales + 4 * j);
          const float s4[4] = {sa.x, sa.y, sa.z, sa.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j + i < rows) finish(p, at + (j + i) * p.ldd, value(p, sum[j + i], cs, s4[i], bias));
        }
      }
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
      cluster_sync();  // every part's sums are in its shared memory
      // after a wait ran out the sums are not complete; the error word says so
      const Tile w = tile_of(first, tiles_n, tiles_m);
      // 512 threads: every other token each
      const int n = w.tn * WN + (tid & (WN - 1)), row0 = w.tm * TM;
      if (first < tiles && !ld_shared_volatile(abort_flag) && n < p.N) {
        const float cs = p.alpha * p.sb[n];
        const float bias = p.bias != nullptr ? p.bias[n] : 0.0f;
        const int j1 = min((part + 1) * TM / split, p.M - row0);
        const uint32_t mine = smem_u32(smem) + static_cast<uint32_t>(tid & (WN - 1)) * 4;
        for (int j = part * TM / split + (tid >> 8); j < j1; j += 2) {
          uint32_t total = 0;
          for (int src = 0; src < split; ++src)
            total += __float_as_uint(ld_shared_cluster_f32(
                mapa_shared(mine + static_cast<uint32_t>(j) * (WN * 4), static_cast<uint32_t>(src))));
          finish(p, (row0 + j) * p.ldd + n, value(p, total, cs, p.sa[row0 + j], bias));
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

// int8 rows -> fp16 rows of pitch ld2 (a multiple of 8; what is behind a row's
// end is zero).  16 values a thread.
__global__ void __launch_bounds__(256) widen_rows_kernel(const int8_t* src, int64_t ld, uint16_t* dst,
                                                         int64_t ld2, int64_t rows, int64_t cols, int vec) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t pieces = (ld2 + 15) / 16, total = rows * pieces;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step) {
    const int64_t r = total < (int64_t{1} << 31) ? static_cast<uint32_t>(i) / static_cast<uint32_t>(pieces) : i / pieces;
    const int64_t c = (i - r * pieces) * 16;
    const int8_t* s = src + r * ld + c;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (vec && c + 16 <= cols) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(s));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < cols) w[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(s[j])) << (8 * (j & 3));
    }
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) widen4(w[j], v[2 * j], v[2 * j + 1]);
    uint4* d = reinterpret_cast<uint4*>(dst + r * ld2 + c);
    d[0] = make_uint4(v[0], v[1], v[2], v[3]);
    if (c + 8 < ld2) d[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
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
  if (ops_allow_smem<int8_kernel<kMaxTokens, kSplit>>(kSmemBytes) == cudaSuccess) {
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
    if (cudaOccupancyMaxActiveClusters(&n, int8_kernel<kMaxTokens, kSplit>, &cfg) != cudaSuccess) n = 0;
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

template <int TM>
cudaError_t launch(int64_t tiles, int num_sms, const Int8Args& a, const CUtensorMap& tmA,
                   const CUtensorMap& tmB, cudaStream_t s) {
  if (a.cluster > 1)
    return ops_launch<int8_kernel<TM, kSplit>>(dim3(static_cast<unsigned>(tiles * a.cluster)), kThreads,
                                             kSmemBytes, a.cluster, s, a, tmA, tmB);
  return ops_launch<int8_kernel<TM, kSingle>>(dim3(static_cast<unsigned>(tiles < num_sms ? tiles : num_sms)),
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
  const int tm = M > 64 ? 128 : (M > 32 ? 64 : (M > 16 ? 32 : 16));
  const int64_t tiles = ((N + WN - 1) / WN) * ((M + tm - 1) / tm);
  if (tiles + sms > kOpsMaxDim) return GEMM_ERR_UNSUPPORTED;
  a.cluster = choose_split(tiles, a.num_kb, sms);
  std::unique_lock<std::mutex> lock;
  CUtensorMap tmA{}, tmB{};
  bool wide = false;
  if (product) {
    ByteOperand oa{A, M, K, lda, 1, 0}, ob{B, N, K, ldb, 1, 0};
    const int64_t need_b = byte_tma_ok(ob) ? 0 : byte_staged(ob);
    const int64_t ld2 = (K + 7) / 8 * 8, wide_a = (2 * M * ld2 + 255) / 256 * 256;
    uint8_t* buf = nullptr;
    // The tokens widened by themselves, if there are enough tiles to share them
    // and memory for them.
    if (tm == kMaxTokens && tiles > sms) {
      st = abi_stage(s, wide_a + need_b, lock, &buf);
      wide = st == GEMM_OK;
      if (!wide) lock = std::unique_lock<std::mutex>();
    }
    const int64_t need_a = wide || byte_tma_ok(oa) ? 0 : byte_staged(oa);
    if (!wide && need_a + need_b > 0) {
      st = abi_stage(s, need_a + need_b, lock, &buf);
      if (st != GEMM_OK) return st;
    }
    cudaError_t e = cudaSuccess;
    if (wide) {
      const int64_t want = (M * ((ld2 + 15) / 16) + 255) / 256, fit = static_cast<int64_t>(sms) * 16;
      uint16_t* to = reinterpret_cast<uint16_t*>(buf);
      const int vec = !ops_misaligned(A, 16) && (M == 1 || lda % 16 == 0);
      e = ops_launch<widen_rows_kernel>(dim3(static_cast<unsigned>(want < fit ? want : fit)), 256, 0, 1, s, A,
                                        lda, to, ld2, M, K, vec);
    } else if (need_a > 0) {
      e = byte_stage(oa, buf, sms, s);
    }
    if (e == cudaSuccess && need_b > 0) e = byte_stage(ob, buf + (wide ? wide_a : need_a), sms, s);
    if (e != cudaSuccess) return abi_from_cuda(e);
    const int64_t da[2] = {K, M}, ta[1] = {wide ? 2 * ld2 : byte_pitch(oa)};
    const int64_t db[2] = {K, N}, tb[1] = {byte_pitch(ob)};
    const uint32_t ba[2] = {wide ? 64u : static_cast<uint32_t>(BK), static_cast<uint32_t>(tm)}, bb[2] = {BK, WN};
    if (!abi_encode_tiled(&tmA, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                          wide ? buf : oa.p, da, ta, ba) ||
        !abi_encode_tiled(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, ob.p, db, tb, bb))
      return GEMM_ERR_LAUNCH;
  }
  if (wide)
    return abi_from_cuda(ops_launch<int8_kernel<kMaxTokens, kWide>>(dim3(static_cast<unsigned>(sms)), kThreads,
                                                                    kSmemBytes, 1, s, a, tmA, tmB));
  switch (tm) {
    case 16: return abi_from_cuda(launch<16>(tiles, sms, a, tmA, tmB, s));
    case 32: return abi_from_cuda(launch<32>(tiles, sms, a, tmA, tmB, s));
    case 64: return abi_from_cuda(launch<64>(tiles, sms, a, tmA, tmB, s));
    default: return abi_from_cuda(launch<128>(tiles, sms, a, tmA, tmB, s));
  }
}
