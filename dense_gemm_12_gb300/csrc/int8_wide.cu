// int8_wide.cu -- large int8 products (int8_tc.cu has the mathematics): both
// operands are widened to fp16 by a kernel of their own, a few microseconds for
// three bytes a value, and meet in a kernel that only sums.
//
// Widening inside the product costs more than it does outside: the int8 values
// pass through shared memory twice and the widened tokens once more, next to the
// MMAs' reads, 1536 cycles of it per 1024 cycles of MMAs, and the accumulator
// fills TMEM together with the widened weights, so the MMAs stand still while it
// is read (8192^3 904 us, of which 590 at the rate of the MMAs).  Measured here:
// 8192^3 605 to 620 us, 38 of them the widening (1.9 PFLOP/s after it), 4096^3 91
// (four full rounds), 3000 x 5000 x 1999 53 (3.7 of four rounds).
//   * CTA pairs take 256 weights x 256 or 224 tokens (cta_group::2, M = 256): each
//     CTA holds half of both, 30 or 32 KB a k-block of 64, in a ring of six stages
//   * warp 0 is the TMA producer, warp 1 of the even CTA the MMA issuer, into two
//     accumulators in turn (up to 256 columns each: all of TMEM)
//   * warps 4..11 carry an accumulator's sums on as integers every 1024 of k, and
//     write a finished tile, while the MMAs fill the other: a thread has one
//     channel and half of the tokens in registers (moved from the first warpgroup).
#include <cstddef>

#include "int8.cuh"

namespace g12 {
namespace {

constexpr int BM = 128, BK = 64;   // a CTA's weights; the pair's tokens are BN
constexpr int STAGES = 6;
constexpr int kChunk = 1024 / BK;  // k-blocks that an accumulator sums exactly
constexpr int kThreads = 384;
constexpr int kSumWarps = 8;
constexpr uint32_t kTmemCols = 512, kSumCols = 256;
constexpr int kFewRegs = 40, kManyRegs = 232;  // 40 + 2 x 232 = 3 x 168

constexpr int kStageBytesA = BM * BK * 2;
constexpr int stage_bytes(int bn) { return kStageBytesA + bn / 2 * BK * 2; }  // multiples of 1024

template <int BN>
struct __align__(16) Tail {
  float scales[kSumWarps][BN / 2];
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t sum_full[2];
  uint64_t sum_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t smem_bytes(int bn) {
  return 1024 + STAGES * stage_bytes(bn) + (bn == 256 ? sizeof(Tail<256>) : sizeof(Tail<224>));
}
static_assert(smem_bytes(256) <= 227 * 1024, "int8 wide kernel shared memory");

// Tile t: bands of 8 column tiles, row tile by row tile within a band.
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

// tmW: the weights (N x K), tmX: the tokens (M x K), boxes of 64 x 128 and 64 x
// BN / 2.
template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    int8_wide_kernel(const __grid_constant__ Int8Args p, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX) {
  using Tail = Tail<BN>;
  constexpr int kStageBytes = stage_bytes(BN);
  constexpr int kSums = BN / 2;  // tokens of a thread
  constexpr uint32_t kIdesc = idesc_f16_f32(2 * BM, BN);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem<1024>(smem_raw);
  Tail* tail = reinterpret_cast<Tail*>(smem + STAGES * kStageBytes);
  const uint32_t tail_at = smem_u32(tail);
  const uint32_t abort_flag = tail_at + offsetof(Tail, abort_flag);
  const uint32_t full_at = tail_at + offsetof(Tail, full), empty_at = tail_at + offsetof(Tail, empty);
  const uint32_t sum_full_at = tail_at + offsetof(Tail, sum_full);
  const uint32_t sum_empty_at = tail_at + offsetof(Tail, sum_empty);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_cta_rank() & 1u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail->sum_full[b], 1);
      mbar_init(&tail->sum_empty[b], 2 * kSumWarps);
    }
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&tail->tmem_base, kTmemCols);
    tmem_relinquish_alloc_permit_pair();
  }
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  // Both CTAs of a pair signal barriers of the even one: all must be
  // initialised first.
  cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = tail->tmem_base;
  const int tiles_n = (p.N + 2 * BM - 1) / (2 * BM), tiles_m = (p.M + BN - 1) / BN;
  const int tiles = tiles_n * tiles_m;
  const int first = static_cast<int>(blockIdx.x) / 2, stride = static_cast<int>(gridDim.x) / 2;

  if (warp < 4) {
    regs_give_back<kFewRegs>();
    if (warp == 0) {
      // ------------------------------------------------------ TMA producer
      if (lane == 0) {
        uint32_t it = 0;
        bool ok = true;
        const uint32_t full0 = mapa_shared(full_at, 0);
        for (int t = first; t < tiles && ok; t += stride) {
          const Tile w = tile_of(t, tiles_n, tiles_m);
          const int n0 = w.tn * (2 * BM) + rank * BM, m0 = w.tm * BN + rank * (BN / 2);
          for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
            const uint32_t s = it % STAGES, round = it / STAGES;
            if (!mbar_wait_at(empty_at + 8 * s, (round & 1u) ^ 1u, abort_flag, p.err)) {
              ok = false;
              break;
            }
            uint8_t* to = smem + s * kStageBytes;
            if (rank == 0) mbar_arrive_expect_tx(&tail->full[s], 2 * kStageBytes);
            tma_load_2d_pair(to, &tmW, kb * BK, n0, full0 + 8 * s);
            tma_load_2d_pair(to + kStageBytesA, &tmX, kb * BK, m0, full0 + 8 * s);
          }
        }
        // Leave only after the MMAs have read every stage this CTA filled: then
        // all of its copies have landed and every commit aimed at its barriers
        // has arrived.
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t j = it > STAGES ? it - STAGES : 0u; j < it; ++j)
          while (!mbar_try_wait_at(empty_at + 8 * (j % STAGES), (j / STAGES) & 1u))
            if (globaltimer_ns() - t0 > kWaitLimitNs) break;
      }
      __syncwarp();
    } else if (warp == 1 && rank == 0) {
      // -------------------------------------------------------- MMA issuer
      uint32_t it = 0, chunk = 0;
      bool ok = true, issued = false;
      // K-major: 8-row groups 1024 bytes apart, a step of 16 of k is 32 bytes
      const uint64_t da0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t db0 = smem_desc_sw128(smem_u32(smem) + kStageBytesA, 16, 1024);
      for (int t = first; t < tiles && ok; t += stride) {
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const uint32_t s = it % STAGES, ab = chunk & 1u;
          const int in_chunk = kb % kChunk;
          bool got = mbar_wait_at(full_at + 8 * s, (it / STAGES) & 1u, abort_flag, p.err);
          if (in_chunk == 0)
            got = got && mbar_wait_at(sum_empty_at + 8 * ab, ((chunk >> 1) & 1u) ^ 1u, abort_flag, p.err);
          if (__any_sync(0xffffffffu, !got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const bool last = in_chunk == kChunk - 1 || kb + 1 == p.num_kb;
          const uint64_t step = static_cast<uint64_t>(s * (kStageBytes >> 4));
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              tc_mma_f16_pair(tmem_base + ab * kSumCols, da0 + step + kk * 2, db0 + step + kk * 2, kIdesc,
                              in_chunk != 0 || kk != 0 ? 1u : 0u);
            tc_commit_pair_multicast(&tail->empty[s], 0x3);
            if (last) tc_commit_pair_multicast(&tail->sum_full[ab], 0x3);
          }
          __syncwarp();
          issued = true;
          if (last) ++chunk;
        }
      }
      if (ok) {
        // no arrival of the odd CTA is still on its way at exit
        for (uint32_t j = chunk > 2 ? chunk - 2 : 0u; j < chunk; ++j) {
          const bool got = mbar_wait_at(sum_empty_at + 8 * (j & 1u), (j >> 1) & 1u, abort_flag, p.err);
          if (__any_sync(0xffffffffu, !got)) break;
        }
      } else if (issued) {
        if (elect_one()) tc_commit_pair(&tail->drain);
        __syncwarp();
        mbar_drain_wait(&tail->drain, 0);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- sums
    regs_take<kManyRegs>();
    const int quarter = warp & 3;      // TMEM lanes this warp may access
    const int half = (warp - 4) >> 2;  // which 128 tokens
    const uint32_t from = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                          static_cast<uint32_t>(half * kSums);
    const uint32_t scales = tail_at + static_cast<uint32_t>((warp - 4) * sizeof(tail->scales[0]));
    const uint32_t empty0 = mapa_shared(sum_empty_at, 0);
    const uint32_t start = 0u - kWholeOff * static_cast<uint32_t>((p.num_kb + kChunk - 1) / kChunk);
    uint32_t chunk = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += stride) {
      const Tile w = tile_of(t, tiles_n, tiles_m);
      const int n = w.tn * (2 * BM) + rank * BM + quarter * 32 + lane, row0 = w.tm * BN + half * kSums;
      fetch_scales<kSums>(p, scales, row0);
      uint32_t sum[kSums];
#pragma unroll
      for (int i = 0; i < kSums; ++i) sum[i] = by_unit(i) ? 0u : start;
      for (int kb = 0; kb < p.num_kb; kb += kChunk, ++chunk) {
        const uint32_t ab = chunk & 1u;
        ok = __all_sync(0xffffffffu,
                        mbar_wait_at(sum_full_at + 8 * ab, (chunk >> 1) & 1u, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after_sync();
        // eight at a time, the next ones on their way
        uint32_t r[2][8];
        tmem_ld_32x32b_x8(from + ab * kSumCols, r[0]);
#pragma unroll
        for (int j = 0; j < kSums; j += 8) {
          const int cur = (j >> 3) & 1;
          tmem_wait_ld(r[cur]);
          if (j + 8 < kSums) tmem_ld_32x32b_x8(from + ab * kSumCols + j + 8, r[cur ^ 1]);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            if (by_unit(j)) {
              sum[j + i] += static_cast<uint32_t>(__float2int_rn(__uint_as_float(r[cur][i])));
              sum[j + i + 1] += static_cast<uint32_t>(__float2int_rn(__uint_as_float(r[cur][i + 1])));
            } else {
              add_whole(sum[j + i], sum[j + i + 1], r[cur][i], r[cur][i + 1]);
            }
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(empty0 + 8 * ab);
      }
      if (!ok) break;
      cp_async_wait_all();
      __syncwarp();
      write_channel<kSums>(p, sum, scales, n, row0);
      __syncwarp();  // the scales have been read
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  // Neither CTA of a pair releases TMEM or exits while the pair's MMAs or copies
  // can still touch it.
  cluster_sync();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// int8 rows -> fp16 rows of pitch ld2 (a multiple of 8; what is behind a row's
// end is zero), of two matrices.  16 values a thread.
struct WidenArgs {
  const int8_t* src[2];
  int64_t ld[2], rows[2];
  int vec[2];       // rows start on 16 bytes
  uint16_t* dst[2];
  int64_t cols, ld2;
};

__global__ void __launch_bounds__(256) widen_kernel(const __grid_constant__ WidenArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t pieces = (a.ld2 + 15) / 16;
  const int64_t mine = a.rows[0] * pieces, total = mine + a.rows[1] * pieces;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step) {
    const int m = i < mine ? 0 : 1;
    const int64_t j = m == 0 ? i : i - mine;
    const int64_t r = total < (int64_t{1} << 31)
                          ? static_cast<uint32_t>(j) / static_cast<uint32_t>(pieces) : j / pieces;
    const int64_t c = (j - r * pieces) * 16;
    const int8_t* s = a.src[m] + r * a.ld[m] + c;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (a.vec[m] && c + 16 <= a.cols) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(s));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
#pragma unroll
      for (int b = 0; b < 16; ++b)
        if (c + b < a.cols) w[b >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(s[b])) << (8 * (b & 3));
    }
    uint32_t v[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) widen4(w[b], v[2 * b], v[2 * b + 1]);
    uint4* d = reinterpret_cast<uint4*>(a.dst[m] + r * a.ld2 + c);
    d[0] = make_uint4(v[0], v[1], v[2], v[3]);
    if (c + 8 < a.ld2) d[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// CTA pairs that can be resident at once on the current device; 0 if unknown.
int max_pairs() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int known = cache[dev].load(std::memory_order_relaxed);
  if (known != 0) return known;
  int n = 0;
  if (ops_allow_smem<int8_wide_kernel<256>>(smem_bytes(256)) == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(256);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, int8_wide_kernel<256>, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  if (n > 0) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

int64_t pitch_of(int64_t K) { return (K + 7) / 8 * 8; }
int64_t copy_bytes(int64_t rows, int64_t K) { return (2 * rows * pitch_of(K) + 255) / 256 * 256; }

// Microseconds of all rounds of tiles of bn tokens: 64 of k in 280 ns for 256 of
// them, or the time of a tile's end, where that is more.
double tiles_us(int bn, int64_t M, int64_t N, int64_t K, int pairs) {
  const int64_t tiles = ((N + 2 * BM - 1) / (2 * BM)) * ((M + bn - 1) / bn);
  const double us = (bn == 256 ? 0.28 : 0.252) * static_cast<double>((K + BK - 1) / BK) + 0.85;
  return static_cast<double>((tiles + pairs - 1) / pairs) * (us < 4.0 ? 4.0 : us);
}
// Tokens of a tile: 224 where that makes better rounds, and does not compute
// many more rows than 256 without a token in them (us, 224 / 256: 3000 x 5000 x
// 1999 52.7 / 58.0, 3000 x 4096 x 4096 71 / 84, 2000 x 8192 x 2048 53 / 60, 4096^3 91 /
// 96, but 4096 x 4096 x 2048 52.3 / 51.0 and x 1024 33.9 / 30.2).
int tokens_of(int64_t M, int64_t N, int64_t K, int pairs) {
  const double few = static_cast<double>((M + 223) / 224 * 224), many = static_cast<double>((M + 255) / 256 * 256);
  const double more = few > many ? few / many - 1.0 : 0.0;
  return tiles_us(224, M, N, K, pairs) < tiles_us(256, M, N, K, pairs) * (1.0 - 2.4 * more) ? 224 : 256;
}

// The widened copies take at most this much of the stream's buffer.
constexpr int64_t kMostBytes = int64_t{1} << 30;

}  // namespace

int64_t int8_wide_bytes(int64_t M, int64_t N, int64_t K) { return copy_bytes(M, K) + copy_bytes(N, K); }

bool int8_wide_pays(int64_t M, int64_t N, int64_t K, double us) {
  const int64_t bytes = int8_wide_bytes(M, N, K);
  const int pairs = max_pairs();
  if (bytes > kMostBytes || pairs <= 0) return false;
  // The tiles, the last one's end, the widening (3 bytes a value at 7 TB/s) and
  // its launch.  Both sides, us here / there: 256 x 4096 x 4096 31 / 17, 512 x
  // 4096 x 4096 31 / 24, 1024 x 4096 x 1024 14.4 / 13.2, 768 x 4096 x 4096 32 / 36,
  // 2048 x 4096 x 512 15.9 / 17.6, 4096^3 96 / 138, 8192 x 8192 x 128 56 / 77,
  // 8192^3 605 / 907.
  return tiles_us(tokens_of(M, N, K, pairs), M, N, K, pairs) + 3.5 +
             1.5e-6 * static_cast<double>(bytes) / 7.0 + 2.5 < us;
}

gemm_status_t int8_wide(const Int8Args& args, int64_t K, const int8_t* A, int64_t lda, const int8_t* B,
                        int64_t ldb, uint8_t* buf, int num_sms, cudaStream_t s) {
  Int8Args p = args;
  p.num_kb = static_cast<int>((K + BK - 1) / BK);
  WidenArgs w{};
  w.src[0] = B;
  w.ld[0] = ldb;
  w.rows[0] = p.N;
  w.src[1] = A;
  w.ld[1] = lda;
  w.rows[1] = p.M;
  for (int i = 0; i < 2; ++i) w.vec[i] = !ops_misaligned(w.src[i], 16) && (w.rows[i] == 1 || w.ld[i] % 16 == 0);
  w.dst[0] = reinterpret_cast<uint16_t*>(buf);
  w.dst[1] = reinterpret_cast<uint16_t*>(buf + copy_bytes(p.N, K));
  w.cols = K;
  w.ld2 = pitch_of(K);
  const int64_t want = ((w.rows[0] + w.rows[1]) * ((w.ld2 + 15) / 16) + 255) / 256;
  const int64_t fit = static_cast<int64_t>(num_sms) * 32;
  const cudaError_t e =
      ops_launch<widen_kernel>(dim3(static_cast<unsigned>(want < fit ? want : fit)), 256, 0, 1, s, w);
  if (e != cudaSuccess) return abi_from_cuda(e);
  const int pairs = max_pairs(), bn = tokens_of(p.M, p.N, K, pairs);
  CUtensorMap tm[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t dims[2] = {K, w.rows[i]}, pitch[1] = {2 * w.ld2};
    const uint32_t box[2] = {BK, static_cast<uint32_t>(i == 0 ? BM : bn / 2)};
    if (!abi_encode_tiled(&tm[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w.dst[i], dims, pitch, box))
      return GEMM_ERR_LAUNCH;
  }
  const int64_t tiles = ((p.N + int64_t{2 * BM - 1}) / (2 * BM)) * ((p.M + bn - int64_t{1}) / bn);
  const dim3 grid(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
  if (bn == 224)
    return abi_from_cuda(
        ops_launch<int8_wide_kernel<224>>(grid, kThreads, smem_bytes(224), 2, s, p, tm[0], tm[1]));
  return abi_from_cuda(
      ops_launch<int8_wide_kernel<256>>(grid, kThreads, smem_bytes(256), 2, s, p, tm[0], tm[1]));
}

}  // namespace g12
