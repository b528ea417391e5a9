// grouped_tc.cu -- bf16 products grouped by expert with ragged row counts, on
// the 5th-generation tensor cores.  Group g has rows offsets[g] ..
// offsets[g + 1] - 1 of A, and a K x N matrix B[g]:
//
//     forward           D[t] = alpha A[t] B[g] + beta D[t]
//     input gradient    the same with B[g]^T (B[g] is then N x K)
//     weight gradient   dB[g] = alpha sum_{t in g} A[t]^T dD[t] + beta dB[g]
//
// The kernel is the dense one's (bf16_tc.cu): a TMA producer, one MMA issuer
// (M = 128, N = 256, K = 16), two accumulators in TMEM, four warps writing
// finished tiles; persistent CTAs walk the tiles of all groups in one order
// (groups.cuh).  What is different:
//   * a group's last row tile reads rows of the next group.  They only reach
//     accumulator rows that are not written.
//   * in the weight gradient the ragged direction is the one summed over, so
//     rows past the group's end must not reach the sum, whatever they hold
//     (NaN included): of a group's last block only the steps of 16 rows that
//     the group reaches run, and the rest of the last one is zeroed in shared
//     memory, in both operands (8001 rows of 24 groups, 1024 x 2048: 44.4 us
//     against 45.6 with the whole block zeroed and summed) -- by the issuing
//     warp, or in a pair by a warp of each CTA's own.
//     Groups are taken as they come: by falling size it took 49.0 us, since the
//     small ones then write their matrices at once, with nothing to compute.
//   * a weight gradient's group without rows is written as beta dB[g].
#include "groups.cuh"
#include "ops.cuh"

namespace g12 {
namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int kRingBytes = 192 * 1024;
constexpr int kStageBytesA = BM * BK * 2;
constexpr int kBoxBytes = BK * 64 * 2;  // one MN-major box: 64 of M or N, 64 of k
// A pair's CTAs hold half of the tile's B each.
constexpr int b_cols(bool pair) { return pair ? BN / 2 : BN; }
constexpr int stage_bytes(bool pair) { return kStageBytesA + BK * b_cols(pair) * 2; }  // 48 or 32 KB
constexpr int ring_stages(bool pair) { return kRingBytes / stage_bytes(pair); }        // 4 or 6
constexpr int kMaxStages = 6;
constexpr int kThreads = 192;
constexpr int kRaggedThreads = 224;  // a pair's weight gradient: a warp for ragged ends
constexpr int kRaggedWarp = 6;
constexpr int kOutThreads = 128;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOutBarAny = 1;
constexpr int kOutWarpBytes = 32 * 32 * 4;

// Layouts: which operands are contiguous along k ("K-major").
enum Mode : int { kForward = 0, kTransB = 1, kWeightGrad = 2 };

struct GroupedArgs {
  int rows;             // of A (and dD)
  int M, N, K;          // kWeightGrad: M x N is one dB[g] and K unused; else N columns, K summed
  int groups;
  const int32_t* offsets;
  float alpha, beta;
  void* D;
  int64_t ldd, stride_d;
  int d_type, d_vec;
  int tile_rows;        // rows of A per tile (not kWeightGrad)
  int band;
  int d_tma;            // beta == 0 and TMA can describe D: whole pieces leave by TMA
  int product;          // 0: alpha == 0 or K == 0, operands are not read
  uint32_t* err;
};

struct __align__(8) Tail {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t landed[kMaxStages];  // a pair's weight gradient, a group's ragged last
  uint64_t ragged[kMaxStages];  // block: it is here / its end is zeroed in both CTAs
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  GroupTable groups;
};

constexpr size_t kSmemBytes = 1024 + kRingBytes + 4 * kOutWarpBytes + sizeof(Tail);
static_assert(kSmemBytes <= 227 * 1024, "grouped kernel shared memory");

// One work item: its k-blocks, where its rows (or, for the weight gradient,
// its M) start, and its output rows.
struct Item {
  int group, tn;
  int row0;      // first row of A read (forward) / first row of the group (weight gradient)
  int m0;        // weight gradient: first row of dB
  int rows;      // output rows
  int num_kb;
  int last;      // weight gradient: rows of the last k-block
};

template <int MODE, bool PAIR>
__device__ __forceinline__ Item item_of(const GroupedArgs& p, const GroupTable& tab, int t,
                                        int tiles_n, int num_kb, int rank, int& g) {
  Item w;
  if (MODE != kWeightGrad) {
    const GroupTile f = group_tile(tab, t, tiles_n, p.band, p.tile_rows, g);
    w.group = f.group;
    w.tn = f.tn;
    // of a pair's 256 rows the CTA takes 128, perhaps none
    w.row0 = f.row0 + (PAIR ? rank * BM : 0);
    w.m0 = 0;
    w.rows = PAIR ? min(f.rows - rank * BM, BM) : f.rows;
    w.num_kb = num_kb;
    w.last = BK;
    return w;
  }
  constexpr int kTileM = PAIR ? 2 * BM : BM;
  const int tiles_m = (p.M + kTileM - 1) / kTileM;
  const int per = tiles_m * tiles_n;
  w.group = t / per;
  const int local = t - w.group * per;
  const int per_band = p.band * tiles_n;
  const int b = local / per_band;
  const int high = min(tiles_m - b * p.band, p.band);
  const int in_band = local - b * per_band;
  w.tn = in_band / high;
  w.m0 = (b * p.band + in_band % high) * kTileM + (PAIR ? rank * BM : 0);
  w.row0 = tab.row[w.group];
  w.rows = min(BM, p.M - w.m0);
  const int n = p.product ? tab.row[w.group + 1] - w.row0 : 0;
  w.num_kb = (n + BK - 1) / BK;
  w.last = n - (w.num_kb - 1) * BK;
  return w;
}

// Whether block kb of a weight gradient holds rows of the next group in its
// last step.
__device__ __forceinline__ bool is_ragged(const Item& w, int kb) {
  return kb == w.num_kb - 1 && (w.last & 15) != 0;
}

// Zeroes those rows in a stage of `boxes` boxes; all lanes of a warp.  Row k of
// a box is its bytes 128 k .. 128 k + 127, whatever the swizzle does inside them.
__device__ __forceinline__ void zero_ragged(uint8_t* stage, const Item& w, int boxes) {
  const int pieces = (16 - (w.last & 15)) * 8;
#pragma unroll
  for (int box = 0; box < boxes; ++box) {
    uint4* z = reinterpret_cast<uint4*>(stage + box * kBoxBytes + w.last * 128);
    for (int i = threadIdx.x & 31; i < pieces; i += 32) z[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// 32 accumulator rows x 64 columns of this warp (r, s: 32 columns each) as
// bf16: packed in registers, turned around in the warp's 4 KB of shared memory
// (128-byte rows, 16-byte pieces XOR-swizzled by row) and written with 8 lanes
// to a row.  All pieces are read back before the first is stored: a load after
// a store to a possibly aliasing address could not be issued early.
__device__ __forceinline__ void write_bf16(const GroupedArgs& p, uint4* stg, const uint32_t (&r)[32],
                                           const uint32_t (&s)[32], float alpha, __nv_bfloat16* D,
                                           int64_t row_base, int rows, int col0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = (q & 3) * 8 + 2 * i;
      w[i] = q < 4 ? pack_bf16(alpha * __uint_as_float(r[k]), alpha * __uint_as_float(r[k + 1]))
                   : pack_bf16(alpha * __uint_as_float(s[k]), alpha * __uint_as_float(s[k + 1]));
    }
    stg[lane * 8 + (q ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  const int piece = lane & 7, rl = lane >> 3;
  const int col = col0 + 8 * piece;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = stg[(i * 4 + rl) * 8 + (piece ^ ((i * 4 + rl) & 7))];
  __nv_bfloat16* d = D + (row_base + rl) * p.ldd + col;
  if (col + 8 <= p.N && p.d_vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 4 + rl < rows) *reinterpret_cast<uint4*>(d + i * 4 * p.ldd) = v[i];
  } else {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      if (i * 4 + rl >= rows) break;
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < p.N)
          reinterpret_cast<uint16_t*>(d + i * 4 * p.ldd)[k] =
              static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    }
  }
  __syncwarp();
}

// 32 accumulator rows x 32 columns of this warp in fp32 through the same 4 KB,
// where D is fp32 or read as well (beta != 0): 4 columns per lane.  The old
// values of D are read before the first store.
__device__ __forceinline__ void write_any(const GroupedArgs& p, float4* stg, const uint32_t (&r)[32],
                                          float alpha, void* D, int64_t row_base, int rows, int col0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    stg[lane * 8 + (q ^ (lane & 7))] =
        make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]),
                    __uint_as_float(r[4 * q + 2]), __uint_as_float(r[4 * q + 3]));
  __syncwarp();
  const int ch = lane & 7, rl = lane >> 3;
  const int col = col0 + 4 * ch;
  const bool whole = col + 4 <= p.N && p.d_vec;
  float4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rr = i * 4 + rl;
    const float4 a = stg[rr * 8 + (ch ^ (rr & 7))];
    v[i] = make_float4(alpha * a.x, alpha * a.y, alpha * a.z, alpha * a.w);
  }
  const int64_t at0 = (row_base + rl) * p.ldd + col, step = 4 * p.ldd;
  if (p.beta != 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i * 4 + rl >= rows) continue;
      float o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = col + k < p.N ? load1(D, p.d_type, at0 + i * step + k) : 0.0f;
      v[i] = make_float4(fmaf(p.beta, o[0], v[i].x), fmaf(p.beta, o[1], v[i].y),
                         fmaf(p.beta, o[2], v[i].z), fmaf(p.beta, o[3], v[i].w));
    }
  }
  if (whole && p.d_type == GEMM_OUT_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 4 + rl < rows)
        *reinterpret_cast<float4*>(static_cast<float*>(D) + at0 + i * step) = v[i];
  } else if (whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 4 + rl < rows)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(D) + at0 + i * step) =
            make_uint2(pack_bf16(v[i].x, v[i].y), pack_bf16(v[i].z, v[i].w));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i * 4 + rl >= rows) continue;
      const float w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < p.N) store1(D, p.d_type, at0 + i * step + k, w[k]);
    }
  }
  __syncwarp();
}

// The same where TMA can describe D and beta is 0: pieces of 32 rows x 64
// bytes (32 columns of bf16, or 16 of fp32) are scaled and packed in registers,
// written to one of the warp's two 2 KB buffers (16-byte pieces XOR-swizzled as
// the tensor map's 64-byte swizzle has them) and stored by one TMA copy, which
// the map clips at D's edges.  The next 32 accumulator columns are read
// meanwhile.  seq: pieces so far; a buffer is rewritten once the copy two
// pieces back has read it.  row, z: coordinates of the first row.
//
// Along a row the copy is clipped to whole 16-byte pieces only: a last piece
// that D's row ends in would be written to its end, over what follows the row.
// Where rows end so, the chunk that holds the end is left to the caller.
// Returns the number of chunks written.
__device__ __forceinline__ void stage_piece(const CUtensorMap* tmD, uint32_t stg, uint32_t& seq,
                                            const uint32_t (&w)[16], int col, int row, int z) {
  const uint32_t lane = threadIdx.x & 31;
  if (lane == 0) bulk_wait_group_read<1>();
  __syncwarp();
  const uint32_t buf = stg + (seq & 1u) * 2048u;
  ++seq;
#pragma unroll
  for (uint32_t q = 0; q < 4; ++q)
    st_shared_u4(buf + lane * 64u + ((q ^ ((lane >> 1) & 3u)) << 4), w[4 * q], w[4 * q + 1],
                 w[4 * q + 2], w[4 * q + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(tmD, buf, col, row, z);
    bulk_commit_group();
  }
}

__device__ __forceinline__ int write_tma(const GroupedArgs& p, const CUtensorMap* tmD, uint32_t taddr,
                                         uint32_t stg, uint32_t& seq, int row, int z, int col0) {
  const bool whole = (p.N & (p.d_type == GEMM_OUT_BF16 ? 7 : 3)) == 0;
  const int chunks = min(BN / 32, (p.N - col0 + (whole ? 31 : 0)) / 32);
  if (chunks == 0) return 0;
  uint32_t r[32], next[32];
  tmem_ld_32x32b_x32(taddr, next);
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    tmem_wait_ld(next);
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = next[i];
    if (c + 1 < chunks) tmem_ld_32x32b_x32(taddr + (c + 1) * 32, next);
    uint32_t w[16];
    if (p.d_type == GEMM_OUT_BF16) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16(p.alpha * __uint_as_float(r[2 * i]), p.alpha * __uint_as_float(r[2 * i + 1]));
      stage_piece(tmD, stg, seq, w, col0 + c * 32, row, z);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = __float_as_uint(p.alpha * __uint_as_float(r[16 * h + i]));
        if (col0 + c * 32 + h * 16 < p.N) stage_piece(tmD, stg, seq, w, col0 + c * 32 + h * 16, row, z);
      }
    }
  }
  return chunks;
}

// The 32 rows x 256 columns of this warp (fewer at the edges), from chunk
// `first` on.  load(c, r): columns 32 c .. 32 c + 31 of its rows.
template <typename Load>
__device__ __forceinline__ void write_tile(const GroupedArgs& p, uint8_t* stg, float alpha, void* D,
                                           int64_t row_base, int rows, int col0, Load load,
                                           int first = 0) {
  const int chunks = min(BN / 32, (p.N - col0 + 31) / 32);
  if (p.d_type == GEMM_OUT_BF16 && p.beta == 0.0f) {
#pragma unroll 1
    for (int c = first; c < chunks; c += 2) {
      uint32_t r[32], s[32];
      load(c, r);
      load(min(c + 1, BN / 32 - 1), s);  // past the last chunk: columns that are not written
      load.wait();
      write_bf16(p, reinterpret_cast<uint4*>(stg), r, s, alpha, static_cast<__nv_bfloat16*>(D),
                 row_base, rows, col0 + c * 32);
    }
    return;
  }
#pragma unroll 1
  for (int c = first; c < chunks; ++c) {
    uint32_t r[32];
    load(c, r);
    load.wait();
    write_any(p, reinterpret_cast<float4*>(stg), r, alpha, D, row_base, rows, col0 + c * 32);
  }
}

struct FromTmem {
  uint32_t taddr;
  __device__ __forceinline__ void operator()(int c, uint32_t (&r)[32]) const {
    tmem_ld_32x32b_x32(taddr + c * 32, r);
  }
  __device__ __forceinline__ void wait() const { tc_wait_ld(); }
};

struct Zeros {
  __device__ __forceinline__ void operator()(int, uint32_t (&r)[32]) const {
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = 0u;
  }
  __device__ __forceinline__ void wait() const {}
};

// PAIR: two CTAs share a 256 x 256 tile and one stream of M = 256 MMAs,
// barriers as in the dense pair kernel (bf16_tc.cu).
// Each SM's shared memory then takes 32 KB of operands per k-block and gives
// the tensor core as much, instead of 48 KB each way: with one CTA per tile
// that traffic (768 cycles at 128 B per cycle) outlasts the MMAs (512).
template <int MODE, bool PAIR>
__global__ void __launch_bounds__(MODE == kWeightGrad && PAIR ? kRaggedThreads : kThreads, 1)
    grouped_kernel(const __grid_constant__ GroupedArgs p, const __grid_constant__ CUtensorMap tmA,
                   const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmD) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = align_smem<1024>(smem_raw);
  uint8_t* out_stage = smem + kRingBytes;
  Tail* tail = reinterpret_cast<Tail*>(out_stage + 4 * kOutWarpBytes);
  int* abort_flag = &tail->abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr bool kGrad = MODE == kWeightGrad;
  constexpr int STAGES = ring_stages(PAIR), kStageBytes = stage_bytes(PAIR);
  const int rank = PAIR ? static_cast<int>(cluster_cta_rank() & 1u) : 0;
  const int first = static_cast<int>(blockIdx.x) / (PAIR ? 2 : 1);
  const int stride = static_cast<int>(gridDim.x) / (PAIR ? 2 : 1);
  constexpr uint32_t kIdesc =
      idesc_bf16_f32(PAIR ? 2 * BM : BM, BN, /*A MN-major*/ kGrad ? 1 : 0, /*B MN-major*/ MODE == kTransB ? 0 : 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&tail->full[s], 1);
      mbar_init(&tail->empty[s], 1);
      if (kGrad && PAIR) {
        mbar_init(&tail->landed[s], 1);
        mbar_init(&tail->ragged[s], 2);
      }
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tail->tmem_full[b], 1);
      mbar_init(&tail->tmem_empty[b], (PAIR ? 2 : 1) * (kOutThreads / 32));
    }
    mbar_init(&tail->drain, 1);
    tail->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(&tail->tmem_base, kTmemCols);
      tmem_relinquish_alloc_permit_pair();
    } else {
      tmem_alloc(&tail->tmem_base, kTmemCols);
      tmem_relinquish_alloc_permit();
    }
  }
  // Everything above touches no global memory and may overlap the previous
  // kernel's last CTAs; every global access below follows its completion.
  grid_dependency_wait();
  if (threadIdx.x == 0) grid_launch_dependents();
  if (warp == 2) build_groups(tail->groups, p.offsets, p.groups, p.rows, kGrad ? 1 : p.tile_rows);
  tc_fence_before_sync();
  __syncthreads();
  // Both CTAs of a pair signal barriers of the even one: all must be
  // initialised first.
  if (PAIR) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = tail->tmem_base;
  const GroupTable& tab = tail->groups;
  const int tiles_n = (p.N + BN - 1) / BN;
  constexpr int kTileM = PAIR ? 2 * BM : BM;  // of the weight gradient
  const int tiles = kGrad ? p.groups * ((p.M + kTileM - 1) / kTileM) * tiles_n
                          : tab.tile[p.groups] * tiles_n;
  const int num_kb = p.product ? (p.K + BK - 1) / BK : 0;

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      int g = 0;
      bool ok = true;
      const uint32_t bytes = PAIR ? 2u * kStageBytes
                                  : static_cast<uint32_t>(((kGrad ? BM : p.tile_rows) + BN) * BK * 2);
      const uint32_t full0 = PAIR ? mapa_shared(smem_u32(&tail->full[0]), 0) : 0u;
      for (int t = first; t < tiles && ok; t += stride) {
        const Item w = item_of<MODE, PAIR>(p, tab, t, tiles_n, num_kb, rank, g);
        for (int kb = 0; kb < w.num_kb; ++kb, ++it) {
          const uint32_t s = it % STAGES, round = it / STAGES;
          if (!mbar_wait_late(&tail->empty[s], (round & 1u) ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * kStageBytes;
          uint8_t* sb = sa + kStageBytesA;
          uint64_t* bar = &tail->full[s];
          if (kGrad && PAIR && is_ragged(w, kb)) {
            // to this CTA's own warp for ragged ends, which passes it on
            if (rank == 0) mbar_arrive(bar);
            bar = &tail->landed[s];
            mbar_arrive_expect_tx(bar, kStageBytes);
            const int k = w.row0 + kb * BK;
#pragma unroll
            for (int j = 0; j < BM / 64; ++j)
              tma_load_2d(sa + j * kBoxBytes, &tmA, w.m0 + j * 64, k, bar);
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_2d(sb + j * kBoxBytes, &tmB, w.tn * BN + rank * (BN / 2) + j * 64, k, bar);
            continue;
          }
          if (rank == 0) mbar_arrive_expect_tx(bar, bytes);
          if (PAIR && kGrad) {
            const uint32_t full = full0 + s * static_cast<uint32_t>(sizeof(uint64_t));
            const int k = w.row0 + kb * BK;
#pragma unroll
            for (int j = 0; j < BM / 64; ++j)
              tma_load_2d_pair(sa + j * kBoxBytes, &tmA, w.m0 + j * 64, k, full);
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_2d_pair(sb + j * kBoxBytes, &tmB, w.tn * BN + rank * (BN / 2) + j * 64, k, full);
          } else if (PAIR) {
            const uint32_t full = full0 + s * static_cast<uint32_t>(sizeof(uint64_t));
            const int n0 = w.tn * BN + rank * (BN / 2);
            tma_load_2d_pair(sa, &tmA, kb * BK, w.row0, full);
            if (MODE == kTransB) {
              tma_load_3d_pair(sb, &tmB, kb * BK, n0, w.group, full);
            } else {
#pragma unroll
              for (int j = 0; j < BN / 128; ++j)
                tma_load_3d_pair(sb + j * kBoxBytes, &tmB, n0 + j * 64, kb * BK, w.group, full);
            }
          } else if (kGrad) {
            const int k = w.row0 + kb * BK;
#pragma unroll
            for (int j = 0; j < BM / 64; ++j)
              tma_load_2d(sa + j * kBoxBytes, &tmA, w.m0 + j * 64, k, bar);
#pragma unroll
            for (int j = 0; j < BN / 64; ++j)
              tma_load_2d(sb + j * kBoxBytes, &tmB, w.tn * BN + j * 64, k, bar);
          } else {
            tma_load_2d(sa, &tmA, kb * BK, w.row0, bar);
            if (MODE == kTransB) {
              tma_load_3d(sb, &tmB, kb * BK, w.tn * BN, w.group, bar);
            } else {
#pragma unroll
              for (int j = 0; j < BN / 64; ++j)
                tma_load_3d(sb + j * kBoxBytes, &tmB, w.tn * BN + j * 64, kb * BK, w.group, bar);
            }
          }
        }
      }
      if (PAIR) {
        // Leave only after the MMAs have read every stage this CTA filled:
        // then all of its copies have landed and every commit aimed at its
        // barriers has arrived.
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t j = it > STAGES ? it - STAGES : 0u; j < it; ++j)
          while (!mbar_try_wait(&tail->empty[j % STAGES], (j / STAGES) & 1u))
            if (globaltimer_ns() - t0 > kWaitLimitNs) break;
      } else if (!ok) {
        for (uint32_t j = it > STAGES ? it - STAGES : 0u; j < it; ++j)
          mbar_drain_wait(&tail->full[j % STAGES], (j / STAGES) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank != 0) {
    // the even CTA issues for both
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer
    // K-major: 8-row groups 1024 B apart, a K step of 16 is 32 B.  MN-major:
    // 64-wide boxes 8 KB apart (LBO), 8-row k groups 1024 B apart (SBO), a K
    // step of 16 rows is 2048 B.
    const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + kStageBytesA;
    const uint64_t da0 = kGrad ? smem_desc_sw128(sa0, kBoxBytes, 1024) : smem_desc_sw128(sa0, 16, 1024);
    const uint64_t db0 = MODE == kTransB ? smem_desc_sw128(sb0, 16, 1024)
                                         : smem_desc_sw128(sb0, kBoxBytes, 1024);
    constexpr uint32_t kStepA = (kGrad ? 2048 : 32) >> 4, kStepB = (MODE == kTransB ? 32 : 2048) >> 4;
    uint32_t it = 0, j = 0, ragged_parity = 0;
    int g = 0;
    bool ok = true, issued = false;
    for (int t = first; t < tiles && ok; t += stride) {
      const Item w = item_of<MODE, PAIR>(p, tab, t, tiles_n, num_kb, rank, g);
      if (w.num_kb == 0) continue;
      const uint32_t ab = j & 1u, ar = j >> 1;
      ++j;
      bool got = mbar_wait_late(&tail->tmem_empty[ab], (ar & 1u) ^ 1u, abort_flag, p.err);
      if (__any_sync(0xffffffffu, !got)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t d_tmem = tmem_base + ab * BN;
      for (int kb = 0; kb < w.num_kb; ++kb, ++it) {
        const uint32_t s = it % STAGES, round = it / STAGES;
        got = mbar_wait_late(&tail->full[s], round & 1u, abort_flag, p.err);
        if (__any_sync(0xffffffffu, !got)) {
          ok = false;
          break;
        }
        // of a weight gradient's last block only the steps of 16 rows that the
        // group reaches
        const int steps = kGrad && kb == w.num_kb - 1 ? (w.last + 15) / 16 : BK / 16;
        if (kGrad && PAIR && is_ragged(w, kb)) {
          got = mbar_wait_late(&tail->ragged[s], ragged_parity >> s & 1u, abort_flag, p.err);
          ragged_parity ^= 1u << s;
          if (__any_sync(0xffffffffu, !got)) {
            ok = false;
            break;
          }
          fence_acq_rel_cluster();
        } else if (kGrad && is_ragged(w, kb)) {
          zero_ragged(smem + s * kStageBytes, w, (BM + BN) / 64);
        }
        tc_fence_after_sync();
        const uint64_t at = static_cast<uint64_t>(s * (kStageBytes >> 4));
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            if (kGrad && kk >= steps) break;
            if (PAIR)
              tc_mma_f16_pair(d_tmem, da0 + at + kk * kStepA, db0 + at + kk * kStepB, kIdesc,
                              (kb != 0 || kk != 0) ? 1u : 0u);
            else
              tc_mma_f16(d_tmem, da0 + at + kk * kStepA, db0 + at + kk * kStepB, kIdesc,
                         (kb != 0 || kk != 0) ? 1u : 0u);
          }
          if (PAIR)
            tc_commit_pair_multicast(&tail->empty[s], 0x3);
          else
            tc_commit(&tail->empty[s]);
        }
        issued = true;
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) {
        if (PAIR)
          tc_commit_pair_multicast(&tail->tmem_full[ab], 0x3);
        else
          tc_commit(&tail->tmem_full[ab]);
      }
      __syncwarp();
    }
    if (ok && PAIR) {
      // no arrival of the odd CTA is still on its way at exit
      for (uint32_t jj = j > 2 ? j - 2 : 0u; jj < j; ++jj)
        if (!mbar_wait_late(&tail->tmem_empty[jj & 1u], (jj >> 1) & 1u, abort_flag, p.err)) break;
    } else if (!ok && issued) {
      // Let every MMA this warp issued finish before TMEM is released.
      if (elect_one()) {
        if (PAIR)
          tc_commit_pair(&tail->drain);
        else
          tc_commit(&tail->drain);
      }
      __syncwarp();
      mbar_drain_wait(&tail->drain, 0);
    }
    __syncwarp();
  } else if (kGrad && PAIR && warp == kRaggedWarp) {
    // ---------------------------------------------------------- ragged ends
    // Zeroed in each CTA as soon as the block has landed there, well before its
    // MMAs; the even CTA's issuer hears of both.
    uint32_t it = 0, parity = 0;  // bits by stage
    int g = 0;
    const uint32_t ragged0 = mapa_shared(smem_u32(&tail->ragged[0]), 0);
    for (int t = first; t < tiles; t += stride) {
      const Item w = item_of<MODE, PAIR>(p, tab, t, tiles_n, num_kb, rank, g);
      it += static_cast<uint32_t>(w.num_kb);
      if (w.num_kb == 0 || !is_ragged(w, w.num_kb - 1)) continue;
      const uint32_t s = (it - 1) % STAGES;
      const bool got = mbar_wait_late(&tail->landed[s], parity >> s & 1u, abort_flag, p.err);
      parity ^= 1u << s;
      if (__any_sync(0xffffffffu, !got)) break;
      zero_ragged(smem + s * kStageBytes, w, (BM + BN / 2) / 64);
      if (lane == 0) mbar_arrive_cluster(ragged0 + s * static_cast<uint32_t>(sizeof(uint64_t)));
    }
  } else {
    // -------------------------------------------------------------- output
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    uint8_t* stg = out_stage + quarter * kOutWarpBytes;
    uint32_t j = 0, seq = 0;
    int g = 0;
    for (int t = first; t < tiles; t += stride) {
      const Item w = item_of<MODE, PAIR>(p, tab, t, tiles_n, num_kb, rank, g);
      const int rows = min(w.rows - quarter * 32, 32);
      const int64_t row_base =
          (kGrad ? w.m0 : w.row0) + quarter * 32;
      void* D = p.D;
      if (kGrad) {
        const int64_t at = w.group * p.stride_d;
        D = p.d_type == GEMM_OUT_F32 ? static_cast<void*>(static_cast<float*>(D) + at)
                                     : static_cast<void*>(static_cast<__nv_bfloat16*>(D) + at);
      }
      if (w.num_kb == 0) {
        if (p.d_tma) {
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
        }
        if (rows > 0) write_tile(p, stg, 0.0f, D, row_base, rows, w.tn * BN, Zeros{});
        continue;
      }
      const uint32_t ab = j & 1u, ar = j >> 1;
      ++j;
      const bool ok = mbar_wait_late(&tail->tmem_full[ab], ar & 1u, abort_flag, p.err);
      // Leave together if a wait ran out anywhere (see named_bar_any).
      if (named_bar_any(kOutBarAny, kOutThreads, !ok)) break;
      tc_fence_after_sync();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + ab * BN;
      // a piece with rows of another group in it (not the weight gradient's:
      // its matrices end where the map clips) is written row by row
      int written = 0;
      if (p.d_tma && rows > 0 && (kGrad || rows == 32))
        written = write_tma(p, &tmD, taddr, smem_u32(stg), seq, static_cast<int>(row_base),
                            kGrad ? w.group : 0, w.tn * BN);
      if (rows > 0 && written < BN / 32 && w.tn * BN + written * 32 < p.N) {
        if (p.d_tma) {  // the copies from the staging area have read it
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
        }
        write_tile(p, stg, p.alpha, D, row_base, rows, w.tn * BN, FromTmem{taddr}, written);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          mbar_arrive_remote(mapa_shared(smem_u32(&tail->tmem_empty[ab]), 0));
        else
          mbar_arrive(&tail->tmem_empty[ab]);
      }
    }
  }
  if (warp >= 2 && p.d_tma && lane == 0) bulk_wait_group_all();  // the stores are complete
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  // Neither CTA of a pair releases TMEM or exits while the pair's MMAs or
  // copies can still touch it.
  if (PAIR) cluster_sync();
  tc_fence_after_sync();
  if (warp == 1) {
    if (PAIR)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
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
  if (ops_allow_smem<grouped_kernel<kForward, true>>(kSmemBytes) == cudaSuccess) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, grouped_kernel<kForward, true>, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  if (n > 0) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

struct Operand {
  const void* p;
  int64_t rows, cols, ld;
  int64_t count, stride;
};

// Row pitch in a tensor map.  A single row has none of its own: any will do.
int64_t map_pitch(const Operand& o) { return o.rows == 1 ? (o.cols + 7) / 8 * 8 : o.ld; }

bool tma_describes(const Operand& o) {
  return !ops_misaligned(o.p, 16) && map_pitch(o) % 8 == 0 &&
         (o.count == 1 || o.stride % 8 == 0);
}

int64_t staged_bytes(const Operand& o) {
  return (o.count * o.rows * ((o.cols + 7) / 8 * 8) * 2 + 255) / 256 * 256;
}

// A copy that TMA can describe: rows padded to 16 bytes, matrices dense.
__global__ void stage_bf16_kernel(const uint16_t* src, int64_t ld, int64_t stride, uint16_t* dst,
                                  int64_t ld2, int64_t rows, int64_t cols, int64_t count) {
  grid_dependency_wait();
  const int64_t pieces = ld2 / 8;
  const int64_t total = count * rows * pieces;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t line = i / pieces, c = (i - line * pieces) * 8;
    const int64_t m = line / rows, r = line - m * rows;
    const uint16_t* s = src + m * stride + r * ld + c;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) w[j >> 1] |= static_cast<uint32_t>(s[j]) << (16 * (j & 1));
    *reinterpret_cast<uint4*>(dst + line * ld2 + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

cudaError_t stage(Operand& o, uint8_t* to, int num_sms, cudaStream_t s) {
  const int64_t ld2 = (o.cols + 7) / 8 * 8;
  const int64_t total = o.count * o.rows * (ld2 / 8);
  const int64_t want = (total + 255) / 256, fit = static_cast<int64_t>(num_sms) * 8;
  const uint16_t* src = static_cast<const uint16_t*>(o.p);
  uint16_t* dst = reinterpret_cast<uint16_t*>(to);
  const int64_t ld = o.ld, stride = o.stride, rows = o.rows, cols = o.cols, count = o.count;
  const cudaError_t e =
      ops_launch<stage_bf16_kernel>(dim3(static_cast<unsigned>(want < fit ? want : fit)), 256, 0, 1,
                                    s, src, ld, stride, dst, ld2, rows, cols, count);
  o.p = dst;
  o.ld = ld2;
  o.stride = o.rows * ld2;
  return e;
}

// The map of D for write_tma: matrices of rows x cols.
bool encode_output(CUtensorMap* tm, void* D, int d_type, int64_t rows, int64_t cols, int64_t ld,
                   int64_t count, int64_t stride) {
  const int bytes = float_type_bytes(d_type);
  const int64_t piece = 16 / bytes;
  if (rows == 1) ld = (cols + piece - 1) / piece * piece;  // a single row's pitch is never used
  if (ops_misaligned(D, 16) || ld * bytes % 16 != 0 || (count > 1 && stride * bytes % 16 != 0))
    return false;
  const int64_t dims[3] = {cols, rows, count};
  const int64_t strides[2] = {ld * bytes, (count > 1 ? stride : ld * rows) * bytes};
  const uint32_t box[3] = {static_cast<uint32_t>(64 / bytes), 32, 1};
  return abi_encode_tiled(tm, d_type == GEMM_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                          3, D, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

bool bad_dim(int64_t v) { return v < 0 || v > kOpsMaxDim; }
bool bad_tiled(int64_t v) { return v < 0 || v > kOpsMaxTiled; }

// Stages the operands that TMA cannot describe and encodes the maps (of B with
// rank_b dimensions); box_a and box_b: elements along the innermost and the
// next dimension.
gemm_status_t operands(Operand a, Operand b, int rank_b, const uint32_t (&box_a)[2], const uint32_t (&box_b)[2],
                       int num_sms, cudaStream_t s, std::unique_lock<std::mutex>& lock,
                       CUtensorMap* tmA, CUtensorMap* tmB) {
  const int64_t need_a = tma_describes(a) ? 0 : staged_bytes(a);
  const int64_t need_b = tma_describes(b) ? 0 : staged_bytes(b);
  if (need_a + need_b > 0) {
    uint8_t* buf = nullptr;
    const gemm_status_t st = abi_stage(s, need_a + need_b, lock, &buf);
    if (st != GEMM_OK) return st;
    cudaError_t e = need_a > 0 ? stage(a, buf, num_sms, s) : cudaSuccess;
    if (e == cudaSuccess && need_b > 0) e = stage(b, buf + need_a, num_sms, s);
    if (e != cudaSuccess) return abi_from_cuda(e);
  }
  const int64_t da[2] = {a.cols, a.rows}, ta[1] = {map_pitch(a) * 2};
  const int64_t db[3] = {b.cols, b.rows, b.count};
  const int64_t tb[2] = {map_pitch(b) * 2,
                         (b.count > 1 ? b.stride : map_pitch(b) * b.rows) * 2};
  const uint32_t bb[3] = {box_b[0], box_b[1], 1};
  if (!abi_encode_tiled(tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.p, da, ta, box_a) ||
      !abi_encode_tiled(tmB, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank_b, b.p, db, tb, bb))
    return GEMM_ERR_LAUNCH;
  return GEMM_OK;
}

}  // namespace
}  // namespace g12

using namespace g12;

extern "C" {

gemm_status_t gemm_bf16gemm_grouped(int64_t G, const int32_t* offsets, int64_t rows, int64_t N,
                                    int64_t K, float alpha, const void* A, int64_t lda,
                                    const void* B, int64_t ldb, int64_t stride_b, int transpose_b,
                                    float beta, void* D, int64_t ldd, int d_type, void* stream) {
  const int d_bytes = float_type_bytes(d_type);
  if (bad_dim(G) || bad_tiled(rows) || bad_tiled(N) || bad_tiled(K) || d_bytes == 0)
    return GEMM_ERR_INVALID_VALUE;
  if (G == 0 || rows == 0 || N == 0) return GEMM_OK;
  const bool product = K > 0 && alpha != 0.0f;
  if (offsets == nullptr || ops_misaligned(offsets, 4) || D == nullptr || ldd < N || bad_dim(ldd) ||
      ops_misaligned(D, d_bytes))
    return GEMM_ERR_INVALID_VALUE;
  const int64_t brows = transpose_b ? N : K, bcols = transpose_b ? K : N;
  if (product) {
    if (A == nullptr || B == nullptr || lda < K || bad_dim(lda) || ldb < bcols || bad_dim(ldb) ||
        (G > 1 && stride_b < (brows - 1) * ldb + bcols))
      return GEMM_ERR_INVALID_VALUE;
    if (ops_misaligned(A, 2) || ops_misaligned(B, 2)) return GEMM_ERR_MISALIGNED;
  }
  if (G > kMaxGroups) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GroupedArgs a{};
  a.rows = static_cast<int>(rows);
  a.N = static_cast<int>(N);
  a.K = static_cast<int>(K);
  a.groups = static_cast<int>(G);
  a.offsets = offsets;
  a.alpha = alpha;
  a.beta = beta;
  a.D = D;
  a.ldd = ldd;
  a.d_type = d_type;
  a.d_vec = !ops_misaligned(D, 16) && (rows == 1 || ldd % (16 / d_bytes) == 0);
  // CTA pairs where their rounds of tiles take less time: a k-block takes a
  // pair 512 cycles (its MMAs) and a single CTA 768 (operands through shared
  // memory), and each group's last row tile is half full on average.
  const int64_t tiles_n = (N + BN - 1) / BN;
  const int64_t tiles_1 = (rows / BM + (G + 1) / 2) * tiles_n;
  const int64_t tiles_2 = (rows / (2 * BM) + (G + 1) / 2) * tiles_n;
  const int pairs = max_pairs();
  const bool pair = pairs > 0 && 2 * ((tiles_2 + pairs - 1) / pairs) < 3 * ((tiles_1 + sms - 1) / sms);
  a.tile_rows = pair ? 2 * BM : rows > 64 ? 128 : (rows > 32 ? 64 : (rows > 16 ? 32 : 16));
  a.band = 8;
  a.product = product ? 1 : 0;
  a.err = err;
  std::unique_lock<std::mutex> lock;
  CUtensorMap tmA{}, tmB{}, tmD{};
  a.d_tma = product && beta == 0.0f && encode_output(&tmD, D, d_type, rows, N, ldd, 1, 0);
  if (product) {
    const uint32_t box_a[2] = {BK, static_cast<uint32_t>(pair ? BM : a.tile_rows)};
    const uint32_t box_b[2] = {BK, static_cast<uint32_t>(transpose_b ? b_cols(pair) : BK)};
    st = operands(Operand{A, rows, K, lda, 1, 0}, Operand{B, brows, bcols, ldb, G, stride_b}, 3,
                  box_a, box_b, sms, s, lock, &tmA, &tmB);
    if (st != GEMM_OK) return st;
  }
  const int64_t row_tiles = (rows + a.tile_rows - 1) / a.tile_rows + (G < rows ? G : rows);
  const int64_t tiles = row_tiles * tiles_n;
  if (tiles + sms > kOpsMaxDim) return GEMM_ERR_UNSUPPORTED;
  if (pair) {
    const dim3 grid(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
    return abi_from_cuda(
        transpose_b
            ? ops_launch<grouped_kernel<kTransB, true>>(grid, kThreads, kSmemBytes, 2, s, a, tmA, tmB,
                                                           tmD)
            : ops_launch<grouped_kernel<kForward, true>>(grid, kThreads, kSmemBytes, 2, s, a, tmA, tmB,
                                                           tmD));
  }
  const dim3 grid(static_cast<unsigned>(tiles < sms ? tiles : sms));
  return abi_from_cuda(
      transpose_b
          ? ops_launch<grouped_kernel<kTransB, false>>(grid, kThreads, kSmemBytes, 1, s, a, tmA, tmB,
                                                           tmD)
          : ops_launch<grouped_kernel<kForward, false>>(grid, kThreads, kSmemBytes, 1, s, a, tmA, tmB,
                                                           tmD));
}

gemm_status_t gemm_bf16gemm_grouped_wgrad(int64_t G, const int32_t* offsets, int64_t rows,
                                          int64_t N, int64_t K, float alpha, const void* A,
                                          int64_t lda, const void* dD, int64_t lddd, float beta,
                                          void* dB, int64_t ldb, int64_t stride_b, int d_type,
                                          void* stream) {
  const int d_bytes = float_type_bytes(d_type);
  if (bad_dim(G) || bad_tiled(rows) || bad_tiled(N) || bad_tiled(K) || d_bytes == 0)
    return GEMM_ERR_INVALID_VALUE;
  if (G == 0 || N == 0 || K == 0) return GEMM_OK;
  const bool product = rows > 0 && alpha != 0.0f;
  if (offsets == nullptr || ops_misaligned(offsets, 4) || dB == nullptr || ldb < N ||
      bad_dim(ldb) || ops_misaligned(dB, d_bytes) || (G > 1 && stride_b < (K - 1) * ldb + N))
    return GEMM_ERR_INVALID_VALUE;
  if (product) {
    if (A == nullptr || dD == nullptr || lda < K || bad_dim(lda) || lddd < N || bad_dim(lddd))
      return GEMM_ERR_INVALID_VALUE;
    if (ops_misaligned(A, 2) || ops_misaligned(dD, 2)) return GEMM_ERR_MISALIGNED;
  }
  const int64_t tiles_n = (N + BN - 1) / BN;
  const int64_t tiles_1 = G * ((K + BM - 1) / BM) * tiles_n;
  const int64_t tiles_2 = G * ((K + 2 * BM - 1) / (2 * BM)) * tiles_n;
  if (G > kMaxGroups || tiles_1 > kOpsMaxDim / 2) return GEMM_ERR_UNSUPPORTED;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GroupedArgs a{};
  a.rows = static_cast<int>(rows);
  a.M = static_cast<int>(K);
  a.N = static_cast<int>(N);
  a.K = 0;
  a.groups = static_cast<int>(G);
  a.offsets = offsets;
  a.alpha = alpha;
  a.beta = beta;
  a.D = dB;
  a.ldd = ldb;
  a.stride_d = stride_b;
  a.d_type = d_type;
  a.d_vec = !ops_misaligned(dB, 16) && (K == 1 || ldb % (16 / d_bytes) == 0) &&
            (G == 1 || stride_b % (16 / d_bytes) == 0);
  a.tile_rows = BM;
  a.band = 8;
  a.product = product ? 1 : 0;
  a.err = err;
  std::unique_lock<std::mutex> lock;
  CUtensorMap tmA{}, tmB{}, tmD{};
  a.d_tma = product && beta == 0.0f && encode_output(&tmD, dB, d_type, K, N, ldb, G, stride_b);
  if (product) {
    const uint32_t box[2] = {64, BK};
    st = operands(Operand{A, rows, K, lda, 1, 0}, Operand{dD, rows, N, lddd, 1, 0}, 2, box, box, sms,
                  s, lock, &tmA, &tmB);
    if (st != GEMM_OK) return st;
  }
  // CTA pairs as for the forward product, but from 512 rows a group on: before
  // that writing the matrices is most of the time, and a pair's tile of 256 rows
  // of them leaves in one piece (8192 rows, 1024 x 2048: 16 groups 33.0 us
  // against 36.2, 64 groups of 78 rows, 512 x 1024, 32.2 against 28.4).
  const int pairs = max_pairs();
  if (pairs > 0 && rows >= 512 * G &&
      2 * ((tiles_2 + pairs - 1) / pairs) < 3 * ((tiles_1 + sms - 1) / sms)) {
    const dim3 grid(static_cast<unsigned>(2 * (tiles_2 < pairs ? tiles_2 : pairs)));
    return abi_from_cuda(ops_launch<grouped_kernel<kWeightGrad, true>>(
        grid, kRaggedThreads, kSmemBytes, 2, s, a, tmA, tmB, tmD));
  }
  const dim3 grid(static_cast<unsigned>(tiles_1 < sms ? tiles_1 : sms));
  return abi_from_cuda(ops_launch<grouped_kernel<kWeightGrad, false>>(
      grid, kThreads, kSmemBytes, 1, s, a, tmA, tmB, tmD));
}

}  // extern "C"
