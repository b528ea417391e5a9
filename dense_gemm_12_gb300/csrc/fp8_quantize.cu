// fp8_quantize.cu -- a matrix, or its transpose, in fp8 (E4M3) with an fp32
// scale per 1 x 128 or 128 x 128 block:
//
//     a = max |x| over the block's finite values
//     scale = max(a / 448, 2^-126)        q = e4m3(x / scale)
//
// Bound by memory: every value is read once, held in registers over its
// block's maximum, and written once.
#include <type_traits>

#include "ops.cuh"

namespace g12 {
namespace {

struct QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;  // of x
  int x_type;
  uint8_t* q;
  int64_t ldq;
  float* scales;
  int64_t ld_scales;
  int q_vec;   // rows of q can be written in 16-byte pieces
  int stages;  // tile kernel: tiles in the ring (0: x cannot be read by TMA)
  uint32_t* err;
};

// 1 x 128 blocks along the rows of x.  A thread's kRowUnits units are loaded
// before the first is reduced.  Three forms: 16 consecutive elements a thread
// and 8 lanes a block (two quotients and the maximum's shuffles per block are
// what the instructions go to: 8192 x 8192 in bf16 takes 38 us, 5.3 TB/s, and
// took 52 us with 8 elements a thread); 8 consecutive elements; and, for rows
// that cannot be moved in vectors, 8 elements 16 apart, which keeps consecutive
// lanes on consecutive elements.
enum RowForm : int { kStrided8 = 0, kVec8 = 1, kVec16 = 2 };
constexpr int kRowUnits = 2;

template <int FORM, int T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __grid_constant__ QuantArgs a) {
  constexpr bool VEC = FORM != kStrided8;
  constexpr int E = FORM == kVec16 ? 16 : 8, LANES = kFp8Block / E, PER_CTA = 256 / LANES;
  grid_dependency_wait();
  grid_launch_dependents();
  const int l = threadIdx.x % LANES;
  const int64_t kb = (a.cols + kFp8Block - 1) / kFp8Block;
  const int64_t units = a.rows * kb;
  const bool small = units < (int64_t{1} << 31);  // 32-bit quotients
  const int64_t stride = static_cast<int64_t>(gridDim.x) * PER_CTA;
  // every lane of a warp takes the same number of turns: the shuffles below
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * PER_CTA; base < units;
       base += stride * kRowUnits) {
    Raw8<T> raw[kRowUnits][E / 8];
    int64_t row[kRowUnits], blk[kRowUnits];
    bool in[kRowUnits];
#pragma unroll
    for (int u = 0; u < kRowUnits; ++u) {
      const int64_t unit = base + u * stride + threadIdx.x / LANES;
      in[u] = unit < units;
      row[u] = !in[u] ? 0 : small ? static_cast<uint32_t>(unit) / static_cast<uint32_t>(kb) : unit / kb;
      blk[u] = in[u] ? unit - row[u] * kb : 0;
      const int64_t c0 = blk[u] * kFp8Block;
      const int n = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(kFp8Block)));
      const int c = VEC ? l * E : l;
#pragma unroll
      for (int h = 0; h < E / 8; ++h)
        raw[u][h] = load8<VEC, T>(a.x, a.x_type, row[u] * a.ldx + c0, c + 8 * h, n, in[u] && c < n);
    }
#pragma unroll
    for (int u = 0; u < kRowUnits; ++u) {
      float v[E];
#pragma unroll
      for (int h = 0; h < E / 8; ++h) {
        float w[8];
        widen8<VEC, T>(raw[u][h], a.x_type, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = w[i];
      }
      const float amax = block_amax<LANES>(v);
      if (!in[u]) continue;
      const float f = fp8_factor(amax);
      const int64_t c0 = blk[u] * kFp8Block;
      uint8_t* q = a.q + row[u] * a.ldq + c0;
      const int n = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(kFp8Block)));
      if constexpr (VEC) {
        uint32_t w[E / 4];
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
          w[i] = pack_e4m3(v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
        if (l * E < n) {
          if constexpr (E == 16)
            *reinterpret_cast<uint4*>(q + l * E) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2*>(q + l * E) = make_uint2(w[0], w[1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (l + 16 * i < n)
            q[l + 16 * i] = __nv_cvt_float_to_fp8(v[i] * f, __NV_SATFINITE, __NV_E4M3);
      }
      if (l == 0) a.scales[blk[u] * a.ld_scales + row[u]] = fp8_scale(amax);
    }
  }
}

template <int FORM, int T>
cudaError_t launch_rows(const QuantArgs& a, int num_sms, cudaStream_t s) {
  constexpr int per_cta = 256 / (kFp8Block / (FORM == kVec16 ? 16 : 8));
  const int64_t units = a.rows * ((a.cols + kFp8Block - 1) / kFp8Block);
  // few units: one per group of lanes; many: kRowUnits each, up to eight CTAs per SM
  int64_t ctas = (units + per_cta - 1) / per_cta;
  const int64_t fit = static_cast<int64_t>(num_sms) * 8;
  if (ctas > fit) {
    const int64_t fewer = (ctas + kRowUnits - 1) / kRowUnits;
    ctas = fewer > fit ? fit : fewer;
  }
  return ops_launch<quantize_rows_kernel<FORM, T>>(dim3(static_cast<unsigned>(ctas)), 256, 0, 1, s, a);
}

// One 128 x 128 tile of x per CTA turn, through shared memory.  Where TMA can
// describe x, one thread keeps `stages` tiles on their way (zeros outside x);
// a thread waiting for its own 16-byte loads instead left too few in flight
// (8192 x 8192 in bf16: 49 us, against 33 with the ring).  Otherwise each warp
// reads 16 rows' elements with consecutive lanes, all before the first is used,
// and through L1, since neighbouring loads share sectors (3000 x 1999: 8.5 us;
// 9.5 in two halves and streaming).  Thread (rg, cg) = (t / 16, t % 16) then holds rows
// 8 rg .. 8 rg + 7 of columns 8 cg .. 8 cg + 7.  The transposed output goes
// through shared memory again: eight values down a column make one 8-byte
// piece of an output row; a row's 16 pieces are XOR-swizzled by its 8-column
// group, so that the 16 lanes of a write fall in distinct banks.
constexpr int kTile = 128;
constexpr int kMaxTileStages = 4;

template <bool TILES, bool TRANSPOSE, int T>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const __grid_constant__ QuantArgs a,
                                                            const __grid_constant__ CUtensorMap tmX) {
  __shared__ __align__(16) uint8_t turned[TRANSPOSE ? 128 * 128 : 16];
  __shared__ float colmax[TILES ? 1 : 8][TILES ? 1 : 128];
  __shared__ __align__(16) float factor[TILES ? 4 : 128];
  __shared__ float tilemax[8];
  __shared__ uint64_t full[kMaxTileStages];
  __shared__ int abort_flag;
  extern __shared__ __align__(128) uint8_t dyn_smem[];
  uint8_t* const ring = align_smem<128>(dyn_smem);
  constexpr int kElem = T == GEMM_OUT_BF16 ? 2 : 4;
  constexpr int kTileBytes = kTile * kTile * kElem;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int cg = t & 15, rg = t >> 4;
  const int64_t tiles_c = (a.cols + 127) / 128, tiles_r = (a.rows + 127) / 128;
  const int64_t tiles = tiles_r * tiles_c;
  auto fetch = [&](int64_t tile, int s) {
    const int64_t tr = tile / tiles_c, tc = tile - tr * tiles_c;
    mbar_arrive_expect_tx(&full[s], kTileBytes);
    tma_load_2d(ring + s * kTileBytes, &tmX, static_cast<int>(tc * kTile),
                static_cast<int>(tr * kTile), &full[s]);
  };
  if (a.stages > 0) {
    if (t == 0) {
      for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
      abort_flag = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (a.stages > 0 && t == 0)
    for (int s = 0; s < a.stages; ++s) {
      const int64_t tile = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
      if (tile < tiles) fetch(tile, s);
    }
  int slot = 0;
  uint32_t parity = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t tr = tile / tiles_c, tc = tile - tr * tiles_c;
    const int64_t r0 = tr * 128 + rg * 8, c0 = tc * 128 + cg * 8;
    if (a.stages > 0) {
      mbar_wait_late(&full[slot], parity, &abort_flag, a.err);
    } else {
      // rows warp, warp + 8, ...; lane l takes columns l, l + 32, l + 64, l + 96
      using E = std::conditional_t<T == GEMM_OUT_BF16, uint16_t, uint32_t>;
      E* to = reinterpret_cast<E*>(ring);
      const E* from = static_cast<const E*>(a.x) + tc * kTile;
      const int n = static_cast<int>(min(a.cols - tc * kTile, static_cast<int64_t>(kTile)));
      E v[16][4];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int64_t r = tr * kTile + i * 8 + warp;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[i][j] = r < a.rows && lane + 32 * j < n ? __ldg(from + r * a.ldx + lane + 32 * j) : E(0);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) to[(i * 8 + warp) * kTile + lane + 32 * j] = v[i][j];
      __syncthreads();
    }
    float v[8][8];  // [row][column]
    {
      const uint8_t* from = ring + slot * kTileBytes + rg * 8 * (kTile * kElem);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        widen_vec<T>(load8_smem<T>(from + i * (kTile * kElem), cg * 8), T, v[i]);
    }
    float f[8];  // factor of each column
    if (TILES) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(v[i][j]));
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
      if (lane == 0) tilemax[warp] = amax;
      __syncthreads();
      amax = tilemax[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) amax = fmaxf(amax, tilemax[i]);
      const float one = fp8_factor(amax);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = one;
      // scale (k-block, row block) of the output: its k runs along its columns
      if (t == 0)
        a.scales[TRANSPOSE ? tr * a.ld_scales + tc : tc * a.ld_scales + tr] = fp8_scale(amax);
    } else {
      // 1 x 128 blocks of the transpose: one per column of the tile
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(v[i][j]));
        f[j] = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      }
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) colmax[warp][cg * 8 + j] = f[j];
      }
      __syncthreads();
      if (t < 128) {  // one thread per column: the quotients are long
        float m = colmax[0][TILES ? 0 : t];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = fmaxf(m, colmax[TILES ? 0 : w][TILES ? 0 : t]);
        const int64_t c = tc * 128 + t;
        if (c < a.cols) a.scales[tr * a.ld_scales + c] = fp8_scale(m);
        factor[TILES ? 0 : t] = fp8_factor(m);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = factor[TILES ? 0 : cg * 8 + j];
    }
    // every thread has read the tile (the barrier among the maxima above)
    if (a.stages > 0) {
      const int64_t next = tile + static_cast<int64_t>(a.stages) * gridDim.x;
      if (t == 0 && next < tiles && !*const_cast<volatile int*>(&abort_flag)) fetch(next, slot);
      if (++slot == a.stages) {
        slot = 0;
        parity ^= 1u;
      }
    }
    if constexpr (!TRANSPOSE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r0 + i >= a.rows) break;
        uint8_t* q = a.q + (r0 + i) * a.ldq + c0;
        const uint2 w = make_uint2(
            pack_e4m3(v[i][0] * f[0], v[i][1] * f[1], v[i][2] * f[2], v[i][3] * f[3]),
            pack_e4m3(v[i][4] * f[4], v[i][5] * f[5], v[i][6] * f[6], v[i][7] * f[7]));
        if (a.q_vec && c0 + 8 <= a.cols) {
          *reinterpret_cast<uint2*>(q) = w;
        } else {
          const uint64_t all = w.x | static_cast<uint64_t>(w.y) << 32;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c0 + j < a.cols) q[j] = static_cast<uint8_t>(all >> (8 * j));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint2 w = make_uint2(
            pack_e4m3(v[0][j] * f[j], v[1][j] * f[j], v[2][j] * f[j], v[3][j] * f[j]),
            pack_e4m3(v[4][j] * f[j], v[5][j] * f[j], v[6][j] * f[j], v[7][j] * f[j]));
        *reinterpret_cast<uint2*>(turned + (cg * 8 + j) * 128 + ((rg ^ cg) << 3)) = w;
      }
      __syncthreads();
      // eight lanes write an output row's 128 bytes, 32 rows per turn
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 32 + (t >> 3);  // column of the tile
        const int piece = t & 7;
        const int swz = row >> 3;
        const uint2 lo = *reinterpret_cast<const uint2*>(turned + row * 128 + (((2 * piece) ^ swz) << 3));
        const uint2 hi =
            *reinterpret_cast<const uint2*>(turned + row * 128 + (((2 * piece + 1) ^ swz) << 3));
        const int64_t orow = tc * 128 + row, ocol = tr * 128 + piece * 16;
        if (orow >= a.cols || ocol >= a.rows) continue;
        uint8_t* q = a.q + orow * a.ldq + ocol;
        if (a.q_vec && ocol + 16 <= a.rows) {
          *reinterpret_cast<uint4*>(q) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (ocol + j < a.rows) q[j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
    __syncthreads();  // `turned` and the maxima are rewritten by the next tile
  }
  if (a.stages > 0 && t == 0 && abort_flag) {
    // after a wait ran out: the copies in flight land before the CTA leaves
    for (int i = 0; i < a.stages; ++i) {
      mbar_drain_wait(&full[slot], parity);
      if (++slot == a.stages) {
        slot = 0;
        parity ^= 1u;
      }
    }
  }
}

template <int T>
cudaError_t launch_tiles(const QuantArgs& a, const CUtensorMap& tmX, int block, bool transpose,
                         int num_sms, cudaStream_t s) {
  const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
  const int64_t fit = static_cast<int64_t>(num_sms) * 2;  // the kernel's registers
  const dim3 grid(static_cast<unsigned>(tiles < fit ? tiles : fit));
  const size_t smem =
      128 + static_cast<size_t>(a.stages > 0 ? a.stages : 1) * kTile * kTile * (T == GEMM_OUT_BF16 ? 2 : 4);
  if (block == GEMM_BLOCK_ROWS)
    return ops_launch<quantize_tile_kernel<false, true, T>>(grid, 256, smem, 1, s, a, tmX);
  if (transpose) return ops_launch<quantize_tile_kernel<true, true, T>>(grid, 256, smem, 1, s, a, tmX);
  return ops_launch<quantize_tile_kernel<true, false, T>>(grid, 256, smem, 1, s, a, tmX);
}

}  // namespace
}  // namespace g12

using namespace g12;

extern "C" gemm_status_t gemm_fp8_quantize(int64_t rows, int64_t cols, const void* x, int64_t ldx,
                                           int x_type, int block, int transpose, void* q,
                                           int64_t ldq, float* scales, int64_t ld_scales,
                                           void* stream) {
  const int bytes = float_type_bytes(x_type);
  if (rows < 0 || cols < 0 || rows > kOpsMaxDim || cols > kOpsMaxDim || bytes == 0)
    return GEMM_ERR_INVALID_VALUE;
  if (block != GEMM_BLOCK_ROWS && block != GEMM_BLOCK_TILES) return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_OK;
  const int64_t qrows = transpose ? cols : rows, qcols = transpose ? rows : cols;
  const int64_t srows = block == GEMM_BLOCK_TILES ? (qrows + 127) / 128 : qrows;
  if (x == nullptr || q == nullptr || scales == nullptr || ldx < cols || ldq < qcols ||
      ld_scales < srows || ldx > kOpsMaxDim || ldq > kOpsMaxDim || ld_scales > kOpsMaxDim ||
      ops_misaligned(x, bytes) || ops_misaligned(scales, 4))
    return GEMM_ERR_INVALID_VALUE;
  int sms = 0;
  uint32_t* err = nullptr;
  const gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  QuantArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.x_type = x_type;
  a.q = static_cast<uint8_t*>(q);
  a.ldq = ldq;
  a.scales = scales;
  a.ld_scales = ld_scales;
  const bool x_vec = !ops_misaligned(x, 16) && ldx % (16 / bytes) == 0;
  a.err = err;
  a.q_vec = !ops_misaligned(q, 16) && ldq % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (block == GEMM_BLOCK_ROWS && !transpose) {
    const bool q16 = !ops_misaligned(q, 16) && ldq % 16 == 0;
    const bool q8 = !ops_misaligned(q, 8) && ldq % 8 == 0;
    const bool half = x_type == GEMM_OUT_BF16;
    cudaError_t e;
    if (x_vec && q16 && cols % 16 == 0)
      e = half ? launch_rows<kVec16, GEMM_OUT_BF16>(a, sms, s) : launch_rows<kVec16, GEMM_OUT_F32>(a, sms, s);
    else if (x_vec && q8 && cols % 8 == 0)
      e = half ? launch_rows<kVec8, GEMM_OUT_BF16>(a, sms, s) : launch_rows<kVec8, GEMM_OUT_F32>(a, sms, s);
    else
      e = launch_rows<kStrided8, kAnyType>(a, sms, s);
    return abi_from_cuda(e);
  }
  CUtensorMap tmX{};
  const int64_t dims[2] = {cols, rows}, pitch[1] = {ldx * bytes};
  const uint32_t box[2] = {kTile, kTile};
  if (x_vec && abi_encode_tiled(&tmX, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                                2, x, dims, pitch, box, CU_TENSOR_MAP_SWIZZLE_NONE))
    a.stages = bytes == 2 ? 2 : 1;
  return abi_from_cuda(x_type == GEMM_OUT_BF16
                           ? launch_tiles<GEMM_OUT_BF16>(a, tmX, block, transpose != 0, sms, s)
                           : launch_tiles<GEMM_OUT_F32>(a, tmX, block, transpose != 0, sms, s));
}
