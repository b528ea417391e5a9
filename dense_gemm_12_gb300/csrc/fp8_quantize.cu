// fp8_quantize.cu -- a matrix, or its transpose, in fp8 (E4M3) with an fp32
// scale per 1 x 128 or 128 x 128 block:
//
//     a = max |x| over the block's finite values
//     scale = max(a / 448, 2^-126)        q = e4m3(x / scale)
//
// Bound by memory: every value is read once, held in registers over its
// block's maximum, and written once.
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
  int x_vec;  // rows of x can be read in 16-byte pieces
  int q_vec;  // rows of q can be written in 16-byte pieces
};

// 1 x 128 blocks along the rows of x: 16 lanes take one block; the thread's
// kRowUnits units are loaded before the first is reduced.  Rows that cannot
// be moved in vectors are read and written by elements 16 apart, which keeps
// consecutive lanes on consecutive elements.
constexpr int kRowUnits = 4;

template <bool VEC, int T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const __grid_constant__ QuantArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int l = threadIdx.x & 15;
  const int64_t kb = (a.cols + kFp8Block - 1) / kFp8Block;
  const int64_t units = a.rows * kb;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 16;
  // every lane of a warp takes the same number of turns: the shuffles below
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * 16; base < units;
       base += stride * kRowUnits) {
    Raw8<T> raw[kRowUnits];
    int64_t row[kRowUnits], blk[kRowUnits];
    bool in[kRowUnits];
#pragma unroll
    for (int u = 0; u < kRowUnits; ++u) {
      const int64_t unit = base + u * stride + (threadIdx.x >> 4);
      in[u] = unit < units;
      row[u] = in[u] ? unit / kb : 0;
      blk[u] = in[u] ? unit - row[u] * kb : 0;
      const int64_t c0 = blk[u] * kFp8Block;
      const int n = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(kFp8Block)));
      const int c = VEC ? l * 8 : l;
      raw[u] = load8<VEC, T>(a.x, a.x_type, row[u] * a.ldx + c0, c, n, in[u] && c < n);
    }
#pragma unroll
    for (int u = 0; u < kRowUnits; ++u) {
      float v[8];
      widen8<VEC, T>(raw[u], a.x_type, v);
      const float amax = block_amax(v);
      if (!in[u]) continue;
      const float f = fp8_factor(amax);
      const int64_t c0 = blk[u] * kFp8Block;
      uint8_t* q = a.q + row[u] * a.ldq + c0;
      if (VEC) {
        if (c0 + l * 8 < a.cols)
          *reinterpret_cast<uint2*>(q + l * 8) =
              make_uint2(pack_e4m3(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                         pack_e4m3(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
      } else {
        const int n = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(kFp8Block)));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (l + 16 * i < n)
            q[l + 16 * i] = __nv_cvt_float_to_fp8(v[i] * f, __NV_SATFINITE, __NV_E4M3);
      }
      if (l == 0) a.scales[blk[u] * a.ld_scales + row[u]] = fp8_scale(amax);
    }
  }
}

// One 128 x 128 tile of x per CTA turn.  Thread (rg, cg) = (t / 16, t % 16)
// holds rows 8 rg .. 8 rg + 7 of columns 8 cg .. 8 cg + 7.  The transposed
// output goes through shared memory: eight values down a column make one
// 8-byte piece of an output row; a row's 16 pieces are XOR-swizzled by its
// 8-column group, so that the 16 lanes of a write fall in distinct banks.
template <bool TILES, bool TRANSPOSE, int T>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ __align__(16) uint8_t turned[TRANSPOSE ? 128 * 128 : 16];
  __shared__ float colmax[TILES ? 1 : 8][TILES ? 1 : 128];
  __shared__ float tilemax[8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int cg = t & 15, rg = t >> 4;
  const int64_t tiles_c = (a.cols + 127) / 128, tiles_r = (a.rows + 127) / 128;
  for (int64_t tile = blockIdx.x; tile < tiles_r * tiles_c; tile += gridDim.x) {
    const int64_t tr = tile / tiles_c, tc = tile - tr * tiles_c;
    const int64_t r0 = tr * 128 + rg * 8, c0 = tc * 128 + cg * 8;
    float v[8][8];  // [row][column]
    if (a.x_vec && c0 + 8 <= a.cols) {
      Raw8<T> raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        raw[i] = load8<true, T>(a.x, a.x_type, (r0 + i) * a.ldx + c0, 0, 8, r0 + i < a.rows);
#pragma unroll
      for (int i = 0; i < 8; ++i) widen8<true, T>(raw[i], a.x_type, v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = r0 + i < a.rows && c0 + j < a.cols
                        ? load1(a.x, T, (r0 + i) * a.ldx + c0 + j) : 0.0f;
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
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = colmax[0][cg * 8 + j];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = fmaxf(m, colmax[w][cg * 8 + j]);
        if (rg == 0 && c0 + j < a.cols) a.scales[tr * a.ld_scales + c0 + j] = fp8_scale(m);
        f[j] = fp8_factor(m);
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
}

template <int T>
cudaError_t launch_tiles(const QuantArgs& a, int block, bool transpose, dim3 grid, cudaStream_t s) {
  if (block == GEMM_BLOCK_ROWS)
    return ops_launch<quantize_tile_kernel<false, true, T>>(grid, 256, 0, 1, s, a);
  if (transpose) return ops_launch<quantize_tile_kernel<true, true, T>>(grid, 256, 0, 1, s, a);
  return ops_launch<quantize_tile_kernel<true, false, T>>(grid, 256, 0, 1, s, a);
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
  a.x_vec = !ops_misaligned(x, 16) && ldx % (16 / bytes) == 0;
  a.q_vec = !ops_misaligned(q, 16) && ldq % 16 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (block == GEMM_BLOCK_ROWS && !transpose) {
    const int64_t units = rows * ((cols + 127) / 128);
    // few units: one per half-warp; many: kRowUnits each, eight CTAs per SM
    int64_t ctas = (units + 15) / 16;
    const int64_t fit = static_cast<int64_t>(sms) * 8;
    if (ctas > fit) ctas = (ctas + kRowUnits - 1) / kRowUnits > fit ? fit : (ctas + kRowUnits - 1) / kRowUnits;
    const dim3 grid(static_cast<unsigned>(ctas));
    const bool vec = a.x_vec && cols % 8 == 0 && !ops_misaligned(q, 8) && ldq % 8 == 0;
    cudaError_t e;
    if (!vec)
      e = ops_launch<quantize_rows_kernel<false, kAnyType>>(grid, 256, 0, 1, s, a);
    else if (x_type == GEMM_OUT_BF16)
      e = ops_launch<quantize_rows_kernel<true, GEMM_OUT_BF16>>(grid, 256, 0, 1, s, a);
    else
      e = ops_launch<quantize_rows_kernel<true, GEMM_OUT_F32>>(grid, 256, 0, 1, s, a);
    return abi_from_cuda(e);
  }
  const int64_t tiles = ((rows + 127) / 128) * ((cols + 127) / 128);
  const int64_t fit = static_cast<int64_t>(sms) * 2;
  const dim3 grid(static_cast<unsigned>(tiles < fit ? tiles : fit));
  return abi_from_cuda(x_type == GEMM_OUT_BF16
                           ? launch_tiles<GEMM_OUT_BF16>(a, block, transpose != 0, grid, s)
                           : launch_tiles<GEMM_OUT_F32>(a, block, transpose != 0, grid, s));
}
