// int8_quantize.cu -- a matrix, or its transpose, in int8 with an fp32 scale for
// each row of the result:
//
//     a = max |x| over the row's finite values
//     scale = max(a / 127, 2^-126)        q = round(x / scale)
//
// Bound by memory.  Along the rows of x a value is read once, held over its
// row's maximum and written once; transposed, a row of the result is a column
// of x, and x is read twice: for the columns' maxima, then for the values.
// A value's byte is the same along the rows and transposed: the factor 127 / a and
// the value's product with it are each rounded to fp32 before the whole number.
// Measured: 8192 x 8192 in bf16 32.5 us (6.2 TB/s), transposed 95.
#include "norm.cuh"

namespace g12 {
namespace {

struct Int8QuantArgs {
  const void* x;
  int64_t rows, cols, ldx;  // of x
  int x_type;
  int8_t* q;
  int64_t ldq;
  float* scales;
  int tpr;       // threads per row (not transposed)
  int q_vec;     // transposed: rows of q can be written in 16-byte pieces
  float* part;   // transposed: maxima of `splits` parts of the rows, cols each
  int splits;
};

// C > 0: a row's values stay in registers, as they were loaded.  C == 0: rows
// longer than that are read twice.  One row (of a CTA with several, one each)
// and no loop: the next row's CTA is there while this one waits.
template <int C, bool VEC, int T>
__global__ void __launch_bounds__(kMaxThreads) int8_rows_kernel(const __grid_constant__ Int8QuantArgs a) {
  __shared__ uint32_t red[2][16], red_finite[2][16];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tpr = a.tpr;
  const int t = threadIdx.x % tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  if (row >= a.rows) return;  // whole warps: rows share no warp
  const int dim = static_cast<int>(a.cols);
  const int chunks = VEC ? dim / 8 : (dim + kFp8Block - 1) / kFp8Block * 16;
  // a chunk's largest magnitude; `only_finite`: infinities and NaN left out
  auto largest = [&](const Raw8<T>& raw, uint32_t& m, bool only_finite) {
    float v[8];
    widen8<VEC, T>(raw, a.x_type, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, only_finite ? __float_as_uint(finite_abs(v[i])) : abs_bits(v[i]));
  };
  auto write = [&](const Raw8<T>& raw, int c, float f, bool finite) {
    float v[8];
    widen8<VEC, T>(raw, a.x_type, v);
    write_s8<VEC>(a.q, a.ldq, row, c, dim, f, finite, v);
  };
  uint32_t amax = 0u;
  if constexpr (C > 0) {
    Raw8<T> raw[C];
    bool in[C];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int chunk = k * tpr + t, c = chunk_col<VEC>(chunk);
      in[k] = chunk < chunks && c < dim;
      raw[k] = load8<VEC, T>(a.x, a.x_type, row * a.ldx, c, dim, in[k]);
    }
#pragma unroll
    for (int k = 0; k < C; ++k) largest(raw[k], amax, false);
    amax = row_max_bits(amax, tpr, 0, red, 0);
    const bool finite = amax < kInfBits;
    if (!finite) {
      amax = 0u;
#pragma unroll
      for (int k = 0; k < C; ++k) largest(raw[k], amax, true);
      amax = row_max_bits(amax, tpr, 0, red_finite, 0);
    }
    const float f = s8_factor(__uint_as_float(amax));
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (in[k]) write(raw[k], chunk_col<VEC>(k * tpr + t), f, finite);
  } else {
    auto search = [&](bool only_finite) {
      uint32_t m = 0u;
      for (int chunk = t; chunk < chunks; chunk += tpr) {
        const int c = chunk_col<VEC>(chunk);
        largest(load8<VEC, T>(a.x, a.x_type, row * a.ldx, c, dim, c < dim), m, only_finite);
      }
      return m;
    };
    amax = row_max_bits(search(false), tpr, 0, red, 0);
    const bool finite = amax < kInfBits;
    if (!finite) amax = row_max_bits(search(true), tpr, 0, red_finite, 0);
    const float f = s8_factor(__uint_as_float(amax));
    for (int chunk = t; chunk < chunks; chunk += tpr) {
      const int c = chunk_col<VEC>(chunk);
      if (c < dim) write(load8<VEC, T>(a.x, a.x_type, row * a.ldx, c, dim, true), c, f, finite);
    }
  }
  if (t == 0) a.scales[row] = s8_scale(__uint_as_float(amax));
}

// Transposed, first: the largest magnitudes of 256 columns over every
// a.splits-th group of 64 rows.  Thread (rl, cl) = (t / 32, t % 32) takes eight
// columns of rows rl, rl + 8, ...
constexpr int kMaxRows = 64;

template <bool VEC, int T>
__global__ void __launch_bounds__(256) int8_column_max_kernel(const __grid_constant__ Int8QuantArgs a) {
  __shared__ float red[8][257];
  grid_dependency_wait();
  grid_launch_dependents();
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 256;
  const int n = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(256)));
  const int c = chunk_col<VEC>(cl);  // within the block
  float m[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t step = static_cast<int64_t>(a.splits) * kMaxRows;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * kMaxRows; r0 < a.rows; r0 += step) {
    Raw8<T> raw[kMaxRows / 8];
#pragma unroll
    for (int k = 0; k < kMaxRows / 8; ++k) {
      const int64_t r = r0 + k * 8 + rl;
      raw[k] = load8<VEC, T>(a.x, a.x_type, r * a.ldx + c0, c, n, r < a.rows && c < n);
    }
#pragma unroll
    for (int k = 0; k < kMaxRows / 8; ++k) {
      float v[8];
      widen8<VEC, T>(raw[k], a.x_type, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], finite_abs(v[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rl][VEC ? c + i : c + 16 * i] = m[i];
  __syncthreads();
  float v = red[0][threadIdx.x];
#pragma unroll
  for (int i = 1; i < 8; ++i) v = fmaxf(v, red[i][threadIdx.x]);
  if (static_cast<int>(threadIdx.x) < n)
    a.part[blockIdx.y * a.cols + c0 + threadIdx.x] = v;
}

// Then 128 x 128 tiles of x, turned around in shared memory: thread (rg, cg) =
// (t / 16, t % 16) holds rows 8 rg .. 8 rg + 7 of eight columns; eight values
// down a column make one 8-byte piece of a row of q, swizzled so that the 16
// lanes of a write fall in distinct banks.
template <bool VEC, int T>
__global__ void __launch_bounds__(256) int8_turn_kernel(const __grid_constant__ Int8QuantArgs a) {
  __shared__ __align__(16) uint8_t turned[128 * 128];
  __shared__ float factor[128];
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4;
  const int64_t tc = blockIdx.x, tr = blockIdx.y;
  const int64_t c0 = tc * 128;
  const int n = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(128)));
  auto swizzle = [](int col) { return (col ^ (col >> 3)) & 15; };
  const int c = VEC ? cg * 8 : cg;
  for (int64_t r0 = tr * 128; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.y) * 128) {
    Raw8<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + rg * 8 + i;
      raw[i] = load8<VEC, T>(a.x, a.x_type, r * a.ldx + c0, c, n, r < a.rows && c < n);
    }
    if (r0 == tr * 128 && t < 128) {
      float m = 0.0f;
      if (t < n) {
#pragma unroll 8
        for (int s = 0; s < a.splits; ++s) m = fmaxf(m, __ldcg(a.part + s * a.cols + c0 + t));
        if (tr == 0) a.scales[c0 + t] = s8_scale(m);
      }
      factor[t] = s8_factor(m);
    }
    __syncthreads();  // the factors are there; the previous tile has been read
    uint2 piece[8];
    {
      float v[8][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) widen8<VEC, T>(raw[i], a.x_type, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = factor[VEC ? c + j : c + 16 * j];
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = static_cast<uint32_t>(round_s8(v[i][j] * f));
        piece[j] = make_uint2(low_bytes(w[0], w[1], w[2], w[3]), low_bytes(w[4], w[5], w[6], w[7]));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = VEC ? c + j : c + 16 * j;
      *reinterpret_cast<uint2*>(turned + col * 128 + ((rg ^ swizzle(col)) << 3)) = piece[j];
    }
    __syncthreads();
    // eight lanes write a row's 128 bytes, 32 rows per turn
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = i * 32 + (t >> 3), p = t & 7;
      const int swz = swizzle(col);
      const uint2 lo = *reinterpret_cast<const uint2*>(turned + col * 128 + (((2 * p) ^ swz) << 3));
      const uint2 hi = *reinterpret_cast<const uint2*>(turned + col * 128 + (((2 * p + 1) ^ swz) << 3));
      const int64_t at = r0 + p * 16;
      if (col >= n || at >= a.rows) continue;
      uint8_t* q = reinterpret_cast<uint8_t*>(a.q) + (c0 + col) * a.ldq + at;
      if (a.q_vec && at + 16 <= a.rows) {
        *reinterpret_cast<uint4*>(q) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (at + j < a.rows) q[j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

template <bool VEC, int T>
cudaError_t launch_int8_rows(const Int8QuantArgs& a, const RowPlan& p, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>((a.rows + p.per_cta - 1) / p.per_cta));
  const int threads = p.tpr * p.per_cta;
  switch (p.chunks_per_thread) {
    case 1: return ops_launch<int8_rows_kernel<1, VEC, T>>(g, threads, 0, 1, s, a);
    case 2: return ops_launch<int8_rows_kernel<2, VEC, T>>(g, threads, 0, 1, s, a);
    case 4: return ops_launch<int8_rows_kernel<4, VEC, T>>(g, threads, 0, 1, s, a);
    default: return ops_launch<int8_rows_kernel<0, VEC, T>>(g, threads, 0, 1, s, a);
  }
}

template <bool VEC, int T>
cudaError_t launch_int8_turned(const Int8QuantArgs& a, cudaStream_t s) {
  const dim3 wide(static_cast<unsigned>((a.cols + 255) / 256), static_cast<unsigned>(a.splits));
  const cudaError_t e = ops_launch<int8_column_max_kernel<VEC, T>>(wide, 256, 0, 1, s, a);
  if (e != cudaSuccess) return e;
  const int64_t high = (a.rows + 127) / 128;
  const dim3 tiles(static_cast<unsigned>((a.cols + 127) / 128), static_cast<unsigned>(high < 65535 ? high : 65535));
  return ops_launch<int8_turn_kernel<VEC, T>>(tiles, 256, 0, 1, s, a);
}

}  // namespace
}  // namespace g12

using namespace g12;

extern "C" gemm_status_t gemm_int8_quantize(int64_t rows, int64_t cols, const void* x, int64_t ldx,
                                            int x_type, int transpose, int8_t* q, int64_t ldq,
                                            float* scales, void* stream) {
  const int bytes = float_type_bytes(x_type);
  if (rows < 0 || cols < 0 || rows > kOpsMaxDim || cols > kOpsMaxDim || bytes == 0)
    return GEMM_ERR_INVALID_VALUE;
  if (!transpose && cols > (int64_t{1} << 30)) return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (x == nullptr || q == nullptr || scales == nullptr || ldx < cols || ldq < (transpose ? rows : cols) ||
      ldx > kOpsMaxDim || ldq > kOpsMaxDim || ops_misaligned(x, bytes) || ops_misaligned(scales, 4))
    return GEMM_ERR_INVALID_VALUE;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  Int8QuantArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.ldx = ldx;
  a.x_type = x_type;
  a.q = q;
  a.ldq = ldq;
  a.scales = scales;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool x_vec = cols % 8 == 0 && !ops_misaligned(x, 16) && (rows == 1 || ldx % (16 / bytes) == 0);
  const bool half = x_type == GEMM_OUT_BF16;
  if (!transpose) {
    const bool vec = x_vec && !ops_misaligned(q, 8) && (rows == 1 || ldq % 8 == 0);
    const int64_t chunks = vec ? cols / 8 : (cols + kFp8Block - 1) / kFp8Block * 16;
    const RowPlan p = plan_rows(rows, chunks, sms, 4, 4);
    a.tpr = p.tpr;
    if (!vec) return abi_from_cuda(launch_int8_rows<false, kAnyType>(a, p, s));
    return abi_from_cuda(half ? launch_int8_rows<true, GEMM_OUT_BF16>(a, p, s)
                              : launch_int8_rows<true, GEMM_OUT_F32>(a, p, s));
  }
  a.q_vec = !ops_misaligned(q, 16) && (cols == 1 || ldq % 16 == 0);
  // as many parts of the rows as fill the GPU a few times, of 256 MB together
  const int64_t groups = (rows + kMaxRows - 1) / kMaxRows, across = (cols + 255) / 256;
  int64_t splits = (static_cast<int64_t>(sms) * 8 + across - 1) / across;
  if (splits > groups) splits = groups;
  if (splits > 64) splits = 64;
  while (splits > 1 && splits * cols > (int64_t{1} << 26)) splits /= 2;
  a.splits = static_cast<int>(splits);
  std::unique_lock<std::mutex> lock;
  st = abi_scratch(s, splits * cols, lock, &a.part);
  if (st != GEMM_OK) return st;
  if (!x_vec) return abi_from_cuda(launch_int8_turned<false, kAnyType>(a, s));
  return abi_from_cuda(half ? launch_int8_turned<true, GEMM_OUT_BF16>(a, s)
                            : launch_int8_turned<true, GEMM_OUT_F32>(a, s));
}
