// norm.cu -- root-mean-square norm with the residual's addition, its output
// in fp32, bf16 or fp8 with block scales, and its gradients.
//
//     h = x + r        v = mean_j h_j^2 + eps        y_j = h_j v^-1/2 w_j
//
// and, with dy the gradient of y, dr that of the stored h (the skip
// connection's), xh = h v^-1/2 and g = dy w:
//
//     dh = v^-1/2 (g - xh mean_j(g_j xh_j)) + dr        dw = sum_rows dy xh
//
// (dh is the gradient of x and of r alike.)  Both directions are bound by
// memory: a row is read once, kept in registers over the row's reduction, and
// written once.
#include "ops.cuh"

namespace g12 {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxRowsPerCta = 8;

struct NormArgs {
  int64_t rows;
  int dim;
  int tpr;  // threads per row, a multiple of 32; > 32: one row at a time per CTA
  gemm_rmsnorm_t p;
};

// Sum over the tpr threads of a row.  red: two rows of 16 floats that
// alternate from call to call (one barrier is then enough: a thread writes a
// row again only after the next call's barrier, which every reader of the
// previous values has passed).
__device__ __forceinline__ float row_sum(float v, int tpr, float (*red)[16], uint32_t& turn) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  if (tpr == 32) return v;
  float* mine = red[turn & 1u];
  ++turn;
  const int lane = threadIdx.x & 31;
  if (lane == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < (tpr >> 5) ? mine[lane] : 0.0f;
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return __shfl_sync(0xffffffffu, v, 0);
}

// Where the eight elements of chunk `chunk` lie: consecutive (VEC), or every
// 16th of a 128-column block from `c` on (see ops.cuh).
template <bool VEC>
__device__ __forceinline__ int chunk_col(int chunk) {
  return VEC ? chunk * 8 : (chunk >> 4) * kFp8Block + (chunk & 15);
}

template <bool VEC>
__device__ __forceinline__ void load_chunk(const void* p, int type, int64_t row_at, int c, int dim,
                                           float (&v)[8]) {
  if (VEC)
    load8_vec(p, type, row_at + c, v);
  else
    load8_strided(p, type, row_at, c, dim, v);
}

template <bool VEC>
__device__ __forceinline__ void store_chunk(void* p, int type, int64_t row_at, int c, int dim,
                                            const float (&v)[8]) {
  if (VEC)
    store8_vec(p, type, row_at + c, v);
  else
    store8_strided(p, type, row_at, c, dim, v);
}

// Weights are read again for every row and stay in L1 and L2.
template <bool VEC>
__device__ __forceinline__ void load_weight(const float* w, int c, int dim, float (&v)[8]) {
  if (VEC) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + c));
    const float4 b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + 16 * i < dim ? __ldg(w + c + 16 * i) : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int c, float (&h)[8]) {
  load_chunk<VEC>(a.p.x, a.p.x_type, row * a.p.ldx, c, a.dim, h);
  if (a.p.residual != nullptr) {
    float r[8];
    load_chunk<VEC>(a.p.residual, a.p.residual_type, row * a.p.ldr, c, a.dim, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += r[i];
  }
}

// Writes a chunk's outputs.  All 32 lanes call it together; lanes without
// elements (in == false) take part in the block's maximum only.
template <bool VEC>
__device__ __forceinline__ void write_y(const NormArgs& a, int64_t row, int c, bool in, float rstd,
                                        const float (&h)[8]) {
  float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (in) {
    load_weight<VEC>(a.p.weight, c, a.dim, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= h[i] * rstd;
    if (a.p.y != nullptr) store_chunk<VEC>(a.p.y, a.p.y_type, row * a.p.ldy, c, a.dim, y);
  }
  if (a.p.q == nullptr) return;
  // the 16 lanes of a 128-column block
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, finite_abs(y[i]));
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
  if (!in) return;
  const float f = fp8_factor(amax);
  uint8_t* q = static_cast<uint8_t*>(a.p.q) + row * a.p.ldq;
  if (VEC) {
    *reinterpret_cast<uint2*>(q + c) = make_uint2(pack_e4m3(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                                                  pack_e4m3(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < a.dim)
        q[c + 16 * i] = __nv_cvt_float_to_fp8(y[i] * f, __NV_SATFINITE, __NV_E4M3);
  }
  if ((threadIdx.x & 15) == 0) a.p.scales[(c >> 7) * a.p.ld_scales + row] = fp8_scale(amax);
}

// C > 0: a thread keeps its C chunks of 8 elements in registers, and the row
// is read once.  C == 0: rows longer than that are read twice (the second
// time mostly from L2).  Nothing of a row is written before its last read, so
// outputs may take the place of inputs element by element.
template <int C, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][16];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tpr = a.tpr;
  const int t = threadIdx.x % tpr;
  const int per_cta = blockDim.x / tpr;
  const int chunks = VEC ? a.dim / 8 : (a.dim + kFp8Block - 1) / kFp8Block * 16;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  uint32_t turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_cta + threadIdx.x / tpr; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * per_cta) {
    float ss = 0.0f;
    if (C > 0) {
      float h[C > 0 ? C : 1][8];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = 0.0f;
        if (chunk < chunks && c < a.dim) load_h<VEC>(a, row, c, h[k]);
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[k][i], h[k][i], ss);
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
        if (a.p.h != nullptr && chunk < chunks && c < a.dim)
          store_chunk<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, h[k]);
      }
      ss = row_sum(ss, tpr, red, turn);
      const float rstd = rsqrtf(fmaf(ss, inv_dim, a.p.eps));
      if (a.p.rstd != nullptr && t == 0) a.p.rstd[row] = rstd;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
        write_y<VEC>(a, row, c, chunk < chunks && c < a.dim, rstd, h[k]);
      }
    } else {
      for (int chunk = t; chunk < chunks; chunk += tpr) {
        const int c = chunk_col<VEC>(chunk);
        if (c >= a.dim) continue;
        float h[8];
        load_h<VEC>(a, row, c, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
      }
      ss = row_sum(ss, tpr, red, turn);
      const float rstd = rsqrtf(fmaf(ss, inv_dim, a.p.eps));
      if (a.p.rstd != nullptr && t == 0) a.p.rstd[row] = rstd;
      for (int base = 0; base < chunks; base += tpr) {  // whole warps: write_y shuffles
        const int chunk = base + t;
        const int c = chunk_col<VEC>(chunk);
        const bool in = chunk < chunks && c < a.dim;
        float h[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (in) {
          load_h<VEC>(a, row, c, h);
          if (a.p.h != nullptr) store_chunk<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, h);
        }
        write_y<VEC>(a, row, c, in, rstd, h);
      }
    }
  }
}

// ---------------------------------------------------------------- backward
struct GradArgs {
  int64_t rows;
  int dim;
  int tpr;
  gemm_rmsnorm_grad_t p;
  float* part;  // partial sums of dw: one row of `dim` floats per CTA, or nullptr
};

// C > 0: as forward; the thread also keeps the sums of its columns' dw over
// the rows that its CTA takes, and the CTA writes them as one row of `part`.
// C == 0: two passes over the row; dw is left to dweight_kernel.
template <int C, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float red[2][16];
  extern __shared__ float4 dyn_smem[];  // several rows per CTA: their dw sums
  grid_dependency_wait();
  grid_launch_dependents();
  const int tpr = a.tpr;
  const int t = threadIdx.x % tpr;
  const int slot = threadIdx.x / tpr;
  const int per_cta = blockDim.x / tpr;
  const int chunks = VEC ? a.dim / 8 : (a.dim + kFp8Block - 1) / kFp8Block * 16;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  constexpr int CR = C > 0 ? C : 1;
  float dw[CR][8];
#pragma unroll
  for (int k = 0; k < CR; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
  uint32_t turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_cta + slot; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * per_cta) {
    const float rstd = a.p.rstd[row];
    float dot = 0.0f;
    if (C > 0) {
      // dy is kept for the second half, or read again (C == 4: registers)
      constexpr bool kKeep = C <= 2;
      float xh[CR][8], g[CR][8];
#pragma unroll
      for (int k = 0; k < CR; ++k) {
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
#pragma unroll
        for (int i = 0; i < 8; ++i) xh[k][i] = g[k][i] = 0.0f;
        if (chunk < chunks && c < a.dim) {
          load_chunk<VEC>(a.p.dy, a.p.dy_type, row * a.p.lddy, c, a.dim, g[k]);
          load_chunk<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, xh[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < CR; ++k) {
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
        if (chunk >= chunks || c >= a.dim) continue;
        float w[8];
        load_weight<VEC>(a.p.weight, c, a.dim, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[k][i] *= rstd;
          dw[k][i] = fmaf(g[k][i], xh[k][i], dw[k][i]);
          g[k][i] *= w[i];
          dot = fmaf(g[k][i], xh[k][i], dot);
        }
      }
      const float mean = row_sum(dot, tpr, red, turn) * inv_dim;
#pragma unroll
      for (int k = 0; k < CR; ++k) {
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
        if (chunk >= chunks || c >= a.dim) continue;
        float r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        float dy[8], w[8];
        if (!kKeep) {
          load_chunk<VEC>(a.p.dy, a.p.dy_type, row * a.p.lddy, c, a.dim, dy);
          load_weight<VEC>(a.p.weight, c, a.dim, w);
        }
        if (a.p.residual_grad != nullptr)
          load_chunk<VEC>(a.p.residual_grad, a.p.residual_grad_type, row * a.p.ldrg, c, a.dim, r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          r[i] = fmaf(rstd, (kKeep ? g[k][i] : dy[i] * w[i]) - xh[k][i] * mean, r[i]);
        store_chunk<VEC>(a.p.dh, a.p.dh_type, row * a.p.lddh, c, a.dim, r);
      }
    } else {
      for (int chunk = t; chunk < chunks; chunk += tpr) {
        const int c = chunk_col<VEC>(chunk);
        if (c >= a.dim) continue;
        float g[8], xh[8], w[8];
        load_chunk<VEC>(a.p.dy, a.p.dy_type, row * a.p.lddy, c, a.dim, g);
        load_chunk<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, xh);
        load_weight<VEC>(a.p.weight, c, a.dim, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(g[i] * w[i], xh[i] * rstd, dot);
      }
      const float mean = row_sum(dot, tpr, red, turn) * inv_dim;
      for (int chunk = t; chunk < chunks; chunk += tpr) {
        const int c = chunk_col<VEC>(chunk);
        if (c >= a.dim) continue;
        float g[8], xh[8], w[8], r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        load_chunk<VEC>(a.p.dy, a.p.dy_type, row * a.p.lddy, c, a.dim, g);
        load_chunk<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, xh);
        load_weight<VEC>(a.p.weight, c, a.dim, w);
        if (a.p.residual_grad != nullptr)
          load_chunk<VEC>(a.p.residual_grad, a.p.residual_grad_type, row * a.p.ldrg, c, a.dim, r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          r[i] = fmaf(rstd, g[i] * w[i] - (xh[i] * rstd) * mean, r[i]);
        store_chunk<VEC>(a.p.dh, a.p.dh_type, row * a.p.lddh, c, a.dim, r);
      }
    }
  }
  if (C == 0 || a.part == nullptr) return;
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * a.dim;
  if (per_cta == 1) {
#pragma unroll
    for (int k = 0; k < CR; ++k) {
      const int chunk = k * tpr + t;
      const int c = chunk_col<VEC>(chunk);
      if (chunk >= chunks || c >= a.dim) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = VEC ? c + i : c + 16 * i;
        if (col < a.dim) out[col] = dw[k][i];
      }
    }
    return;
  }
  float* sums = reinterpret_cast<float*>(dyn_smem);
#pragma unroll
  for (int k = 0; k < CR; ++k) {
    const int chunk = k * tpr + t;
    const int c = chunk_col<VEC>(chunk);
    if (chunk >= chunks || c >= a.dim) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = VEC ? c + i : c + 16 * i;
      if (col < a.dim) sums[slot * a.dim + col] = dw[k][i];
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < a.dim; col += blockDim.x) {
    float s = 0.0f;
    for (int r = 0; r < per_cta; ++r) s += sums[r * a.dim + col];
    out[col] = s;
  }
}

// dw of rows too long for norm_grad_kernel's registers: one column per
// thread, the rows cut into gridDim.y parts, one row of `part` each.
__global__ void __launch_bounds__(256) dweight_kernel(const __grid_constant__ GradArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (col >= a.dim) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
    s = fmaf(load1(a.p.dy, a.p.dy_type, row * a.p.lddy + col),
             load1(a.p.h, a.p.h_type, row * a.p.ldh + col) * a.p.rstd[row], s);
  a.part[blockIdx.y * static_cast<int64_t>(a.dim) + col] = s;
}

// dw[col] = sum of the `parts` partial sums, always in the same order: a
// warp's lanes take 32 columns, the block's 8 warps every 8th part.
__global__ void __launch_bounds__(256) add_parts_kernel(const float* part, int parts, int dim,
                                                        float* dw) {
  __shared__ float sums[8][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (col < dim) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 8) s += __ldcg(part + static_cast<int64_t>(p) * dim + col);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < dim) {
    for (int r = 1; r < 8; ++r) s += sums[r][lane];
    dw[col] = s;
  }
}

struct RowPlan {
  int chunks_per_thread;  // 0: the row does not fit the registers
  int tpr, per_cta;
};

// Threads per row.  Few rows: one chunk a thread, for the shortest time of a
// row.  Many rows: up to `most` chunks a thread, for more loads in flight per
// thread and fewer threads per reduction; short rows take one warp each,
// eight to a CTA.  Long rows: up to `limit` chunks a thread; beyond that the
// looping instance.
RowPlan plan_rows(int64_t rows, int64_t chunks, int num_sms, int most, int limit) {
  RowPlan p{1, 32, 1};
  const bool many = rows > 2 * static_cast<int64_t>(num_sms);
  int c = 1;
  while (c < most && chunks > (many ? 32 : kMaxThreads) * c) c *= 2;
  while (c < limit && chunks > static_cast<int64_t>(kMaxThreads) * c) c *= 2;
  const int64_t threads = ((chunks + c - 1) / c + 31) / 32 * 32;
  if (threads > kMaxThreads) return RowPlan{0, kMaxThreads, 1};
  p.chunks_per_thread = c;
  p.tpr = static_cast<int>(threads);
  if (p.tpr == 32 && many) p.per_cta = kMaxRowsPerCta;
  return p;
}

template <bool VEC>
cudaError_t launch_norm(const NormArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid));
  const int threads = p.tpr * p.per_cta;
  switch (p.chunks_per_thread) {
    case 1: return ops_launch<norm_kernel<1, VEC>>(g, threads, 0, 1, s, a);
    case 2: return ops_launch<norm_kernel<2, VEC>>(g, threads, 0, 1, s, a);
    case 4: return ops_launch<norm_kernel<4, VEC>>(g, threads, 0, 1, s, a);
    default: return ops_launch<norm_kernel<0, VEC>>(g, threads, 0, 1, s, a);
  }
}

template <bool VEC>
cudaError_t launch_grad(const GradArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid));
  const int threads = p.tpr * p.per_cta;
  const size_t smem = p.per_cta > 1 ? sizeof(float) * p.per_cta * a.dim : 0;
  switch (p.chunks_per_thread) {
    case 1: return ops_launch<norm_grad_kernel<1, VEC>>(g, threads, smem, 1, s, a);
    case 2: return ops_launch<norm_grad_kernel<2, VEC>>(g, threads, smem, 1, s, a);
    case 4: return ops_launch<norm_grad_kernel<VEC ? 4 : 0, VEC>>(g, threads, smem, 1, s, a);
    default: return ops_launch<norm_grad_kernel<0, VEC>>(g, threads, 0, 1, s, a);
  }
}

int row_grid(int64_t rows, const RowPlan& p, int num_sms) {
  const int64_t ctas = (rows + p.per_cta - 1) / p.per_cta;
  const int64_t fit = static_cast<int64_t>(num_sms) * (1024 / (p.tpr * p.per_cta));
  return static_cast<int>(ctas < fit ? ctas : fit);
}

// A row-major array of the operator: NULL where `need` is false is fine;
// vec is cleared where its rows cannot be moved in 16-byte pieces.
bool array_ok(const void* p, int type, int64_t ld, int64_t dim, bool need, bool& vec) {
  if (p == nullptr) return !need;
  const int bytes = float_type_bytes(type);
  if (bytes == 0 || ld < dim || ld > kOpsMaxDim || ops_misaligned(p, bytes)) return false;
  if (ops_misaligned(p, 16) || ld % (16 / bytes) != 0) vec = false;
  return true;
}

}  // namespace
}  // namespace g12

using namespace g12;

extern "C" {

gemm_status_t gemm_rmsnorm(int64_t rows, int64_t dim, const gemm_rmsnorm_t* args, void* stream) {
  if (args == nullptr || rows < 0 || dim < 0 || rows > kOpsMaxDim || dim > (int64_t{1} << 30))
    return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || dim == 0) return GEMM_OK;
  const gemm_rmsnorm_t& p = *args;
  bool vec = dim % 8 == 0;
  if (!array_ok(p.x, p.x_type, p.ldx, dim, true, vec) ||
      !array_ok(p.residual, p.residual_type, p.ldr, dim, false, vec) ||
      !array_ok(p.h, p.h_type, p.ldh, dim, false, vec) ||
      !array_ok(p.y, p.y_type, p.ldy, dim, false, vec) ||
      !array_ok(p.weight, GEMM_OUT_F32, dim, dim, true, vec))
    return GEMM_ERR_INVALID_VALUE;
  if ((p.q == nullptr) != (p.scales == nullptr)) return GEMM_ERR_INVALID_VALUE;
  if (p.q != nullptr) {
    if (p.ldq < dim || p.ldq > kOpsMaxDim || p.ld_scales < rows || p.ld_scales > kOpsMaxDim ||
        ops_misaligned(p.scales, 4))
      return GEMM_ERR_INVALID_VALUE;
    if (ops_misaligned(p.q, 8) || p.ldq % 8 != 0) vec = false;
  }
  if (p.rstd != nullptr && ops_misaligned(p.rstd, 4)) return GEMM_ERR_INVALID_VALUE;
  if (p.h == nullptr && p.y == nullptr && p.q == nullptr && p.rstd == nullptr) return GEMM_OK;
  int sms = 0;
  uint32_t* err = nullptr;
  const gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  NormArgs a{};
  a.rows = rows;
  a.dim = static_cast<int>(dim);
  a.p = p;
  const int64_t chunks = vec ? dim / 8 : (dim + kFp8Block - 1) / kFp8Block * 16;
  const RowPlan pl = plan_rows(rows, chunks, sms, 4, 4);
  a.tpr = pl.tpr;
  const int grid = row_grid(rows, pl, sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return abi_from_cuda(vec ? launch_norm<true>(a, pl, grid, s) : launch_norm<false>(a, pl, grid, s));
}

gemm_status_t gemm_rmsnorm_backward(int64_t rows, int64_t dim, const gemm_rmsnorm_grad_t* args,
                                    void* stream) {
  if (args == nullptr || rows < 0 || dim < 0 || rows > kOpsMaxDim || dim > (int64_t{1} << 30))
    return GEMM_ERR_INVALID_VALUE;
  if (dim == 0) return GEMM_OK;
  const gemm_rmsnorm_grad_t& p = *args;
  bool vec = dim % 8 == 0;
  const bool some = rows > 0;
  if (!array_ok(p.dy, p.dy_type, p.lddy, dim, some, vec) ||
      !array_ok(p.h, p.h_type, p.ldh, dim, some, vec) ||
      !array_ok(p.residual_grad, p.residual_grad_type, p.ldrg, dim, false, vec) ||
      !array_ok(p.dh, p.dh_type, p.lddh, dim, some, vec) ||
      !array_ok(p.weight, GEMM_OUT_F32, dim, dim, some, vec))
    return GEMM_ERR_INVALID_VALUE;
  if (some && (p.rstd == nullptr || ops_misaligned(p.rstd, 4))) return GEMM_ERR_INVALID_VALUE;
  if (p.dweight != nullptr && ops_misaligned(p.dweight, 4)) return GEMM_ERR_INVALID_VALUE;
  if (!some && p.dweight == nullptr) return GEMM_OK;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!some) {
    const cudaError_t e = cudaMemsetAsync(p.dweight, 0, sizeof(float) * dim, s);
    return abi_from_cuda(e);
  }
  GradArgs a{};
  a.rows = rows;
  a.dim = static_cast<int>(dim);
  a.p = p;
  const int64_t chunks = vec ? dim / 8 : (dim + kFp8Block - 1) / kFp8Block * 16;
  const RowPlan pl = plan_rows(rows, chunks, sms, 2, vec ? 4 : 2);
  a.tpr = pl.tpr;
  const int grid = row_grid(rows, pl, sms);
  const bool by_column = pl.chunks_per_thread == 0;
  int parts = grid;
  if (by_column) parts = static_cast<int>(rows < 64 ? rows : 64);
  std::unique_lock<std::mutex> lock;
  if (p.dweight != nullptr) {
    st = abi_scratch(s, static_cast<int64_t>(parts) * dim, lock, &a.part);
    if (st != GEMM_OK) return st;
  }
  cudaError_t e = vec ? launch_grad<true>(a, pl, grid, s) : launch_grad<false>(a, pl, grid, s);
  if (e != cudaSuccess || p.dweight == nullptr) return abi_from_cuda(e);
  if (by_column) {
    const dim3 g(static_cast<unsigned>((dim + 255) / 256), static_cast<unsigned>(parts));
    e = ops_launch<dweight_kernel>(g, 256, 0, 1, s, a);
    if (e != cudaSuccess) return abi_from_cuda(e);
  }
  const dim3 g(static_cast<unsigned>((dim + 31) / 32));
  const float* part = a.part;
  return abi_from_cuda(
      ops_launch<add_parts_kernel>(g, 256, 0, 1, s, part, parts, a.dim, p.dweight));
}

}  // extern "C"
