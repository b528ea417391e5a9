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
#include "norm.cuh"

namespace g12 {
namespace {

struct NormArgs {
  int64_t rows;
  int dim;
  int tpr;  // threads per row, a multiple of 32; > 32: one row at a time per CTA
  RingArgs ring;
  gemm_rmsnorm_t p;
};

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
    if (a.p.y != nullptr) store8<VEC>(a.p.y, a.p.y_type, row * a.p.ldy, c, a.dim, y);
  }
  if (a.p.q == nullptr) return;
  write_fp8<VEC>(a.p.q, a.p.ldq, a.p.scales, a.p.ld_scales, row, c, a.dim, in, y);
}

// C > 0: a thread keeps its C chunks of 8 elements in registers, and the row
// is read once.  C == 0: rows longer than that are read twice (the second
// time mostly from L2).  Nothing of a row is written before its last read, so
// outputs may take the place of inputs element by element.
template <int C, bool VEC, int TX, int TR, bool RING = false>
__global__ void __launch_bounds__(kMaxThreads, RING ? 2 : 1) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][16];
  __shared__ Ring ring;
  extern __shared__ uint4 dyn_smem[];
  uint8_t* const stages = reinterpret_cast<uint8_t*>(dyn_smem);
  const int stage_bytes = RING ? a.dim * (type_bytes(TX) + (TR < 0 ? 0 : type_bytes(TR))) : 0;
  // thread 0: copies `row` into stage s
  auto fetch = [&](int64_t row, int s) {
    uint8_t* to = stages + s * stage_bytes;
    mbar_arrive_expect_tx(&ring.full[s], static_cast<uint32_t>(stage_bytes));
    bulk_load(to, static_cast<const uint8_t*>(a.p.x) + row * a.p.ldx * type_bytes(TX),
              static_cast<uint32_t>(a.dim * type_bytes(TX)), &ring.full[s]);
    if constexpr (TR >= 0)
      bulk_load(to + a.dim * type_bytes(TX),
                static_cast<const uint8_t*>(a.p.residual) + row * a.p.ldr * type_bytes(TR),
                static_cast<uint32_t>(a.dim * type_bytes(TR)), &ring.full[s]);
  };
  if (RING) ring_init(ring, a.ring.stages);
  grid_dependency_wait();
  grid_launch_dependents();
  if (RING && threadIdx.x == 0)
    for (int s = 0; s < a.ring.stages; ++s) {
      const int64_t row = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
      if (row < a.rows) fetch(row, s);
    }
  int slot = 0;
  uint32_t parity = 0;
  const int tpr = a.tpr;
  const int t = threadIdx.x % tpr;
  const int per_cta = blockDim.x / tpr;
  const int chunks = VEC ? a.dim / 8 : (a.dim + kFp8Block - 1) / kFp8Block * 16;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  uint32_t turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_cta + threadIdx.x / tpr; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * per_cta) {
    float ss = 0.0f;
    if constexpr (C > 0) {
      Inputs<VEC, TX, TR> raw[C];
      bool in[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
        in[k] = chunk < chunks && c < a.dim;
        if constexpr (RING) {
          if (k == 0) mbar_wait_late(&ring.full[slot], parity, &ring.abort_flag, a.ring.err);
          raw[k].from_ring(a, stages + slot * stage_bytes, c, in[k]);
        } else {
          raw[k].load(a, row, c, in[k]);
        }
      }
      float h[C][8];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        raw[k].sum(a, h[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[k][i], h[k][i], ss);
        if (a.p.h != nullptr && in[k])
          store8<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, chunk_col<VEC>(k * tpr + t), a.dim, h[k]);
      }
      ss = row_sum(ss, tpr, red, turn);
      if constexpr (RING) {
        // every thread has read the stage (row_sum's barrier): the next row
        // for it.  After a wait ran out nothing more is fetched; the error
        // word says that the results are not to be used.
        const int64_t next = row + static_cast<int64_t>(a.ring.stages) * gridDim.x;
        if (threadIdx.x == 0 && next < a.rows && !*const_cast<volatile int*>(&ring.abort_flag))
          fetch(next, slot);
        if (++slot == a.ring.stages) {
          slot = 0;
          parity ^= 1u;
        }
      }
      const float rstd = rsqrtf(fmaf(ss, inv_dim, a.p.eps));
      if (a.p.rstd != nullptr && t == 0) a.p.rstd[row] = rstd;
#pragma unroll
      for (int k = 0; k < C; ++k) write_y<VEC>(a, row, chunk_col<VEC>(k * tpr + t), in[k], rstd, h[k]);
    } else {
      for (int chunk = t; chunk < chunks; chunk += tpr) {
        const int c = chunk_col<VEC>(chunk);
        Inputs<VEC, TX, TR> raw;
        raw.load(a, row, c, c < a.dim);
        float h[8];
        raw.sum(a, h);
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
        Inputs<VEC, TX, TR> raw;
        raw.load(a, row, c, in);
        float h[8];
        raw.sum(a, h);
        if (in && a.p.h != nullptr) store8<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, h);
        write_y<VEC>(a, row, c, in, rstd, h);
      }
    }
  }
  if (RING && threadIdx.x == 0 && ring.abort_flag) drain(ring, a.ring.stages, slot, parity);
}

// ---------------------------------------------------------------- backward
struct GradArgs {
  int64_t rows;
  int dim;
  int tpr;
  RingArgs ring;
  gemm_rmsnorm_grad_t p;
  float* part;  // partial sums of dw: one row of `dim` floats per CTA, or nullptr
};

// C > 0: as forward; the thread also keeps the sums of its columns' dw over
// the rows that its CTA takes, and the CTA writes them as one row of `part`.
// C == 0: two passes over the row; dw is left to dweight_kernel.
template <int C, bool VEC, int TD, int TH, bool RING = false>
__global__ void __launch_bounds__(RING && C == 1 ? 1024 : kMaxThreads, 1)
    norm_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float red[2][16];
  __shared__ Ring ring;
  extern __shared__ uint4 dyn_smem[];  // the ring, or several rows' dw sums
  uint8_t* const stages = reinterpret_cast<uint8_t*>(dyn_smem);
  const int ring_dim = RING ? a.dim : 0;
  const int bytes_d = ring_dim * type_bytes(TD), bytes_h = ring_dim * type_bytes(TH);
  const int bytes_r = a.p.residual_grad == nullptr ? 0 : ring_dim * type_bytes(a.p.residual_grad_type);
  const int stage_bytes = bytes_d + bytes_h + bytes_r;
  auto fetch = [&](int64_t row, int s) {
    uint8_t* to = stages + s * stage_bytes;
    uint64_t* bar = &ring.full[s];
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(stage_bytes));
    bulk_load(to, static_cast<const uint8_t*>(a.p.dy) + row * a.p.lddy * type_bytes(TD), bytes_d, bar);
    bulk_load(to + bytes_d, static_cast<const uint8_t*>(a.p.h) + row * a.p.ldh * type_bytes(TH),
              bytes_h, bar);
    if (bytes_r > 0)
      bulk_load(to + bytes_d + bytes_h,
                static_cast<const uint8_t*>(a.p.residual_grad) +
                    row * a.p.ldrg * type_bytes(a.p.residual_grad_type),
                bytes_r, bar);
  };
  if (RING) ring_init(ring, a.ring.stages);
  grid_dependency_wait();
  grid_launch_dependents();
  if (RING && threadIdx.x == 0)
    for (int s = 0; s < a.ring.stages; ++s) {
      const int64_t row = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
      if (row < a.rows) fetch(row, s);
    }
  int slot = 0;
  uint32_t parity = 0;
  const int tpr = a.tpr;
  const int t = threadIdx.x % tpr;
  const int sub = threadIdx.x / tpr;
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
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * per_cta;
  int64_t row = static_cast<int64_t>(blockIdx.x) * per_cta + sub;
  float next_rstd = row < a.rows ? a.p.rstd[row] : 0.0f;  // loaded a row ahead
  for (; row < a.rows; row += row_step) {
    const float rstd = next_rstd;
    if (row + row_step < a.rows) next_rstd = a.p.rstd[row + row_step];
    float dot = 0.0f;
    if constexpr (C > 0) {
      // RING: both halves read the stage, which keeps registers free for more
      // threads; it is filled again at the next row's barrier.  Otherwise dy
      // and h stay as they were loaded.
      Raw8<TD> dy[C];
      Raw8<TH> rh[C];
      const uint8_t* from = stages + slot * stage_bytes;
      if (RING) mbar_wait_late(&ring.full[slot], parity, &ring.abort_flag, a.ring.err);
      auto get = [&](int k, int c, bool in) {
        if constexpr (RING) {
          dy[k] = {};
          rh[k] = {};
          if (!in) return;
          dy[k] = load8_smem<TD>(from, c);
          rh[k] = load8_smem<TH>(from + bytes_d, c);
        } else {
          dy[k] = load8<VEC, TD>(a.p.dy, a.p.dy_type, row * a.p.lddy, c, a.dim, in);
          rh[k] = load8<VEC, TH>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, in);
        }
      };
      auto inside = [&](int k) {
        const int chunk = k * tpr + t;
        return chunk < chunks && chunk_col<VEC>(chunk) < a.dim;
      };
      if (!RING) {
#pragma unroll
        for (int k = 0; k < C; ++k) get(k, chunk_col<VEC>(k * tpr + t), inside(k));
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = chunk_col<VEC>(k * tpr + t);
        if (RING) get(k, c, inside(k));
        if (!inside(k)) continue;
        float w[8], g[8], xh[8];
        load_weight<VEC>(a.p.weight, c, a.dim, w);
        widen8<VEC, TD>(dy[k], a.p.dy_type, g);
        widen8<VEC, TH>(rh[k], a.p.h_type, xh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[i] *= rstd;
          dw[k][i] = fmaf(g[i], xh[i], dw[k][i]);
          dot = fmaf(g[i] * w[i], xh[i], dot);
        }
      }
      const float mean = row_sum(dot, tpr, red, turn) * inv_dim;
      if (RING && threadIdx.x == 0 && row >= static_cast<int64_t>(gridDim.x)) {
        // every thread has left the previous row (row_sum's barrier)
        const int64_t next = row + static_cast<int64_t>(a.ring.stages - 1) * gridDim.x;
        if (next < a.rows && !*const_cast<volatile int*>(&ring.abort_flag))
          fetch(next, slot == 0 ? a.ring.stages - 1 : slot - 1);
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = chunk_col<VEC>(k * tpr + t);
        if (!inside(k)) continue;
        if (RING) get(k, c, true);
        float w[8], g[8], xh[8], r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (a.p.residual_grad != nullptr) {
          const int type = a.p.residual_grad_type;
          if constexpr (RING) {
            const uint8_t* rg = from + bytes_d + bytes_h;
            if (type == GEMM_OUT_BF16)
              widen8<true, GEMM_OUT_BF16>(load8_smem<GEMM_OUT_BF16>(rg, c), type, r);
            else
              widen8<true, GEMM_OUT_F32>(load8_smem<GEMM_OUT_F32>(rg, c), type, r);
          } else {
            widen8<VEC, kAnyType>(load8<VEC, kAnyType>(a.p.residual_grad, type, row * a.p.ldrg, c,
                                                       a.dim, true), type, r);
          }
        }
        load_weight<VEC>(a.p.weight, c, a.dim, w);
        widen8<VEC, TD>(dy[k], a.p.dy_type, g);
        widen8<VEC, TH>(rh[k], a.p.h_type, xh);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          r[i] = fmaf(rstd, g[i] * w[i] - (xh[i] * rstd) * mean, r[i]);
        store8<VEC>(a.p.dh, a.p.dh_type, row * a.p.lddh, c, a.dim, r);
      }
      if (RING && ++slot == a.ring.stages) {
        slot = 0;
        parity ^= 1u;
      }
    } else {
      for (int half = 0; half < 2; ++half) {
        const float mean = half == 0 ? 0.0f : row_sum(dot, tpr, red, turn) * inv_dim;
        for (int chunk = t; chunk < chunks; chunk += tpr) {
          const int c = chunk_col<VEC>(chunk);
          if (c >= a.dim) continue;
          float w[8], g[8], xh[8], r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
          const Raw8<TD> dy = load8<VEC, TD>(a.p.dy, a.p.dy_type, row * a.p.lddy, c, a.dim, true);
          const Raw8<TH> rh = load8<VEC, TH>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, true);
          if (half == 1 && a.p.residual_grad != nullptr)
            widen8<VEC, kAnyType>(load8<VEC, kAnyType>(a.p.residual_grad, a.p.residual_grad_type,
                                                       row * a.p.ldrg, c, a.dim, true),
                                  a.p.residual_grad_type, r);
          load_weight<VEC>(a.p.weight, c, a.dim, w);
          widen8<VEC, TD>(dy, a.p.dy_type, g);
          widen8<VEC, TH>(rh, a.p.h_type, xh);
          if (half == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = fmaf(g[i] * w[i], xh[i] * rstd, dot);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              r[i] = fmaf(rstd, g[i] * w[i] - (xh[i] * rstd) * mean, r[i]);
            store8<VEC>(a.p.dh, a.p.dh_type, row * a.p.lddh, c, a.dim, r);
          }
        }
      }
    }
  }
  if (RING && threadIdx.x == 0 && ring.abort_flag) drain(ring, a.ring.stages, slot, parity);
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
      if (col < a.dim) sums[sub * a.dim + col] = dw[k][i];
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

// Rows moved in vectors have an instance for each pair of input types; the
// others look at the types as they go.
template <bool VEC, int TX, int TR>
cudaError_t launch_norm(const NormArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid));
  const int threads = p.tpr * p.per_cta;
  if constexpr (VEC) {
    if (a.ring.stages > 0) {  // more than one warp a row: two chunks a thread (plan_rows)
      const size_t smem = static_cast<size_t>(a.ring.stages) * a.dim *
                          (type_bytes(TX) + (TR < 0 ? 0 : type_bytes(TR)));
      return ops_launch<norm_kernel<2, VEC, TX, TR, true>>(g, threads, smem, 1, s, a);
    }
  }
  switch (p.chunks_per_thread) {
    case 1: return ops_launch<norm_kernel<1, VEC, TX, TR>>(g, threads, 0, 1, s, a);
    case 2: return ops_launch<norm_kernel<2, VEC, TX, TR>>(g, threads, 0, 1, s, a);
    case 4: return ops_launch<norm_kernel<4, VEC, TX, TR>>(g, threads, 0, 1, s, a);
    default: return ops_launch<norm_kernel<0, VEC, TX, TR>>(g, threads, 0, 1, s, a);
  }
}

template <int TX>
cudaError_t launch_norm_vec(const NormArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  if (a.p.residual == nullptr) return launch_norm<true, TX, -1>(a, p, grid, s);
  return a.p.residual_type == GEMM_OUT_BF16 ? launch_norm<true, TX, GEMM_OUT_BF16>(a, p, grid, s)
                                            : launch_norm<true, TX, GEMM_OUT_F32>(a, p, grid, s);
}

cudaError_t launch_norm_any(const NormArgs& a, const RowPlan& p, bool vec, int grid, cudaStream_t s) {
  if (vec)
    return a.p.x_type == GEMM_OUT_BF16 ? launch_norm_vec<GEMM_OUT_BF16>(a, p, grid, s)
                                       : launch_norm_vec<GEMM_OUT_F32>(a, p, grid, s);
  return a.p.residual == nullptr ? launch_norm<false, kAnyType, -1>(a, p, grid, s)
                                 : launch_norm<false, kAnyType, kAnyType>(a, p, grid, s);
}

template <bool VEC, int TD, int TH>
cudaError_t launch_grad(const GradArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid));
  const int threads = p.tpr * p.per_cta;
  const size_t smem = p.per_cta > 1 ? sizeof(float) * p.per_cta * a.dim : 0;
  if constexpr (VEC) {
    if (a.ring.stages > 0) {
      const int rg = a.p.residual_grad == nullptr ? 0 : type_bytes(a.p.residual_grad_type);
      const size_t bytes = static_cast<size_t>(a.ring.stages) * a.dim * (type_bytes(TD) + type_bytes(TH) + rg);
      switch (p.chunks_per_thread) {
        case 1: return ops_launch<norm_grad_kernel<1, VEC, TD, TH, true>>(g, threads, bytes, 1, s, a);
        default: return ops_launch<norm_grad_kernel<2, VEC, TD, TH, true>>(g, threads, bytes, 1, s, a);
      }
    }
  }
  switch (p.chunks_per_thread) {
    case 1: return ops_launch<norm_grad_kernel<1, VEC, TD, TH>>(g, threads, smem, 1, s, a);
    case 2: return ops_launch<norm_grad_kernel<2, VEC, TD, TH>>(g, threads, smem, 1, s, a);
    case 4:
      return ops_launch<norm_grad_kernel<VEC && TD == GEMM_OUT_BF16 && TH == GEMM_OUT_BF16 ? 4 : 0,
                                         VEC, TD, TH>>(g, threads, smem, 1, s, a);
    default: return ops_launch<norm_grad_kernel<0, VEC, TD, TH>>(g, threads, 0, 1, s, a);
  }
}

cudaError_t launch_grad_any(const GradArgs& a, const RowPlan& p, bool vec, int grid, cudaStream_t s) {
  constexpr int B = GEMM_OUT_BF16, F = GEMM_OUT_F32;
  if (!vec) return launch_grad<false, kAnyType, kAnyType>(a, p, grid, s);
  if (a.p.dy_type == B)
    return a.p.h_type == B ? launch_grad<true, B, B>(a, p, grid, s) : launch_grad<true, B, F>(a, p, grid, s);
  return a.p.h_type == B ? launch_grad<true, F, B>(a, p, grid, s) : launch_grad<true, F, F>(a, p, grid, s);
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
  RowPlan pl = plan_rows(rows, chunks, sms, 4, 4);
  a.tpr = pl.tpr;
  a.ring.err = err;
  int grid = row_grid(rows, pl, sms, 1024);
  if (vec) {
    const int64_t bytes = dim * (type_bytes(p.x_type) +
                                 (p.residual == nullptr ? 0 : type_bytes(p.residual_type)));
    const RowPlan pr = plan_rows(rows, chunks, sms, 2, 2);
    const int ring_grid = plan_ring(pr, rows, bytes, sms, 1024, a.ring);
    if (ring_grid > 0) {
      grid = ring_grid;
      pl = pr;
      a.tpr = pl.tpr;
    }
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return abi_from_cuda(launch_norm_any(a, pl, vec, grid, s));
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
  // the registers hold four chunks of dw and of both inputs only in bf16
  const bool both_bf16 = vec && p.dy_type == GEMM_OUT_BF16 && p.h_type == GEMM_OUT_BF16;
  // Two chunks a thread where one would leave threads over or not reach: short
  // rows of few threads, long ones.  Otherwise one, for more threads an SM (bf16
  // with the skip connection's gradient, 8192 x 4096 54 us against 57, 16384 x
  // 1024 33 against 37; but 16384 x 512 22 with two, 24 with one) and always
  // where rows are not moved in vectors (4000 x 3001 36 us against 54).
  const bool two = vec && (chunks <= 64 || chunks > kMaxThreads);
  const RowPlan pl = plan_rows(rows, chunks, sms, two ? 2 : 1, both_bf16 ? 4 : 2);
  a.tpr = pl.tpr;
  a.ring.err = err;
  int grid = row_grid(rows, pl, sms, pl.chunks_per_thread == 1 ? 768 : 512);
  if (vec && pl.chunks_per_thread <= 2) {
    const int64_t bytes =
        dim * (type_bytes(p.dy_type) + type_bytes(p.h_type) +
               (p.residual_grad == nullptr ? 0 : type_bytes(p.residual_grad_type)));
    const int ring_grid =
        plan_ring(pl, rows, bytes, sms, pl.chunks_per_thread == 1 ? 1024 : 640, a.ring);
    if (ring_grid > 0) grid = ring_grid;
  }
  const bool by_column = pl.chunks_per_thread == 0;
  int parts = grid;
  if (by_column) {  // up to 64, of 256 MB together
    parts = static_cast<int>(rows < 64 ? rows : 64);
    while (parts > 1 && parts * dim > (int64_t{1} << 26)) parts /= 2;
  }
  std::unique_lock<std::mutex> lock;
  if (p.dweight != nullptr) {
    st = abi_scratch(s, static_cast<int64_t>(parts) * dim, lock, &a.part);
    if (st != GEMM_OK) return st;
  }
  cudaError_t e = cudaSuccess;
  if (by_column && p.dweight != nullptr) {  // first: dh may take the place of dy or h
    const dim3 g(static_cast<unsigned>((dim + 255) / 256), static_cast<unsigned>(parts));
    e = ops_launch<dweight_kernel>(g, 256, 0, 1, s, a);
  }
  if (e == cudaSuccess) e = launch_grad_any(a, pl, vec, grid, s);
  if (e != cudaSuccess || p.dweight == nullptr) return abi_from_cuda(e);
  const dim3 g(static_cast<unsigned>((dim + 31) / 32));
  const float* part = a.part;
  float* const none = nullptr;
  return abi_from_cuda(ops_launch<add_parts_kernel>(g, 1024, 0, 1, s, part, parts, a.dim,
                                                    static_cast<int64_t>(a.dim), p.dweight, none));
}

}  // extern "C"
