// layernorm.cu -- layer norm with the residual's addition, its output in fp32,
// bf16, fp8 with block scales or int8 with a scale per row, and its gradients.
//
//     h = x + r      m = mean_j h_j      s = (mean_j (h_j - m)^2 + eps)^-1/2
//     y_j = (h_j - m) s w_j + b_j
//
// and, with dy the gradient of y, dr that of the stored h, xh = (h - m) s and
// g = dy w:
//
//     dh = s (g - mean_j g_j - xh mean_j(g_j xh_j)) + dr
//     dw = sum_rows dy xh        db = sum_rows dy
//
// Bound by memory: a row is read once, kept in registers over its sums, and
// written once.  Many rows come through rings in shared memory as in norm.cu,
// but a CTA fills an SM: up to eight groups of threads, each with a row and a
// ring of its own, around one copy of the weight and the bias.  Read anew for
// each row those are as many bytes as the row itself, and with shared memory
// full of rows they do not stay in L1 (8192 rows of 8192 in bf16: 104 us with a
// group to a CTA and weights from L2, 87 here, 6.2 TB/s; into fp8 106, int8 107; the
// gradient of 8192 rows of 4096 54, 5.0 TB/s).  Rows that 16-byte pieces do not fit
// come element by element, one to a CTA's turn: 8000 x 1999 46 us (2.8 TB/s), the
// gradient 65.  Rows too long for the registers are read three times, by the
// gradient too: 2048 x 20000 156 us, the gradient of 2048 x 16384 212.
//
// The squares are summed about the mean, never as mean(h^2) - m^2, which loses
// everything when the mean is large.  The mean itself is only known to fp32's
// rounding; what it is off by is the mean of the differences from it, which
// comes with the second sum and is taken off both the squares' mean and the
// values.
#include "norm.cuh"

namespace g12 {
namespace {

constexpr int kMaxRings = 8;      // groups of a CTA
constexpr int kLnCtaBytes = 6144;  // shared memory of a CTA besides weights and rings

struct LnRings {
  uint64_t full[kMaxRings * kMaxStages];
  int abort_flag;
};

struct LnArgs {
  int64_t rows;
  int dim;
  int tpr;
  RingArgs ring;
  gemm_layernorm_t p;
};

// Sums of N values over the tpr threads of a group.  red: two rows
// of a value per warp, used in turn, one call a row.
template <int N>
__device__ __forceinline__ void over_row(float (&v)[N], int tpr, int group, float (*red)[16][N], uint32_t turn) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], s);
  if (tpr == 32) return;
  const int lane = threadIdx.x & 31, warps = tpr >> 5;
  float(*mine)[N] = red[turn & 1u];
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) mine[(threadIdx.x >> 5) % warps][i] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? mine[lane & 15][i] : 0.0f;
#pragma unroll
  for (int s = 8; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], s);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
}

// After a wait ran out: a group's copies in flight land before the CTA leaves.
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, int slot, uint32_t parity) {
  for (int i = 0; i < stages; ++i) {
    mbar_drain_wait(&full[slot], parity);
    if (++slot == stages) {
      slot = 0;
      parity ^= 1u;
    }
  }
}

// The weight, and the bias behind it, to shared memory; all threads of the CTA.
__device__ __forceinline__ void stage_weights(float* to, const float* weight, const float* bias, int dim,
                                              bool with_bias) {
  for (int i = threadIdx.x * 4; i < dim; i += blockDim.x * 4) {
    *reinterpret_cast<float4*>(to + i) = weight != nullptr ? __ldg(reinterpret_cast<const float4*>(weight + i))
                                                           : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (with_bias)
      *reinterpret_cast<float4*>(to + dim + i) =
          bias != nullptr ? __ldg(reinterpret_cast<const float4*>(bias + i)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
}
// Eight of them from there.
__device__ __forceinline__ void staged_pairs(const float* from, uint64_t (&p)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
  p[0] = f32x2(a.x, a.y);
  p[1] = f32x2(a.z, a.w);
  p[2] = f32x2(b.x, b.y);
  p[3] = f32x2(b.z, b.w);
}

// Elements of chunk column c, and (not VEC) 16 i further, inside the row.
template <bool VEC>
__device__ __forceinline__ bool inside(int c, int i, int dim) {
  return VEC || c + 16 * i < dim;
}

__device__ __forceinline__ void to_pairs(const float (&v)[8], uint64_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = f32x2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void from_pairs(const uint64_t (&p)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = f32x2_parts(p[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ float both(uint64_t p) {
  const float2 f = f32x2_parts(p);
  return f.x + f.y;
}

// A chunk's differences from the mean, zero where nothing is, and what they and
// their squares add to the sums.
template <bool VEC>
__device__ __forceinline__ void center(uint64_t (&h)[4], uint64_t minus_mean, int c, int dim, bool in,
                                       uint64_t& sum, uint64_t& squares) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = add2(h[i], minus_mean);
    if (!VEC) {
      const float2 f = f32x2_parts(h[i]);
      h[i] = f32x2(inside<VEC>(c, 2 * i, dim) ? f.x : 0.0f, inside<VEC>(c, 2 * i + 1, dim) ? f.y : 0.0f);
    }
    if (!in) h[i] = 0ull;
    sum = add2(sum, h[i]);
    squares = fma2(h[i], h[i], squares);
  }
}

// y of one chunk from its differences d from the mean; 0 where nothing is.
// STAGED: weight and bias are in shared memory, one behind the other.
template <bool VEC, bool STAGED = false>
__device__ __forceinline__ void affine(const float* weight, const float* bias, int c, int dim, bool in,
                                       float rstd, float off, const uint64_t (&d)[4], float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = 0.0f;
  if (!in) return;
  const float o = -off * rstd;
  if constexpr (STAGED) {  // four elements at a time: registers
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 w = *reinterpret_cast<const float4*>(weight + c + 4 * i);
      const float4 b = *reinterpret_cast<const float4*>(weight + dim + c + 4 * i);
      const float2 d0 = f32x2_parts(d[2 * i]), d1 = f32x2_parts(d[2 * i + 1]);
      y[4 * i] = fmaf(fmaf(d0.x, rstd, o), w.x, b.x);
      y[4 * i + 1] = fmaf(fmaf(d0.y, rstd, o), w.y, b.y);
      y[4 * i + 2] = fmaf(fmaf(d1.x, rstd, o), w.z, b.z);
      y[4 * i + 3] = fmaf(fmaf(d1.y, rstd, o), w.w, b.w);
    }
  } else {
    uint64_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = fma2(d[i], f32x2(rstd, rstd), f32x2(o, o));
    float v[8];
    uint64_t q[4];
    if (weight != nullptr) {
      load_weight<VEC>(weight, c, dim, v);
      to_pairs(v, q);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = mul2(p[i], q[i]);
    }
    if (bias != nullptr) {
      load_weight<VEC>(bias, c, dim, v);
      to_pairs(v, q);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = add2(p[i], q[i]);
    }
    from_pairs(p, y);
    if (!VEC) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = inside<VEC>(c, i, dim) ? y[i] : 0.0f;
    }
  }
}

__device__ __forceinline__ uint32_t chunk_max(const float (&y)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(y[i]));
  return m;
}
// The same over the finite values only.
__device__ __forceinline__ uint32_t chunk_finite_max(const float (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(y[i]));
  return __float_as_uint(m);
}

// C > 0: a row in registers.  C == 0: rows longer than that are read three
// times, and once more where their largest value is needed before the first is
// written.  Nothing of a row is written before its last read.
// Q: the 8-bit output's type, kNoQ for none, or kAnyQ for one known at run time.
constexpr int kNoQ = 0, kAnyQ = -1;

template <int C, bool VEC, int TX, int TR, bool RING = false, int Q = kAnyQ>
__global__ void __launch_bounds__(RING ? 1024 : kMaxThreads, 1)
    layernorm_kernel(const __grid_constant__ LnArgs a) {
  __shared__ float red_mean[kMaxRings][2][16][1];
  __shared__ uint32_t red_max[kMaxRings][2][16], red_finite[kMaxRings][2][16];
  __shared__ float red_var[kMaxRings][2][16][2];
  __shared__ LnRings ring;
  extern __shared__ uint4 dyn_smem[];
  float* const weights = reinterpret_cast<float*>(dyn_smem);  // RING: and the bias, then the rings
  const int tpr = a.tpr;
  const int t = threadIdx.x % tpr, group = threadIdx.x / tpr;
  const int per_cta = blockDim.x / tpr;
  const uint32_t rows = static_cast<uint32_t>(a.rows), row_step = gridDim.x * per_cta;  // below 2^31
  const uint32_t row0 = blockIdx.x * per_cta + group;
  const int stage_bytes = RING ? a.dim * (type_bytes(TX) + (TR < 0 ? 0 : type_bytes(TR))) : 0;
  // offsets of the group's ring and barriers: short, for the registers
  const int ring_off = RING ? 8 * a.dim + group * a.ring.stages * stage_bytes : 0;
  const int bar_off = RING ? group * kMaxStages : 0;
  auto stage = [&](int s) { return reinterpret_cast<uint8_t*>(dyn_smem) + ring_off + s * stage_bytes; };
  // a group's first thread: copies `row` into stage s
  auto fetch = [&](uint32_t at, int s) {
    const int64_t row = at;
    uint8_t* to = stage(s);
    uint64_t* bar = &ring.full[bar_off + s];
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(stage_bytes));
    bulk_load(to, static_cast<const uint8_t*>(a.p.x) + row * a.p.ldx * type_bytes(TX),
              static_cast<uint32_t>(a.dim * type_bytes(TX)), bar);
    if constexpr (TR >= 0)
      bulk_load(to + a.dim * type_bytes(TX),
                static_cast<const uint8_t*>(a.p.residual) + row * a.p.ldr * type_bytes(TR),
                static_cast<uint32_t>(a.dim * type_bytes(TR)), bar);
  };
  if (RING) {
    if (t == 0) {
      for (int s = 0; s < a.ring.stages; ++s) mbar_init(&ring.full[bar_off + s], 1);
      if (group == 0) ring.abort_flag = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (RING) {
    if (t == 0)
      for (int s = 0; s < a.ring.stages; ++s)
        if (row0 + s * row_step < rows) fetch(row0 + s * row_step, s);
    stage_weights(weights, a.p.weight, a.p.bias, a.dim, true);
    __syncthreads();
  }
  int slot = 0;
  uint32_t parity = 0;
  const int chunks = VEC ? a.dim / 8 : (a.dim + kFp8Block - 1) / kFp8Block * 16;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  uint32_t turn = 0;  // of all three sums
  const bool s8 = Q == kAnyQ ? a.p.q != nullptr && a.p.q_type == GEMM_OUT_S8 : Q == GEMM_OUT_S8;
  const bool f8 = Q == kAnyQ ? a.p.q != nullptr && !s8 : Q == GEMM_OUT_F8E4M3;
  // given a thread's sums of the differences from `mean` and of their squares
  auto statistics = [&](int64_t row, float mean, float left, float squares, float& off, float& rstd) {
    float v[2] = {left, squares};
    over_row<2>(v, tpr, group, red_var[RING ? group : 0], turn);
    off = v[0] * inv_dim;
    const float var = fmaf(v[1], inv_dim, -off * off);
    rstd = rsqrtf((var < 0.0f ? 0.0f : var) + a.p.eps);  // (NaN stays)
    if (t == 0) {
      if (a.p.mean != nullptr) a.p.mean[row] = mean + off;
      if (a.p.rstd != nullptr) a.p.rstd[row] = rstd;
    }
  };
  for (uint32_t at = row0; at < rows; at += row_step, ++turn) {
    const int64_t row = at;
    float sum = 0.0f, off, rstd;
    auto mean_of = [&]() {
      float v[1] = {sum};
      over_row<1>(v, tpr, group, red_mean[RING ? group : 0], turn);
      return v[0] * inv_dim;
    };
    auto largest_of = [&](uint32_t m) {
      return row_max_bits(m, tpr, group, red_max[RING ? group : 0], turn);
    };
    auto largest_finite_of = [&](uint32_t m) {
      return row_max_bits(m, tpr, group, red_finite[RING ? group : 0], turn);
    };
    if constexpr (C > 0) {
      // RING: a chunk at a time; else all chunks' loads are on their way together
      Inputs<VEC, TX, TR> raw[RING ? 1 : C];
      bool in[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int chunk = k * tpr + t;
        const int c = chunk_col<VEC>(chunk);
        in[k] = chunk < chunks && c < a.dim;
        if constexpr (!RING) raw[k].load(a, row, c, in[k]);
      }
      if constexpr (RING) mbar_wait_late(&ring.full[bar_off + slot], parity, &ring.abort_flag, a.ring.err);
      uint64_t h[C][4], total = 0ull;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = chunk_col<VEC>(k * tpr + t);
        float v[8];
        if constexpr (RING) raw[0].from_ring(a, stage(slot), c, in[k]);
        raw[RING ? 0 : k].sum(a, v);  // zeros where nothing is
        to_pairs(v, h[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) total = add2(total, h[k][i]);
        if (a.p.h != nullptr && in[k]) store8<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, v);
      }
      sum = both(total);
      const float mean = mean_of();
      if constexpr (RING) {
        // every thread has read the stage (the sum's barrier): the next row
        const uint32_t next = at + a.ring.stages * row_step;
        if (t == 0 && next < rows && !*const_cast<volatile int*>(&ring.abort_flag))
          fetch(next, slot);
        if (++slot == a.ring.stages) {
          slot = 0;
          parity ^= 1u;
        }
      }
      uint64_t left = 0ull, squares = 0ull;
#pragma unroll
      for (int k = 0; k < C; ++k)
        center<VEC>(h[k], f32x2(-mean, -mean), chunk_col<VEC>(k * tpr + t), a.dim, in[k], left, squares);
      statistics(row, mean, both(left), both(squares), off, rstd);
      uint32_t amax = 0u;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = chunk_col<VEC>(k * tpr + t);
        float y[8];
        affine<VEC, RING>(RING ? weights : a.p.weight, a.p.bias, c, a.dim, in[k], rstd, off, h[k], y);
        if (a.p.y != nullptr && in[k]) store8<VEC>(a.p.y, a.p.y_type, row * a.p.ldy, c, a.dim, y);
        if (f8) write_fp8<VEC>(a.p.q, a.p.ldq, a.p.scales, a.p.ld_scales, row, c, a.dim, in[k], y);
        if (s8) {
          amax = max(amax, chunk_max(y));
          to_pairs(y, h[k]);
        }
      }
      if (!s8) continue;
      amax = largest_of(amax);
      const bool finite = amax < kInfBits;
      if (!finite) {
        amax = 0u;
#pragma unroll
        for (int k = 0; k < C; ++k) {
          float y[8];
          from_pairs(h[k], y);
          amax = max(amax, chunk_finite_max(y));
        }
        amax = largest_finite_of(amax);
      }
      const float f = s8_factor(__uint_as_float(amax));
#pragma unroll
      for (int k = 0; k < C; ++k) {
        float y[8];
        from_pairs(h[k], y);
        if (in[k]) write_s8<VEC>(a.p.q, a.p.ldq, row, chunk_col<VEC>(k * tpr + t), a.dim, f, finite, y);
      }
      if (t == 0) a.p.scales[row] = s8_scale(__uint_as_float(amax));
    } else {
      auto load = [&](int c, bool in, float (&h)[8]) {
        Inputs<VEC, TX, TR> raw;
        raw.load(a, row, c, in);
        raw.sum(a, h);
      };
      for (int chunk = t; chunk < chunks; chunk += tpr) {
        const int c = chunk_col<VEC>(chunk);
        float h[8];
        load(c, c < a.dim, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += h[i];
      }
      const float mean = mean_of();
      const uint64_t minus_mean = f32x2(-mean, -mean);
      uint64_t left = 0ull, squares = 0ull;
      // the differences from the mean of one chunk
      auto differences = [&](int c, bool in, uint64_t (&d)[4], uint64_t& s, uint64_t& ss) {
        float h[8];
        load(c, in, h);
        to_pairs(h, d);
        center<VEC>(d, minus_mean, c, a.dim, in, s, ss);
      };
      for (int chunk = t; chunk < chunks; chunk += tpr) {
        uint64_t d[4];
        const int c = chunk_col<VEC>(chunk);
        differences(c, c < a.dim, d, left, squares);
      }
      statistics(row, mean, both(left), both(squares), off, rstd);
      uint64_t unused = 0ull;
      float f = 0.0f;
      bool finite = true;
      if (s8) {
        uint32_t amax = 0u;
        auto search = [&](bool only_finite) {
          uint32_t m = 0u;
          for (int chunk = t; chunk < chunks; chunk += tpr) {
            const int c = chunk_col<VEC>(chunk);
            uint64_t d[4];
            float y[8];
            differences(c, c < a.dim, d, unused, unused);
            affine<VEC>(a.p.weight, a.p.bias, c, a.dim, c < a.dim, rstd, off, d, y);
            m = max(m, only_finite ? chunk_finite_max(y) : chunk_max(y));
          }
          return m;
        };
        amax = largest_of(search(false));
        finite = amax < kInfBits;
        if (!finite) amax = largest_finite_of(search(true));
        f = s8_factor(__uint_as_float(amax));
        if (t == 0) a.p.scales[row] = s8_scale(__uint_as_float(amax));
      }
      for (int base = 0; base < chunks; base += tpr) {  // whole warps: write_fp8 shuffles
        const int chunk = base + t;
        const int c = chunk_col<VEC>(chunk);
        const bool in = chunk < chunks && c < a.dim;
        float h[8], y[8];
        load(c, in, h);
        if (in && a.p.h != nullptr) store8<VEC>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, h);
        uint64_t d[4];
        to_pairs(h, d);
        center<VEC>(d, minus_mean, c, a.dim, in, unused, unused);
        affine<VEC>(a.p.weight, a.p.bias, c, a.dim, in, rstd, off, d, y);
        if (in && a.p.y != nullptr) store8<VEC>(a.p.y, a.p.y_type, row * a.p.ldy, c, a.dim, y);
        if (f8) write_fp8<VEC>(a.p.q, a.p.ldq, a.p.scales, a.p.ld_scales, row, c, a.dim, in, y);
        if (s8 && in) write_s8<VEC>(a.p.q, a.p.ldq, row, c, a.dim, f, finite, y);
      }
    }
  }
  if (RING && t == 0 && ring.abort_flag) drain_ring(ring.full + bar_off, a.ring.stages, slot, parity);
}

// ---------------------------------------------------------------- backward
struct LnGradArgs {
  int64_t rows;
  int dim;
  int tpr;
  RingArgs ring;
  gemm_layernorm_grad_t p;
  float* part;  // partial sums of dw and db: a row of 2 dim floats per CTA, or nullptr
};

// As norm_grad_kernel, with the two sums of a row taken together.
template <int C, bool VEC, int TD, int TH, bool RING = false>
__global__ void __launch_bounds__(kMaxThreads, 1)
    layernorm_grad_kernel(const __grid_constant__ LnGradArgs a) {
  __shared__ float red[kMaxRings][2][16][2];
  __shared__ LnRings ring;
  extern __shared__ uint4 dyn_smem[];  // the weight and the rings, or several rows' sums
  float* const weights = reinterpret_cast<float*>(dyn_smem);
  const int tpr = a.tpr;
  const int t = threadIdx.x % tpr, group = threadIdx.x / tpr;
  const int per_cta = blockDim.x / tpr;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * per_cta;
  int64_t row = static_cast<int64_t>(blockIdx.x) * per_cta + group;
  const int ring_dim = RING ? a.dim : 0;
  const int bytes_d = ring_dim * type_bytes(TD), bytes_h = ring_dim * type_bytes(TH);
  const int bytes_r = a.p.residual_grad == nullptr ? 0 : ring_dim * type_bytes(a.p.residual_grad_type);
  const int stage_bytes = bytes_d + bytes_h + bytes_r;
  uint8_t* const stages = reinterpret_cast<uint8_t*>(weights + ring_dim) + group * a.ring.stages * stage_bytes;
  uint64_t* const full = ring.full + (RING ? group * kMaxStages : 0);
  auto fetch = [&](int64_t row, int s) {
    uint8_t* to = stages + s * stage_bytes;
    uint64_t* bar = &full[s];
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
  if (RING) {
    if (t == 0) {
      for (int s = 0; s < a.ring.stages; ++s) mbar_init(&full[s], 1);
      if (group == 0) ring.abort_flag = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (RING) {
    if (t == 0)
      for (int s = 0; s < a.ring.stages; ++s)
        if (row + s * row_step < a.rows) fetch(row + s * row_step, s);
    stage_weights(weights, a.p.weight, nullptr, a.dim, false);
    __syncthreads();
  }
  int slot = 0;
  uint32_t parity = 0;
  const int chunks = VEC ? a.dim / 8 : (a.dim + kFp8Block - 1) / kFp8Block * 16;
  const float inv_dim = 1.0f / static_cast<float>(a.dim);
  constexpr int CR = C > 0 ? C : 1;
  uint64_t dw[CR][4], db[CR][4];
#pragma unroll
  for (int k = 0; k < CR; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[k][i] = db[k][i] = 0ull;
  uint32_t turn = 0;
  // dy times the weight
  auto weighted = [&](int c, uint64_t (&g)[4]) {
    float v[8];
    uint64_t w[4];
    if constexpr (RING) {
      staged_pairs(weights + c, w);
    } else {
      if (a.p.weight == nullptr) return;
      load_weight<VEC>(a.p.weight, c, a.dim, v);
      to_pairs(v, w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = mul2(g[i], w[i]);
  };
  // (h - mean) * rstd, zero past the row's end; g is zero there
  auto normal = [&](int c, float rstd, float mean, uint64_t (&xh)[4]) {
    const uint64_t m = f32x2(-mean, -mean), s = f32x2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xh[i] = mul2(add2(xh[i], m), s);
      if (!VEC) {
        const float2 f = f32x2_parts(xh[i]);
        xh[i] = f32x2(inside<VEC>(c, 2 * i, a.dim) ? f.x : 0.0f, inside<VEC>(c, 2 * i + 1, a.dim) ? f.y : 0.0f);
      }
    }
  };
  // the gradient of h: r + rstd * (g - mean_g - xh * mean_x)
  auto gradient = [&](const uint64_t (&g)[4], const uint64_t (&xh)[4], float rstd, float2 means, float (&r)[8]) {
    float gv[8], xv[8];
    from_pairs(g, gv);
    from_pairs(xh, xv);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = fmaf(rstd, fmaf(-xv[i], means.y, gv[i] - means.x), r[i]);
  };
  float next_rstd = row < a.rows ? a.p.rstd[row] : 0.0f;  // loaded a row ahead
  float next_mean = row < a.rows ? a.p.mean[row] : 0.0f;
  // the row's means of g and of g xh, given a thread's sums
  auto means_of = [&](uint64_t sum_g, uint64_t sum_x) {
    float v[2] = {both(sum_g), both(sum_x)};
    over_row<2>(v, tpr, group, red[RING ? group : 0], turn);
    return make_float2(v[0] * inv_dim, v[1] * inv_dim);
  };
  for (; row < a.rows; row += row_step, ++turn) {
    const float rstd = next_rstd, mean = next_mean;
    if (row + row_step < a.rows) {
      next_rstd = a.p.rstd[row + row_step];
      next_mean = a.p.mean[row + row_step];
    }
    uint64_t sum_g = 0ull, sum_x = 0ull;  // of g, and of g xh
    if constexpr (C > 0) {
      Raw8<TD> dy[C];
      Raw8<TH> rh[C];
      const uint8_t* from = stages + slot * stage_bytes;
      if (RING) mbar_wait_late(&full[slot], parity, &ring.abort_flag, a.ring.err);
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
      auto has = [&](int k) {
        const int chunk = k * tpr + t;
        return chunk < chunks && chunk_col<VEC>(chunk) < a.dim;
      };
      // the registers hold both inputs but for two chunks loaded one by one
      constexpr bool kHeld = !RING && (VEC || C == 1);
      if (kHeld) {
#pragma unroll
        for (int k = 0; k < C; ++k) get(k, chunk_col<VEC>(k * tpr + t), has(k));
      }
      // From a ring of bf16 rows, the first pass's g and xh stay for the second
      // (8192 x 4096 55.5 us against 61.7 with the rows read again); in fp32 those
      // registers cost more than the reads (106 us against 98).
      constexpr bool kKept = RING && TD == GEMM_OUT_BF16 && TH == GEMM_OUT_BF16;
      uint64_t gs[kKept ? C : 1][4], xs[kKept ? C : 1][4];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = chunk_col<VEC>(k * tpr + t);
        if (!kHeld) get(k, c, has(k));
        if (!has(k)) continue;
        float v[8];
        uint64_t(&g)[4] = gs[kKept ? k : 0];
        uint64_t(&xh)[4] = xs[kKept ? k : 0];
        widen8<VEC, TD>(dy[k], a.p.dy_type, v);  // zeros past the row's end
        to_pairs(v, g);
        widen8<VEC, TH>(rh[k], a.p.h_type, v);
        to_pairs(v, xh);
        normal(c, rstd, mean, xh);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          db[k][i] = add2(db[k][i], g[i]);
          dw[k][i] = fma2(g[i], xh[i], dw[k][i]);
        }
        weighted(c, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum_g = add2(sum_g, g[i]);
          sum_x = fma2(g[i], xh[i], sum_x);
        }
      }
      const float2 means = means_of(sum_g, sum_x);
      if (RING && t == 0 && turn > 0) {
        // every thread has left the previous row (the sums' barrier)
        const int64_t next = row + (a.ring.stages - 1) * row_step;
        if (next < a.rows && !*const_cast<volatile int*>(&ring.abort_flag))
          fetch(next, slot == 0 ? a.ring.stages - 1 : slot - 1);
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int c = chunk_col<VEC>(k * tpr + t);
        if (!has(k)) continue;
        if (!kHeld && !kKept) get(k, c, true);
        float r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
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
        uint64_t(&g)[4] = gs[kKept ? k : 0];
        uint64_t(&xh)[4] = xs[kKept ? k : 0];
        if (!kKept) {
          float v[8];
          widen8<VEC, TD>(dy[k], a.p.dy_type, v);
          to_pairs(v, g);
          weighted(c, g);
          widen8<VEC, TH>(rh[k], a.p.h_type, v);
          to_pairs(v, xh);
          normal(c, rstd, mean, xh);
        }
        gradient(g, xh, rstd, means, r);
        store8<VEC>(a.p.dh, a.p.dh_type, row * a.p.lddh, c, a.dim, r);
      }
      if (RING && ++slot == a.ring.stages) {
        slot = 0;
        parity ^= 1u;
      }
    } else {
      float2 means = make_float2(0.0f, 0.0f);
      for (int half = 0; half < 2; ++half) {
        if (half == 1) means = means_of(sum_g, sum_x);
        for (int chunk = t; chunk < chunks; chunk += tpr) {
          const int c = chunk_col<VEC>(chunk);
          if (c >= a.dim) continue;
          float v[8], r[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
          uint64_t g[4], xh[4];
          const Raw8<TD> dy = load8<VEC, TD>(a.p.dy, a.p.dy_type, row * a.p.lddy, c, a.dim, true);
          const Raw8<TH> rh = load8<VEC, TH>(a.p.h, a.p.h_type, row * a.p.ldh, c, a.dim, true);
          if (half == 1 && a.p.residual_grad != nullptr)
            widen8<VEC, kAnyType>(load8<VEC, kAnyType>(a.p.residual_grad, a.p.residual_grad_type,
                                                       row * a.p.ldrg, c, a.dim, true),
                                  a.p.residual_grad_type, r);
          widen8<VEC, TD>(dy, a.p.dy_type, v);
          to_pairs(v, g);
          weighted(c, g);
          widen8<VEC, TH>(rh, a.p.h_type, v);
          to_pairs(v, xh);
          normal(c, rstd, mean, xh);
          if (half == 1) {
            gradient(g, xh, rstd, means, r);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sum_g = add2(sum_g, g[i]);
              sum_x = fma2(g[i], xh[i], sum_x);
            }
          }
          if (half == 1) store8<VEC>(a.p.dh, a.p.dh_type, row * a.p.lddh, c, a.dim, r);
        }
      }
    }
  }
  if (RING && t == 0 && ring.abort_flag) drain_ring(full, a.ring.stages, slot, parity);
  if (C == 0 || a.part == nullptr) return;
  if (RING && per_cta > 1) __syncthreads();  // the rings make room for the sums
  // dw in the first dim columns of the CTA's row of `part`, db in the others
  float* out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.dim;
  float* sums = reinterpret_cast<float*>(dyn_smem);
#pragma unroll
  for (int k = 0; k < CR; ++k) {
    const int chunk = k * tpr + t;
    const int c = chunk_col<VEC>(chunk);
    if (chunk >= chunks || c >= a.dim) continue;
    float* to = per_cta == 1 ? out : sums + static_cast<int64_t>(group) * 2 * a.dim;
    float w[8], b[8];
    from_pairs(dw[k], w);
    from_pairs(db[k], b);
    if constexpr (VEC) {  // (value by value a CTA's sums would take 4 us to leave it)
      float4* to_w = reinterpret_cast<float4*>(to + c);
      float4* to_b = reinterpret_cast<float4*>(to + a.dim + c);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        to_w[i] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        to_b[i] = make_float4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = c + 16 * i;
        if (col < a.dim) {
          to[col] = w[i];
          to[a.dim + col] = b[i];
        }
      }
    }
  }
  if (per_cta == 1) return;
  __syncthreads();
  for (int col = threadIdx.x; col < 2 * a.dim; col += blockDim.x) {
    float s = 0.0f;
    for (int r = 0; r < per_cta; ++r) s += sums[r * 2 * a.dim + col];
    out[col] = s;
  }
}

// dw and db of rows too long for layernorm_grad_kernel's registers: one column
// per thread, the rows cut into gridDim.y parts, one row of `part` each.
__global__ void __launch_bounds__(256) layernorm_dweight_kernel(const __grid_constant__ LnGradArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (col >= a.dim) return;
  float w = 0.0f, b = 0.0f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float dy = load1(a.p.dy, a.p.dy_type, row * a.p.lddy + col);
    b += dy;
    w = fmaf(dy, (load1(a.p.h, a.p.h_type, row * a.p.ldh + col) - a.p.mean[row]) * a.p.rstd[row], w);
  }
  float* out = a.part + blockIdx.y * 2 * static_cast<int64_t>(a.dim) + col;
  out[0] = w;
  out[a.dim] = b;
}

// Adds the parts of dw and db, 128 of their 2 dim columns to a CTA (dim % 4 == 0),
// every eighth part to a warp: for few parts, with fewer threads to launch than
// add_parts_kernel (64 rows of 8192 7.7 us against 9.4).
__global__ void __launch_bounds__(256) layernorm_parts_kernel(const float* part, int parts, int dim,
                                                              float* dweight, float* dbias) {
  __shared__ float4 sums[8][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t pitch = 2 * static_cast<int64_t>(dim), first = static_cast<int64_t>(blockIdx.x) * 128;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (first + lane * 4 < pitch) {
    const float4* from = reinterpret_cast<const float4*>(part + first) + lane;
#pragma unroll 8
    for (int p = warp; p < parts; p += 8) {
      const float4 v = __ldcg(from + p * (pitch / 4));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  const int64_t col = first + threadIdx.x;
  if (threadIdx.x >= 128 || col >= pitch) return;
  float total = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) total += reinterpret_cast<const float*>(sums[w])[threadIdx.x];
  if (col < dim) {
    if (dweight != nullptr) dweight[col] = total;
  } else if (dbias != nullptr) {
    dbias[col - dim] = total;
  }
}

// Groups per CTA (p.per_cta), CTAs per SM (the return value; 0: no rings) and
// stages of each group's ring of rows of `bytes`, next to `weights` bytes of
// weights, if there are enough rows.  sm_threads: what the instance's registers
// let an SM hold.  Groups need a barrier each, so short rows take two CTAs.
// fewer: fewer groups than that where there are too few rows for them.
int plan_groups(RowPlan& p, int64_t rows, int64_t bytes, int64_t weights, int num_sms, int sm_threads,
                bool fewer, RingArgs& ring) {
  if (p.per_cta != 1 || p.chunks_per_thread == 0 || p.tpr == 32) return 0;
  const int per_sm = 2 * kMaxRings * p.tpr <= sm_threads ? 2 : 1;
  int groups = sm_threads / per_sm / p.tpr;
  if (groups > kMaxRings) groups = kMaxRings;
  for (; groups >= 1; --groups) {
    const int64_t stages = (kSmBytes / per_sm - kLnCtaBytes - weights) / (groups * bytes);
    if (stages < 2) continue;
    if (rows < 2 * static_cast<int64_t>(per_sm) * num_sms * groups) {
      if (fewer) continue;
      return 0;
    }
    ring.stages = static_cast<int>(stages < kMaxStages ? stages : kMaxStages);
    p.per_cta = groups;
    return per_sm;
  }
  return 0;
}

// Rows moved in vectors have an instance for each pair of input types; the
// others look at the types as they go.
template <bool VEC, int TX, int TR>
cudaError_t launch_ln(const LnArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid));
  const int threads = p.tpr * p.per_cta;
  if constexpr (VEC) {
    if (a.ring.stages > 0) {  // more than one warp a row: two chunks a thread (plan_rows)
      const size_t row = static_cast<size_t>(a.dim) * (type_bytes(TX) + (TR < 0 ? 0 : type_bytes(TR)));
      const size_t smem = 8 * static_cast<size_t>(a.dim) + p.per_cta * a.ring.stages * row;
      if (a.p.q == nullptr) return ops_launch<layernorm_kernel<2, VEC, TX, TR, true, kNoQ>>(g, threads, smem, 1, s, a);
      if (a.p.q_type == GEMM_OUT_S8)
        return ops_launch<layernorm_kernel<2, VEC, TX, TR, true, GEMM_OUT_S8>>(g, threads, smem, 1, s, a);
      return ops_launch<layernorm_kernel<2, VEC, TX, TR, true, GEMM_OUT_F8E4M3>>(g, threads, smem, 1, s, a);
    }
  }
  switch (p.chunks_per_thread) {
    case 1: return ops_launch<layernorm_kernel<1, VEC, TX, TR>>(g, threads, 0, 1, s, a);
    case 2: return ops_launch<layernorm_kernel<2, VEC, TX, TR>>(g, threads, 0, 1, s, a);
    case 4: return ops_launch<layernorm_kernel<4, VEC, TX, TR>>(g, threads, 0, 1, s, a);
    default: return ops_launch<layernorm_kernel<0, VEC, TX, TR>>(g, threads, 0, 1, s, a);
  }
}

template <int TX>
cudaError_t launch_ln_vec(const LnArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  if (a.p.residual == nullptr) return launch_ln<true, TX, -1>(a, p, grid, s);
  return a.p.residual_type == GEMM_OUT_BF16 ? launch_ln<true, TX, GEMM_OUT_BF16>(a, p, grid, s)
                                            : launch_ln<true, TX, GEMM_OUT_F32>(a, p, grid, s);
}

cudaError_t launch_ln_any(const LnArgs& a, const RowPlan& p, bool vec, int grid, cudaStream_t s) {
  if (vec)
    return a.p.x_type == GEMM_OUT_BF16 ? launch_ln_vec<GEMM_OUT_BF16>(a, p, grid, s)
                                       : launch_ln_vec<GEMM_OUT_F32>(a, p, grid, s);
  return a.p.residual == nullptr ? launch_ln<false, kAnyType, -1>(a, p, grid, s)
                                 : launch_ln<false, kAnyType, kAnyType>(a, p, grid, s);
}

template <bool VEC, int TD, int TH>
cudaError_t launch_ln_grad(const LnGradArgs& a, const RowPlan& p, int grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid));
  const int threads = p.tpr * p.per_cta;
  const size_t smem = p.per_cta > 1 ? sizeof(float) * 2 * p.per_cta * a.dim : 0;
  if constexpr (VEC) {
    if (a.ring.stages > 0) {
      const int rg = a.p.residual_grad == nullptr ? 0 : type_bytes(a.p.residual_grad_type);
      const size_t row = static_cast<size_t>(a.dim) * (type_bytes(TD) + type_bytes(TH) + rg);
      const size_t bytes = 4 * static_cast<size_t>(a.dim) + p.per_cta * a.ring.stages * row;
      return ops_launch<layernorm_grad_kernel<2, VEC, TD, TH, true>>(g, threads, bytes, 1, s, a);
    }
  }
  switch (p.chunks_per_thread) {
    case 1: return ops_launch<layernorm_grad_kernel<1, VEC, TD, TH>>(g, threads, smem, 1, s, a);
    case 2: return ops_launch<layernorm_grad_kernel<2, VEC, TD, TH>>(g, threads, smem, 1, s, a);
    default: return ops_launch<layernorm_grad_kernel<0, VEC, TD, TH>>(g, threads, 0, 1, s, a);
  }
}

cudaError_t launch_ln_grad_any(const LnGradArgs& a, const RowPlan& p, bool vec, int grid, cudaStream_t s) {
  constexpr int B = GEMM_OUT_BF16, F = GEMM_OUT_F32;
  if (!vec) return launch_ln_grad<false, kAnyType, kAnyType>(a, p, grid, s);
  if (a.p.dy_type == B)
    return a.p.h_type == B ? launch_ln_grad<true, B, B>(a, p, grid, s) : launch_ln_grad<true, B, F>(a, p, grid, s);
  return a.p.h_type == B ? launch_ln_grad<true, F, B>(a, p, grid, s) : launch_ln_grad<true, F, F>(a, p, grid, s);
}

}  // namespace
}  // namespace g12

using namespace g12;

extern "C" {

gemm_status_t gemm_layernorm(int64_t rows, int64_t dim, const gemm_layernorm_t* args, void* stream) {
  if (args == nullptr || rows < 0 || dim < 0 || rows > kOpsMaxDim || dim > (int64_t{1} << 30))
    return GEMM_ERR_INVALID_VALUE;
  if (rows == 0 || dim == 0) return GEMM_OK;
  const gemm_layernorm_t& p = *args;
  bool vec = dim % 8 == 0;
  if (!array_ok(p.x, p.x_type, p.ldx, dim, true, vec) ||
      !array_ok(p.residual, p.residual_type, p.ldr, dim, false, vec) ||
      !array_ok(p.h, p.h_type, p.ldh, dim, false, vec) ||
      !array_ok(p.y, p.y_type, p.ldy, dim, false, vec) ||
      !array_ok(p.weight, GEMM_OUT_F32, dim, dim, false, vec) ||
      !array_ok(p.bias, GEMM_OUT_F32, dim, dim, false, vec))
    return GEMM_ERR_INVALID_VALUE;
  if ((p.q == nullptr) != (p.scales == nullptr)) return GEMM_ERR_INVALID_VALUE;
  if (p.q != nullptr) {
    if ((p.q_type != GEMM_OUT_F8E4M3 && p.q_type != GEMM_OUT_S8) || p.ldq < dim || p.ldq > kOpsMaxDim ||
        ops_misaligned(p.scales, 4) ||
        (p.q_type == GEMM_OUT_F8E4M3 && (p.ld_scales < rows || p.ld_scales > kOpsMaxDim)))
      return GEMM_ERR_INVALID_VALUE;
    if (ops_misaligned(p.q, 8) || p.ldq % 8 != 0) vec = false;
  }
  if ((p.mean != nullptr && ops_misaligned(p.mean, 4)) || (p.rstd != nullptr && ops_misaligned(p.rstd, 4)))
    return GEMM_ERR_INVALID_VALUE;
  if (p.h == nullptr && p.y == nullptr && p.q == nullptr && p.mean == nullptr && p.rstd == nullptr)
    return GEMM_OK;
  int sms = 0;
  uint32_t* err = nullptr;
  const gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  LnArgs a{};
  a.rows = rows;
  a.dim = static_cast<int>(dim);
  a.p = p;
  const int64_t chunks = vec ? dim / 8 : (dim + kFp8Block - 1) / kFp8Block * 16;
  // Four chunks a thread, but one where four leave 33 to 64 threads a row, 1025 to
  // 2048 elements (us, one / four: 400 x 1032 2.9 / 3.9, 1000 x 1280 5.0 / 6.7, 1000 x
  // 2048 5.8 / 7.5, 2400 x 1536 11.3 / 12.1, 2400 x 2048 10.0 / 13.0, ragged 1000 x 1100
  // 6.3 / 10.3, 8000 x 1999 46 / 66; 150 x 1032 to 2048 alike; shorter rows fit a warp:
  // 2000 x 1024 7.2 / 4.5).
  RowPlan pl = plan_rows(rows, chunks, sms, chunks > 128 && chunks <= 256 ? 1 : 4, 4);
  a.tpr = pl.tpr;
  a.ring.err = err;
  int grid = row_grid(rows, pl, sms, 1024);
  if (vec) {
    const int64_t bytes = dim * (type_bytes(p.x_type) +
                                 (p.residual == nullptr ? 0 : type_bytes(p.residual_type)));
    RowPlan pr = plan_rows(rows, chunks, sms, 2, 2);
    const int per_sm = plan_groups(pr, rows, bytes, 8 * dim, sms, 1024, false, a.ring);
    if (per_sm > 0) {
      grid = per_sm * sms;
      pl = pr;
      a.tpr = pl.tpr;
    }
  }
  return abi_from_cuda(launch_ln_any(a, pl, vec, grid, static_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_layernorm_backward(int64_t rows, int64_t dim, const gemm_layernorm_grad_t* args,
                                      void* stream) {
  if (args == nullptr || rows < 0 || dim < 0 || rows > kOpsMaxDim || dim > (int64_t{1} << 30))
    return GEMM_ERR_INVALID_VALUE;
  if (dim == 0) return GEMM_OK;
  const gemm_layernorm_grad_t& p = *args;
  bool vec = dim % 8 == 0;
  const bool some = rows > 0;
  if (!array_ok(p.dy, p.dy_type, p.lddy, dim, some, vec) ||
      !array_ok(p.h, p.h_type, p.ldh, dim, some, vec) ||
      !array_ok(p.residual_grad, p.residual_grad_type, p.ldrg, dim, false, vec) ||
      !array_ok(p.dh, p.dh_type, p.lddh, dim, some, vec) ||
      !array_ok(p.weight, GEMM_OUT_F32, dim, dim, false, vec))
    return GEMM_ERR_INVALID_VALUE;
  if (some && (p.rstd == nullptr || ops_misaligned(p.rstd, 4) || p.mean == nullptr ||
               ops_misaligned(p.mean, 4)))
    return GEMM_ERR_INVALID_VALUE;
  if ((p.dweight != nullptr && ops_misaligned(p.dweight, 4)) ||
      (p.dbias != nullptr && ops_misaligned(p.dbias, 4)))
    return GEMM_ERR_INVALID_VALUE;
  const bool params = p.dweight != nullptr || p.dbias != nullptr;
  if (!some && !params) return GEMM_OK;
  int sms = 0;
  uint32_t* err = nullptr;
  gemm_status_t st = abi_device(&sms, &err);
  if (st != GEMM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!some) {
    cudaError_t e = cudaSuccess;
    for (float* d : {p.dweight, p.dbias})
      if (d != nullptr && e == cudaSuccess) e = cudaMemsetAsync(d, 0, sizeof(float) * dim, s);
    return abi_from_cuda(e);
  }
  LnGradArgs a{};
  a.rows = rows;
  a.dim = static_cast<int>(dim);
  a.p = p;
  const int64_t chunks = vec ? dim / 8 : (dim + kFp8Block - 1) / kFp8Block * 16;
  // From rings, and where a row takes one warp, two chunks a thread (one and twice
  // the threads: 8192 x 4096 66 us against 61, 16384 x 1024 41 against 36, 3000 x 512
  // 16 against 9), else one.  Rings even with fewer groups (1000 x 1024 10 us, 18
  // without, 2000 x 1024 11 and 22; the forward pass is faster without).
  RowPlan pl = plan_rows(rows, chunks, sms, vec ? 2 : 1, 2);
  a.ring.err = err;
  int per_sm = 0;
  if (vec && pl.chunks_per_thread == 2) {
    const int64_t bytes =
        dim * (type_bytes(p.dy_type) + type_bytes(p.h_type) +
               (p.residual_grad == nullptr ? 0 : type_bytes(p.residual_grad_type)));
    per_sm = plan_groups(pl, rows, bytes, 4 * dim, sms, kMaxThreads, true, a.ring);
  }
  if (per_sm == 0 && pl.tpr > 32) pl = plan_rows(rows, chunks, sms, 1, 2);
  a.tpr = pl.tpr;
  const int grid = per_sm > 0 ? per_sm * sms : row_grid(rows, pl, sms, 512);
  const bool by_column = pl.chunks_per_thread == 0;
  int parts = grid;
  if (by_column) {  // up to 64, of 256 MB together
    parts = static_cast<int>(rows < 64 ? rows : 64);
    while (parts > 1 && 2 * parts * dim > (int64_t{1} << 26)) parts /= 2;
  }
  std::unique_lock<std::mutex> lock;
  if (params) {
    st = abi_scratch(s, static_cast<int64_t>(parts) * 2 * dim, lock, &a.part);
    if (st != GEMM_OK) return st;
  }
  cudaError_t e = cudaSuccess;
  if (by_column && params) {  // first: dh may take the place of dy or h
    const dim3 g(static_cast<unsigned>((dim + 255) / 256), static_cast<unsigned>(parts));
    e = ops_launch<layernorm_dweight_kernel>(g, 256, 0, 1, s, a);
  }
  if (e == cudaSuccess) e = launch_ln_grad_any(a, pl, vec, grid, s);
  if (e != cudaSuccess || !params) return abi_from_cuda(e);
  const float* part = a.part;
  if (dim % 4 == 0 && parts <= 64)
    return abi_from_cuda(ops_launch<layernorm_parts_kernel>(dim3(static_cast<unsigned>((2 * dim + 127) / 128)), 256,
                                                            0, 1, s, part, parts, a.dim, p.dweight, p.dbias));
  const dim3 g(static_cast<unsigned>((dim + 31) / 32), 2);
  return abi_from_cuda(ops_launch<add_parts_kernel>(g, 1024, 0, 1, s, part, parts, a.dim, 2 * dim,
                                                    p.dweight, p.dbias));
}

}  // extern "C"
