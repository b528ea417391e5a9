// norm.cuh -- what the norms over rows share (norm.cu, layernorm.cu): sums over
// a row, the ring that rows come through, where a thread's elements lie, the
// last step of the weight's gradient, and how rows are shared out.
#pragma once

#include "ops.cuh"

namespace g12 {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxRowsPerCta = 8;

// Many rows that fit the registers come through a ring in shared memory: one
// thread copies whole rows (bulk copies, so no registers wait for them) up to
// `stages` rows ahead of the one that the CTA works on.  Without it the loads
// of a row wait for the CTA's previous row, and too few bytes are in flight:
// 8192 rows of 8192 in bf16 took 110 us (63 % of the copy rate, 25 %
// occupancy); with it they take 78 us (88 %).
constexpr int kMaxStages = 4;
constexpr int kSmBytes = 227 * 1024;  // an SM's shared memory, for all its CTAs
constexpr int kCtaBytes = 1536;       // of it taken by a CTA besides the ring

struct RingArgs {
  int stages;        // 0: rows are loaded from global memory
  uint32_t* err;
};

struct Ring {
  uint64_t full[kMaxStages];
  int abort_flag;
};

// Starts the barriers; all threads, before the first copy.
__device__ __forceinline__ void ring_init(Ring& r, int stages) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&r.full[s], 1);
    r.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
}

// After a wait ran out: the copies in flight land before the CTA leaves.
__device__ __forceinline__ void drain(Ring& r, int stages, int slot, uint32_t parity) {
  for (int i = 0; i < stages; ++i) {
    mbar_drain_wait(&r.full[slot], parity);
    if (++slot == stages) {
      slot = 0;
      parity ^= 1u;
    }
  }
}

constexpr int type_bytes(int t) { return t == GEMM_OUT_BF16 ? 2 : 4; }

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

// Bits of |v|: they order like the values, infinities and NaN above all.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// Largest of the bits over the tpr threads of a row, which are group `group` of
// the CTA's.  red: two rows of a value per warp, used in turn, one call a row.
__device__ __forceinline__ uint32_t row_max_bits(uint32_t m, int tpr, int group, uint32_t (*red)[16],
                                                 uint32_t turn) {
  m = __reduce_max_sync(0xffffffffu, m);
  if (tpr == 32) return m;
  const int lane = threadIdx.x & 31, warps = tpr >> 5;
  uint32_t* mine = red[turn & 1u];
  if (lane == 0) mine[(threadIdx.x >> 5) % warps] = m;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
  return __reduce_max_sync(0xffffffffu, lane < warps ? mine[lane & 15] : 0u);
}

// Where the eight elements of chunk `chunk` lie: consecutive (VEC), or every
// 16th of a 128-column block from `c` on (see ops.cuh).
template <bool VEC>
__device__ __forceinline__ int chunk_col(int chunk) {
  return VEC ? chunk * 8 : (chunk >> 4) * kFp8Block + (chunk & 15);
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

// A chunk of a row in fp8.  All 32 lanes call it together; lanes without
// elements (in == false) take part in the block's maximum only.
template <bool VEC>
__device__ __forceinline__ void write_fp8(void* q_rows, int64_t ldq, float* scales, int64_t ld_scales,
                                          int64_t row, int c, int dim, bool in, const float (&y)[8]) {
  const float amax = block_amax<16>(y);
  if (!in) return;
  const float f = fp8_factor(amax);
  uint8_t* q = static_cast<uint8_t*>(q_rows) + row * ldq;
  if (VEC) {
    *reinterpret_cast<uint2*>(q + c) = make_uint2(pack_e4m3(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                                                  pack_e4m3(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < dim)
        q[c + 16 * i] = __nv_cvt_float_to_fp8(y[i] * f, __NV_SATFINITE, __NV_E4M3);
  }
  if ((threadIdx.x & 15) == 0) scales[(c >> 7) * ld_scales + row] = fp8_scale(amax);
}

// A chunk of a row in int8, given the factor of the row.  finite: neither
// infinities nor NaN in the row.  Its products then lie within +-127.001, and
// adding 1.5 * 2^23 rounds them to whole numbers in the last bits, two's
// complement (the conversion instruction takes 16 a cycle).  The product is
// rounded before that, as round_s8's is: a value's byte is the same whatever else
// is in its row, and whichever kernel makes it.  Both in one fused operation
// would decide ties by the factor's own rounding, and half of a row's largest
// value, 63.5 steps, is common in bf16; so the product is __fmul_rn's, which is
// never joined to an addition (see mul2).
template <bool VEC>
__device__ __forceinline__ void write_s8(void* q_rows, int64_t ldq, int64_t row, int c, int dim, float f,
                                         bool finite, const float (&y)[8]) {
  int8_t* q = static_cast<int8_t*>(q_rows) + row * ldq;
  uint32_t w[8];
  if (finite) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t p = f32x2(__fmul_rn(y[i], f), __fmul_rn(y[i + 1], f));
      const float2 r = f32x2_parts(add2(p, f32x2(12582912.0f, 12582912.0f)));
      w[i] = __float_as_uint(r.x);
      w[i + 1] = __float_as_uint(r.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = static_cast<uint32_t>(round_s8(y[i] * f));
  }
  if (VEC) {
    *reinterpret_cast<uint2*>(q + c) = make_uint2(low_bytes(w[0], w[1], w[2], w[3]),
                                                  low_bytes(w[4], w[5], w[6], w[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < dim) q[c + 16 * i] = static_cast<int8_t>(w[i]);
  }
}

// x and the residual (TR < 0: none) of one chunk.
template <bool VEC, int TX, int TR>
struct Inputs {
  Raw8<TX> x;
  Raw8<TR < 0 ? int{GEMM_OUT_BF16} : TR> r;
  template <typename A>
  __device__ __forceinline__ void load(const A& a, int64_t row, int c, bool in) {
    x = load8<VEC, TX>(a.p.x, a.p.x_type, row * a.p.ldx, c, a.dim, in);
    if constexpr (TR >= 0)
      r = load8<VEC, TR>(a.p.residual, a.p.residual_type, row * a.p.ldr, c, a.dim, in);
  }
  template <typename A>
  __device__ __forceinline__ void from_ring(const A& a, const uint8_t* stage, int c, bool in) {
    x = Raw8<TX>{};
    r = {};
    if (!in) return;
    x = load8_smem<TX>(stage, c);
    if constexpr (TR >= 0) r = load8_smem<TR>(stage + a.dim * type_bytes(TX), c);
  }
  template <typename A>
  __device__ __forceinline__ void sum(const A& a, float (&h)[8]) const {
    widen8<VEC, TX>(x, a.p.x_type, h);
    if constexpr (TR >= 0) {
      float v[8];
      widen8<VEC, TR>(r, a.p.residual_type, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] += v[i];
    }
  }
};

// out[col] = sum of the `parts` partial sums, always in the same order: a
// warp's lanes take 32 columns, the block's 32 warps every 32nd part (few
// loads one after the other: the time of this kernel is their latency).
// Two sums of `dim` columns may share a row of the parts (`pitch` apart): the
// second, for blockIdx.y == 1, goes to out1.  An output may be nullptr.
__global__ void __launch_bounds__(1024) add_parts_kernel(const float* part, int parts, int dim,
                                                         int64_t pitch, float* out0, float* out1) {
  __shared__ float sums[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  float* out = blockIdx.y == 0 ? out0 : out1;
  if (out == nullptr) return;
  part += static_cast<int64_t>(blockIdx.y) * dim;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (col < dim) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 32) s += __ldcg(part + p * pitch + col);
  }
  sums[warp][lane] = s;
  __syncthreads();
  // warp w adds column w's 32 sums
  s = sums[lane][warp];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const int64_t to = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && to < dim) out[to] = s;
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

// CTAs per SM and stages of a ring of rows of `bytes`, if there are enough
// rows to use it; leaves ring.stages at 0 otherwise.  sm_threads: what the
// instance's registers let an SM hold.
int plan_ring(const RowPlan& p, int64_t rows, int64_t bytes, int num_sms, int sm_threads,
              RingArgs& ring) {
  if (p.per_cta != 1 || p.chunks_per_thread == 0 || p.tpr == 32) return 0;
  for (int per_sm = sm_threads / p.tpr; per_sm >= 1; --per_sm) {
    const int64_t stages = (kSmBytes / per_sm - kCtaBytes) / bytes;
    if (stages < 3 && per_sm > 1) continue;
    if (stages < 2 || rows < 2 * static_cast<int64_t>(per_sm) * num_sms) return 0;
    ring.stages = static_cast<int>(stages < kMaxStages ? stages : kMaxStages);
    return per_sm * num_sms;
  }
  return 0;
}

// sm_threads: how many threads' worth of CTAs an SM is given.  Forward 1024:
// where the registers hold fewer at a time, a second wave takes no longer.
// Backward what they hold, since each CTA writes a row of partial dw (16384 x
// 512: 21 us against 24).
int row_grid(int64_t rows, const RowPlan& p, int num_sms, int sm_threads) {
  const int64_t ctas = (rows + p.per_cta - 1) / p.per_cta;
  const int64_t fit = static_cast<int64_t>(num_sms) * (sm_threads / (p.tpr * p.per_cta));
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
