// ops.cuh -- what the operators around the GEMMs share (normalisation, fp8
// quantisation, block-scaled fp8 products, products grouped by expert):
// pieces of the C ABI they borrow from api.cu, element types, fp8 block
// scales, and the PTX wrappers that the plain GEMM kernels do not need.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>
#include <mutex>

#include "../../include/gemm12.h"
#include "ptx.cuh"

namespace g12 {

// ------------------------------------------------------------ host pieces
// (defined in api.cu)
gemm_status_t abi_device(int* num_sms, uint32_t** err_word);
// `lock` is taken (on the device's scratch mutex) and must be held until the
// kernels that use the buffer are queued.  GEMM_ERR_NO_MEMORY inside a stream
// capture when the stream's buffer is too small.
gemm_status_t abi_scratch(cudaStream_t stream, int64_t floats, std::unique_lock<std::mutex>& lock,
                          float** ws);
gemm_status_t abi_stage(cudaStream_t stream, int64_t bytes, std::unique_lock<std::mutex>& lock,
                        uint8_t** buf);
// Tensor map of `rank` (2 or 3) dimensions, innermost first; strides in bytes
// of dimensions 1 .. rank - 1; zeros outside.
bool abi_encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base,
                      const int64_t* dims, const int64_t* strides, const uint32_t* box,
                      CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);
gemm_status_t abi_from_cuda(cudaError_t e);

constexpr int64_t kOpsMaxDim = (int64_t{1} << 31) - 1;
// Largest extent that a product cuts into tiles: its kernels keep rows, columns
// and tile counts in 32 bits, and go up to 255 past a position when they round
// up to a tile or step to a tile's end.
constexpr int64_t kOpsMaxTiled = kOpsMaxDim - 255;

inline bool ops_misaligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}
// A row-major array of `type` (gemm_out_t): element bytes, 0 for a type that
// the operator does not take.
inline int float_type_bytes(int type) {
  return type == GEMM_OUT_F32 ? 4 : (type == GEMM_OUT_BF16 ? 2 : 0);
}

// Raises a kernel's dynamic shared memory limit to at least `bytes` (once per
// device and size; the limit only ever grows).
template <auto Kernel>
cudaError_t ops_allow_smem(size_t bytes) {
  static std::mutex mutex;
  static std::atomic<size_t> limit[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (limit[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  std::lock_guard<std::mutex> lock(mutex);
  if (limit[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) limit[dev].store(bytes, std::memory_order_release);
  return e;
}

// Launches with programmatic stream serialization, as the GEMM kernels are:
// every kernel here waits in grid_dependency_wait() before its first global
// access.  cluster > 1: in clusters of that many CTAs along x.
template <auto Kernel, typename... Args>
cudaError_t ops_launch(dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                       const Args&... args) {
  if (smem > 16 * 1024) {  // with what the kernel has statically, perhaps over the default
    const cudaError_t e = ops_allow_smem<Kernel>(smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster > 1 ? cluster : 1);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, Kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------- fp8 block scales
constexpr float kFp8Max = 448.0f;             // largest finite E4M3 value
constexpr float kFp8ScaleMin = FLT_MIN;       // 2^-126: blocks of zeros keep a usable scale
constexpr int kFp8Block = 128;

// |v| if finite, else 0: infinities and NaN do not set a block's scale.
__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a <= FLT_MAX ? a : 0.0f;
}

// Largest finite magnitude of a thread's values over the LANES lanes of a block
// (16 or 8); all 32 lanes call it together.  fmaxf passes over NaN; infinities
// are rare, and only when one shows up are the values looked at one by one.
template <int LANES, int E>
__device__ __forceinline__ float block_amax(const float (&v)[E]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) m = fmaxf(m, fabsf(v[i]));
  if (__any_sync(0xffffffffu, m > FLT_MAX)) {
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) m = fmaxf(m, finite_abs(v[i]));
  }
#pragma unroll
  for (int s = LANES / 2; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  return m;
}

// Scale of a block whose largest finite magnitude is amax, and the factor
// that its values are multiplied by before rounding.  The factor is one
// correctly rounded quotient, so a value's product with it has the same two
// roundings as its quotient by the scale.
__device__ __forceinline__ float fp8_scale(float amax) {
  return fmaxf(__fdiv_rn(amax, kFp8Max), kFp8ScaleMin);
}
__device__ __forceinline__ float fp8_factor(float amax) {
  return fminf(__fdiv_rn(kFp8Max, amax), 1.0f / kFp8ScaleMin);
}

// Four values -> four E4M3 bytes (nearest even, saturating, NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// ------------------------------------------------ eight elements of a row
// A thread moves eight elements of a row at a time.  Vector form: they are
// consecutive, 16-byte aligned.  Strided form (rows that cannot be moved in
// vectors): elements c, c + 16, ..., c + 112 of a 128-column block, so that
// the 16 lanes of a block read consecutive elements; those at or past `n` read
// as zero and are not written.  Loading (Raw8) and widening are apart, so that
// a thread's loads are all on their way before the first is used, and are
// marked as read once (evict first).
//
// T: GEMM_OUT_F32, GEMM_OUT_BF16, or kAnyType for a type known at run time.
constexpr int kAnyType = 2;

template <int T>
struct Raw8 {
  uint32_t w[T == GEMM_OUT_BF16 ? 4 : 8];
};

__device__ __forceinline__ float load1(const void* p, int type, int64_t at) {
  return type == GEMM_OUT_BF16 ? __bfloat162float(__ldcs(static_cast<const __nv_bfloat16*>(p) + at))
                               : __ldcs(static_cast<const float*>(p) + at);
}

__device__ __forceinline__ void store1(void* p, int type, int64_t at, float v) {
  if (type == GEMM_OUT_BF16)
    static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[at] = v;
}

template <int T>
__device__ __forceinline__ Raw8<T> load8_vec(const void* p, int type, int64_t at) {
  Raw8<T> r;
  const bool half = T == GEMM_OUT_BF16 || (T == kAnyType && type == GEMM_OUT_BF16);
  const uint4* src = half ? reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at)
                          : reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
  const uint4 a = __ldcs(src);
  r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
  if constexpr (T != GEMM_OUT_BF16) {
    uint4 b = make_uint4(0u, 0u, 0u, 0u);
    if (!half) b = __ldcs(src + 1);
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  }
  return r;
}

template <int T>
__device__ __forceinline__ void widen_vec(const Raw8<T>& r, int type, float (&v)[8]) {
  if (T == GEMM_OUT_BF16 || (T == kAnyType && type == GEMM_OUT_BF16)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  } else if constexpr (T != GEMM_OUT_BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
  }
}

// Strided forms (types at run time).  The words stay as they were loaded:
// anything done to them here would wait for them before the next chunk's loads
// (a norm of 4000 x 5001 in bf16: 131 us with the shift to fp32 here, 48 without).
__device__ __forceinline__ Raw8<kAnyType> load8_strided(const void* p, int type, int64_t row_at,
                                                        int c, int n) {
  Raw8<kAnyType> r;
  if (type == GEMM_OUT_BF16) {
    const unsigned short* src = static_cast<const unsigned short*>(p) + row_at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r.w[i] = c + 16 * i < n ? static_cast<uint32_t>(__ldcs(src + c + 16 * i)) : 0u;
  } else {
    const uint32_t* src = static_cast<const uint32_t*>(p) + row_at;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = c + 16 * i < n ? __ldcs(src + c + 16 * i) : 0u;
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store8_vec(void* p, int type, int64_t at, const float (&v)[8]) {
  if (type == GEMM_OUT_BF16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                   pack_bf16(v[6], v[7]));
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ void store8_strided(void* p, int type, int64_t row_at, int c, int n,
                                               const float (&v)[8]) {
  if (type == GEMM_OUT_BF16) {
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p) + row_at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < n) to[c + 16 * i] = __float2bfloat16_rn(v[i]);
  } else {
    float* to = static_cast<float*>(p) + row_at;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 16 * i < n) to[c + 16 * i] = v[i];
  }
}

// Eight consecutive elements from shared memory (16-byte aligned).
template <int T>
__device__ __forceinline__ Raw8<T> load8_smem(const uint8_t* row, int c) {
  static_assert(T != kAnyType, "the type is known");
  Raw8<T> r;
  const uint4* src = reinterpret_cast<const uint4*>(row + c * (T == GEMM_OUT_BF16 ? 2 : 4));
  const uint4 a = src[0];
  r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
  if constexpr (T != GEMM_OUT_BF16) {
    const uint4 b = src[1];
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  }
  return r;
}

// Either form, zero where `in` is false.
template <bool VEC, int T>
__device__ __forceinline__ Raw8<T> load8(const void* p, int type, int64_t row_at, int c, int n,
                                         bool in) {
  Raw8<T> r{};
  if constexpr (VEC) {
    if (in) r = load8_vec<T>(p, type, row_at + c);
  } else {
    if (in) r = load8_strided(p, type, row_at, c, n);
  }
  return r;
}

template <bool VEC, int T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, int type, float (&v)[8]) {
  if constexpr (VEC) {
    widen_vec<T>(r, type, v);
  } else {
    const int up = type == GEMM_OUT_BF16 ? 16 : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i] << up);
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(void* p, int type, int64_t row_at, int c, int n,
                                       const float (&v)[8]) {
  if (VEC)
    store8_vec(p, type, row_at + c, v);
  else
    store8_strided(p, type, row_at, c, n, v);
}

// --------------------------------------------------------- PTX additions
// 3-D tiled copy global -> shared; x is the innermost coordinate.
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int32_t x,
                                            int32_t y, int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Asks L2 to fetch a box (no shared-memory destination, nothing to wait for).
__device__ __forceinline__ void tma_prefetch_l2_3d(const CUtensorMap* map, int32_t x, int32_t y,
                                                   int32_t z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// The same, completion signalled on an mbarrier that may live in the peer CTA
// of a pair (shared::cluster address).
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, int32_t x,
                                                 int32_t y, int32_t z, uint32_t mbar_cluster_addr) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar_cluster_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// True in one lane of the (converged) warp.  The roles that issue MMAs and TMA
// copies run their loops with the whole warp and only issue under this:
// their operands are then known to be the same in all lanes and stay in
// uniform registers.  In a branch of one lane every operand of every MMA is
// first moved there, 400 cycles for the four MMAs of a k-block.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// mbar_wait and its companions by 32-bit shared addresses: all barriers of a
// kernel are then one base register and constants.
__device__ __forceinline__ bool mbar_try_wait_at(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ int ld_shared_volatile(uint32_t addr) {
  int v;
  asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ bool mbar_wait_at(uint32_t bar, uint32_t parity, uint32_t abort_flag,
                                             uint32_t* err_word) {
  if (mbar_try_wait_at(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) { if (mbar_try_wait_at(bar, parity)) return true; }
    if (ld_shared_volatile(abort_flag)) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(abort_flag), "r"(1) : "memory");
      atomicOr(err_word, kErrWaitTimeout);
      return false;
    }
  }
}

__device__ __forceinline__ bool mbar_wait_late(uint64_t* bar, uint32_t parity, int* abort_flag,
                                               uint32_t* err_word) {
  return mbar_wait_at(smem_u32(bar), parity, smem_u32(abort_flag), err_word);
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cp_async_4_at(uint32_t smem_dst, const void* gmem_src,
                                              uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_dst), "l"(gmem_src),
               "r"(src_bytes)
               : "memory");
}

__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int4 ld_shared_i4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Arrive on an mbarrier given by its shared::cluster address, releasing at CTA
// scope only: for arrivals that publish nothing in memory (the accumulator's
// reads are complete, tcgen05.wait::ld).  The cluster-scope release of
// mbar_arrive_cluster waits for the thread's outstanding memory operations,
// 1000 cycles and more.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ void fence_acq_rel_cluster() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// 3-D tiled copy shared -> global of one box, in the issuing thread's bulk
// group; elements outside the tensor are not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t smem_src, int32_t x,
                                             int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_src), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Contiguous copy global -> shared; both addresses 16-byte aligned, `bytes` a
// multiple of 16, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[smem] x B[smem] with 8-bit floating operands, single CTA.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of tcgen05.mma kind::f8f6f4 with E4M3 A and B (format
// 0), both K-major, and an fp32 accumulator: fields as in idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Waits for this thread's TMEM loads; r is tied to the wait so that no use of
// the loaded registers is scheduled before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Two fp32 values in one register pair.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f32x2_parts(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// Registers per thread of the calling warpgroup after launch.  The shares of
// a block's warpgroups add up to at most what it was launched with.
template <int N>
__device__ __forceinline__ void regs_give_back() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace g12
