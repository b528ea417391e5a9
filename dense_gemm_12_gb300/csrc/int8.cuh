// int8.cuh -- what the kernels of the int8 product share: its arguments, int8 to
// fp16, exact sums, and a finished tile's way to D.
#pragma once

#include "ops.cuh"

namespace g12 {

struct Int8Args {
  int M, N;
  int num_kb;          // k-blocks; 0: D <- bias + beta * D
  float alpha, beta;
  const float* sa;
  const float* sb;
  const float* bias;   // or nullptr
  void* D;
  int64_t ldd;
  int d_type;
  int d_pair;          // bf16, beta == 0: two channels can be written at once
  int cluster;         // > 1: CTAs that split one tile's k-blocks
  uint32_t* err;
};

// Four int8 -> four fp16: with the sign bit turned over, a byte is its value +
// 128, and as the low byte of 0x6400 it is the fp16 number 1024 + that.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Adds two whole numbers of at most 2^24, as fp32, to 32-bit integers, each with
// kWholeOff on top.  Adding kRound leaves f rounded to a multiple of 2^13, which
// its last bits then count; what is left, less than 2^13, is counted by the last
// bits of its sum with 1.5 * 2^23 (the constants are chosen so that the second
// and third sums are exact).  The conversion instruction, 16 a cycle, would take
// as long as two k-blocks' MMAs for a tile's accumulator.
constexpr float kRound = 103079215104.0f;               // 1.5 * 2^36
constexpr float kRoundLeft = 103079215104.0f + 12582912.0f;  // and 1.5 * 2^23
constexpr uint32_t kWholeOff = 0x51c00000u * 8192u + 0x4b400000u;  // their bits, as added below
__device__ __forceinline__ void add_whole(uint32_t& a, uint32_t& b, uint32_t f, uint32_t g) {
  uint32_t t0, t1, u0, u1;
  asm("{\n\t.reg .b64 f, c, d, m, t, u;\n\t"
      "mov.b64 f, {%4, %5};\n\t"
      "mov.b64 c, {%6, %6};\n\t"
      "mov.b64 d, {%7, %7};\n\t"
      "mov.b64 m, {%8, %8};\n\t"
      "add.rn.f32x2 t, f, c;\n\t"
      "fma.rn.f32x2 u, t, m, d;\n\t"
      "add.rn.f32x2 u, u, f;\n\t"
      "mov.b64 {%0, %1}, t;\n\t"
      "mov.b64 {%2, %3}, u;\n\t}"
      : "=r"(t0), "=r"(t1), "=r"(u0), "=r"(u1)
      : "r"(f), "r"(g), "f"(kRound), "f"(kRoundLeft), "f"(-1.0f));
  a += (t0 << 13) + u0;
  b += (t1 << 13) + u1;
}
// Which of a thread's sums go through the conversion instruction all the same:
// some 16 of 64, as long as the others take on the other units.
__host__ __device__ constexpr bool by_unit(int j) { return (j & 48) == 48; }

// A value of D without beta's part, given its integer sum.  cs: alpha times the
// channel's scale.
__device__ __forceinline__ float value(const Int8Args& p, uint32_t sum, float cs, float sa, float bias) {
  return p.num_kb > 0 ? fmaf(static_cast<float>(static_cast<int>(sum)) * sa, cs, bias) : bias;
}
__device__ __forceinline__ void finish(const Int8Args& p, int64_t at, float v) {
  if (p.beta != 0.0f) v = fmaf(p.beta, load1(p.D, p.d_type, at), v);
  store1(p.D, p.d_type, at, v);
}

// A thread's sums of S tokens from row0 on, for channel n (32 neighbouring ones
// to a warp), to D.  scales: shared address of the tokens' scales.
template <int S>
__device__ __forceinline__ void write_channel(const Int8Args& p, const uint32_t (&sum)[S], uint32_t scales,
                                              int n, int row0) {
  const int lane = threadIdx.x & 31;
  const int rows = min(p.M - row0, S);  // below 1: none
  const bool in = n < p.N;
  const float cs = in && p.num_kb > 0 ? p.alpha * p.sb[n] : 0.0f;
  const float bias = in && p.bias != nullptr ? p.bias[n] : 0.0f;
  const int64_t at = row0 * p.ldd + n;
  if (p.d_pair && n - lane + 32 <= p.N && rows == S) {
    // Two tokens' values of a channel become two channels' of a token: even
    // lanes take the first token's, odd ones the second's.
    const bool odd = lane & 1;
    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.D) + at + (odd ? p.ldd - 1 : 0);
#pragma unroll
    for (int j = 0; j < S; j += 4) {
      const float4 sa = ld_shared_v4(scales + 4 * j);
      const float v0 = value(p, sum[j], cs, sa.x, bias), v1 = value(p, sum[j + 1], cs, sa.y, bias);
      const float v2 = value(p, sum[j + 2], cs, sa.z, bias), v3 = value(p, sum[j + 3], cs, sa.w, bias);
      const float x = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
      const float y = __shfl_xor_sync(0xffffffffu, odd ? v2 : v3, 1);
      *reinterpret_cast<uint32_t*>(d) = odd ? pack_bf16(x, v1) : pack_bf16(v0, x);
      d += 2 * p.ldd;
      *reinterpret_cast<uint32_t*>(d) = odd ? pack_bf16(y, v3) : pack_bf16(v2, y);
      d += 2 * p.ldd;
    }
  } else if (in) {
#pragma unroll
    for (int j = 0; j < S; j += 4) {
      const float4 sa = ld_shared_v4(scales + 4 * j);
      const float s4[4] = {sa.x, sa.y, sa.z, sa.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < rows) finish(p, at + (j + i) * p.ldd, value(p, sum[j + i], cs, s4[i], bias));
    }
  }
}

// Scales of S tokens from row0 on to shared memory; whole warps.
template <int S>
__device__ __forceinline__ void fetch_scales(const Int8Args& p, uint32_t to, int row0) {
  for (int j = threadIdx.x & 31; j < S; j += 32)
    cp_async_4_at(to + 4 * j, row0 + j < p.M ? p.sa + row0 + j : p.sa, row0 + j < p.M ? 4u : 0u);
}

// The product with both operands widened to fp16 beforehand (int8_wide.cu): the
// bytes of the widened copies, and whether that takes less than `us`
// microseconds; then the product, with the copies in `buf`.
int64_t int8_wide_bytes(int64_t M, int64_t N, int64_t K);
bool int8_wide_pays(int64_t M, int64_t N, int64_t K, double us);
gemm_status_t int8_wide(const Int8Args& a, int64_t K, const int8_t* A, int64_t lda, const int8_t* B,
                        int64_t ldb, uint8_t* buf, int num_sms, cudaStream_t s);

}  // namespace g12
