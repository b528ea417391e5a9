// bytes.cu -- copies of operands of bytes (fp8, int8) with rows padded to 16
// bytes, which TMA can describe.
#include "ops.cuh"

namespace g12 {
namespace {

__global__ void stage_bytes_kernel(const uint8_t* src, int64_t ld, int64_t stride, uint8_t* dst,
                                   int64_t ld2, int64_t rows, int64_t cols, int64_t count) {
  grid_dependency_wait();
  const int64_t pieces = ld2 / 16;
  const int64_t total = count * rows * pieces;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t line = i / pieces, c = (i - line * pieces) * 16;
    const int64_t m = line / rows, r = line - m * rows;
    const uint8_t* s = src + m * stride + r * ld + c;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c + j < cols) w[j >> 2] |= static_cast<uint32_t>(s[j]) << (8 * (j & 3));
    *reinterpret_cast<uint4*>(dst + line * ld2 + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t byte_stage(ByteOperand& o, uint8_t* dst, int num_sms, cudaStream_t s) {
  const int64_t ld2 = (o.cols + 15) / 16 * 16;
  const int64_t total = o.count * o.rows * (ld2 / 16);
  const int64_t want = (total + 255) / 256, fit = static_cast<int64_t>(num_sms) * 8;
  const uint8_t* src = static_cast<const uint8_t*>(o.p);
  const int64_t ld = o.ld, stride = o.stride, rows = o.rows, cols = o.cols, count = o.count;
  const cudaError_t e = ops_launch<stage_bytes_kernel>(
      dim3(static_cast<unsigned>(want < fit ? want : fit)), 256, 0, 1, s, src, ld, stride, dst, ld2,
      rows, cols, count);
  o.p = dst;
  o.ld = ld2;
  o.stride = o.rows * ld2;
  return e;
}

}  // namespace g12
