// repitch_kernel.cu -- the copy that makes an operand addressable by TMA.
#include "expert.h"

namespace gemmlib {
namespace {

// A lane loads the eight elements that it stores: 2-byte loads (the source's rows
// start anywhere) whose lines the warp uses whole, one 16-byte store.
__global__ void __launch_bounds__(256) repitch_kernel(const uint16_t* src, int64_t ld, int64_t stride, uint16_t* dst,
                                                      int64_t ldd, int64_t stride_d, int64_t rows, int64_t cols,
                                                      const int32_t* offsets) {
  const int64_t z = blockIdx.y;
  if (offsets != nullptr && offsets[z + 1] <= offsets[z]) return;
  src += z * stride;
  dst += z * stride_d;
  const int64_t per_row = ldd / 8, total = rows * per_row;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / per_row, c = i % per_row * 8;
    uint16_t v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = c + u < cols ? src[r * ld + c + u] : (uint16_t)0;
    *reinterpret_cast<uint4*>(dst + r * ldd + c) = *reinterpret_cast<uint4*>(v);
  }
}

}  // namespace

cudaError_t launch_repitch(const void* src, int64_t ld, int64_t stride, void* dst, int64_t ldd, int64_t stride_d,
                           int64_t rows, int64_t cols, int64_t batch, const int32_t* offsets, cudaStream_t stream) {
  const int64_t per = (rows * (ldd / 8) + 255) / 256;
  const dim3 grid((unsigned)std::min<int64_t>(per, std::max<int64_t>(1, 2432 / batch)), (unsigned)batch);
  repitch_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(src), ld, stride, static_cast<uint16_t*>(dst),
                                           ldd, stride_d, rows, cols, offsets);
  return cudaGetLastError();
}

}  // namespace gemmlib
