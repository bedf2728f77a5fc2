// repitch_kernel.cu -- the copy that makes an operand addressable by TMA.
#include "expert.h"

namespace gemmlib {
namespace {

// A lane loads the elements that it stores: narrow loads (the source's rows start
// anywhere) whose lines the warp uses whole, one 16-byte store.
template <typename T>
__global__ void __launch_bounds__(256) repitch_kernel(const T* src, int64_t ld, int64_t stride, T* dst, int64_t ldd,
                                                      int64_t stride_d, int64_t rows, int64_t cols,
                                                      const int32_t* offsets) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t z = blockIdx.y;
  if (offsets != nullptr && offsets[z + 1] <= offsets[z]) return;
  src += z * stride;
  dst += z * stride_d;
  const int64_t per_row = ldd / V, total = rows * per_row;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / per_row, c = (i - r * per_row) * V;
    __align__(16) T v[V];
#pragma unroll
    for (int u = 0; u < V; ++u) v[u] = c + u < cols ? src[r * ld + c + u] : T(0);
    *reinterpret_cast<uint4*>(dst + r * ldd + c) = *reinterpret_cast<uint4*>(v);
  }
}

}  // namespace

cudaError_t launch_repitch(const void* src, int64_t ld, int64_t stride, void* dst, int64_t ldd, int64_t stride_d,
                           int64_t rows, int64_t cols, int64_t batch, const int32_t* offsets, int elem_bytes,
                           cudaStream_t stream) {
  const int64_t per = (rows * ldd * elem_bytes / 16 + 255) / 256;
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(per, std::max<int64_t>(1, 2432 / batch))), (unsigned)batch);
  if (elem_bytes == 1)
    repitch_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint8_t*>(src), ld, stride, static_cast<uint8_t*>(dst), ldd,
                                             stride_d, rows, cols, offsets);
  else
    repitch_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(src), ld, stride, static_cast<uint16_t*>(dst),
                                             ldd, stride_d, rows, cols, offsets);
  return cudaGetLastError();
}

}  // namespace gemmlib
