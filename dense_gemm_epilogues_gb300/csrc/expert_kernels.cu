// expert_kernels.cu -- kernels of the expert-layer operators.
#include "expert.h"

namespace gemmlib {
namespace {

__device__ __forceinline__ void finish(const EpiParams& e, void* D, const void* C, const void* bias, int64_t i,
                                       int64_t j, float acc) {
  float v = e.alpha * acc;
  if (e.read_c) {
    float c = load_as_float(C, e.c_dtype, i * e.ldc + j);
    v = fmaf(e.beta, c, v);
  }
  if (e.bias_mode == GEMM_BIAS_COL) v += load_as_float(bias, e.bias_dtype, j);
  if (e.relu) v = fmaxf(v, 0.0f);
  store_float_as(D, e.d_dtype, i * e.ldd + j, v);
}

// One warp per output: lanes stride over K.
__global__ void __launch_bounds__(256) q4_kernel(const Q4Params p) {
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (n >= p.N) return;
  for (int64_t r = blockIdx.y; r < p.g.rows; r += gridDim.y) {
    int e = 0, lo = 0, hi = 0;
    for (; e < p.g.count; ++e) {
      group_range(p.g, e, lo, hi);
      if (r >= lo && r < hi) break;
    }
    if (e == p.g.count) continue;
    const uint8_t* q = p.q + e * p.stride_q + n * p.ldq;
    const char* sc = static_cast<const char*>(p.scales) + e * p.stride_s * dtype_bytes(p.scale_dtype);
    float acc = 0.0f;
    for (int64_t k = lane; k < p.K; k += 32) {
      const int64_t gk = k / p.group;
      const int v = (q[k >> 1] >> (4 * (k & 1))) & 15;
      const int z = p.zeros ? p.zeros[e * p.stride_z + n * p.ldz + gk] : 8;
      const float w = load_as_float(sc, p.scale_dtype, n * p.lds + gk) * (float)(v - z);
      acc = fmaf(load_as_float(p.A, p.ab_dtype, r * p.lda + k), w, acc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) finish(p.epi, p.epi.D, nullptr, epi_ptrs(p.epi, e).bias, r, n, acc);
  }
}

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

cudaError_t launch_q4(const Q4Params& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.N + 7) / 8), (unsigned)std::min(p.g.rows, 65535));
  q4_kernel<<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gemmlib
