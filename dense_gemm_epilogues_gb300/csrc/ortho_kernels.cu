// ortho_kernels.cu -- what the Newton-Schulz steps need around their products: the
// norm of each matrix, the normalised fp16 copy that the products read, and the
// cast of a result that no product writes itself.
#include "expert.h"

namespace gemmlib {
namespace {

// Both passes over G work on TILE x TILE tiles of the wide matrix X (G or its
// transpose): a tile is loaded along G's rows and turned around in shared
// memory, so that every thread meets the same entries of X whichever way G
// lies.  The sum of squares then has one order, fixed by X's shape alone: a
// matrix, its transpose, and any batch around it give the same bits.
// Bound by memory: G is read twice (the second time from L2 when it fits) and X
// written once.
constexpr int TILE = 64;

template <typename T>
__device__ __forceinline__ float widen(T v) { return (float)v; }
template <>
__device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// tile[r][c] = X[r0 + r, c0 + c] (zero outside).  vec: G's rows can be read 16 bytes at a time.
template <typename T>
__device__ __forceinline__ void load_tile(const T* g, int64_t m, int64_t n, int64_t ld, bool transpose, bool vec,
                                          int64_t r0, int64_t c0, float (&tile)[TILE][TILE + 1]) {
  constexpr int V = 16 / (int)sizeof(T), PER_ROW = TILE / V;
  // In G: rows i (outer), entries j (contiguous).
  const int64_t i0 = transpose ? c0 : r0, j0 = transpose ? r0 : c0;
  const int64_t ni = transpose ? n : m, nj = transpose ? m : n;
  for (int q = threadIdx.x; q < TILE * PER_ROW; q += blockDim.x) {
    const int i = q / PER_ROW, j = q % PER_ROW * V;
    T v[V];
    const T* src = g + (i0 + i) * ld + j0 + j;
    if (vec && i0 + i < ni && j0 + j + V <= nj) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(src);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u) v[u] = (i0 + i < ni && j0 + j + u < nj) ? src[u] : T(0.0f);
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if (transpose) tile[j + u][i] = widen(v[u]);
      else tile[i][j + u] = widen(v[u]);
    }
  }
}

// Sum over a block of 256 threads, in a fixed order; the result in every thread.
__device__ __forceinline__ float block_sum(float s) {
  __shared__ float warp_sums[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += warp_sums[w];
  return s;
}

// partials[matrix][slot]: the squares of tiles slot, slot + slots, ... of X.
template <typename T>
__global__ void __launch_bounds__(256) sumsq_kernel(const OrthoInput in, float* partials, int32_t* counters,
                                                    int64_t num_counters) {
  for (int64_t i = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * 256 + threadIdx.x; i < num_counters;
       i += (int64_t)gridDim.x * gridDim.y * 256)
    counters[i] = 0;
  __shared__ float tile[TILE][TILE + 1];
  const T* g = static_cast<const T*>(in.g) + blockIdx.y * in.stride;
  const int64_t tiles_n = (in.n + TILE - 1) / TILE, tiles = (in.m + TILE - 1) / TILE * tiles_n;
  float s = 0.0f;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    __syncthreads();
    load_tile(g, in.m, in.n, in.ld, in.transpose, in.vec, t / tiles_n * TILE, t % tiles_n * TILE, tile);
    __syncthreads();
    float p = 0.0f;   // per tile first: a long sum loses less
#pragma unroll
    for (int r = 0; r < TILE; r += 4) {
      const float v = tile[r + (threadIdx.x >> 6)][threadIdx.x & 63];
      p = fmaf(v, v, p);
    }
    s += p;
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partials[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// X = G * (scale / (norm + eps)) in fp16, rows pitched to ldx with zeros past n.
template <typename T>
__global__ void __launch_bounds__(256) normalize_kernel(const OrthoInput in, const float* partials, int slots,
                                                        float eps, float scale, __half* x, int64_t ldx,
                                                        int64_t stride_x) {
  __shared__ float tile[TILE][TILE + 1];
  float s = 0.0f;
  for (int i = threadIdx.x; i < slots; i += 256) s += partials[blockIdx.y * slots + i];
  const float f = scale / (sqrtf(block_sum(s)) + eps);
  const T* g = static_cast<const T*>(in.g) + blockIdx.y * in.stride;
  x += blockIdx.y * stride_x;
  const int64_t tiles_n = (ldx + TILE - 1) / TILE, tiles = (in.m + TILE - 1) / TILE * tiles_n;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t r0 = t / tiles_n * TILE, c0 = t % tiles_n * TILE;
    __syncthreads();
    load_tile(g, in.m, in.n, in.ld, in.transpose, in.vec, r0, c0, tile);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = h * 32 + (threadIdx.x >> 3), c = (threadIdx.x & 7) * 8;
      if (r0 + r >= in.m || c0 + c >= ldx) continue;
      __half2 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = __floats2half2_rn(tile[r][c + 2 * u] * f, tile[r][c + 2 * u + 1] * f);
      *reinterpret_cast<uint4*>(x + (r0 + r) * ldx + c0 + c) = *reinterpret_cast<uint4*>(v);
    }
  }
}

__global__ void __launch_bounds__(256) unscale_kernel(const __half* x, int64_t M, int64_t N, int64_t ldx,
                                                      int64_t stride_x, int transpose, float scale, void* D, int dtype,
                                                      int64_t ldd, int64_t stride_d) {
  x += blockIdx.y * stride_x;
  char* d = static_cast<char*>(D) + blockIdx.y * stride_d * dtype_bytes(dtype);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / N, c = i % N;
    store_float_as(d, dtype, r * ldd + c, __half2float(x[transpose ? c * ldx + r : r * ldx + c]) * scale);
  }
}

template <typename T>
cudaError_t launch_ortho_input(const OrthoInput& in, int64_t batch, float* partials, float eps, float scale, __half* x,
                               int64_t ldx, int64_t stride_x, int32_t* counters, int64_t num_counters,
                               cudaStream_t stream) {
  const int64_t tiles = ((in.m + TILE - 1) / TILE) * ((ldx + TILE - 1) / TILE);
  const int slots = ortho_slots(in.m, in.n);
  sumsq_kernel<T><<<dim3((unsigned)slots, (unsigned)batch), 256, 0, stream>>>(in, partials, counters, num_counters);
  normalize_kernel<T><<<dim3((unsigned)std::min<int64_t>(tiles, 1216), (unsigned)batch), 256, 0, stream>>>(
      in, partials, slots, eps, scale, x, ldx, stride_x);
  return cudaGetLastError();
}

}  // namespace

int ortho_slots(int64_t m, int64_t n) {
  return (int)std::min<int64_t>(((m + TILE - 1) / TILE) * ((n + TILE - 1) / TILE), 608);
}

cudaError_t launch_ortho_input(const OrthoInput& in, int dtype, int64_t batch, float* partials, float eps, float scale,
                               __half* x, int64_t ldx, int64_t stride_x, int32_t* counters, int64_t num_counters,
                               cudaStream_t stream) {
  if (dtype == GEMM_F32) return launch_ortho_input<float>(in, batch, partials, eps, scale, x, ldx, stride_x, counters, num_counters, stream);
  if (dtype == GEMM_F16) return launch_ortho_input<__half>(in, batch, partials, eps, scale, x, ldx, stride_x, counters, num_counters, stream);
  return launch_ortho_input<__nv_bfloat16>(in, batch, partials, eps, scale, x, ldx, stride_x, counters, num_counters, stream);
}

cudaError_t launch_unscale(const __half* x, int64_t batch, int64_t M, int64_t N, int64_t ldx, int64_t stride_x,
                           int transpose, float scale, void* D, int dtype, int64_t ldd, int64_t stride_d,
                           cudaStream_t stream) {
  const int64_t per = (M * N + 255) / 256;
  unscale_kernel<<<dim3((unsigned)std::min<int64_t>(per, 2048), (unsigned)batch), 256, 0, stream>>>(
      x, M, N, ldx, stride_x, transpose, scale, D, dtype, ldd, stride_d);
  return cudaGetLastError();
}

}  // namespace gemmlib
