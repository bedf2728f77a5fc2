// ortho_kernels.cu -- what the Newton-Schulz steps need around their products: the
// norm of each matrix, the normalised copy that the products read (pairs of fp16 halves),
// and the cast of a result that no product writes itself.
#include "expert.h"

namespace gemmlib {
namespace {

// Both passes over G work on TILE x TILE tiles of the wide matrix X (G or its
// transpose), in units of 8 consecutive entries of a row of X, two units per thread.  A
// unit lies contiguous in G when X is G, at any alignment (then it is put together from
// aligned words); when X is G's transpose, the tile is loaded along G's rows and arranged
// in shared memory.  Either way every thread meets the
// same units in the same order, so the sum of squares has one order, fixed by X's shape
// alone: a matrix, its transpose, and any batch around it give the same bits.
// Bound by memory: G is read twice (the second time from L2 when it fits) and both halves
// of X written once.  Many light threads; the next tile's units are under way while one
// tile is worked on, and the first of the second pass while the norm is added up: 25 and 42
// us for 4096 x 11008 in bf16 (3.6 and 6.4 TB/s), 20 and 28 for 16 x 768 x 2001, whose rows
// lie at every alignment.
constexpr int TILE = 64;

template <typename T>
__device__ __forceinline__ float widen(T v) { return (float)v; }
template <>
__device__ __forceinline__ float widen<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Unit u (0, 1) of this thread in a tile: row 32 u + thread / 8, columns 8 (thread % 8) ...
__device__ __forceinline__ int unit_row(int u) { return 32 * u + (int)(threadIdx.x >> 3); }
__device__ __forceinline__ int unit_col() { return (int)(threadIdx.x & 7) * 8; }

// The eight entries of X at (r, c) ..., X being G; zero outside.
template <typename T>
__device__ __forceinline__ void load_unit(const T* g, const OrthoInput& in, int64_t r, int64_t c, T (&v)[8]) {
  const T* src = g + r * in.ld + c;
  uint32_t* w = reinterpret_cast<uint32_t*>(v);
  // (aligned words around a 16-bit unit reach two bytes past it: not at the matrix's ends)
  if (in.vec && r < in.m && c + 8 <= in.n) {
    constexpr int W = (int)sizeof(T) * 8 / 16;
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(v)[i] = reinterpret_cast<const uint4*>(src)[i];
  } else if (!in.vec && r < in.m && c + 8 < in.n && r + c > 0) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(src);
    const uint32_t* p = reinterpret_cast<const uint32_t*>(at & ~uintptr_t(3));
    constexpr int W = (int)sizeof(T) * 8 / 4;
    uint32_t u[W + 1];
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = p[i];
    if constexpr (sizeof(T) == 2) {
      const uint32_t shift = (uint32_t)(at & 3) * 8;
      u[W] = shift ? p[W] : 0u;
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(u[i], u[i + 1], shift);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = u[i];
    }
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = r < in.m && c + u < in.n ? src[u] : T(0.0f);
  }
}

// This thread's units of tile t.
template <typename T>
__device__ __forceinline__ void load_units(const T* g, const OrthoInput& in, int t, int tiles_n, T (&v)[2][8]) {
  const int64_t r0 = (int64_t)(t / tiles_n) * TILE, c = (int64_t)(t % tiles_n) * TILE + unit_col();
#pragma unroll
  for (int u = 0; u < 2; ++u) load_unit(g, in, r0 + unit_row(u), c, v[u]);
}

// tile[r][c] = X[r0 + r, c0 + c] (zero outside), X being G's transpose: G's rows 16 bytes
// at a time where they lie on 16 bytes, else element by element, 64 to a row.
template <typename T>
__device__ __forceinline__ void load_turned(const T* g, const OrthoInput& in, int64_t r0, int64_t c0,
                                            float (&tile)[TILE][TILE + 1]) {
  constexpr int V = 16 / (int)sizeof(T), PER_ROW = TILE / V;
  if (!in.vec) {
    const int j = (int)threadIdx.x & 63;
    T v[16];
#pragma unroll
    for (int h = 0; h < 16; ++h) {
      const int i = 4 * h + (int)(threadIdx.x >> 6);
      v[h] = c0 + i < in.n && r0 + j < in.m ? g[(c0 + i) * in.ld + r0 + j] : T(0.0f);
    }
#pragma unroll
    for (int h = 0; h < 16; ++h) {
      const int i = 4 * h + (int)(threadIdx.x >> 6);
      tile[j][i] = widen(v[h]);
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < TILE * PER_ROW / 256; ++h) {
    const int q = h * 256 + (int)threadIdx.x, i = q / PER_ROW, j = q % PER_ROW * V;
    __align__(16) T v[V];
    const T* src = g + (c0 + i) * in.ld + r0 + j;   // G's row c0 + i, entries r0 + j ...
    if (c0 + i < in.n && r0 + j + V <= in.m) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(src);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u) v[u] = c0 + i < in.n && r0 + j + u < in.m ? src[u] : T(0.0f);
    }
#pragma unroll
    for (int u = 0; u < V; ++u) tile[j + u][i] = widen(v[u]);
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

// The sum of the squares of a tile's two units.
__device__ __forceinline__ float squares(const float (&x)[2][8]) {
  float p = 0.0f;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int k = 0; k < 8; ++k) p = fmaf(x[u][k], x[u][k], p);
  return p;
}

// partials[matrix][slot]: the squares of tiles slot, slot + slots, ... of X, each tile's
// first (a long sum loses less).
template <typename T>
__global__ void __launch_bounds__(256) sumsq_kernel(const OrthoInput in, float* partials, int32_t* counters,
                                                    int64_t num_counters) {
  __shared__ float tile[TILE][TILE + 1];
  pdl_wait();
  for (int64_t i = (blockIdx.y * (int64_t)gridDim.x + blockIdx.x) * 256 + threadIdx.x; i < num_counters;
       i += (int64_t)gridDim.x * gridDim.y * 256)
    counters[i] = 0;
  const T* g = static_cast<const T*>(in.g) + blockIdx.y * in.stride;
  const int tiles_n = (int)((in.n + TILE - 1) / TILE), tiles = (int)((in.m + TILE - 1) / TILE) * tiles_n;
  float s = 0.0f, x[2][8];
  if (in.transpose) {
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      __syncthreads();
      load_turned(g, in, (int64_t)(t / tiles_n) * TILE, (int64_t)(t % tiles_n) * TILE, tile);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u][k] = tile[unit_row(u)][unit_col() + k];
      s += squares(x);
    }
  } else {
    __align__(16) T v[2][8];
    load_units(g, in, blockIdx.x, tiles_n, v);
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[u][k] = widen(v[u][k]);
      if (t + (int)gridDim.x < tiles) load_units(g, in, t + (int)gridDim.x, tiles_n, v);
      s += squares(x);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partials[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// X = G * (scale / (norm + eps)) as x + xlo, both fp16, xlo what x rounds away; rows
// pitched to ldx with zeros past n.
template <typename T>
__global__ void __launch_bounds__(256) normalize_kernel(const OrthoInput in, const float* partials, int slots,
                                                        float eps, float scale, __half* x, __half* xlo, int64_t ldx,
                                                        int64_t stride_x) {
  __shared__ float tile[TILE][TILE + 1];
  pdl_wait();
  const T* g = static_cast<const T*>(in.g) + blockIdx.y * in.stride;
  const int tiles_n = (int)((ldx + TILE - 1) / TILE), tiles = (int)((in.m + TILE - 1) / TILE) * tiles_n;
  __align__(16) T v[2][8];
  if (!in.transpose) load_units(g, in, blockIdx.x, tiles_n, v);
  float s = 0.0f;
  for (int i = threadIdx.x; i < slots; i += 256) s += partials[blockIdx.y * slots + i];
  const float f = scale / (sqrtf(block_sum(s)) + eps);
  x += blockIdx.y * stride_x;
  xlo += blockIdx.y * stride_x;
  auto store = [&](int64_t r, int64_t c, const float (&e)[8]) {
    if (r >= in.m || c >= ldx) return;
    __align__(16) __half2 h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float v0 = __fmul_rn(e[2 * k], f), v1 = __fmul_rn(e[2 * k + 1], f);
      h[k] = __floats2half2_rn(v0, v1);
      const float2 w = __half22float2(h[k]);
      l[k] = __floats2half2_rn(v0 - w.x, v1 - w.y);
    }
    *reinterpret_cast<uint4*>(x + r * ldx + c) = *reinterpret_cast<uint4*>(h);
    *reinterpret_cast<uint4*>(xlo + r * ldx + c) = *reinterpret_cast<uint4*>(l);
  };
  float e[2][8];
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t r0 = (int64_t)(t / tiles_n) * TILE, c0 = (int64_t)(t % tiles_n) * TILE;
    if (in.transpose) {
      __syncthreads();
      load_turned(g, in, r0, c0, tile);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 8; ++k) e[u][k] = tile[unit_row(u)][unit_col() + k];
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 8; ++k) e[u][k] = widen(v[u][k]);
      if (t + (int)gridDim.x < tiles) load_units(g, in, t + (int)gridDim.x, tiles_n, v);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) store(r0 + unit_row(u), c0 + unit_col(), e[u]);
  }
}

__global__ void __launch_bounds__(256) unscale_kernel(const __half* x, const __half* xlo, int64_t M, int64_t N, int64_t ldx,
                                                      int64_t stride_x, int transpose, float scale, void* D, int dtype,
                                                      int64_t ldd, int64_t stride_d) {
  x += blockIdx.y * stride_x;
  xlo += blockIdx.y * stride_x;
  char* d = static_cast<char*>(D) + blockIdx.y * stride_d * dtype_bytes(dtype);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / N, c = i % N;
    const int64_t at = transpose ? c * ldx + r : r * ldx + c;
    store_float_as(d, dtype, r * ldd + c, (__half2float(x[at]) + __half2float(xlo[at])) * scale);
  }
}

template <typename T>
cudaError_t launch_ortho_input(const OrthoInput& in, int64_t batch, float* partials, float eps, float scale, __half* x,
                               __half* xlo, int64_t ldx, int64_t stride_x, int32_t* counters, int64_t num_counters,
                               cudaStream_t stream) {
  const int64_t tiles = ((in.m + TILE - 1) / TILE) * ((ldx + TILE - 1) / TILE);
  const int slots = ortho_slots(in.m, in.n);
  cudaError_t e = launch_dependent(sumsq_kernel<T>, dim3((unsigned)slots, (unsigned)batch), 256, stream, in, partials,
                                   counters, num_counters);
  if (e != cudaSuccess) return e;
  return launch_dependent(normalize_kernel<T>, dim3((unsigned)std::min<int64_t>(tiles, std::max<int64_t>(1216 / batch, 76)), (unsigned)batch), 256, stream,
                          in, (const float*)partials, slots, eps, scale, x, xlo, ldx, stride_x);
}

}  // namespace

int ortho_slots(int64_t m, int64_t n) {
  // (by the shape alone, whatever the batch) four tiles each, once that fills the chip
  const int64_t tiles = ((m + TILE - 1) / TILE) * ((n + TILE - 1) / TILE);
  return (int)std::min<int64_t>(1216, std::max<int64_t>(std::min<int64_t>(tiles, 152), (tiles + 3) / 4));
}

cudaError_t launch_ortho_input(const OrthoInput& in, int dtype, int64_t batch, float* partials, float eps, float scale,
                               __half* x, __half* xlo, int64_t ldx, int64_t stride_x, int32_t* counters,
                               int64_t num_counters, cudaStream_t stream) {
  if (dtype == GEMM_F32) return launch_ortho_input<float>(in, batch, partials, eps, scale, x, xlo, ldx, stride_x, counters, num_counters, stream);
  if (dtype == GEMM_F16) return launch_ortho_input<__half>(in, batch, partials, eps, scale, x, xlo, ldx, stride_x, counters, num_counters, stream);
  return launch_ortho_input<__nv_bfloat16>(in, batch, partials, eps, scale, x, xlo, ldx, stride_x, counters, num_counters, stream);
}

cudaError_t launch_unscale(const __half* x, const __half* xlo, int64_t batch, int64_t M, int64_t N, int64_t ldx, int64_t stride_x,
                           int transpose, float scale, void* D, int dtype, int64_t ldd, int64_t stride_d,
                           cudaStream_t stream) {
  const int64_t per = (M * N + 255) / 256;
  unscale_kernel<<<dim3((unsigned)std::min<int64_t>(per, 2048), (unsigned)batch), 256, 0, stream>>>(
      x, xlo, M, N, ldx, stride_x, transpose, scale, D, dtype, ldd, stride_d);
  return cudaGetLastError();
}

}  // namespace gemmlib
