// expert_kernels.cu -- kernels of the expert-layer operators.
#include "expert.h"

namespace gemmlib {
namespace {

constexpr int ST = 64;    // output tile edge of the plain tile kernel
constexpr int SK = 16;    // its depth per step

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

// One ST x ST tile: rows [m0, m1) and columns [n0, n0 + ST) with element (i, k) of A at
// a_i * i + a_k * k and (k, j) of B at b_k * k + b_j * j, k in [k0, k1).
__device__ void tile_product(const void* A, int64_t a_i, int64_t a_k, const void* B, int64_t b_k, int64_t b_j,
                             int ab, int64_t m0, int64_t m1, int64_t n0, int64_t N, int64_t k0, int64_t k1,
                             float (&acc)[4][4]) {
  __shared__ float sa[SK][ST + 1], sb[SK][ST + 1];
  const int tx = threadIdx.x, ty = threadIdx.y, t = ty * 16 + tx;
  for (int64_t k = k0; k < k1; k += SK) {
    for (int q = t; q < SK * ST; q += 256) {
      // Consecutive threads run along the operand's contiguous dimension.
      const int ai = a_k == 1 ? q / SK : q % ST, ak = a_k == 1 ? q % SK : q / ST;
      const int bj = b_k == 1 ? q / SK : q % ST, bk = b_k == 1 ? q % SK : q / ST;
      sa[ak][ai] = (m0 + ai < m1 && k + ak < k1) ? load_as_float(A, ab, (m0 + ai) * a_i + (k + ak) * a_k) : 0.0f;
      sb[bk][bj] = (n0 + bj < N && k + bk < k1) ? load_as_float(B, ab, (k + bk) * b_k + (n0 + bj) * b_j) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < SK; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = sa[kk][ty + 16 * i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = sb[kk][tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) grouped_kernel(const GroupedParams p) {
  // Tile row blockIdx.y of all groups' tile rows, one group after the other.
  __shared__ int s_e, s_lo, s_hi, s_t;
  if (threadIdx.x == 0 && threadIdx.y == 0) {
    int left = (int)blockIdx.y;
    s_e = -1;
    for (int e = 0; e < p.g.count; ++e) {
      int lo, hi;
      group_range(p.g, e, lo, hi);
      const int t = (hi - lo + ST - 1) / ST;
      if (left < t) {
        s_e = e;
        s_lo = lo;
        s_hi = hi;
        s_t = left;
        break;
      }
      left -= t;
    }
  }
  __syncthreads();
  if (s_e < 0) return;
  const int64_t m0 = s_lo + (int64_t)s_t * ST, n0 = (int64_t)blockIdx.x * ST;
  float acc[4][4] = {};
  const char* B = static_cast<const char*>(p.B) + s_e * p.stride_b * dtype_bytes(p.ab_dtype);
  tile_product(p.A, p.lda, 1, B, p.b_k, p.b_n, p.ab_dtype, m0, s_hi, n0, p.N, 0, p.K, acc);
  const char* bias = static_cast<const char*>(p.epi.bias) + s_e * p.epi.stride_bias * dtype_bytes(p.epi.bias_dtype);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = m0 + threadIdx.y + 16 * i, n = n0 + threadIdx.x + 16 * j;
      if (r < s_hi && n < p.N) finish(p.epi, p.epi.D, nullptr, bias, r, n, acc[i][j]);
    }
}

__global__ void __launch_bounds__(256) wgrad_kernel(const WgradParams p) {
  const int e = (int)blockIdx.z;
  int lo, hi;
  group_range(p.g, e, lo, hi);
  const int64_t m0 = (int64_t)blockIdx.y * ST, n0 = (int64_t)blockIdx.x * ST;
  float acc[4][4] = {};
  tile_product(p.A, 1, p.lda, p.B, p.ldb, 1, p.ab_dtype, m0, p.M, n0, p.N, lo, hi, acc);
  const EpiPtrs ptr = epi_ptrs(p.epi, e);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + threadIdx.y + 16 * i, n = n0 + threadIdx.x + 16 * j;
      if (m < p.M && n < p.N) finish(p.epi, ptr.D, ptr.C, nullptr, m, n, acc[i][j]);
    }
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

}  // namespace

cudaError_t launch_grouped(const GroupedParams& p, cudaStream_t stream) {
  const int64_t gy = (int64_t)(p.g.rows + ST - 1) / ST + p.g.count, gx = (p.N + ST - 1) / ST;
  for (int64_t y = 0; y < 1; ++y) {
    if (gy > 65535) return cudaErrorInvalidValue;
    grouped_kernel<<<dim3((unsigned)gx, (unsigned)gy), dim3(16, 16), 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_wgrad(const WgradParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.N + ST - 1) / ST), (unsigned)((p.M + ST - 1) / ST), (unsigned)p.g.count);
  if (grid.y > 65535) return cudaErrorInvalidValue;
  wgrad_kernel<<<grid, dim3(16, 16), 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_q4(const Q4Params& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.N + 7) / 8), (unsigned)std::min(p.g.rows, 65535));
  q4_kernel<<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gemmlib
