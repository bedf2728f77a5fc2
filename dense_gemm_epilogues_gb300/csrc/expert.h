// expert.h -- launch interface of the expert-layer kernels: products grouped by
// expert, products with 4-bit weights, orthogonalised updates (internal).
#pragma once

#include "kernels.h"

namespace gemmlib {

constexpr int kMaxGroups = 1024;   // experts of one call (their tile counts are kept in shared memory)

// Rows [offsets[g], offsets[g + 1]) of a buffer of `rows` rows belong to group g.
// Bad offsets (decreasing, or outside the buffer) are clamped, so that no access
// leaves the buffers, and reported through the error word.
struct Groups {
  const int32_t* offsets;   // device, count + 1 entries; null: one group of all rows
  int32_t count;
  int32_t rows;
  int32_t* err;
};

#if defined(__CUDACC__)
__device__ __forceinline__ void group_range(const Groups& g, int e, int& lo, int& hi) {
  if (g.offsets == nullptr) {
    lo = 0;
    hi = g.rows;
    return;
  }
  const int a = g.offsets[e], b = g.offsets[e + 1];
  lo = min(max(a, 0), g.rows);
  hi = min(max(b, lo), g.rows);
  if (lo != a || hi != b) atomicCAS(g.err, 0, (int32_t)GEMM_ERR_INVALID_ARG);
}
#endif

// D[r, :] = act(alpha * A[r, :] * op(B_g) + bias_g) for the rows r of each group g.
struct GroupedParams {
  Groups g;
  const void* A;                 // rows x K, row-major
  int64_t lda;
  const void* B;                 // per group: element (k, n) at k * b_k + n * b_n
  int64_t b_k, b_n, stride_b;
  int32_t N, K;
  int32_t ab_dtype;
  EpiParams epi;                 // D: rows x N; bias: stride_bias elements from group to group
};
cudaError_t launch_grouped(const GroupedParams& p, cudaStream_t stream);

// D_g = alpha * A_g' * B_g + beta * C_g over the rows of each group g (A: rows x M, B: rows x N).
struct WgradParams {
  Groups g;
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  int32_t M, N;
  int32_t ab_dtype;
  EpiParams epi;                 // C, D: M x N per group, stride_c / stride_d from group to group
};
cudaError_t launch_wgrad(const WgradParams& p, cudaStream_t stream);

// D[r, n] = act(alpha * sum_k A[r, k] * scale[n, k / group] * (q[n, k] - zero[n, k / group]) + bias[n])
// with the q, scales and zeros of the row's group.
struct Q4Params {
  Groups g;
  const void* A;                 // rows x K, row-major
  int64_t lda;
  const uint8_t* q;              // N rows of ceil(K / 2) bytes, the lower k in the low half
  int64_t ldq, stride_q;         // bytes
  const void* scales;
  int64_t lds, stride_s;
  int32_t scale_dtype;
  const uint8_t* zeros;          // null: 8 everywhere
  int64_t ldz, stride_z;
  int32_t N, K, group;
  int32_t ab_dtype;
  EpiParams epi;
};
cudaError_t launch_q4(const Q4Params& p, cudaStream_t stream);

// Newton-Schulz: the wide matrix X (m <= n) of each input matrix G.
struct OrthoInput {
  const void* g;
  int64_t m, n;             // of X
  int64_t ld, stride;       // of G
  int32_t transpose;        // X is G's transpose
  int32_t vec;              // G's rows can be read 16 bytes at a time
};
int ortho_slots(int64_t m, int64_t n);   // partial sums per matrix
// X = G / (||G|| + eps) times `scale`, in fp16; partials: batch * ortho_slots(m, n) floats.
cudaError_t launch_ortho_input(const OrthoInput& in, int dtype, int64_t batch, float* partials, float eps, float scale,
                               __half* x, int64_t ldx, int64_t stride_x, cudaStream_t stream);
cudaError_t launch_identity(__half* d, int64_t m, int64_t ld, cudaStream_t stream);
// D (M x N) = scale * X (or its transpose), cast.
cudaError_t launch_unscale(const __half* x, int64_t batch, int64_t M, int64_t N, int64_t ldx, int64_t stride_x,
                           int transpose, float scale, void* D, int dtype, int64_t ldd, int64_t stride_d,
                           cudaStream_t stream);

}  // namespace gemmlib
