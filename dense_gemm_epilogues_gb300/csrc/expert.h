// expert.h -- launch interface of the expert-layer kernels: products grouped by
// expert, products with 4-bit weights, orthogonalised updates (internal).
#pragma once

#include "kernels.h"

namespace gemmlib {

#if defined(__CUDACC__)
// Launch a kernel as a programmatic dependent of the stream's last one (it calls
// pdl_wait before it touches global memory).
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
#endif

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

// f(type tag) for an output type: f's argument has it as a constant `value`.
template <int V>
struct TypeTag {
  static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void with_type(int dtype, F&& f) {
  if (dtype == GEMM_F32) f(TypeTag<GEMM_F32>{});
  else if (dtype == GEMM_F16) f(TypeTag<GEMM_F16>{});
  else f(TypeTag<GEMM_BF16>{});
}

// ReLU that keeps NaN (fmaxf would make it 0 and hide it from the layers that follow).
__device__ __forceinline__ float relu_keep_nan(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}

// Order this thread's use of a tensor map after its making by another kernel.
__device__ __forceinline__ void tensormap_acquire(const CUtensorMap* tm) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(tm) : "memory");
}
#endif

// What seg_kernel.cu computes (its head says how).
enum { SEG_TOKENS = 0, SEG_WGRAD = 1, SEG_CHAIN = 2 };
// CHAIN's maps in tmB, beside E as M side in tmA: both X buffers as M side of E, as N side
// of E, as N side of F X; F as M side; E as N side.
enum { CHAIN_XK = 0, CHAIN_XB = 2, CHAIN_XN = 4, CHAIN_F = 6, CHAIN_EB = 7, SEG_MAPS = 8 };
struct SegParams {
  CUtensorMap tmA;              // M side (WGRAD: the template of every group's map)
  CUtensorMap tmB[SEG_MAPS];    // N side; TOKENS: boxes of 128, 64, 32, 16 and 8 rows
  Groups groups;                // TOKENS, WGRAD
  const CUtensorMap* group_maps;   // WGRAD: two per group, made by launch_wgrad_maps
  uint64_t a_base, b_base;      // WGRAD: the operands' addresses and row pitches in bytes
  uint64_t a_pitch, b_pitch;
  int64_t M;                    // rows of the M side
  int32_t N, K;                 // rows of the N side and depth (what the groups do not give)
  int32_t tiles_m, tiles_n;     // 128- or 256-wide tiles
  int32_t tiles_per_group, num_tiles;
  int32_t a_batched;            // TOKENS: the M side has one slice per group
  uint32_t idesc;               // instruction descriptor without N
  const float* m_scale;         // TOKENS: factors of the M side's rows, M per group; null: 1
  // CHAIN: X is M x N, E and F are M x M; tiles_per_group tiles of E or F (bns columns
  // each), tiles_m x tiles_n of X (bn columns each) per matrix; num_tiles over all steps.
  int32_t batch, steps, bns, bn;
  int32_t store_t;              // the result (epi.D) is stored transposed
  // Matrices as pairs of fp16 halves (the second one is what the first rounds away): X
  // always for a X; with `pairs`, X, E and F in the products too, as the sum of three,
  // hi lo + lo hi + hi hi (the second halves then lie `batch` slices behind the first).
  int32_t pairs;
  int32_t* counters;            // 3 * steps * batch * tiles_m, zero at the start
  struct {
    __half *x[2], *e, *f;       // step s reads x[s % 2]
    __half* xlo[2];             // second halves of X (without `pairs` one buffer: read in place)
    int64_t ldx, stride_x, lde, stride_e;
    float a[2], b[2], c;        // early steps, the last two (see gemm_orthogonalize)
    float inv_x, scale_e, inv_e;   // X is held times 1 / inv_x, E and F times scale_e = 1 / inv_e
  } chain;
  EpiParams epi;
  int32_t* err;
  uint64_t timeout_ns;
};
// workers: CTAs (cg 1) or CTA pairs (cg 2).
cudaError_t launch_seg(const SegParams& p, int mode, int cg, bool a_mn, int workers, cudaStream_t stream);
cudaError_t launch_wgrad_maps(const SegParams& p, CUtensorMap* maps, cudaStream_t stream);

// dst[z][r][c] = src[z][r][c] for elements of one or two bytes, with a pitch that TMA
// can address (ldd * elem_bytes a multiple of 16; columns up to ldd are zero).  offsets != null: the z-th matrix
// is skipped when group z has no rows.
cudaError_t launch_repitch(const void* src, int64_t ld, int64_t stride, void* dst, int64_t ldd, int64_t stride_d,
                           int64_t rows, int64_t cols, int64_t batch, const int32_t* offsets, int elem_bytes,
                           cudaStream_t stream);

// D[r, n] = act(alpha * sum_k A[r, k] * scale[n, k / group] * (q[n, k] - zero[n, k / group]) + bias[n])
// with the q, scales and zeros of the row's group.
struct Q4Params {
  CUtensorMap tm_q;              // q: boxes of 64 bytes (128 k) x cta_rows columns, 64-byte swizzle
  CUtensorMap tm_x;              // A: boxes of 64 k x 8 nt rows, 128-byte swizzle
  Groups g;
  const uint8_t* q;              // N rows of ceil(K / 2) bytes, the lower k in the low half
  int64_t ldq, stride_q;         // bytes
  const void* scales;
  int64_t lds, stride_s;
  int32_t scale_dtype;
  const uint8_t* zeros;          // null: 8 everywhere
  int64_t ldz, stride_z;
  int32_t N, K, group;
  int32_t ab_dtype;
  int32_t q_batched;             // tm_q has one slice per group
  int32_t cta_rows;              // columns of weights per CTA
  const float* col_scale;        // decoded weights are s (q - z) / col_scale, N per group; null: 1
  int32_t group_units, group_shift, vec_s, scale_cols;   // set by launch_q4
  EpiParams epi;
  uint64_t timeout_ns;
};
// How q4_kernel runs a call: blocks of 8 rows per pass over the weights (1, 2, 4) and
// columns per CTA.  rows_per_group: of an average group; groups_used: at most so many
// groups have rows.
struct Q4Shape {
  int nt, cta_rows;
};
Q4Shape q4_shape(int64_t N, int64_t rows_per_group, int64_t groups_used, int sm_count);
cudaError_t launch_q4(const Q4Params& p, int nt, cudaStream_t stream);
// out[group][n]: the power of two near 2^-11 times the largest scale of column n.
cudaError_t launch_q4_range(const Q4Params& p, float* out, cudaStream_t stream);
cudaError_t launch_q4_dequant(const Q4Params& p, void* out, int64_t ldw, int64_t stride_w, cudaStream_t stream);

// Newton-Schulz: the wide matrix X (m <= n) of each input matrix G.
struct OrthoInput {
  const void* g;
  int64_t m, n;             // of X
  int64_t ld, stride;       // of G
  int32_t transpose;        // X is G's transpose
  int32_t vec;              // G's rows can be read 16 bytes at a time
};
int ortho_slots(int64_t m, int64_t n);   // partial sums per matrix
// X = G / (||G|| + eps) times `scale`, as pairs of fp16 halves x + xlo; partials: batch *
// ortho_slots(m, n) floats.
// counters[0 .. num_counters) are set to zero.
cudaError_t launch_ortho_input(const OrthoInput& in, int dtype, int64_t batch, float* partials, float eps, float scale,
                               __half* x, __half* xlo, int64_t ldx, int64_t stride_x, int32_t* counters,
                               int64_t num_counters, cudaStream_t stream);
// D (M x N) = scale * (x + xlo) (or its transpose), cast.
cudaError_t launch_unscale(const __half* x, const __half* xlo, int64_t batch, int64_t M, int64_t N, int64_t ldx, int64_t stride_x,
                           int transpose, float scale, void* D, int dtype, int64_t ldd, int64_t stride_d,
                           cudaStream_t stream);

}  // namespace gemmlib
