// expert_api.cu -- the C entry points of the expert-layer operators (declared in
// include/gemm.h): argument checks, workspaces and launches.  Host code only.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "expert.h"
#include "plan.h"

using namespace gemmlib;

namespace {

// The fused epilogue that the grouped operators take: a column bias, an
// activation and the output type (no C, no operand transforms).
gemm_status_t check_epilogue(const gemm_epilogue_t* epi, gemm_dtype_t out) {
  if (!is_float_out(out)) return GEMM_ERR_INVALID_ARG;
  if (!epi) return GEMM_OK;
  if (epi->act != GEMM_ACT_NONE && epi->act != GEMM_ACT_RELU) return GEMM_ERR_INVALID_ARG;
  if (epi->bias_mode != GEMM_BIAS_NONE && epi->bias_mode != GEMM_BIAS_COL && epi->bias_mode != GEMM_BIAS_ROW)
    return GEMM_ERR_INVALID_ARG;
  if (epi->bias_mode == GEMM_BIAS_ROW || epi->load_xf != 0) return GEMM_ERR_UNSUPPORTED;
  if (epi->bias_mode == GEMM_BIAS_COL && (!epi->bias || !is_float_out(epi->bias_dtype))) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

EpiParams epilogue_of(const gemm_epilogue_t* epi, gemm_dtype_t out, double alpha, void* D, int64_t ldd) {
  EpiParams e{};
  e.alpha = (float)alpha;
  e.D = D;
  e.ldd = ldd;
  e.d_dtype = out;
  e.bias_mode = epi ? epi->bias_mode : GEMM_BIAS_NONE;
  e.bias = e.bias_mode != GEMM_BIAS_NONE ? epi->bias : nullptr;
  e.bias_dtype = e.bias ? epi->bias_dtype : GEMM_F32;
  e.relu = (epi && epi->act == GEMM_ACT_RELU) ? 1 : 0;
  e.out_scale = 1.0f;
  e.vec_d = (aligned16(D) && (ldd * dtype_bytes(out)) % 16 == 0) ? 1 : 0;
  return e;
}

bool too_large(std::initializer_list<int64_t> dims) {
  for (int64_t d : dims)
    if (d > kMaxDim - 512) return true;   // tile edges past a size stay within 32 bits
  return false;
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_grouped(gemm_plan_t plan, gemm_layout_t lb, int64_t groups, int64_t M, int64_t N, int64_t K,
                               double alpha, const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b,
                               void* D, int64_t ldd, const int32_t* offsets, const gemm_epilogue_t* epi,
                               int64_t stride_bias, gemm_stream_t stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_grouped");
  if (!is_f16ish(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (lb != GEMM_OP_N && lb != GEMM_OP_T) return GEMM_ERR_INVALID_ARG;
  if (groups < 0 || M < 0 || N < 0 || K < 0 || stride_b < 0 || stride_bias < 0) return GEMM_ERR_INVALID_ARG;
  if (groups > kMaxGroups || too_large({M, N, K})) return GEMM_ERR_UNSUPPORTED;
  const gemm_dtype_t out = epi ? epi->out_dtype : plan->c;
  gemm_status_t s = check_epilogue(epi, out);
  if (s != GEMM_OK) return s;
  if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
  if (!offsets || !D || ldd < N) return GEMM_ERR_INVALID_ARG;
  if (K > 0 && (!A || !B || lda < K || ldb < (lb == GEMM_OP_N ? K : N))) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  GroupedParams p{};
  p.g = Groups{offsets, (int32_t)groups, (int32_t)M, plan->d_err};
  p.A = A;
  p.lda = lda;
  p.B = B;
  p.b_k = lb == GEMM_OP_N ? 1 : ldb;
  p.b_n = lb == GEMM_OP_N ? ldb : 1;
  p.stride_b = stride_b;
  p.N = (int32_t)N;
  p.K = (int32_t)K;
  p.ab_dtype = plan->ab;
  p.epi = epilogue_of(epi, out, alpha, D, ldd);
  p.epi.stride_bias = stride_bias;
  return launch_grouped(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_run_grouped_wgrad(gemm_plan_t plan, int64_t groups, int64_t M, int64_t N, int64_t K, double alpha,
                                     const void* A, int64_t lda, const void* B, int64_t ldb, double beta,
                                     const void* C, int64_t ldc, int64_t stride_c, void* D, int64_t ldd,
                                     int64_t stride_d, const int32_t* offsets, gemm_dtype_t out_dtype,
                                     gemm_stream_t stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_grouped_wgrad");
  if (!is_f16ish(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (groups < 0 || M < 0 || N < 0 || K < 0 || stride_c < 0 || stride_d < 0) return GEMM_ERR_INVALID_ARG;
  if (groups > kMaxGroups || too_large({M, N, K})) return GEMM_ERR_UNSUPPORTED;
  if (!is_float_out(out_dtype)) return GEMM_ERR_INVALID_ARG;
  if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
  if (!offsets || !D || ldd < N) return GEMM_ERR_INVALID_ARG;
  if (groups > 1 && stride_d < (M - 1) * ldd + N) return GEMM_ERR_INVALID_ARG;
  if (K > 0 && (!A || !B || lda < M || ldb < N)) return GEMM_ERR_INVALID_ARG;
  if (beta != 0.0) {
    if (!C || ldc < N) return GEMM_ERR_INVALID_ARG;
    if (C == D && (ldc != ldd || plan->c != out_dtype || (groups > 1 && stride_c != stride_d)))
      return GEMM_ERR_INVALID_ARG;
  }
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  WgradParams p{};
  p.g = Groups{offsets, (int32_t)groups, (int32_t)K, plan->d_err};
  p.A = A;
  p.lda = lda;
  p.B = B;
  p.ldb = ldb;
  p.M = (int32_t)M;
  p.N = (int32_t)N;
  p.ab_dtype = plan->ab;
  p.epi = epilogue_of(nullptr, out_dtype, alpha, D, ldd);
  p.epi.stride_d = stride_d;
  p.epi.beta = (float)beta;
  p.epi.read_c = beta != 0.0 ? 1 : 0;
  p.epi.C = p.epi.read_c ? C : nullptr;
  p.epi.ldc = ldc;
  p.epi.c_dtype = plan->c;
  p.epi.stride_c = stride_c;
  p.epi.vec_c = (p.epi.read_c && aligned16(C) && (ldc * dtype_bytes(plan->c)) % 16 == 0) ? 1 : 0;
  return launch_wgrad(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_run_q4(gemm_plan_t plan, int64_t groups, int64_t M, int64_t N, int64_t K, double alpha,
                          const void* A, int64_t lda, const gemm_q4_t* B, void* D, int64_t ldd,
                          const int32_t* offsets, const gemm_epilogue_t* epi, int64_t stride_bias,
                          gemm_stream_t stream) {
  if (!plan || !B) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_q4");
  if (!is_f16ish(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (groups < 0 || M < 0 || N < 0 || K < 0 || stride_bias < 0) return GEMM_ERR_INVALID_ARG;
  if (B->group_size <= 0 || B->group_size % 32 != 0 || !is_float_out(B->scale_dtype)) return GEMM_ERR_INVALID_ARG;
  if (B->stride_values < 0 || B->stride_scales < 0 || B->stride_zeros < 0) return GEMM_ERR_INVALID_ARG;
  if (groups > kMaxGroups || too_large({M, N, K})) return GEMM_ERR_UNSUPPORTED;
  const gemm_dtype_t out = epi ? epi->out_dtype : plan->c;
  gemm_status_t s = check_epilogue(epi, out);
  if (s != GEMM_OK) return s;
  if (groups == 0 || M == 0 || N == 0) return GEMM_OK;
  if (!D || ldd < N || (groups > 1 && !offsets)) return GEMM_ERR_INVALID_ARG;
  const int64_t kg = (K + B->group_size - 1) / B->group_size;
  if (K > 0 && (!A || lda < K || !B->values || B->ld_values < (K + 1) / 2 || !B->scales || B->ld_scales < kg ||
                (B->zeros && B->ld_zeros < kg)))
    return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  Q4Params p{};
  p.g = Groups{offsets, (int32_t)groups, (int32_t)M, plan->d_err};
  p.A = A;
  p.lda = lda;
  p.q = static_cast<const uint8_t*>(B->values);
  p.ldq = B->ld_values;
  p.stride_q = B->stride_values;
  p.scales = B->scales;
  p.lds = B->ld_scales;
  p.stride_s = B->stride_scales;
  p.scale_dtype = B->scale_dtype;
  p.zeros = B->zeros;
  p.ldz = B->ld_zeros;
  p.stride_z = B->stride_zeros;
  p.N = (int32_t)N;
  p.K = (int32_t)K;
  p.group = (int32_t)std::min<int64_t>(B->group_size, kMaxDim);
  p.ab_dtype = plan->ab;
  p.epi = epilogue_of(epi, out, alpha, D, ldd);
  p.epi.stride_bias = stride_bias;
  return launch_q4(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_orthogonalize(gemm_plan_t plan, int64_t batch, int64_t M, int64_t N, int steps,
                                 const double* coeffs, double eps, const void* G, int64_t ldg, int64_t stride_g,
                                 void* D, int64_t ldd, int64_t stride_d, gemm_dtype_t out_dtype,
                                 gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_orthogonalize");
  if (plan->ab == GEMM_S8) return GEMM_ERR_UNSUPPORTED;
  if (batch < 0 || M < 0 || N < 0 || stride_g < 0 || stride_d < 0 || steps < 0 || steps > 64 || !(eps >= 0.0) ||
      !std::isfinite(eps))
    return GEMM_ERR_INVALID_ARG;
  if (steps > 0 && (!coeffs || !std::isfinite(coeffs[0]) || !std::isfinite(coeffs[1]) || !std::isfinite(coeffs[2])))
    return GEMM_ERR_INVALID_ARG;
  if (out_dtype != GEMM_F16 && out_dtype != GEMM_BF16 && out_dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
  if (batch > 65535 || too_large({M, N})) return GEMM_ERR_UNSUPPORTED;
  if (batch == 0 || M == 0 || N == 0) return GEMM_OK;
  if (!G || !D || ldg < N || ldd < N) return GEMM_ERR_INVALID_ARG;
  if (batch > 1 && stride_d < (M - 1) * ldd + N) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);

  // X is kept as the wide one of the matrix and its transpose: m <= n.
  const bool tall = M > N;
  const int64_t m = tall ? N : M, n = tall ? M : N;
  const int64_t ldx = (n + 7) / 8 * 8, lde = (m + 7) / 8 * 8;
  const int64_t sx = m * ldx, se = m * lde;
  const size_t xb = align_up((size_t)(batch * sx) * 2, 256), eb = align_up((size_t)(batch * se) * 2, 256);
  const size_t sb = align_up((size_t)batch * ortho_slots(m, n) * sizeof(float), 256);
  gemm_status_t s = ensure_ws(plan, 2 * xb + 2 * eb + sb + (size_t)se * 2, stream);
  if (s != GEMM_OK) return s;
  char* ws = static_cast<char*>(plan->ws);
  __half* X[2] = {reinterpret_cast<__half*>(ws), reinterpret_cast<__half*>(ws + xb)};
  __half* E = reinterpret_cast<__half*>(ws + 2 * xb);
  __half* F = reinterpret_cast<__half*>(ws + 2 * xb + eb);
  float* sums = reinterpret_cast<float*>(ws + 2 * xb + 2 * eb);
  // fp16 keeps 11 bits; entries of X are at most ~1 and as small as 1 / sqrt(m n), so
  // they are held times 256, which keeps the small ones out of fp16's subnormals.
  const double scale = 256.0;
  __half* I = reinterpret_cast<__half*>(ws + 2 * xb + 2 * eb + sb);
  const int es = dtype_bytes(plan->ab);
  const OrthoInput in{G, m, n, ldg, stride_g, tall ? 1 : 0,
                      aligned16(G) && (ldg * es) % 16 == 0 && (batch == 1 || (stride_g * es) % 16 == 0) ? 1 : 0};
  if (launch_ortho_input(in, plan->ab, batch, sums, (float)eps, (float)scale, X[0], ldx, sx, stream) != cudaSuccess ||
      launch_identity(I, m, lde, stream) != cudaSuccess)
    return GEMM_ERR_CUDA;
  for (int k = 0; k < steps; ++k) {
    // E = X X' - h I with h = 1 once the singular values have come near one (the
    // last two steps): E is then small and its rounding with it.  With X X' = E + h I,
    //   a X + (b X X' + c (X X')^2) X = (a + b h + c h^2) X + ((b + 2 c h) E + c E^2) X.
    const double h = k >= steps - 2 ? 1.0 : 0.0;
    const double c = coeffs[2], b = coeffs[1] + 2 * c * h, a = coeffs[0] + coeffs[1] * h + c * h * h;
    s = run_product(plan, GEMM_F16, GEMM_F16, GEMM_F16, GEMM_OP_T, GEMM_OP_N, m, m, n, 1.0 / (scale * scale), X[0],
                    ldx, sx, X[0], ldx, sx, -h, I, lde, 0, E, lde, se, batch, stream_);
    if (s == GEMM_OK)
      s = run_product(plan, GEMM_F16, GEMM_F16, GEMM_F16, GEMM_OP_T, GEMM_OP_N, m, m, m, c, E, lde, se, E, lde, se, b,
                      E, lde, se, F, lde, se, batch, stream_);
    if (s == GEMM_OK)
      s = run_product(plan, GEMM_F16, GEMM_F16, GEMM_F16, GEMM_OP_T, GEMM_OP_T, m, n, m, 1.0, F, lde, se, X[0], ldx,
                      sx, a, X[0], ldx, sx, X[1], ldx, sx, batch, stream_);
    if (s != GEMM_OK) return s;
    std::swap(X[0], X[1]);
  }
  return launch_unscale(X[0], batch, M, N, ldx, sx, tall, (float)(1.0 / scale), D, out_dtype, ldd, stride_d, stream) ==
                 cudaSuccess
             ? GEMM_OK
             : GEMM_ERR_CUDA;
}

}  // extern "C"
