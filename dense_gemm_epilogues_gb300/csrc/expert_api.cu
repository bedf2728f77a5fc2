// expert_api.cu -- the C entry points of the expert-layer operators (declared in
// include/gemm.h): argument checks, workspaces and launches.  Host code only.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "expert.h"
#include "operands.h"

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

// Are 4-bit weights decoded once into scratch and multiplied on the tensor-core kernel,
// rather than inside the product, once per 32 rows?  Up to 32 rows never (one pass over
// the weights, exact integers).  Beyond, by the times that both take, in us: a pass inside
// the product 3 and 0.4 per million weights; decoding once 0.38 per million, and each
// wave of 128 x 128 tiles 0.45 per 128 k.  Measured, inside / once:
//                                 33 rows        64             96             128 per expert
//   4096 -> 11008                 44.8 / 36.4    46.9 / 37.3    68.6 / 38.5    90.3 / 40.5
//   4096 -> 4096                  17.2 / 21.6    17.8 / 22.2    25.7 / 23.4    33.6 / 25.7
//   1024 -> 1024                  8.2 / 7.5      7.8 / 7.7      11.2 / 8.2     14.6 / 9.9
//   11008 -> 4096                 33.5 / 54.8    34.2 / 56.5    50.3 / 59.1    66.5 / 62.5
//   2048 -> 1408, 16 experts      42.9 / 39.8    70.4 / 41.3    97.6 / 42.3    123 / 46.7
// The estimate takes the slower side by 17 per cent for 96 rows of 11008 -> 4096 and by 9 for
// 33 rows of 1024 -> 1024, elsewhere the faster one or one within 2 per cent.
bool q4_decode_once(int64_t N, int64_t K, int64_t rows, int64_t groups, int sm_count) {
  if (rows <= 32 || K == 0) return false;
  const double millions = 1e-6 * (double)N * (double)K * (double)groups;
  const int64_t tiles = (N + 127) / 128 * ((rows + 127) / 128) * groups, waves = (tiles + sm_count - 1) / sm_count;
  const double inside = (3.0 + 0.4 * millions) * (double)((rows + 31) / 32);
  const double once = 0.38 * millions + 0.45 * (double)((K + 127) / 128) * (double)waves + 3.0;
  return once < inside;
}

// D[r, :] = epilogue(x[r, :] * W_g) on seg_kernel: x M x K row-major, W_g K x N (w_mn: N
// contiguous, else K); TMA can address both.  w_scale: factors of W_g's columns, N per group,
// or null.
gemm_status_t tokens_product(gemm_plan* plan, const Groups& groups, int64_t M, int64_t N, int64_t K, const Operand& x,
                             const Operand& w, bool w_mn, const float* w_scale, const EpiParams& epi, const char* entry,
                             cudaStream_t stream) {
  const int64_t nw = w.stride != 0 ? groups.count : 1;   // matrices of weights
  SegParams p;
  std::memset(&p, 0, sizeof(p));
  p.groups = groups;
  // CTA pairs from 128 rows per expert on, if their tiles (256 x 256) occupy three quarters
  // of the chip or single ones need a second wave.  Single CTAs / pairs, us: 64 experts of
  // 256 rows (2048 to 4096) 348 / 240, 32 of 128 100 / 94, of 64 86.0 / 86.6; 16 of 300 (1000
  // to 2048) 32.0 / 26.1, of 96 18.1 / 18.3; 8 of 128 (1024 to 2048) 13.4 / 12.4; one matrix
  // 4096 to 11008, 256 rows 36.8 / 29.2; 4096 to 4096, 300 rows 18.1 / 21.5.
  const int64_t groups_used = std::min<int64_t>(groups.count, M);
  const int64_t tiles256 = (N + 255) / 256 * std::max((M + 255) / 256, groups_used);
  const int64_t tiles128 = (N + 127) / 128 * std::max((M + 127) / 128, groups_used);
  const bool fill = 4 * tiles256 >= 3 * plan->pair_clusters || tiles128 > plan->sm_count;
  const int cg = plan->pair_clusters > 0 && M >= 128 * (int64_t)groups.count && fill ? 2 : 1;
  const int64_t tiles = ((N + 128 * cg - 1) / (128 * cg)) * (M / (128 * cg) + std::min<int64_t>(groups.count, M));
  if (tiles > kMaxTiles) return GEMM_ERR_UNSUPPORTED;
  if (K > 0) {
    const CUtensorMapDataType dt = map_type(plan->ab);
    bool ok = w_mn ? encode_3d(&p.tmA, dt, w.p, N, K, w.ld, nw, w.stride, 64, 2 * TC_BK)
                   : encode_3d(&p.tmA, dt, w.p, K, N, w.ld, nw, w.stride, TC_BK, 128);
    for (int b = 0; b < 5; ++b) ok = ok && encode_3d(&p.tmB[b], dt, x.p, K, M, x.ld, 1, 0, TC_BK, 128u >> b);
    if (!ok) return GEMM_ERR_CUDA;
  }
  p.a_batched = nw > 1 ? 1 : 0;
  p.m_scale = w_scale;
  p.M = N;
  p.K = (int32_t)K;
  p.tiles_m = (int32_t)((N + 128 * cg - 1) / (128 * cg));
  p.idesc = make_idesc(plan->ab == GEMM_BF16, 0, w_mn, false, 128 * cg);
  p.epi = epi;
  p.err = plan->d_err;
  p.timeout_ns = plan->timeout_ns;
  const int workers = workers_of(plan, cg, tiles);
  if (launch_seg(p, SEG_TOKENS, cg, w_mn, workers, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  plan->last = seg_config(cg, tiles, workers);
  log_config(entry, M, N, K, groups.count, plan->last);
  return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_grouped(gemm_plan_t plan, gemm_layout_t lb, int64_t groups, int64_t M, int64_t N, int64_t K,
                               double alpha, const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b,
                               void* D, int64_t ldd, const int32_t* offsets, const gemm_epilogue_t* epi,
                               int64_t stride_bias, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_grouped");
  if (!is_f16ish(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (lb != GEMM_OP_N && lb != GEMM_OP_T) return GEMM_ERR_INVALID_ARG;
  if (groups < 0 || M < 0 || N < 0 || K < 0 || stride_b < 0 || stride_bias < 0) return GEMM_ERR_INVALID_ARG;
  if (groups > kMaxGroups || too_large({M, N, K})) return GEMM_ERR_UNSUPPORTED;
  const gemm_dtype_t out = epi ? epi->out_dtype : plan->c;
  gemm_status_t s = check_epilogue(epi, out);
  if (s != GEMM_OK) return s;
  if (groups == 0 || M == 0 || N == 0) return nothing(plan);
  if (!offsets || !D || ldd < N) return GEMM_ERR_INVALID_ARG;
  if (K > 0 && (!A || !B || lda < K || ldb < (lb == GEMM_OP_N ? K : N))) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  EpiParams e = epilogue_of(epi, out, alpha, D, ldd);
  e.stride_bias = stride_bias;
  Operand x{A, lda, 0}, w{B, ldb, stride_b};
  const bool w_mn = lb == GEMM_OP_T;
  if (K > 0) {   // operands that TMA cannot address are copied to a pitch it can
    const int64_t wrows = w_mn ? K : N, wcols = w_mn ? N : K, nw = stride_b != 0 ? groups : 1;
    const size_t xb = repitch_bytes(x, M, K, 1), wb = repitch_bytes(w, wrows, wcols, nw);
    if (xb + wb > 0) {
      s = ensure_ws(plan, xb + wb, stream);
      char* ws = static_cast<char*>(plan->ws.p);
      if (s == GEMM_OK) s = repitch(&x, M, K, 1, nullptr, ws, stream);
      if (s == GEMM_OK) s = repitch(&w, wrows, wcols, nw, nw > 1 ? offsets : nullptr, ws + xb, stream);
      if (s != GEMM_OK) return s;
    }
  }
  return tokens_product(plan, Groups{offsets, (int32_t)groups, (int32_t)M, plan->d_err}, M, N, K, x, w, w_mn, nullptr, e,
                        "grouped", stream);
}

gemm_status_t gemm_run_grouped_wgrad(gemm_plan_t plan, int64_t groups, int64_t M, int64_t N, int64_t K, double alpha,
                                     const void* A, int64_t lda, const void* B, int64_t ldb, double beta,
                                     const void* C, int64_t ldc, int64_t stride_c, void* D, int64_t ldd,
                                     int64_t stride_d, const int32_t* offsets, gemm_dtype_t out_dtype,
                                     gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_grouped_wgrad");
  if (!is_f16ish(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (groups < 0 || M < 0 || N < 0 || K < 0 || stride_c < 0 || stride_d < 0) return GEMM_ERR_INVALID_ARG;
  if (groups > kMaxGroups || too_large({M, N, K})) return GEMM_ERR_UNSUPPORTED;
  if (!is_float_out(out_dtype)) return GEMM_ERR_INVALID_ARG;
  if (groups == 0 || M == 0 || N == 0) return nothing(plan);
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
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  Operand x{A, lda, 0}, y{B, ldb, 0};
  SegParams p;
  std::memset(&p, 0, sizeof(p));
  // CTA pairs (tiles of 256 x 256) from 256 rows per expert on.  Both gradients on single
  // CTAs / pairs, us: 32 experts of 512 rows (4096 x 2048) 646 / 427, 16 of 300 (1000 x 2048)
  // 74.2 / 69.3, of 192 61.6 / 61.3, of 96 51.2 / 53.6; 8 of 192 (1024 x 2048) 35.4 / 41.7.
  const int cg = plan->pair_clusters > 0 && M > 128 && N > 128 && K >= 256 * groups ? 2 : 1;
  p.tiles_m = (int32_t)((M + 128 * cg - 1) / (128 * cg));
  p.tiles_n = (int32_t)((N + 128 * cg - 1) / (128 * cg));
  const int64_t tiles = groups * p.tiles_m * (int64_t)p.tiles_n;
  if (tiles > kMaxTiles) return GEMM_ERR_UNSUPPORTED;
  p.tiles_per_group = p.tiles_m * p.tiles_n;
  p.num_tiles = (int32_t)tiles;
  p.groups = Groups{offsets, (int32_t)groups, (int32_t)K, plan->d_err};
  const size_t mb = align_up((size_t)groups * 2 * sizeof(CUtensorMap), 256);
  const size_t xb = K > 0 ? repitch_bytes(x, K, M, 1) : 0, yb = K > 0 ? repitch_bytes(y, K, N, 1) : 0;
  gemm_status_t s = ensure_ws(plan, mb + xb + yb, stream);
  if (s != GEMM_OK) return s;
  char* ws = static_cast<char*>(plan->ws.p);
  CUtensorMap* maps = reinterpret_cast<CUtensorMap*>(ws);
  if (K > 0) {
    s = repitch(&x, K, M, 1, nullptr, ws + mb, stream);
    if (s == GEMM_OK) s = repitch(&y, K, N, 1, nullptr, ws + mb + xb, stream);
    if (s != GEMM_OK) return s;
    const CUtensorMapDataType dt = map_type(plan->ab);
    if (!encode_3d(&p.tmA, dt, x.p, M, K, x.ld, 1, 0, 64, 2 * TC_BK) ||
        !encode_3d(&p.tmB[0], dt, y.p, N, K, y.ld, 1, 0, 64, 2 * TC_BK))
      return GEMM_ERR_CUDA;
    p.a_base = reinterpret_cast<uint64_t>(x.p);
    p.b_base = reinterpret_cast<uint64_t>(y.p);
    p.a_pitch = (uint64_t)x.ld * 2;
    p.b_pitch = (uint64_t)y.ld * 2;
    if (launch_wgrad_maps(p, maps, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  }
  p.group_maps = maps;
  p.M = M;
  p.N = (int32_t)N;
  p.idesc = make_idesc(plan->ab == GEMM_BF16, 0, true, true, 128 * cg);
  p.epi = epilogue_of(nullptr, out_dtype, alpha, D, ldd);
  p.epi.stride_d = stride_d;
  p.epi.beta = (float)beta;
  p.epi.read_c = beta != 0.0 ? 1 : 0;
  p.epi.C = p.epi.read_c ? C : nullptr;
  p.epi.ldc = ldc;
  p.epi.c_dtype = plan->c;
  p.epi.stride_c = stride_c;
  const int cs = dtype_bytes(plan->c);
  p.epi.vec_c = (p.epi.read_c && aligned16(C) && (ldc * cs) % 16 == 0 && (stride_c * cs) % 16 == 0) ? 1 : 0;
  if (groups > 1 && (stride_d * dtype_bytes(out_dtype)) % 16 != 0) p.epi.vec_d = 0;
  p.err = plan->d_err;
  p.timeout_ns = plan->timeout_ns;
  const int workers = workers_of(plan, cg, tiles);
  if (launch_seg(p, SEG_WGRAD, cg, true, workers, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  plan->last = seg_config(cg, tiles, workers);
  log_config("grouped_wgrad", M, N, K, groups, plan->last);
  return GEMM_OK;
}

gemm_status_t gemm_run_q4(gemm_plan_t plan, int64_t groups, int64_t M, int64_t N, int64_t K, double alpha,
                          const void* A, int64_t lda, const gemm_q4_t* B, void* D, int64_t ldd,
                          const int32_t* offsets, const gemm_epilogue_t* epi, int64_t stride_bias,
                          gemm_stream_t stream_) {
  if (!plan || !B) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_q4");
  if (!is_f16ish(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (groups < 0 || M < 0 || N < 0 || K < 0 || stride_bias < 0) return GEMM_ERR_INVALID_ARG;
  if (B->group_size <= 0 || B->group_size % 32 != 0 || !is_float_out(B->scale_dtype)) return GEMM_ERR_INVALID_ARG;
  if (B->stride_values < 0 || B->stride_scales < 0 || B->stride_zeros < 0) return GEMM_ERR_INVALID_ARG;
  if (groups > kMaxGroups || too_large({M, N, K})) return GEMM_ERR_UNSUPPORTED;
  if (B->ld_scales >= (1 << 23) || B->ld_zeros >= (1 << 23)) return GEMM_ERR_UNSUPPORTED;   // 32-bit offsets in a CTA
  const gemm_dtype_t out = epi ? epi->out_dtype : plan->c;
  gemm_status_t s = check_epilogue(epi, out);
  if (s != GEMM_OK) return s;
  if (groups == 0 || M == 0 || N == 0) return nothing(plan);
  if (!D || ldd < N || (groups > 1 && !offsets)) return GEMM_ERR_INVALID_ARG;
  const int64_t kg = (K + B->group_size - 1) / B->group_size;
  if (K > 0 && (!A || lda < K || !B->values || B->ld_values < (K + 1) / 2 || !B->scales || B->ld_scales < kg ||
                (B->zeros && B->ld_zeros < kg)))
    return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  Q4Params p;
  std::memset(&p, 0, sizeof(p));
  p.g = Groups{offsets, (int32_t)groups, (int32_t)M, plan->d_err};
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
  p.timeout_ns = plan->timeout_ns;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int64_t per_group = (M + groups - 1) / groups;   // rows of an average group
  Operand x{A, lda, 0};
  const bool q_ok = aligned16(p.q) && p.ldq % 16 == 0 && (groups == 1 || p.stride_q % 16 == 0);
  const int64_t ldq = align_up((size_t)(K + 1) / 2, 16);
  const size_t qb = K == 0 || q_ok ? 0 : align_up((size_t)(groups * N * ldq), 256);
  const size_t xb = K == 0 ? 0 : repitch_bytes(x, M, K, 1);
  bool prompt = q4_decode_once(N, K, per_group, std::min(groups, M), plan->sm_count);
  const int64_t ldw = (K + 15) / 16 * 16;
  size_t wb = prompt ? align_up((size_t)(groups * N * ldw) * 2, 256) : 0;
  // Weights with scales of a wider type are decoded into fp16 relative to their column's
  // largest scale (2000 rows of 4096 to 11008, fp32 scales: 140 us, with bf16 x 135); bf16 has the
  // range of every scale.
  bool ranged = prompt && plan->ab == GEMM_F16 && B->scale_dtype != GEMM_F16;
  size_t fb = ranged ? (size_t)(groups * N) * sizeof(float) : 0;
  if (prompt && ensure_ws(plan, qb + xb + wb + fb, stream) != GEMM_OK) {
    prompt = ranged = false;   // no memory for the decoded weights of all experts: decode inside the product
    wb = fb = 0;
  }
  if (!prompt && qb + xb > 0) {
    s = ensure_ws(plan, qb + xb, stream);
    if (s != GEMM_OK) return s;
  }
  char* ws = static_cast<char*>(plan->ws.p);
  if (qb > 0) {   // packed weights that TMA cannot address are copied to a pitch it can
    if (launch_repitch(p.q, p.ldq, p.stride_q, ws, ldq, N * ldq, N, (K + 1) / 2, groups, offsets, 1, stream) != cudaSuccess)
      return GEMM_ERR_CUDA;
    p.q = reinterpret_cast<const uint8_t*>(ws);
    p.ldq = ldq;
    p.stride_q = N * ldq;
  }
  s = K == 0 ? GEMM_OK : repitch(&x, M, K, 1, nullptr, ws + qb, stream);
  if (s != GEMM_OK) return s;
  if (prompt) {
    if (ranged) {
      float* range = reinterpret_cast<float*>(ws + qb + xb + wb);
      if (launch_q4_range(p, range, stream) != cudaSuccess) return GEMM_ERR_CUDA;
      p.col_scale = range;
    }
    if (launch_q4_dequant(p, ws + qb + xb, ldw, N * ldw, stream) != cudaSuccess) return GEMM_ERR_CUDA;
    return tokens_product(plan, p.g, M, N, K, x, Operand{ws + qb + xb, ldw, groups > 1 ? N * ldw : 0}, false,
                          p.col_scale, p.epi, "q4", stream);
  }
  const Q4Shape shape = q4_shape(N, per_group, std::min(groups, M), plan->sm_count);
  p.cta_rows = shape.cta_rows;
  p.q_batched = groups > 1 && p.stride_q != 0 ? 1 : 0;
  if (K > 0 &&
      (!encode_tiled(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.q, (K + 1) / 2, N, p.ldq, p.q_batched ? groups : 1,
                     p.q_batched ? p.stride_q : N * p.ldq, 64, (uint32_t)shape.cta_rows, CU_TENSOR_MAP_SWIZZLE_64B) ||
       !encode_tiled(&p.tm_x, map_type(plan->ab), x.p, K, M, x.ld * 2, 1, 0, 64, 8u * shape.nt,
                     CU_TENSOR_MAP_SWIZZLE_128B)))
    return GEMM_ERR_CUDA;
  if (launch_q4(p, shape.nt, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  gemm_config_t cfg{};
  cfg.kernel = GEMM_KERNEL_SIMT;
  cfg.bm = 8 * shape.nt;
  cfg.bn = shape.cta_rows;
  cfg.bk = 128;
  cfg.cta_group = cfg.cluster = cfg.split_k = 1;
  cfg.grid = cfg.tiles = (int32_t)((N + shape.cta_rows - 1) / shape.cta_rows * groups);
  plan->last = cfg;
  log_config("q4", M, N, K, groups, cfg);
  return GEMM_OK;
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
  if (batch == 0 || M == 0 || N == 0) return nothing(plan);
  if (!G || !D || ldg < N || ldd < N) return GEMM_ERR_INVALID_ARG;
  if (batch > 1 && stride_d < (M - 1) * ldd + N) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);

  // X is kept as the wide one of the matrix and its transpose: m <= n.
  const bool tall = M > N;
  const int64_t m = tall ? N : M, n = tall ? M : N;
  const int64_t ldx = (n + 15) / 16 * 16, lde = (m + 15) / 16 * 16;   // rows on 32 bytes
  const int64_t sx = m * ldx, se = m * lde;
  // Tiles: CTA pairs with 256 columns cost the least per product; with too few of them
  // for all pairs, narrower ones on E and F fill the chip, and small problems (whose time
  // is the chain of tile latencies) run narrow tiles on single CTAs.  Measured, us, bf16
  // result, single CTAs / pairs with E and F tiles of 64 / 128 / 256 columns:
  //   256 x 384 80 / 105 / 116 / 138;  1024^2 116 / 151 / 169 / 213;  700 x 2800 153 / 162 / 184 / 234;
  //   1024 x 4096 211 / 194 / 220 / 288;  2048^2 299 / 267 / 241 / 294;  32 of 300 x 500
  //   238 / 274 / 209 / 205;  16 of 768 x 2001 642 / 566 / 480 / 476;  4096 x 11008 - / - / 2331 / 2103.
  // fp32 result (three products for one): 256 x 384 113 / 140 / 159 / 202;  700 x 2800 290 / 287 /
  // 335 / 452;  1024 x 4096 434 / 358 / 416 / 593;  2048^2 680 / 548 / 458 / 588;  16 of 768 x 2001
  // 1397 / 1077 / 907 / 889;  4096 x 11008 - / - / 6730 / 6291.
  const int64_t m256 = (m + 255) / 256, sym256 = batch * m256 * (m256 + 1) / 2, dense256 = batch * m256 * ((n + 255) / 256);
  int cg = 1, bns = 64, bn = 64;   // columns of a tile of E and F, and of X
  if (plan->pair_clusters > 0 && (sym256 >= 24 || dense256 >= 48)) {
    cg = 2;
    bn = 256;
    bns = 2 * sym256 >= 3 * plan->pair_clusters ? 256 : sym256 >= 24 ? 128 : 64;
  }
  const int64_t bm = 128 * cg, tm = (m + bm - 1) / bm, tn = (n + bn - 1) / bn;
  const int64_t per_sym = tm * (tm + 1) / 2 * (bm / bns), per_step = batch * (2 * per_sym + tm * tn);
  if (per_step > kMaxTiles / std::max(1, steps)) return GEMM_ERR_UNSUPPORTED;
  const int64_t num_counters = 3 * (int64_t)steps * batch * tm;
  const size_t sb = align_up((size_t)batch * ortho_slots(m, n) * sizeof(float), 256);
  // X is held as a pair of fp16 halves for a X, and X, E and F as one half each in the
  // products: that leaves 0.7 to 1.4e-3 of the result's norm for a full-rank matrix and up to
  // 3.1e-3 for one of low rank, beside the 1.7e-3 of a rounding to bf16.  A finer result
  // takes products of pairs, three for one: 2e-6 to 4e-5.  So does one of at most 16 singular
  // values, over which the roundings do not average out (1 x 2: up to 1e-2 from one half).
  // Times of one half / pairs, us: 16 x 64 68 / 78, 16 x 2048 90 / 143, 64 of 16 x 2048 309 / 410.
  const bool pairs = out_dtype != GEMM_BF16 || m <= 16;
  const int64_t halves = pairs ? 2 : 1;   // second halves behind the first ones, as further slices
  const size_t xs = align_up((size_t)(halves * batch * sx) * 2, 256), es_b = align_up((size_t)(halves * batch * se) * 2, 256);
  const size_t ls = pairs ? 0 : xs;   // without pairs one buffer of second halves: a tile reads and writes only its own part
  gemm_status_t s = ensure_ws(plan, 2 * xs + ls + 2 * es_b + sb + (size_t)num_counters * sizeof(int32_t), stream);
  if (s != GEMM_OK) return s;
  char* ws = static_cast<char*>(plan->ws.p);
  __half* X[2] = {reinterpret_cast<__half*>(ws), reinterpret_cast<__half*>(ws + xs)};
  __half* one_lo = reinterpret_cast<__half*>(ws + 2 * xs);
  __half* Xlo[2] = {pairs ? X[0] + batch * sx : one_lo, pairs ? X[1] + batch * sx : one_lo};
  __half* E = reinterpret_cast<__half*>(ws + 2 * xs + ls);
  __half* F = reinterpret_cast<__half*>(ws + 2 * xs + ls + es_b);
  float* sums = reinterpret_cast<float*>(ws + 2 * xs + ls + 2 * es_b);
  int32_t* counters = reinterpret_cast<int32_t*>(ws + 2 * xs + ls + 2 * es_b + sb);
  // Entries of X are at most ~1 and as small as 1 / sqrt(m n), so they are held times 1024,
  // which keeps the second halves' units (2^-24) below 2^-20 of an entry up to m n = 2^26.
  // In pairs E and F are held times 256 for the same reason (entries of 1 / m).
  const float scale = 1024.0f, scale_e = pairs ? 256.0f : 1.0f;
  const int es = dtype_bytes(plan->ab);
  const OrthoInput in{G, m, n, ldg, stride_g, tall ? 1 : 0,
                      aligned16(G) && (ldg * es) % 16 == 0 && (batch == 1 || (stride_g * es) % 16 == 0) ? 1 : 0};
  if (launch_ortho_input(in, plan->ab, batch, sums, (float)eps, scale, X[0], Xlo[0], ldx, sx, counters, num_counters,
                         stream) != cudaSuccess)
    return GEMM_ERR_CUDA;
  if (steps == 0) {
    if (launch_unscale(X[0], Xlo[0], batch, M, N, ldx, sx, tall, 1.0f / scale, D, out_dtype, ldd, stride_d, stream) !=
        cudaSuccess)
      return GEMM_ERR_CUDA;
    return nothing(plan);   // (no product)
  }
  SegParams p;
  std::memset(&p, 0, sizeof(p));
  const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int64_t slices = halves * batch;
  bool ok = encode_3d(&p.tmA, dt, E, m, m, lde, slices, se, TC_BK, 128) &&
            encode_3d(&p.tmB[CHAIN_F], dt, F, m, m, lde, slices, se, TC_BK, 128);
  ok = ok && encode_3d(&p.tmB[CHAIN_EB], dt, E, m, m, lde, slices, se, TC_BK, (uint32_t)(bns / cg));
  for (int i = 0; i < 2; ++i)
    ok = ok && encode_3d(&p.tmB[CHAIN_XK + i], dt, X[i], n, m, ldx, slices, sx, TC_BK, 128) &&
         encode_3d(&p.tmB[CHAIN_XB + i], dt, X[i], n, m, ldx, slices, sx, TC_BK, (uint32_t)(bns / cg)) &&
         encode_3d(&p.tmB[CHAIN_XN + i], dt, X[i], n, m, ldx, slices, sx, 64, 2 * TC_BK);
  if (!ok) return GEMM_ERR_CUDA;
  p.M = m;
  p.N = (int32_t)n;
  p.tiles_m = (int32_t)tm;
  p.tiles_n = (int32_t)tn;
  p.tiles_per_group = (int32_t)per_sym;
  p.num_tiles = (int32_t)(per_step * steps);
  p.idesc = make_idesc(false, 0, false, false, 128 * cg);
  p.batch = (int32_t)batch;
  p.steps = steps;
  p.bns = bns;
  p.bn = bn;
  p.store_t = tall ? 1 : 0;
  p.counters = counters;
  p.pairs = pairs ? 1 : 0;
  for (int i = 0; i < 2; ++i) {
    p.chain.x[i] = X[i];
    p.chain.xlo[i] = Xlo[i];
  }
  p.chain.e = E;
  p.chain.f = F;
  p.chain.ldx = ldx;
  p.chain.stride_x = sx;
  p.chain.lde = lde;
  p.chain.stride_e = se;
  // E = X X' - h I with h = 1 once the singular values have come near one (the last two
  // steps): E is then small and its rounding with it.  With X X' = E + h I,
  //   a X + (b X X' + c (X X')^2) X = (a + b h + c h^2) X + ((b + 2 c h) E + c E^2) X.
  for (int h = 0; h < 2; ++h) {
    p.chain.a[h] = (float)(coeffs[0] + coeffs[1] * h + coeffs[2] * h);
    p.chain.b[h] = (float)(coeffs[1] + 2 * coeffs[2] * h);
  }
  p.chain.c = (float)coeffs[2];
  p.chain.inv_x = 1.0f / scale;
  p.chain.scale_e = scale_e;
  p.chain.inv_e = 1.0f / scale_e;
  p.epi = epilogue_of(nullptr, out_dtype, 1.0, D, ldd);
  if (batch > 1 && (stride_d * dtype_bytes(out_dtype)) % 16 != 0) p.epi.vec_d = 0;
  p.epi.stride_d = stride_d;
  p.epi.read_c = 1;
  p.epi.c_dtype = GEMM_F16;
  p.epi.vec_c = 1;   // the matrices in scratch start on 16 bytes, and so do their rows
  p.err = plan->d_err;
  p.timeout_ns = plan->timeout_ns;
  const int workers = workers_of(plan, cg, batch * std::max(per_sym, tm * tn));
  if (launch_seg(p, SEG_CHAIN, cg, false, workers, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  plan->last = seg_config(cg, p.num_tiles, workers);
  plan->last.bn = bns;
  log_config("orthogonalize", m, n, steps, batch, plan->last);
  return GEMM_OK;
}

}  // extern "C"
