// layer_api.cu -- the C entry points of the operators around the products (declared in
// include/gemm.h): argument checks, workspaces and launches.  Host code only.
#include <cmath>
#include <cstring>

#include "layer.h"
#include "operands.h"

using namespace gemmlib;

namespace {

bool is_type(int t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }

// Rows that can be read and written 16 bytes at a time.
bool wide_rows(const void* p, int64_t ld, int es) { return aligned16(p) && (ld * es) % 16 == 0; }

// What gemm_plan_last_config reports of a call without a product, and its log line.
gemm_status_t launched(gemm_plan* plan, cudaError_t e, const char* entry, int64_t M, int64_t N, int64_t K, int64_t batch,
                       int grid) {
  if (e != cudaSuccess) return GEMM_ERR_CUDA;
  gemm_config_t c{};
  c.kernel = GEMM_KERNEL_SIMT;
  c.cta_group = c.cluster = c.split_k = 1;
  c.grid = grid;
  plan->last = c;
  log_config(entry, M, N, K, batch, c);
  return GEMM_OK;
}

gemm_status_t check_routing(const gemm_plan* plan, int64_t tokens, int64_t experts, const void* logits, int64_t ld,
                            const gemm_routing_t* r) {
  if (!is_type(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (!r || tokens < 0 || experts <= 0 || r->top <= 0 || r->top > experts) return GEMM_ERR_INVALID_ARG;
  if (r->top > kMaxTop || experts > kMaxGroups || tokens > kMaxDim / r->top) return GEMM_ERR_UNSUPPORTED;
  if (!r->counts || !r->offsets || !r->routed) return GEMM_ERR_INVALID_ARG;
  if (tokens > 0 && (!logits || ld < experts || !r->weights || !r->experts)) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

RouteParams routing_of(const gemm_plan* plan, int64_t tokens, int64_t experts, const void* logits, int64_t ld,
                       const gemm_routing_t* r) {
  RouteParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.ld = ld;
  p.dtype = plan->ab;
  p.tokens = tokens;
  p.experts = (int32_t)experts;
  p.top = r->top;
  p.renormalize = r->renormalize != 0 ? 1 : 0;
  p.weights = r->weights;
  p.chosen = r->experts;
  p.slots = r->slots;
  p.counts = r->counts;
  p.offsets = r->offsets;
  p.routed = r->routed;
  p.loss = r->loss;
  return p;
}

// What the exchange's three entry points check alike, and their parameters.
gemm_status_t exchange_of(const gemm_plan* plan, int64_t tokens, int64_t top, int64_t rows, int64_t width,
                          const int32_t* slots, ExchangeParams* p) {
  if (!is_type(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if (tokens < 0 || top <= 0 || rows < 0 || width < 0) return GEMM_ERR_INVALID_ARG;
  if (top > kMaxTop || rows > kMaxDim || width > (int64_t(1) << 30) || tokens > kMaxDim / top) return GEMM_ERR_UNSUPPORTED;
  if (tokens > 0 && !slots) return GEMM_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  p->tokens = tokens;
  p->rows = rows;
  p->width = width;
  p->top = (int32_t)top;
  p->dtype = plan->ab;
  p->slots = slots;
  p->err = plan->d_err;
  return GEMM_OK;
}

// ------------------------------ fully connected layers ------------------------------

gemm_status_t check_linear(const gemm_plan* plan, gemm_layout_t lb, int64_t M, int64_t N, int64_t K) {
  if (!is_f16ish(plan->ab)) return GEMM_ERR_UNSUPPORTED;
  if ((lb != GEMM_OP_N && lb != GEMM_OP_T) || M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (too_large({M, N, K})) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// How linear_split_kernel runs a product: rows of a tile, and CTAs that share a tile's K (0: the
// product runs on seg_kernel).  A CTA takes 1024 k, or less down to 128 as long as four share a
// tile, and two CTAs have room on an SM.  Up to 32 rows always: the weights' stream bounds the
// product.  Beyond, tiles of 64 rows wherever they are few enough to be split; a tile's partial
// sums cost a CTA 1 us per 16 KB, so tiles of 128 rows only where K is long beside their number.
// Measured with a residual, tiles of 64 rows / of 128 / seg_kernel, us: 128 rows, 1024 to 1024
// 6.5 / 7.9 / 8.8, 4096 to 11008 29.9 / 24.7 / 27.0, 512 to 4096 7.4 / 8.9 / 7.8; 200 rows, 2048 to
// 2048 10.0 / 12.0 / 12.2; 256 rows, 4096 to 4096 17.5 / 18.5 / 20.2; 512 rows, 11008 to 1024 20.3
// / 24.0 / 43.7; 1000 rows, 2048 to 1024 12.3 / 13.8 / 12.9, 1000 to 2048 14.9 / 15.1 / 11.2.
// Fewer rows, split / seg_kernel: 1 row, 4096 to 4096 9.5 / 16.1, 1024 to 20000 (not split) 10.8
// / 13.6; 64 rows, 4096 to 20000 (not split) 33.5 / 42, 4096 to 4096 12.9 / 17.2.
struct SplitShape {
  int box_rows, splits;
};
SplitShape split_shape(int64_t M, int64_t N, int64_t K, int sm_count) {
  const int64_t num_kb = (K + TC_BK - 1) / TC_BK, cols = (N + 127) / 128;
  if (num_kb == 0 || cols > 65535) return {0, 0};
  const int64_t want = std::max<int64_t>({1, num_kb / 16, std::min<int64_t>(4, num_kb / 2)});
  auto splits = [&](int64_t tiles) {
    return (int)std::min<int64_t>({8, want, std::max<int64_t>(1, 2 * (int64_t)sm_count / tiles)});
  };
  const int box = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  const int64_t tiles = cols * ((M + box - 1) / box), tiles128 = cols * ((M + 127) / 128);
  if (M <= 32 || splits(tiles) >= 2 || (M <= 64 && tiles <= 4 * num_kb)) return {box, splits(tiles)};
  if (splits(tiles128) >= 2 && 2 * tiles128 <= 3 * num_kb) return {128, splits(tiles128)};
  return {0, 0};
}

// D = act(x W + bias) + residual: x M x K row-major, W K x N (w_mn: N contiguous, else K);
// TMA can address both.
gemm_status_t linear_product(gemm_plan* plan, int64_t M, int64_t N, int64_t K, const Operand& x, const Operand& w,
                             bool w_mn, const EpiParams& epi, const LinearEpilogue& lin, const char* entry,
                             cudaStream_t stream) {
  const CUtensorMapDataType dt = map_type(plan->ab);
  const SplitShape shape = split_shape(M, N, K, plan->sm_count);
  const int box = shape.box_rows, splits = shape.splits;
  if (splits > 0) {
    LinearSplitParams p;
    std::memset(&p, 0, sizeof(p));
    const bool ok = (w_mn ? encode_3d(&p.tmW, dt, w.p, N, K, w.ld, 1, 0, 64, TC_BK)
                          : encode_3d(&p.tmW, dt, w.p, K, N, w.ld, 1, 0, TC_BK, 128)) &&
                    encode_3d(&p.tmX, dt, x.p, K, M, x.ld, 1, 0, TC_BK, (uint32_t)box);
    if (!ok) return GEMM_ERR_CUDA;
    p.rows = M;
    p.K = K;
    p.epi_n = N;
    p.box_rows = box;
    p.stages = split_stages(box);
    auto by_four = [&](const void* q, int64_t ld) {
      return reinterpret_cast<uintptr_t>(q) % (4 * dtype_bytes(epi.d_dtype)) == 0 && ld % 4 == 0;
    };
    p.vec = by_four(epi.D, epi.ldd) && (!lin.pre || by_four(lin.pre, lin.ldp)) &&
                    (!lin.residual || by_four(lin.residual, lin.ldr))
                ? 1
                : 0;
    p.idesc = make_idesc(plan->ab == GEMM_BF16, 0, w_mn, false, 128);
    p.linear = lin;
    p.epi = epi;
    p.err = plan->d_err;
    p.timeout_ns = plan->timeout_ns;
    if (launch_linear_split(p, w_mn, splits, stream) != cudaSuccess) return GEMM_ERR_CUDA;
    const int64_t tiles = (N + 127) / 128 * ((M + box - 1) / box);
    gemm_config_t c = seg_config(1, tiles, (int)tiles * splits);
    c.bn = box;
    c.bk = TC_BK;
    c.stages = p.stages;
    c.split_k = splits;
    c.cluster = splits;
    plan->last = c;
    log_config(entry, M, N, K, 1, plan->last);
    return GEMM_OK;
  }
  SegParams p;
  std::memset(&p, 0, sizeof(p));
  // Single CTAs (128 x 128) or CTA pairs (256 x 256) by the times that both take, in us: single ones
  // share the operands' supply, so part of a wave costs its part; a pair's tile costs 0.33 per 64 k
  // like a single one's, but its epilogue and first loads more, and its waves are whole.  Measured,
  // single / pairs (with GELU and residual): 4096 rows, 1024 to 1024 15.7 / 16.9; 1500 rows, 1024 to
  // 4096 20.3 / 24.4; 1000 rows, 1000 to 2048 11.0 / 15.6, 2048 to 4096 21.1 / 21.2; 2000 rows, 2000 to
  // 2000 23.9 / 22.1; 512 rows, 4096 to 11008 50.7 / 51.3; 1929 rows, 10288 to 4184 208 / 125; 200
  // rows, 256 to 12000 11.1 / 11.6.  The estimate takes the faster side of all these.
  const int64_t tiles256 = (N + 255) / 256 * ((M + 255) / 256), tiles128 = (N + 127) / 128 * ((M + 127) / 128);
  int cg = 1;
  if (plan->pair_clusters > 0 && M >= 128) {
    const double per_tile = 0.33 * (double)((K + TC_BK - 1) / TC_BK);
    const double single = 4.5 + std::max(1.0, (double)tiles128 / plan->sm_count) * (per_tile + 0.9);
    const double pairs = 9.0 + (double)((tiles256 + plan->pair_clusters - 1) / plan->pair_clusters) * (per_tile + 1.7);
    cg = pairs < single ? 2 : 1;
  }
  const int64_t tiles = cg == 2 ? tiles256 : tiles128;
  if (tiles > kMaxTiles) return GEMM_ERR_UNSUPPORTED;
  if (K > 0) {
    bool ok = w_mn ? encode_3d(&p.tmA, dt, w.p, N, K, w.ld, 1, 0, 64, 2 * TC_BK)
                   : encode_3d(&p.tmA, dt, w.p, K, N, w.ld, 1, 0, TC_BK, 128);
    // The boxes that the tiles' rows take: all tiles but the last have equally many.
    const int64_t n_tiles = (M + 128 * cg - 1) / (128 * cg), per = ((M + n_tiles - 1) / n_tiles + 15) / 16 * 16;
    for (const int64_t rows : {per, (M - (n_tiles - 1) * per + 15) / 16 * 16}) {
      int b = 0;
      while (b < 4 && (64 >> b) >= rows / cg) ++b;
      ok = ok && encode_3d(&p.tmB[b], dt, x.p, K, M, x.ld, 1, 0, TC_BK, 128u >> b);
    }
    if (!ok) return GEMM_ERR_CUDA;
  }
  p.groups = Groups{nullptr, 1, (int32_t)M, plan->d_err};
  p.M = N;
  p.K = (int32_t)K;
  p.tiles_m = (int32_t)((N + 128 * cg - 1) / (128 * cg));
  p.idesc = make_idesc(plan->ab == GEMM_BF16, 0, w_mn, false, 128 * cg);
  p.epi = epi;
  p.linear = lin;
  p.err = plan->d_err;
  p.timeout_ns = plan->timeout_ns;
  const int workers = workers_of(plan, cg, tiles);
  if (launch_seg(p, SEG_LINEAR, cg, w_mn, workers, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  plan->last = seg_config(cg, tiles, workers);
  log_config(entry, M, N, K, 1, plan->last);
  return GEMM_OK;
}

EpiParams plain_epilogue(void* D, int64_t ldd, gemm_dtype_t type) {
  EpiParams e{};
  e.alpha = 1.0f;
  e.D = D;
  e.ldd = ldd;
  e.d_dtype = type;
  e.bias_dtype = GEMM_F32;
  e.out_scale = 1.0f;
  e.vec_d = wide_rows(D, ldd, dtype_bytes(type)) ? 1 : 0;
  return e;
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_linear(gemm_plan_t plan, gemm_layout_t lb, int64_t M, int64_t N, int64_t K, const void* A,
                              int64_t lda, const void* B, int64_t ldb, void* D, int64_t ldd, const gemm_linear_t* epi,
                              gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_linear");
  gemm_status_t s = check_linear(plan, lb, M, N, K);
  if (s != GEMM_OK) return s;
  const gemm_dtype_t out = epi ? epi->out_dtype : plan->ab;
  if (!is_type(out) || (epi && (epi->act < GEMM_LINEAR_NONE || epi->act > GEMM_LINEAR_SILU))) return GEMM_ERR_INVALID_ARG;
  if (epi && epi->bias && !is_type(epi->bias_dtype)) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return nothing(plan);
  if (!D || ldd < N) return GEMM_ERR_INVALID_ARG;
  if (epi && ((epi->residual && epi->ld_residual < N) || (epi->pre && epi->ld_pre < N))) return GEMM_ERR_INVALID_ARG;
  if (K > 0 && (!A || !B || lda < K || ldb < (lb == GEMM_OP_N ? K : N) || D == A || D == B)) return GEMM_ERR_INVALID_ARG;
  if (epi && epi->pre && (epi->pre == D || epi->pre == epi->residual || (K > 0 && (epi->pre == A || epi->pre == B))))
    return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  EpiParams e = plain_epilogue(D, ldd, out);
  LinearEpilogue lin{};
  if (epi) {
    if (epi->bias) {
      e.bias_mode = GEMM_BIAS_COL;
      e.bias = epi->bias;
      e.bias_dtype = epi->bias_dtype;
    }
    lin.residual = epi->residual;
    lin.ldr = epi->ld_residual;
    lin.pre = epi->pre;
    lin.ldp = epi->ld_pre;
    lin.act = epi->act;
    lin.vec_r = epi->residual && out != GEMM_F32 && wide_rows(epi->residual, epi->ld_residual, 2) ? 1 : 0;
    lin.vec_p = epi->pre && wide_rows(epi->pre, epi->ld_pre, dtype_bytes(out)) ? 1 : 0;
  }
  Operand x{A, lda, 0}, w{B, ldb, 0};
  const bool w_mn = lb == GEMM_OP_T;
  if (K > 0) {   // operands that TMA cannot address are copied to a pitch it can
    const int64_t wrows = w_mn ? K : N, wcols = w_mn ? N : K;
    const size_t xb = repitch_bytes(x, M, K, 1), wb = repitch_bytes(w, wrows, wcols, 1);
    if (xb + wb > 0) {
      s = ensure_ws(plan, xb + wb, stream);
      char* ws = static_cast<char*>(plan->ws.p);
      if (s == GEMM_OK) s = repitch(&x, M, K, 1, nullptr, ws, stream);
      if (s == GEMM_OK) s = repitch(&w, wrows, wcols, 1, nullptr, ws + xb, stream);
      if (s != GEMM_OK) return s;
    }
  }
  return linear_product(plan, M, N, K, x, w, w_mn, e, lin, "linear", stream);
}

gemm_status_t gemm_run_linear_grad(gemm_plan_t plan, gemm_layout_t lb, int64_t M, int64_t N, int64_t K, const void* dY,
                                   int64_t lddy, const void* pre, int64_t ldp, gemm_linear_act_t act, const void* A,
                                   int64_t lda, const void* B, int64_t ldb, void* dA, int64_t ldda, void* dB,
                                   int64_t lddb, gemm_dtype_t db_dtype, float* dbias, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_run_linear_grad");
  gemm_status_t s = check_linear(plan, lb, M, N, K);
  if (s != GEMM_OK) return s;
  if (act < GEMM_LINEAR_NONE || act > GEMM_LINEAR_SILU || (dB && !is_type(db_dtype))) return GEMM_ERR_INVALID_ARG;
  const int64_t wld = lb == GEMM_OP_N ? K : N;
  if (M > 0 && N > 0 && (!dY || lddy < N || (act != GEMM_LINEAR_NONE && (!pre || ldp < N)))) return GEMM_ERR_INVALID_ARG;
  if (dA && (ldda < K || (N > 0 && K > 0 && (!B || ldb < wld)))) return GEMM_ERR_INVALID_ARG;
  if (dB && (lddb < wld || (M > 0 && K > 0 && (!A || lda < K)))) return GEMM_ERR_INVALID_ARG;
  const bool want_a = dA && M > 0 && K > 0, want_b = dB && N > 0 && K > 0, want_bias = dbias && N > 0;
  if (!want_a && !want_b && !want_bias) return nothing(plan);
  auto is_input = [&](const void* p) { return p == dY || p == A || p == B || (act != GEMM_LINEAR_NONE && p == pre); };
  if (M > 0 && N > 0 && ((want_a && is_input(dA)) || (want_b && is_input(dB)) || (want_bias && is_input(dbias))))
    return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const bool w_mn = lb == GEMM_OP_T, acts = act != GEMM_LINEAR_NONE && M > 0 && N > 0;
  Operand dy{dY, lddy, 0}, x{A, lda, 0}, w{B, ldb, 0};
  const int64_t wrows = w_mn ? K : N, wcols = w_mn ? N : K;
  // dz (or dy at a pitch that TMA can address), x and w where they need a copy, partial sums.
  const int64_t ldz = (N + 7) / 8 * 8;
  const size_t zb = M == 0 || N == 0 ? 0 : acts ? align_up((size_t)(M * ldz) * 2, 256) : repitch_bytes(dy, M, N, 1);
  const size_t xb = want_b && M > 0 ? repitch_bytes(x, M, K, 1) : 0;
  const size_t wb = want_a && N > 0 ? repitch_bytes(w, wrows, wcols, 1) : 0;
  // Blocks of rows: CTAs for four per SM, at least 32 rows each.  One block (up to 64 rows) writes
  // the bias's gradient itself, one launch less: blocks of 32 / one, us: 64 x 11008 5.3 / 3.7, 128 x
  // 4096 5.4 / 5.7, 256 x 1024 3.7 / 10.1.
  const int64_t strips = (N + 255) / 256;
  const int64_t want = std::max<int64_t>(1, 4 * (int64_t)plan->sm_count / std::max<int64_t>(1, strips));
  const int64_t block_rows = M <= 64 ? std::max<int64_t>(M, 1) : std::max<int64_t>(32, (M + want - 1) / want);
  const int blocks = (int)((M + block_rows - 1) / block_rows);
  const size_t pb = want_bias && blocks > 1 ? (size_t)blocks * (size_t)N * sizeof(float) : 0;
  if (zb + xb + wb + pb > 0) {
    s = ensure_ws(plan, zb + xb + wb + pb, stream);
    if (s != GEMM_OK) return s;
  }
  char* ws = static_cast<char*>(plan->ws.p);
  float* partials = !want_bias ? nullptr : blocks == 1 ? dbias : reinterpret_cast<float*>(ws + zb + xb + wb);
  if (M > 0 && N > 0 && (acts || want_bias)) {
    ActGradParams p{};
    p.dy = dY;
    p.pre = pre;
    p.dz = acts ? ws : nullptr;
    p.M = M;
    p.N = N;
    p.ldy = lddy;
    p.ldp = ldp;
    p.ldz = ldz;
    p.block_rows = block_rows;
    p.act = act;
    p.vec = wide_rows(dY, lddy, 2) && (!acts || wide_rows(pre, ldp, 2)) ? 1 : 0;
    p.partials = partials;
    if (launch_act_grad(p, plan->ab, blocks, stream) != cudaSuccess) return GEMM_ERR_CUDA;
  }
  if (want_bias && blocks != 1 && launch_column_sums(partials, blocks, N, dbias, stream) != cudaSuccess)
    return GEMM_ERR_CUDA;
  if (acts) dy = Operand{ws, ldz, 0};
  else if (zb > 0) s = repitch(&dy, M, N, 1, nullptr, ws, stream);
  if (s == GEMM_OK && xb > 0) s = repitch(&x, M, K, 1, nullptr, ws + zb, stream);
  if (s == GEMM_OK && wb > 0) s = repitch(&w, wrows, wcols, 1, nullptr, ws + zb + xb, stream);
  if (s != GEMM_OK) return s;
  if (!want_a && !want_b)   // (the products report themselves)
    return launched(plan, cudaSuccess, "linear_grad", M, N, K, 1, (int)strips * std::max(1, blocks));
  if (want_a) {   // dA = dz W': W' is N x K, N contiguous where W's K is
    s = linear_product(plan, M, K, N, dy, w, !w_mn, plain_epilogue(dA, ldda, plan->ab), LinearEpilogue{}, "linear_grad",
                       stream);
    if (s != GEMM_OK) return s;
  }
  if (want_b) {   // dB = x' dz, or its transpose dz' x
    gemm_epilogue_t e{};
    e.out_dtype = db_dtype;
    const gemm_kernel_t forced = plan->forced;
    plan->forced = GEMM_KERNEL_AUTO;
    s = w_mn ? gemm_run(plan, GEMM_OP_N, GEMM_OP_T, K, N, M, 1.0, x.p, std::max(x.ld, K), dy.p, std::max(dy.ld, N), 0.0,
                        nullptr, 0, dB, lddb, &e, stream_)
             : gemm_run(plan, GEMM_OP_N, GEMM_OP_T, N, K, M, 1.0, dy.p, std::max(dy.ld, N), x.p, std::max(x.ld, K), 0.0,
                        nullptr, 0, dB, lddb, &e, stream_);
    plan->forced = forced;
  }
  return s;
}

gemm_status_t gemm_route(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ld,
                         const uint8_t* mask, const gemm_routing_t* routing, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_route");
  gemm_status_t s = check_routing(plan, tokens, experts, logits, ld, routing);
  if (s != GEMM_OK) return s;
  if (tokens > 0 && !routing->slots) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  RouteParams p = routing_of(plan, tokens, experts, logits, ld, routing);
  p.mask = mask;
  p.blocks = route_blocks(tokens, experts, plan->sm_count);
  p.warps = route_warps(experts);
  p.per_warp = (int32_t)((tokens + (int64_t)p.blocks * p.warps - 1) / ((int64_t)p.blocks * p.warps));
  if (p.blocks > 1) {
    const size_t hist = align_up((size_t)p.blocks * (size_t)route_pitch((int)experts) * sizeof(int32_t), 256);
    s = ensure_ws(plan, 2 * hist, stream);
    if (s != GEMM_OK) return s;
    p.hist = static_cast<int32_t*>(plan->ws.p);
    p.mass = reinterpret_cast<float*>(static_cast<char*>(plan->ws.p) + hist);
  }
  return launched(plan, launch_route(p, stream), "route", tokens, experts, p.top, 1, p.blocks);
}

gemm_status_t gemm_route_grad(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ld,
                              const gemm_routing_t* routing, const float* dweights, double dloss_scale,
                              const float* dloss, void* dlogits, int64_t ldd, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_route_grad");
  gemm_status_t s = check_routing(plan, tokens, experts, logits, ld, routing);
  if (s != GEMM_OK) return s;
  if (tokens == 0) return nothing(plan);
  if (!dlogits || ldd < experts) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  RouteParams p = routing_of(plan, tokens, experts, logits, ld, routing);
  p.dweights = dweights;
  p.dloss = dloss;
  p.dloss_scale = (float)dloss_scale;
  p.dlogits = dlogits;
  p.ldd = ldd;
  int grid = 0;
  const cudaError_t e = launch_route_grad(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_), &grid);
  return launched(plan, e, "route_grad", tokens, experts, p.top, 1, grid);
}

gemm_status_t gemm_dispatch(gemm_plan_t plan, int64_t tokens, int64_t top, int64_t rows, int64_t width, const void* X,
                            int64_t ldx, const int32_t* slots, const int32_t* used, void* D, int64_t ldd,
                            gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_dispatch");
  ExchangeParams p;
  const gemm_status_t s = exchange_of(plan, tokens, top, rows, width, slots, &p);
  if (s != GEMM_OK) return s;
  if (rows == 0 || width == 0) return nothing(plan);
  if (!D || ldd < width || (tokens > 0 && (!X || ldx < width || D == X))) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const int es = dtype_bytes(plan->ab);
  p.used = used;
  p.x = X;
  p.ldx = ldx;
  p.out = D;
  p.ldo = ldd;
  p.vec = (width * es) % 16 == 0 && wide_rows(X, ldx, es) && wide_rows(D, ldd, es) ? 1 : 0;
  int grid = 0;
  const cudaError_t e = launch_dispatch(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_), &grid);
  return launched(plan, e, "dispatch", tokens, width, top, 1, grid);
}

gemm_status_t gemm_combine(gemm_plan_t plan, int64_t tokens, int64_t top, int64_t rows, int64_t width, const void* Y,
                           int64_t ldy, const int32_t* slots, const float* weights, const void* residual, int64_t ldr,
                           void* D, int64_t ldd, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_combine");
  ExchangeParams p;
  const gemm_status_t s = exchange_of(plan, tokens, top, rows, width, slots, &p);
  if (s != GEMM_OK) return s;
  if (tokens == 0 || width == 0) return nothing(plan);
  if (!D || ldd < width || (rows > 0 && (!Y || ldy < width || D == Y)) || (residual && ldr < width))
    return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const int es = dtype_bytes(plan->ab);
  p.weights = weights;
  p.y = Y;
  p.ldy = ldy;
  p.residual = residual;
  p.ldr = ldr;
  p.out = D;
  p.ldo = ldd;
  p.vec = (width * es) % 16 == 0 && wide_rows(Y, ldy, es) && wide_rows(D, ldd, es) &&
                  (!residual || wide_rows(residual, ldr, es))
              ? 1
              : 0;
  int grid = 0;
  const cudaError_t e = launch_combine(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_), &grid);
  return launched(plan, e, "combine", tokens, width, top, 1, grid);
}

gemm_status_t gemm_combine_grad(gemm_plan_t plan, int64_t tokens, int64_t top, int64_t rows, int64_t width,
                                const void* dout, int64_t ldo, const void* Y, int64_t ldy, const int32_t* slots,
                                const int32_t* used, const float* weights, void* dY, int64_t lddy, float* dweights,
                                gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_combine_grad");
  ExchangeParams p;
  const gemm_status_t s = exchange_of(plan, tokens, top, rows, width, slots, &p);
  if (s != GEMM_OK) return s;
  if (tokens > 0 && (!dweights || (width > 0 && (!dout || ldo < width)))) return GEMM_ERR_INVALID_ARG;
  if (rows > 0 && width > 0 && (!Y || ldy < width || !dY || lddy < width || dY == Y || (tokens > 0 && dY == dout)))
    return GEMM_ERR_INVALID_ARG;
  if (tokens == 0 && (rows == 0 || width == 0)) return nothing(plan);
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const int es = dtype_bytes(plan->ab);
  p.used = used;
  p.weights = weights;
  p.x = dout;
  p.ldx = ldo;
  p.y = Y;
  p.ldy = ldy;
  p.out = dY;
  p.ldo = lddy;
  p.dweights = dweights;
  p.vec = (width * es) % 16 == 0 && wide_rows(dout, ldo, es) && wide_rows(Y, ldy, es) && wide_rows(dY, lddy, es) ? 1 : 0;
  int grid = 0;
  const cudaError_t e = launch_combine_grad(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_), &grid);
  return launched(plan, e, "combine_grad", tokens, width, top, 1, grid);
}

gemm_status_t gemm_clip_norm(gemm_plan_t plan, int64_t count, const gemm_tensor_t* tensors, double max_norm, double eps,
                             float* norm, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_clip_norm");
  if (count < 0 || (count > 0 && !tensors) || !norm) return GEMM_ERR_INVALID_ARG;
  if (!(max_norm >= 0.0) || !(eps >= 0.0) || !std::isfinite(eps)) return GEMM_ERR_INVALID_ARG;
  if (count > (int64_t(1) << 20)) return GEMM_ERR_UNSUPPORTED;
  int64_t total = 0;
  bool scales = false;
  for (int64_t i = 0; i < count; ++i) {
    const gemm_tensor_t& t = tensors[i];
    if (t.count < 0 || t.count > (int64_t(1) << 40) || !is_type(t.src_type)) return GEMM_ERR_INVALID_ARG;
    if (t.count > 0 && (!t.src || reinterpret_cast<uintptr_t>(t.src) % dtype_bytes(t.src_type) != 0))
      return GEMM_ERR_INVALID_ARG;
    if (t.dst && (!is_type(t.dst_type) || reinterpret_cast<uintptr_t>(t.dst) % dtype_bytes(t.dst_type) != 0 ||
                  (t.dst == t.src && t.dst_type != t.src_type)))
      return GEMM_ERR_INVALID_ARG;
    total += t.count;
    scales = scales || t.dst != nullptr;
  }
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  constexpr int64_t PART = ClipTensors::LARGE;
  const int64_t parts = std::max<int64_t>(1, (count + PART - 1) / PART);
  gemm_status_t s = ensure_ws(plan, (size_t)parts * 2 * (size_t)plan->sm_count * sizeof(double), stream);
  if (s != GEMM_OK) return s;
  ClipPass p{};
  p.chunk = clip_chunk(total, plan->sm_count);
  p.partials = static_cast<double*>(plan->ws.p);
  p.max_norm = (float)max_norm;
  p.eps = (float)eps;
  p.norm = norm;
  p.scales = scales ? 1 : 0;
  ClipTensor part[PART];
  auto fill = [&](int64_t i) {
    const int n = (int)std::min<int64_t>(PART, count - i * PART);
    for (int k = 0; k < n; ++k) {
      const gemm_tensor_t& t = tensors[i * PART + k];
      part[k] = ClipTensor{t.src, t.dst, t.count, t.src_type, t.dst ? t.dst_type : GEMM_F32};
    }
    return n;
  };
  for (int64_t i = 0; i < parts; ++i) {
    const int n = fill(i), blocks = clip_blocks(part, n, p.chunk, plan->sm_count);
    if (launch_clip_norm(part, n, p, p.num_partials, blocks, stream) != cudaSuccess) return GEMM_ERR_CUDA;
    p.num_partials += blocks;
  }
  for (int64_t i = 0; i < parts && (scales || i == 0); ++i) {
    const int64_t at = parts - 1 - i;   // (the last tensors first)
    const int n = parts > 1 ? fill(at) : (int)count;
    if (launch_clip_scale(part, n, p, i == 0, scales ? clip_blocks(part, n, p.chunk, plan->sm_count) : 1, stream) !=
        cudaSuccess)
      return GEMM_ERR_CUDA;
  }
  return launched(plan, cudaSuccess, "clip_norm", total, 1, 1, count, p.num_partials);
}

}  // extern "C"
