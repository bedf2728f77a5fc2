// layer_api.cu -- the C entry points of the operators around the products (declared in
// include/gemm.h): argument checks, workspaces and launches.  Host code only.
#include <cmath>
#include <cstring>

#include "layer.h"
#include "plan.h"

using namespace gemmlib;

namespace {

bool is_type(int t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }

// Rows that can be read and written 16 bytes at a time.
bool wide_rows(const void* p, int64_t ld, int es) { return aligned16(p) && (ld * es) % 16 == 0; }

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
  if (top > kMaxTop || rows > kMaxDim || width > kMaxDim || tokens > kMaxDim / top) return GEMM_ERR_UNSUPPORTED;
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

}  // namespace

extern "C" {

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
  if (p.blocks > 1) {
    const size_t hist = align_up((size_t)p.blocks * (size_t)(experts + 1) * sizeof(int32_t), 256);
    s = ensure_ws(plan, hist + (size_t)p.blocks * (size_t)experts * sizeof(float), stream);
    if (s != GEMM_OK) return s;
    p.hist = static_cast<int32_t*>(plan->ws.p);
    p.mass = reinterpret_cast<float*>(static_cast<char*>(plan->ws.p) + hist);
  }
  return launch_route(p, stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

gemm_status_t gemm_route_grad(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ld,
                              const gemm_routing_t* routing, const float* dweights, double dloss_scale,
                              const float* dloss, void* dlogits, int64_t ldd, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_route_grad");
  gemm_status_t s = check_routing(plan, tokens, experts, logits, ld, routing);
  if (s != GEMM_OK) return s;
  if (tokens == 0) return GEMM_OK;
  if (!dlogits || ldd < experts) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  RouteParams p = routing_of(plan, tokens, experts, logits, ld, routing);
  p.dweights = dweights;
  p.dloss = dloss;
  p.dloss_scale = (float)dloss_scale;
  p.dlogits = dlogits;
  p.ldd = ldd;
  return launch_route_grad(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess ? GEMM_OK
                                                                                                     : GEMM_ERR_CUDA;
}

gemm_status_t gemm_dispatch(gemm_plan_t plan, int64_t tokens, int64_t top, int64_t rows, int64_t width, const void* X,
                            int64_t ldx, const int32_t* slots, const int32_t* used, void* D, int64_t ldd,
                            gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_dispatch");
  ExchangeParams p;
  const gemm_status_t s = exchange_of(plan, tokens, top, rows, width, slots, &p);
  if (s != GEMM_OK) return s;
  if (rows == 0 || width == 0) return GEMM_OK;
  if (!D || ldd < width || (tokens > 0 && (!X || ldx < width))) return GEMM_ERR_INVALID_ARG;
  DeviceGuard g(plan->device);
  if (!g.ok) return GEMM_ERR_CUDA;
  const int es = dtype_bytes(plan->ab);
  p.used = used;
  p.x = X;
  p.ldx = ldx;
  p.out = D;
  p.ldo = ldd;
  p.vec = (width * es) % 16 == 0 && wide_rows(X, ldx, es) && wide_rows(D, ldd, es) ? 1 : 0;
  return launch_dispatch(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess ? GEMM_OK
                                                                                                   : GEMM_ERR_CUDA;
}

gemm_status_t gemm_combine(gemm_plan_t plan, int64_t tokens, int64_t top, int64_t rows, int64_t width, const void* Y,
                           int64_t ldy, const int32_t* slots, const float* weights, const void* residual, int64_t ldr,
                           void* D, int64_t ldd, gemm_stream_t stream_) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  NvtxRange range("gemm_combine");
  ExchangeParams p;
  const gemm_status_t s = exchange_of(plan, tokens, top, rows, width, slots, &p);
  if (s != GEMM_OK) return s;
  if (tokens == 0 || width == 0) return GEMM_OK;
  if (!D || ldd < width || (rows > 0 && (!Y || ldy < width)) || (residual && ldr < width)) return GEMM_ERR_INVALID_ARG;
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
  return launch_combine(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess ? GEMM_OK
                                                                                                  : GEMM_ERR_CUDA;
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
  if (rows > 0 && width > 0 && (!Y || ldy < width || !dY || lddy < width || dY == Y)) return GEMM_ERR_INVALID_ARG;
  if (tokens == 0 && (rows == 0 || width == 0)) return GEMM_OK;
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
  return launch_combine_grad(p, plan->sm_count, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess
             ? GEMM_OK
             : GEMM_ERR_CUDA;
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
  gemm_status_t s = ensure_ws(plan, (size_t)parts * 4 * (size_t)plan->sm_count * sizeof(double), stream);
  if (s != GEMM_OK) return s;
  ClipPass p{};
  p.chunk = clip_chunk(total, plan->sm_count);
  p.partials = static_cast<double*>(plan->ws.p);
  p.max_norm = (float)max_norm;
  p.eps = (float)eps;
  p.norm = norm;
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
  return GEMM_OK;
}

}  // extern "C"
