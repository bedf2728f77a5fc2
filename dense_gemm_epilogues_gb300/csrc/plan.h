// plan.h -- the plan's state and the host helpers that the entry points share (internal).
#pragma once

#include <cstdint>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "kernels.h"

namespace gemmlib {
// Device scratch that grows on demand (ensure_buffer).
struct PlanBuffer {
  void* p = nullptr;
  size_t bytes = 0;
  bool captured = false;   // a captured call holds its address
};
}  // namespace gemmlib

struct gemm_plan {
  int device = 0;
  gemm_dtype_t ab = GEMM_F16;
  gemm_dtype_t c = GEMM_F32;
  int sm_count = 0;
  int32_t* d_err = nullptr;          // device error word
  gemmlib::PlanBuffer ws;            // staged operands, partial sums, the expert layers' intermediates
  // Blocks that a larger one has replaced but captured graphs still use (of sk1_flags: apart,
  // since a launch that gave up leaves its arrival counters other than zero).
  std::vector<gemmlib::PlanBuffer> kept, kept_counters;
  void* stage = nullptr;             // gemm_run_host device buffers
  size_t stage_bytes = 0;
  gemm_kernel_t forced = GEMM_KERNEL_AUTO;
  int pair_clusters = 0;             // co-resident CTA-pair clusters (0: pair kernel unavailable)
  void* sk_ws = nullptr;             // stream-K partial accumulators and flags (per cluster and CTA)
  size_t sk_ws_bytes = 0;
  int32_t sk_epoch = 0;
  // Stream-K of the single-CTA kernel: two fp32 partial slots per CTA, and one arrival
  // counter per tile (zero between launches; each tile's last arriver resets its
  // counter).  The counters have a buffer of their own: the slots' size goes with the
  // tile width, and counters behind them would lie in an earlier launch's partial sums.
  gemmlib::PlanBuffer sk1_ws, sk1_flags;
  gemm_config_t last{};
  uint64_t timeout_ns = 4000000000ull;
  // gemm_run_host's row-panel pipeline: copy-in and copy-out streams and the
  // events that order them with the caller's stream (created on first use).
  cudaStream_t host_in = nullptr, host_out = nullptr;
  cudaEvent_t host_ev[36] = {};
  bool host_pipe = false;
};

namespace gemmlib {

constexpr int64_t kMaxDim = 0x7fffffffLL;   // tile indices and TMA coordinates are 32-bit

// NVTX range around a public entry point (a profiler's timeline shows each call;
// without a tool attached a push or pop costs a predictable branch).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

inline bool is_f16ish(int t) { return t == GEMM_F16 || t == GEMM_BF16; }
inline bool is_float_out(int t) { return t == GEMM_F32 || t == GEMM_F16 || t == GEMM_BF16; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Can TMA describe this operand (16-byte aligned base, 16-byte multiple row pitch)?
inline bool tma_ok(const void* p, int64_t ld, int esize) {
  return aligned16(p) && ((ld * esize) % 16) == 0 && ld * esize < (int64_t(1) << 40);
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// tcgen05 instruction descriptor, kind::f16 with fp32 accumulation:
//   bits 4-5 D format (1 = f32), 7-9 A format, 10-12 B format (0 = f16, 1 = bf16),
//   15 / 16 A / B MN-major, 17-22 N >> 3, 24-28 M >> 4.
inline uint32_t make_idesc(bool bf16, int bn, bool a_mn_major, bool b_mn_major, int bm = TC_BM) {
  const uint32_t f = bf16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(bm >> 4) << 24);
}

struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
    if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

// GEMM_LOG=1: print the configuration of a launch to stderr.
void log_config(const char* entry, int64_t M, int64_t N, int64_t K, int64_t batch, const gemm_config_t& c);

// Grow plan scratch to at least `bytes`, in stream order.  A captured graph keeps the
// addresses of its calls: a block that a captured call uses is never freed before the
// plan, and what a capture has to allocate is ordinary memory, not the graph's.
// zero: a new block starts as zeros.
gemm_status_t ensure_buffer(gemm_plan* plan, PlanBuffer& b, size_t bytes, bool zero,
                            std::vector<PlanBuffer>& kept, cudaStream_t stream);
inline gemm_status_t ensure_ws(gemm_plan* plan, size_t bytes, cudaStream_t stream) {
  return ensure_buffer(plan, plan->ws, bytes, false, plan->kept, stream);
}

// A row-pitched tensor of 16-bit elements (inner elements contiguous, `ld`
// elements between rows of the outer dimension) with a third, outermost
// dimension: `nbatch` problems `bstride` elements apart (one problem when
// nbatch == 1).  128-byte swizzle; out-of-bounds elements read as zero.
bool encode_3d(CUtensorMap* tm, CUtensorMapDataType dt, const void* ptr, uint64_t inner, uint64_t outer,
               uint64_t ld, uint64_t nbatch, uint64_t bstride, uint32_t box_inner, uint32_t box_outer);

// The same for any element type: `inner` contiguous elements, pitches in bytes
// (multiples of 16); two dimensions when nbatch <= 1 and bstride is 0, else three.
bool encode_tiled(CUtensorMap* tm, CUtensorMapDataType dt, const void* ptr, uint64_t inner, uint64_t outer,
                  uint64_t pitch_bytes, uint64_t nbatch, uint64_t bstride_bytes, uint32_t box_inner, uint32_t box_outer,
                  CUtensorMapSwizzle swizzle);

}  // namespace gemmlib
