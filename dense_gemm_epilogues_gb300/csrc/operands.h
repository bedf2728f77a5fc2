// operands.h -- host helpers that the entry points of the expert layers and of the operators
// around the products share (internal).
#pragma once

#include <algorithm>
#include <initializer_list>

#include "expert.h"
#include "plan.h"

namespace gemmlib {

// A 16-bit operand as TMA can read it: itself, or a copy with another pitch in scratch.
struct Operand {
  const void* p;
  int64_t ld, stride;
};

inline bool addressable(const Operand& x, int64_t batch) {
  return tma_ok(x.p, x.ld, 2) && (batch <= 1 || x.stride % 8 == 0);
}

// Scratch bytes of the copy of `batch` rows x cols matrices (0: none needed).
inline size_t repitch_bytes(const Operand& x, int64_t rows, int64_t cols, int64_t batch) {
  return addressable(x, batch) ? 0 : align_up((size_t)(batch * rows * ((cols + 7) / 8 * 8)) * 2, 256);
}

inline gemm_status_t repitch(Operand* x, int64_t rows, int64_t cols, int64_t batch, const int32_t* offsets, char* to,
                      cudaStream_t stream) {
  if (addressable(*x, batch)) return GEMM_OK;
  const int64_t ld = (cols + 7) / 8 * 8;
  if (launch_repitch(x->p, x->ld, x->stride, to, ld, rows * ld, rows, cols, batch, offsets, 2, stream) !=
      cudaSuccess)
    return GEMM_ERR_CUDA;
  *x = Operand{to, ld, batch > 1 ? rows * ld : 0};
  return GEMM_OK;
}

inline int workers_of(const gemm_plan* plan, int cg, int64_t tiles) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(tiles, cg == 2 ? plan->pair_clusters : plan->sm_count));
}

inline CUtensorMapDataType map_type(gemm_dtype_t t) {
  return t == GEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

constexpr int64_t kMaxTiles = int64_t(1) << 28;   // tile numbers are 32-bit

// What gemm_plan_last_config reports for a product on seg_kernel.
inline gemm_config_t seg_config(int cg, int64_t tiles, int workers) {
  gemm_config_t c{};
  c.kernel = cg == 2 ? GEMM_KERNEL_TC_PAIR : GEMM_KERNEL_TC;
  c.bm = c.bn = 128 * cg;
  c.bk = 2 * TC_BK;
  c.stages = 3;
  c.cta_group = c.cluster = cg;
  c.split_k = 1;
  c.raster = 8;
  c.grid = workers * cg;
  c.tiles = (int32_t)tiles;
  return c;
}

// A call that launches nothing.
inline gemm_status_t nothing(gemm_plan* plan) {
  plan->last = gemm_config_t{};
  plan->last.kernel = GEMM_KERNEL_NONE;
  return GEMM_OK;
}

inline bool too_large(std::initializer_list<int64_t> dims) {
  for (int64_t d : dims)
    if (d > kMaxDim - 512) return true;   // tile edges past a size stay within 32 bits
  return false;
}

}  // namespace gemmlib
