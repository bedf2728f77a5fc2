// layer.h -- launch interface of the kernels around the products: fully connected layers of few
// tiles and the elementwise pass of their gradient, routing, the exchange of rows between tokens
// and experts, clipping by a global norm (internal).
#pragma once

#include "expert.h"

namespace gemmlib {

// ---- fully connected layers (linear_kernel.cu; products of many tiles: seg_kernel.cu) ----
constexpr int SPLIT_SMEM = 112 * 1024;   // of a CTA: two on an SM
struct LinearSplitParams {
  CUtensorMap tmW;           // weights: boxes of 64 k x 128 columns of D, or 64 columns x 64 k
  CUtensorMap tmX;           // rows: boxes of 64 k x box_rows
  int64_t rows, K, epi_n;    // epi_n: columns of D
  int32_t box_rows;          // rows of a tile: 16, 32, 64 or 128
  int32_t stages;            // split_stages(box_rows)
  int32_t vec;               // D, pre and residual can be accessed four entries at a time
  uint32_t idesc;            // instruction descriptor without N
  LinearEpilogue linear;
  EpiParams epi;             // bias and D
  int32_t* err;
  uint64_t timeout_ns;
};
int split_stages(int box_rows);
// splits: CTAs that share a tile's K, 1 .. 8 and at most ceil(K / 64).
cudaError_t launch_linear_split(const LinearSplitParams& p, bool a_mn, int splits, cudaStream_t stream);

// dz = dy act'(pre) (16-bit types, rows of dz padded to whole 16 bytes), and the sums of dz's
// columns over blocks of rows.  No activation: only the sums, of dy.
struct ActGradParams {
  const void *dy, *pre;
  void* dz;
  int64_t M, N, ldy, ldp, ldz;
  int64_t block_rows;
  int32_t act;
  int32_t vec;               // rows of dy and pre can be read 16 bytes at a time
  float* partials;           // blocks x N, or null
};
cudaError_t launch_act_grad(const ActGradParams& p, int dtype, int blocks, cudaStream_t stream);
cudaError_t launch_column_sums(const float* partials, int blocks, int64_t N, float* out, cudaStream_t stream);

// ---- routing (route_kernels.cu) ----
constexpr int kMaxTop = 32;   // experts of one token
struct RouteParams {
  const void* logits;        // tokens x experts, pitch ld
  int64_t ld;
  int32_t dtype;
  int64_t tokens;
  int32_t experts, top, renormalize;
  const uint8_t* mask;       // tokens entries, 0: the token does not count; or null
  // What the forward pass writes and the gradient reads.
  float* weights;            // tokens x top
  int32_t* chosen;           // tokens x top: experts, -1 behind the last one
  int32_t* slots;            // tokens x top: places among the sorted rows, -1 for none
  int32_t *counts, *offsets, *routed;   // experts, experts + 1 and 1 entries
  float* loss;               // or null
  // Of the forward pass.
  int32_t blocks, warps;     // CTAs that choose, and their warps
  int32_t per_warp;          // tokens of a warp
  int32_t* hist;             // blocks x route_pitch: rows of every expert, tokens with any
  float* mass;               // blocks x route_pitch: sums of the probabilities
  // Of the gradient.
  const float* dweights;     // tokens x top, or null
  const float* dloss;        // or null: 1
  float dloss_scale;
  void* dlogits;             // tokens x experts, pitch ldd, logits' type
  int64_t ldd;
};
__host__ __device__ inline int route_pitch(int experts) { return (experts + 4) / 4 * 4; }   // experts + 1, whole 16 bytes
int route_blocks(int64_t tokens, int64_t experts, int sm_count);   // RouteParams::blocks
int route_warps(int64_t experts);                                  // RouteParams::warps
cudaError_t launch_route(const RouteParams& p, cudaStream_t stream);
cudaError_t launch_route_grad(const RouteParams& p, int sm_count, cudaStream_t stream, int* grid);   // grid: CTAs launched

// ---- rows between tokens and experts (exchange_kernels.cu) ----
struct ExchangeParams {
  int64_t tokens, rows, width;   // rows: of the sorted buffer
  int32_t top, dtype;
  const int32_t* slots;      // tokens x top; outside 0 .. rows - 1: no row (and an error but for -1)
  const int32_t* used;       // rows in use (those behind are written as zeros), or null: all
  const float* weights;      // tokens x top, or null: 1
  const void *x, *y, *residual;   // token rows (x: dispatch's input, combine_grad's dout), sorted rows, or null
  int64_t ldx, ldy, ldr;
  void *out, *dweights;      // dispatch, combine_grad: sorted rows; combine: token rows
  int64_t ldo;
  int32_t vec;               // all rows can be read and written 16 bytes at a time
  int32_t parts_shift;       // log2 of the warps that share a token (set by the launch)
  int32_t* err;
};
// grid: CTAs launched.
cudaError_t launch_dispatch(const ExchangeParams& p, int sm_count, cudaStream_t stream, int* grid);
cudaError_t launch_combine(const ExchangeParams& p, int sm_count, cudaStream_t stream, int* grid);
cudaError_t launch_combine_grad(const ExchangeParams& p, int sm_count, cudaStream_t stream, int* grid);

// ---- global norm and clipping (clip_kernels.cu) ----
// A part of the list of tensors, as one launch takes it (by value: a captured launch keeps
// its own, and nothing has to outlive the call).
struct ClipTensors {
  static constexpr int SMALL = 48, LARGE = 1024;
};
struct ClipTensor {
  const void* src;
  void* dst;                 // null: only the norm
  int64_t count;
  int32_t src_type, dst_type;
};
struct ClipPass {
  int64_t chunk;             // entries that a CTA takes at a time (a multiple of 8)
  double* partials;          // one per CTA of every norm launch
  int32_t num_partials;
  int32_t scales;            // some tensor has a place for its scaled values
  float max_norm, eps;
  float* norm;
};
int64_t clip_chunk(int64_t total, int sm_count);
// CTAs of the launch that adds up the squares of tensors [0, count).
int clip_blocks(const ClipTensor* t, int count, int64_t chunk, int sm_count);
cudaError_t launch_clip_norm(const ClipTensor* t, int count, const ClipPass& p, int first_partial, int blocks,
                             cudaStream_t stream);
// Writes the norm (first) and the scaled tensors.
cudaError_t launch_clip_scale(const ClipTensor* t, int count, const ClipPass& p, bool first, int blocks,
                              cudaStream_t stream);

}  // namespace gemmlib
