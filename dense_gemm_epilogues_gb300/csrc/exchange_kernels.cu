// exchange_kernels.cu -- rows between tokens and experts:
//     dispatch      out[slot(t, j)] = x[t];  rows behind the last used one are zero
//     combine       out[t] = residual[t] + sum_j w(t, j) y[slot(t, j)]
//     combine_grad  out[slot(t, j)] = w(t, j) x[t],  dweights(t, j) = <x[t], y[slot(t, j)]>
// (dispatch's own gradient is combine without weights and residual.)  All three go by
// tokens: a token's row is read or written once and its `top` sorted rows lie anywhere, each
// a long run of bytes; so memory moves every byte once (combine_grad reads a token's row again
// from the caches for every four choices beyond the first four), no atomics decide an order, and
// the sums over a token's rows and over a row's entries have one order.
//
// Bound by memory.  A warp takes a token -- of few tokens with long rows, a part of one, up to
// eight warps of a CTA together -- with its slots and weights in its lanes, and goes along the
// row in pieces of 16 bytes per lane, several pieces and rows under way.  16384 tokens, top 2,
// width 2048, bf16: dispatch and combine 68 us, 5.9 TB/s of what they have to move (with half the
// loads under way 93); 8191 tokens, top 4, width 4096: combine_grad and dispatch's gradient 143
// us, 6.6 TB/s.
//
// A slot outside the sorted buffer is no row; one that is not -1 either is reported through
// the error word.
#include "layer.h"

namespace gemmlib {
namespace {

constexpr int THREADS = 256;

// A piece of a row: 16 bytes as they lie in memory (half the registers of their values, so
// that more are under way), or a single entry where rows are not aligned.
template <int DT, bool WIDE>
struct Piece {
  static constexpr int N = !WIDE ? 1 : DT == GEMM_F32 ? 4 : 8;
  uint32_t w[WIDE ? 4 : 1];

  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (!WIDE) {
      w[0] = __float_as_uint(load_as_float(p, DT, i));
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (16 / N));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    if constexpr (!WIDE) store_float_as(p, DT, i, __uint_as_float(w[0]));
    else *reinterpret_cast<uint4*>(static_cast<char*>(p) + i * (16 / N)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int h = 0; h < (WIDE ? 4 : 1); ++h) w[h] = 0u;
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
    if constexpr (!WIDE || DT == GEMM_F32) {
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = __uint_as_float(w[k]);
    } else {
#pragma unroll
      for (int h = 0; h < N / 2; ++h) unpack2<DT>(w[h], x[2 * h], x[2 * h + 1]);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
    if constexpr (!WIDE || DT == GEMM_F32) {
#pragma unroll
      for (int k = 0; k < N; ++k) w[k] = __float_as_uint(x[k]);
    } else {
#pragma unroll
      for (int h = 0; h < N / 2; ++h) w[h] = pack2<DT>(x[2 * h], x[2 * h + 1]);
    }
  }
};

constexpr int WARPS = THREADS / 32;

// What warp `index` works on: a token and its part of the row, pieces first, first + stride, ...
struct Part {
  int64_t token;
  int first, stride;
};
__device__ __forceinline__ Part part_of(const ExchangeParams& p, int64_t index) {
  const int lane = threadIdx.x & 31;
  return Part{index >> p.parts_shift, (int)(index & ((1 << p.parts_shift) - 1)) * 32 + lane, 32 << p.parts_shift};
}

// Lane j: the row of the token's j-th choice, -1 for none.
__device__ __forceinline__ int row_of(const ExchangeParams& p, int64_t t) {
  const int lane = threadIdx.x & 31;
  if (lane >= p.top) return -1;
  const int s = p.slots[t * p.top + lane];
  if (s >= 0 && s < p.rows) return s;
  if (s != -1) atomicCAS(p.err, 0, (int32_t)GEMM_ERR_INVALID_ARG);
  return -1;
}

// Rows from the last used one on, as zeros: all warps share them.
template <int DT, bool WIDE>
__device__ __forceinline__ void clear_rest(const ExchangeParams& p) {
  if (p.used == nullptr) return;
  using P = Piece<DT, WIDE>;
  const int per = (int)(p.width / P::N);
  P z;
  z.clear();
  const int64_t first = min(p.rows, max((int64_t)0, (int64_t)*p.used));
  for (int64_t r = first + (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); r < p.rows; r += (int64_t)gridDim.x * WARPS)
    for (int v = (int)threadIdx.x & 31; v < per; v += 32) z.store(p.out, r * p.ldo + (int64_t)v * P::N);
}

template <int DT, bool WIDE>
__global__ void __launch_bounds__(THREADS) dispatch_kernel(const __grid_constant__ ExchangeParams p) {
  using P = Piece<DT, WIDE>;
  constexpr int U = 4;   // pieces under way
  pdl_launch_dependents();
  pdl_wait();
  const int per = (int)(p.width / P::N);
  const int64_t warps = (int64_t)gridDim.x * WARPS;
  for (int64_t i = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); i >> p.parts_shift < p.tokens; i += warps) {
    const Part a = part_of(p, i);
    const int mine = row_of(p, a.token);
    const int64_t at = a.token * p.ldx;
    for (int v0 = a.first; v0 - (int)(threadIdx.x & 31) < per; v0 += U * a.stride) {
      P x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v0 + u * a.stride < per) x[u].load(p.x, at + (int64_t)(v0 + u * a.stride) * P::N);
      for (int j = 0; j < p.top; ++j) {
        const int r = __shfl_sync(0xffffffffu, mine, j);
        if (r < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * a.stride < per) x[u].store(p.out, r * p.ldo + (int64_t)(v0 + u * a.stride) * P::N);
      }
    }
  }
  clear_rest<DT, WIDE>(p);
}

// Eight loads of sorted rows per lane under way, and as many of the residual as pieces: all
// ROWS rows of 8 / ROWS pieces.  ROWS is the least of 2, 4 and 8 that holds top, or 8: 16384 tokens,
// top 2, 2048 wide 41, 44 and 59 us with ROWS of 2, 4 and 8.
template <int DT, bool WIDE, int ROWS>
__global__ void __launch_bounds__(THREADS) combine_kernel(const __grid_constant__ ExchangeParams p) {
  using P = Piece<DT, WIDE>;
  constexpr int U = 8 / ROWS;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int per = (int)(p.width / P::N);
  const int64_t warps = (int64_t)gridDim.x * WARPS;
  for (int64_t i = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); i >> p.parts_shift < p.tokens; i += warps) {
    const Part a = part_of(p, i);
    const float weight = p.weights != nullptr && lane < p.top ? p.weights[a.token * p.top + lane] : 1.0f;
    const int mine = row_of(p, a.token);
    int r[ROWS];
    float w[ROWS];
    auto choices = [&](int j0) {
#pragma unroll
      for (int q = 0; q < ROWS; ++q) {
        r[q] = __shfl_sync(0xffffffffu, mine, (j0 + q) & 31);
        w[q] = __shfl_sync(0xffffffffu, weight, (j0 + q) & 31);
        if (j0 + q >= p.top) r[q] = -1;
      }
    };
    choices(0);
    for (int v0 = a.first; v0 - lane < per; v0 += U * a.stride) {
      P y[U][ROWS], z[U];
      auto load_rows = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < ROWS; ++q)
            if (r[q] >= 0 && v0 + u * a.stride < per) y[u][q].load(p.y, r[q] * p.ldy + (int64_t)(v0 + u * a.stride) * P::N);
      };
      auto add_rows = [&](int u, float (&sum)[P::N]) {
#pragma unroll
        for (int q = 0; q < ROWS; ++q)
          if (r[q] >= 0) {
            float x[P::N];
            y[u][q].get(x);
#pragma unroll
            for (int k = 0; k < P::N; ++k) sum[k] = fmaf(w[q], x[k], sum[k]);
          }
      };
      if (ROWS == 8 && p.top > 8) choices(0);
      load_rows();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        z[u].clear();
        if (p.residual != nullptr && v0 + u * a.stride < per)
          z[u].load(p.residual, a.token * p.ldr + (int64_t)(v0 + u * a.stride) * P::N);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float sum[P::N];
        z[u].get(sum);
        add_rows(u, sum);
        if constexpr (ROWS == 8) {
          for (int j0 = 8; j0 < p.top; j0 += 8) {
            choices(j0);
            load_rows();
            add_rows(u, sum);
          }
        }
        z[u].set(sum);
        if (v0 + u * a.stride < per) z[u].store(p.out, a.token * p.ldo + (int64_t)(v0 + u * a.stride) * P::N);
      }
    }
  }
}

template <int DT, bool WIDE>
__global__ void __launch_bounds__(THREADS) combine_grad_kernel(const __grid_constant__ ExchangeParams p) {
  using P = Piece<DT, WIDE>;
  constexpr int ROWS = 4;
  __shared__ float parts[WARPS][32];   // a token's parts: the warps' sums
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int per = (int)(p.width / P::N);
  const int64_t warps = (int64_t)gridDim.x * WARPS;
  // (all warps of a CTA take the same turns: those of a token meet at a barrier)
  for (int64_t i0 = (int64_t)blockIdx.x * WARPS; i0 >> p.parts_shift < p.tokens; i0 += warps) {
    const Part a = part_of(p, i0 + warp);
    const bool in = a.token < p.tokens;
    const int mine = in ? row_of(p, a.token) : -1;
    const float weight = mine >= 0 && p.weights != nullptr ? p.weights[a.token * p.top + lane] : 1.0f;
    float result = 0.0f;   // lane j: the j-th sum
    for (int j0 = 0; j0 < p.top; j0 += ROWS) {
      int r[ROWS];
      float w[ROWS], dot[ROWS];
#pragma unroll
      for (int q = 0; q < ROWS; ++q) {
        r[q] = __shfl_sync(0xffffffffu, mine, (j0 + q) & 31);
        if (j0 + q >= p.top) r[q] = -1;
        w[q] = __shfl_sync(0xffffffffu, weight, (j0 + q) & 31);
        dot[q] = 0.0f;
      }
#pragma unroll 2
      for (int v = a.first; in && v < per; v += a.stride) {
        P x, y[ROWS];
        x.load(p.x, a.token * p.ldx + (int64_t)v * P::N);
#pragma unroll
        for (int q = 0; q < ROWS; ++q)
          if (r[q] >= 0) y[q].load(p.y, r[q] * p.ldy + (int64_t)v * P::N);
#pragma unroll
        for (int q = 0; q < ROWS; ++q)
          if (r[q] >= 0) {
            P d;
            float g[P::N], v_y[P::N];
            x.get(g);
            y[q].get(v_y);
#pragma unroll
            for (int k = 0; k < P::N; ++k) {
              dot[q] = fmaf(g[k], v_y[k], dot[q]);
              g[k] *= w[q];
            }
            d.set(g);
            d.store(p.out, r[q] * p.ldo + (int64_t)v * P::N);
          }
      }
#pragma unroll
      for (int q = 0; q < ROWS; ++q) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[q] += __shfl_xor_sync(0xffffffffu, dot[q], o);
        if (lane == j0 + q) result = dot[q];
      }
    }
    const int group = 1 << p.parts_shift;
    if (group > 1) {
      __syncthreads();
      parts[warp][lane] = result;
      __syncthreads();
      if ((warp & (group - 1)) == 0)
        for (int h = 1; h < group; ++h) result += parts[warp + h][lane];
    }
    if (in && (warp & (group - 1)) == 0 && lane < p.top) static_cast<float*>(p.dweights)[a.token * p.top + lane] = result;
  }
  clear_rest<DT, WIDE>(p);
}

enum { DISPATCH, COMBINE, COMBINE_GRAD };

template <int WHAT, int DT, bool WIDE>
cudaError_t launch_as(ExchangeParams p, int sm_count, cudaStream_t stream, int* ctas) {
  // Warps of a token: as many as leave each lane two turns of its loads (four pieces of dispatch,
  // eight of combine_grad), so that a row's bytes are asked for closer together; more,
  // down to one piece per lane, while the chip has less than 16 warps per SM.  At most eight.
  // Measured with one warp / the rule's, us: dispatch of 3000 tokens, top 2, 4096 wide 11.7 / 10.7
  // (four), 6000 of 8192 52.3 / 45.7 (eight), 16 tokens of 8192 6.6 / 2.4 (eight); combine of 8191,
  // top 4, 4096 63.6 / 59.7 (four), of 16384, top 2, 2048 41.0 with one, 48.5 with four; combine_grad
  // of 6000, top 2, 8192 88.9 / 78.4 (four), of 16384, top 2, 1024 31.7 with one, 34.1 with two.
  const int64_t per = p.width / Piece<DT, WIDE>::N;
  const int64_t keep = WHAT == DISPATCH ? 4 : WHAT == COMBINE_GRAD ? 8 : p.top <= 2 ? 8 : p.top <= 4 ? 4 : 2;
  p.parts_shift = 0;
  while (p.parts_shift < 3 && per >= (32 * keep << (p.parts_shift + 1))) ++p.parts_shift;
  while (p.parts_shift < 3 && (p.tokens << p.parts_shift) < 16 * (int64_t)sm_count && per > (int64_t)(32 << p.parts_shift))
    ++p.parts_shift;
  const int64_t work = ((p.tokens << p.parts_shift) + WARPS - 1) / WARPS;
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(work, 16 * (int64_t)sm_count)));
  *ctas = (int)grid.x;
  if constexpr (WHAT == DISPATCH) return launch_dependent(dispatch_kernel<DT, WIDE>, grid, THREADS, stream, p);
  else if constexpr (WHAT == COMBINE) return p.top <= 2 ? launch_dependent(combine_kernel<DT, WIDE, 2>, grid, THREADS, stream, p)
                                      : p.top <= 4 ? launch_dependent(combine_kernel<DT, WIDE, 4>, grid, THREADS, stream, p)
                                                   : launch_dependent(combine_kernel<DT, WIDE, 8>, grid, THREADS, stream, p);
  else return launch_dependent(combine_grad_kernel<DT, WIDE>, grid, THREADS, stream, p);
}

template <int WHAT>
cudaError_t launch_any(const ExchangeParams& p, int sm_count, cudaStream_t stream, int* grid) {
  if (p.dtype == GEMM_F32)
    return p.vec ? launch_as<WHAT, GEMM_F32, true>(p, sm_count, stream, grid)
                 : launch_as<WHAT, GEMM_F32, false>(p, sm_count, stream, grid);
  if (p.dtype == GEMM_F16)
    return p.vec ? launch_as<WHAT, GEMM_F16, true>(p, sm_count, stream, grid)
                 : launch_as<WHAT, GEMM_F16, false>(p, sm_count, stream, grid);
  return p.vec ? launch_as<WHAT, GEMM_BF16, true>(p, sm_count, stream, grid)
               : launch_as<WHAT, GEMM_BF16, false>(p, sm_count, stream, grid);
}

}  // namespace

cudaError_t launch_dispatch(const ExchangeParams& p, int sm_count, cudaStream_t stream, int* grid) {
  return launch_any<DISPATCH>(p, sm_count, stream, grid);
}
cudaError_t launch_combine(const ExchangeParams& p, int sm_count, cudaStream_t stream, int* grid) {
  return launch_any<COMBINE>(p, sm_count, stream, grid);
}
cudaError_t launch_combine_grad(const ExchangeParams& p, int sm_count, cudaStream_t stream, int* grid) {
  return launch_any<COMBINE_GRAD>(p, sm_count, stream, grid);
}

}  // namespace gemmlib
