// exchange_kernels.cu -- rows between tokens and experts:
//     dispatch      out[slot(t, j)] = x[t];  rows behind the last used one are zero
//     combine       out[t] = residual[t] + sum_j w(t, j) y[slot(t, j)]
//     combine_grad  out[slot(t, j)] = w(t, j) x[t],  dweights(t, j) = <x[t], y[slot(t, j)]>
// (dispatch's own gradient is combine without weights and residual.)  All three go by
// tokens: a token's row is read or written once and its `top` sorted rows lie anywhere, each
// a long run of bytes; so every byte moves once, no atomics decide an order, and the sums
// over a token's rows and over a row's entries have one order.
//
// Bound by memory.  dispatch and combine: a thread takes 16 bytes of a token and all of its
// rows' (four rows' loads under way), and as many such pieces as the chip has room for.
// combine_grad: a warp takes a token, four of its rows at a time.
//
// A slot outside the sorted buffer is no row; one that is not -1 either is reported through
// the error word.
#include "layer.h"

namespace gemmlib {
namespace {

constexpr int THREADS = 256;

// Piece v of a row: VEC entries (16 bytes), or a single entry where rows are not aligned.
template <int DT, bool WIDE>
struct Piece {
  static constexpr int N = !WIDE ? 1 : DT == GEMM_F32 ? 4 : 8;
  float x[N];

  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (!WIDE) {
      x[0] = load_as_float(p, DT, i);
    } else if constexpr (DT == GEMM_F32) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      set(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    }
  }
  __device__ __forceinline__ void set(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int h = 0; h < N / 2; ++h) {
      if constexpr (DT == GEMM_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[h]));
        x[2 * h] = f.x, x[2 * h + 1] = f.y;
      } else {
        x[2 * h] = __uint_as_float(w[h] << 16), x[2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    if constexpr (!WIDE) {
      store_float_as(p, DT, i, x[0]);
    } else if constexpr (DT == GEMM_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < N / 2; ++h) {
        if constexpr (DT == GEMM_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[h]) : "f"(x[2 * h + 1]), "f"(x[2 * h]));
        else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[h]) : "f"(x[2 * h + 1]), "f"(x[2 * h]));
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// The row of (t, j), -1 for none.
__device__ __forceinline__ int64_t row_of(const ExchangeParams& p, int64_t i) {
  const int s = p.slots[i];
  if (s >= 0 && s < p.rows) return s;
  if (s != -1) atomicCAS(p.err, 0, (int32_t)GEMM_ERR_INVALID_ARG);
  return -1;
}

// Rows from the last used one on, as zeros.
template <int DT, bool WIDE>
__device__ __forceinline__ void clear_rest(const ExchangeParams& p) {
  if (p.used == nullptr) return;
  using P = Piece<DT, WIDE>;
  const int64_t first = min(p.rows, max((int64_t)0, (int64_t)*p.used)), per = p.width / P::N;
  P z;
#pragma unroll
  for (int k = 0; k < P::N; ++k) z.x[k] = 0.0f;
  const int64_t stride = (int64_t)gridDim.x * THREADS;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < (p.rows - first) * per; i += stride) {
    const int64_t r = i / per;
    z.store(p.out, (first + r) * p.ldo + (i - r * per) * P::N);
  }
}

template <int DT, bool WIDE>
__global__ void __launch_bounds__(THREADS) dispatch_kernel(const __grid_constant__ ExchangeParams p) {
  using P = Piece<DT, WIDE>;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t per = p.width / P::N, stride = (int64_t)gridDim.x * THREADS;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < p.tokens * per; i += stride) {
    const int64_t t = i / per, c = (i - t * per) * P::N;
    P x;
    x.load(p.x, t * p.ldx + c);
    for (int j = 0; j < p.top; ++j) {
      const int64_t r = row_of(p, t * p.top + j);
      if (r >= 0) x.store(p.out, r * p.ldo + c);
    }
  }
  clear_rest<DT, WIDE>(p);
}

template <int DT, bool WIDE>
__global__ void __launch_bounds__(THREADS) combine_kernel(const __grid_constant__ ExchangeParams p) {
  using P = Piece<DT, WIDE>;
  constexpr int ROWS = 4;   // loads under way
  pdl_launch_dependents();
  pdl_wait();
  const int64_t per = p.width / P::N, stride = (int64_t)gridDim.x * THREADS;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < p.tokens * per; i += stride) {
    const int64_t t = i / per, c = (i - t * per) * P::N;
    P sum;
    if (p.residual != nullptr) {
      sum.load(p.residual, t * p.ldr + c);
    } else {
#pragma unroll
      for (int k = 0; k < P::N; ++k) sum.x[k] = 0.0f;
    }
    for (int j0 = 0; j0 < p.top; j0 += ROWS) {
      P y[ROWS];
      float w[ROWS];
      bool ok[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int64_t r = j0 + u < p.top ? row_of(p, t * p.top + j0 + u) : -1;
        ok[u] = r >= 0;
        if (ok[u]) {
          w[u] = p.weights != nullptr ? p.weights[t * p.top + j0 + u] : 1.0f;
          y[u].load(p.y, r * p.ldy + c);
        }
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u)
        if (ok[u]) {
#pragma unroll
          for (int k = 0; k < P::N; ++k) sum.x[k] = fmaf(w[u], y[u].x[k], sum.x[k]);
        }
    }
    sum.store(p.out, t * p.ldo + c);
  }
}

template <int DT, bool WIDE>
__global__ void __launch_bounds__(THREADS) combine_grad_kernel(const __grid_constant__ ExchangeParams p) {
  using P = Piece<DT, WIDE>;
  constexpr int ROWS = 4;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32), per = p.width / P::N;
  for (int64_t t = (int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5); t < p.tokens; t += warps) {
    for (int j0 = 0; j0 < p.top; j0 += ROWS) {
      int64_t r[ROWS];
      float w[ROWS], dot[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int64_t i = t * p.top + j0 + u;
        r[u] = j0 + u < p.top ? row_of(p, i) : -1;
        w[u] = r[u] >= 0 && p.weights != nullptr ? p.weights[i] : 1.0f;
        dot[u] = 0.0f;
      }
#pragma unroll 2
      for (int64_t v = lane; v < per; v += 32) {
        P x, y[ROWS];
        x.load(p.x, t * p.ldx + v * P::N);
#pragma unroll
        for (int u = 0; u < ROWS; ++u)
          if (r[u] >= 0) y[u].load(p.y, r[u] * p.ldy + v * P::N);
#pragma unroll
        for (int u = 0; u < ROWS; ++u)
          if (r[u] >= 0) {
            P d;
#pragma unroll
            for (int k = 0; k < P::N; ++k) {
              dot[u] = fmaf(x.x[k], y[u].x[k], dot[u]);
              d.x[k] = w[u] * x.x[k];
            }
            d.store(p.out, r[u] * p.ldo + v * P::N);
          }
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
        if (lane == 0 && j0 + u < p.top) static_cast<float*>(p.dweights)[t * p.top + j0 + u] = dot[u];
      }
    }
  }
  clear_rest<DT, WIDE>(p);
}

enum { DISPATCH, COMBINE, COMBINE_GRAD };

template <int WHAT, int DT, bool WIDE>
cudaError_t launch_as(const ExchangeParams& p, int sm_count, cudaStream_t stream) {
  const int64_t per = p.width / Piece<DT, WIDE>::N;
  const int64_t work = WHAT == COMBINE_GRAD ? p.tokens * 32 : p.tokens * per;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((work + THREADS - 1) / THREADS, 16 * (int64_t)sm_count));
  if constexpr (WHAT == DISPATCH) return launch_dependent(dispatch_kernel<DT, WIDE>, dim3((unsigned)grid), THREADS, stream, p);
  else if constexpr (WHAT == COMBINE) return launch_dependent(combine_kernel<DT, WIDE>, dim3((unsigned)grid), THREADS, stream, p);
  else return launch_dependent(combine_grad_kernel<DT, WIDE>, dim3((unsigned)grid), THREADS, stream, p);
}

template <int WHAT>
cudaError_t launch_any(const ExchangeParams& p, int sm_count, cudaStream_t stream) {
  if (p.dtype == GEMM_F32)
    return p.vec ? launch_as<WHAT, GEMM_F32, true>(p, sm_count, stream) : launch_as<WHAT, GEMM_F32, false>(p, sm_count, stream);
  if (p.dtype == GEMM_F16)
    return p.vec ? launch_as<WHAT, GEMM_F16, true>(p, sm_count, stream) : launch_as<WHAT, GEMM_F16, false>(p, sm_count, stream);
  return p.vec ? launch_as<WHAT, GEMM_BF16, true>(p, sm_count, stream) : launch_as<WHAT, GEMM_BF16, false>(p, sm_count, stream);
}

}  // namespace

cudaError_t launch_dispatch(const ExchangeParams& p, int sm_count, cudaStream_t stream) {
  return launch_any<DISPATCH>(p, sm_count, stream);
}
cudaError_t launch_combine(const ExchangeParams& p, int sm_count, cudaStream_t stream) {
  return launch_any<COMBINE>(p, sm_count, stream);
}
cudaError_t launch_combine_grad(const ExchangeParams& p, int sm_count, cudaStream_t stream) {
  return launch_any<COMBINE_GRAD>(p, sm_count, stream);
}

}  // namespace gemmlib
