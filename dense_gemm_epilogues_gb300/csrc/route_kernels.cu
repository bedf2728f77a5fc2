// route_kernels.cu -- the routing of tokens to experts, its balance loss, and the gradient.
//
//   p = softmax(z),  the experts of a token are its `top` largest z (the lower index first
//   where they are equal; one whose z is -inf is never taken);
//   w = p at them, or p at them over their sum;
//   c_e = rows of expert e,  C = sum c_e,  n = tokens with any expert;
//   loss = E / (C n) * sum_e c_e * sum_t p_te.
// Rows are numbered expert by expert, in the order of tokens (and of a token's choices)
// within one: a stable counting sort by expert.
//
// Two launches.  The first chooses: a warp takes one token at a time, a lane experts lane,
// lane + 32, ...; each of the `top` turns is one warp maximum of a key that orders like the
// logits and one warp minimum of the index.  A lane keeps the counts and the sums of p of
// its own experts in registers over all tokens of its warp, so a choice's number among its
// warp's rows is known when it is made.  Warps take tokens in order, CTAs too; a CTA adds up
// its warps' counts and leaves its own in scratch.  The second launch places: every CTA adds
// the counts of the CTAs before it (B x E integers, from L2) to its tokens' numbers, and one
// more CTA adds up the loss.  Nothing waits for another CTA and no atomics decide an order,
// so a routing is the same bits every time.  A batch that one CTA takes whole is one launch.
// Bound by latency: the data are a few megabytes.
#include "layer.h"

namespace gemmlib {
namespace {

constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;
constexpr uint32_t LOWEST = 0x007fffffu;   // the key of -inf

// Orders like the float: -inf lowest, zeros alike, NaN highest.
__device__ __forceinline__ uint32_t key_of(float z) {
  if (z != z) return 0xffffffffu;
  const uint32_t b = __float_as_uint(z + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The tokens of warp `w` of `warps`: in order, equal parts.
__device__ __forceinline__ void token_range(int64_t tokens, int64_t warps, int64_t w, int64_t& lo, int64_t& hi) {
  const int64_t per = (tokens + warps - 1) / warps;
  lo = min(tokens, w * per);
  hi = min(tokens, lo + per);
}

// z of a token: lane's experts; -inf where there is none.
template <int V>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float (&z)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 32 * v;
    z[v] = e < p.experts ? load_as_float(p.logits, p.dtype, t * p.ld + e) : -INFINITY;
  }
}

// exp(z - m) of a lane's experts and 1 / sum over the warp; m is the largest of them.
template <int V>
__device__ __forceinline__ float softmax(const float (&z)[V], float m, float (&e)[V]) {
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    e[v] = expf(z[v] - m);
    s += e[v];
  }
  return 1.0f / warp_sum(s);
}

// Where experts begin: an exclusive sum of counts[0 .. E) into starts[0 .. E], by one warp.
__device__ __forceinline__ void scan_counts(const int* counts, int* starts, int E, int lane) {
  int sum = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    int v = e0 + lane < E ? counts[e0 + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (e0 + lane < E) starts[e0 + lane + 1] = sum + v;
    sum += __shfl_sync(0xffffffffu, v, 31);
  }
  if (lane == 0) starts[0] = 0;
}

// The loss from the counts and the sums of p over all tokens, by one warp.
__device__ __forceinline__ void write_loss(const RouteParams& p, const int* counts, const double* mass, int rows,
                                           int routed, int lane) {
  double s = 0.0;
  for (int e = lane; e < p.experts; e += 32) s += (double)counts[e] * mass[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && p.loss != nullptr)
    *p.loss = rows > 0 ? (float)(s * (double)p.experts / ((double)rows * (double)routed)) : 0.0f;
}

// Chooses.  Dynamic shared memory: WARPS x E counts, then sums of p.
template <int V>
__global__ void __launch_bounds__(THREADS) route_choose_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int smem[];
  const int E = p.experts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* counts = smem;                                             // [WARPS][E]
  float* mass = reinterpret_cast<float*>(smem + WARPS * E);       // [WARPS][E]
  __shared__ int tokens_of[WARPS];
  pdl_launch_dependents();
  pdl_wait();
  int64_t lo, hi;
  token_range(p.tokens, (int64_t)gridDim.x * WARPS, (int64_t)blockIdx.x * WARPS + warp, lo, hi);
  int cnt[V];
  float sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) cnt[v] = 0, sum[v] = 0.0f;
  int routed = 0;
  constexpr bool AHEAD = V <= 8;   // the next token's logits come in during this one's turns (registers allow it)
  float z[V], ahead[AHEAD ? V : 1];
  if constexpr (AHEAD) {
    if (lo < hi) load_logits<V>(p, lo, lane, ahead);
  }
  for (int64_t t = lo; t < hi; ++t) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = ahead[v];
      if (t + 1 < hi) load_logits<V>(p, t + 1, lane, ahead);
    } else {
      load_logits<V>(p, t, lane, z);
    }
    // Choice j is kept by lane j.
    int expert = -1, number = -1;
    float value = -INFINITY, first = 0.0f;
    const bool counts_in = p.mask == nullptr || p.mask[t] != 0;
    if (counts_in) {
      uint32_t key[V];
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = lane + 32 * v < E ? key_of(z[v]) : 0u;
      for (int j = 0; j < p.top; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int v = 1; v < V; ++v) best = max(best, key[v]);
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        if (most <= LOWEST) break;
        int mine = 0x7fffffff;
        float at = 0.0f;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          if (key[v] == most) mine = lane + 32 * v, at = z[v];
        const int e = (int)__reduce_min_sync(0xffffffffu, (unsigned)mine);
        int rank = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (e == lane + 32 * v) {
            rank = cnt[v]++;
            key[v] = 0u;
          }
        rank = __shfl_sync(0xffffffffu, rank, e & 31);
        at = __shfl_sync(0xffffffffu, at, e & 31);
        if (j == 0) first = at;
        if (lane == j) expert = e, number = rank, value = at;
      }
    }
    const bool any = __shfl_sync(0xffffffffu, expert, 0) >= 0;
    float w = 0.0f;
    if (any) {
      ++routed;
      float e[V];
      const float inv = softmax<V>(z, first, e);
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] += e[v] * inv;
      w = expert >= 0 ? expf(value - first) : 0.0f;
      w = p.renormalize ? w / warp_sum(w) : w * inv;
    }
    if (lane < p.top) {
      const int64_t i = t * p.top + lane;
      p.weights[i] = expert >= 0 ? w : 0.0f;
      p.chosen[i] = expert;
      p.slots[i] = number;   // (its number among the warp's rows of that expert)
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 32 * v;
    if (e < E) {
      counts[warp * E + e] = cnt[v];
      mass[warp * E + e] = sum[v];
    }
  }
  if (lane == 0) tokens_of[warp] = routed;
  __syncthreads();
  // The warps' counts become the numbers that their rows start at; row 0 takes the CTA's.
  const bool alone = gridDim.x == 1;
  int* starts = reinterpret_cast<int*>(mass + WARPS * E);         // alone: [E + 1]
  int* all = starts + E + 1;                                      // alone: [E]
  double* dmass = reinterpret_cast<double*>(smem + ((2 * WARPS * E + 2 * E + 2) & ~1));   // alone: [E]
  for (int e = threadIdx.x; e < E; e += THREADS) {
    int n = 0;
    double m = 0.0;
    for (int w = 0; w < WARPS; ++w) {
      const int c = counts[w * E + e];
      counts[w * E + e] = n;
      n += c;
      m += (double)mass[w * E + e];
    }
    if (alone) {
      all[e] = n;
      dmass[e] = m;
      p.counts[e] = n;
    } else {
      p.hist[(int64_t)blockIdx.x * (E + 1) + e] = n;
      p.mass[(int64_t)blockIdx.x * E + e] = (float)m;
    }
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < WARPS; ++w) n += tokens_of[w];
    if (alone) *p.routed = n;
    else p.hist[(int64_t)blockIdx.x * (E + 1) + E] = n;
    tokens_of[0] = n;
  }
  __syncthreads();
  if (alone) {
    if (warp == 0) {
      scan_counts(all, starts, E, lane);
      __syncwarp();
      write_loss(p, all, dmass, starts[E], tokens_of[0], lane);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += THREADS) p.offsets[e] = starts[e];
  }
  // (a warp's own slots: the lane that wrote an entry reads it)
  for (int64_t t = lo; t < hi; ++t) {
    if (lane < p.top) {
      const int64_t i = t * p.top + lane;
      const int e = p.chosen[i];
      if (e >= 0) p.slots[i] += counts[warp * E + e] + (alone ? starts[e] : 0);
    }
  }
}

// Places.  CTA b < p.blocks adds what lies before its rows to its tokens' numbers; the last
// CTA writes the counts, offsets and the loss.
__global__ void __launch_bounds__(THREADS) route_place_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int smem[];
  const int E = p.experts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const bool last = b == p.blocks;
  int* all = smem;             // [E + 1] all rows of an expert; tokens with any
  int* before = all + E + 1;   // [E] those of the CTAs before this one
  int* starts = before + E;    // [E + 1]
  double* dmass = reinterpret_cast<double*>(smem + ((3 * E + 3) & ~1));   // last CTA: [E]
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < 2 * E + 1; e += THREADS) smem[e] = 0;
  __syncthreads();
  pdl_wait();
  // Rows of the table are shared out over groups of threads as wide as the table.
  const int cols = E + 1, width = (cols + 31) / 32 * 32, groups = max(1, THREADS / width);
  const int g = (int)threadIdx.x / width;
  for (int c = (int)threadIdx.x % width; g < groups && c < cols; c += width * groups >= THREADS ? THREADS : width) {
    int sum = 0, part = 0;
#pragma unroll 8
    for (int r = g; r < p.blocks; r += groups) {
      const int n = __ldcg(p.hist + (int64_t)r * cols + c);
      sum += n;
      part += r < b ? n : 0;
    }
    atomicAdd(&all[c], sum);   // (integers: any order)
    if (c < E) atomicAdd(&before[c], part);
  }
  if (last) {
    for (int e = threadIdx.x; e < E; e += THREADS) {
      double m = 0.0;
#pragma unroll 8
      for (int r = 0; r < p.blocks; ++r) m += (double)__ldcg(p.mass + (int64_t)r * E + e);
      dmass[e] = m;
    }
  }
  __syncthreads();
  if (warp == 0) {
    scan_counts(all, starts, E, lane);
    __syncwarp();
    if (last) write_loss(p, all, dmass, starts[E], all[E], lane);
  }
  __syncthreads();
  if (last) {
    for (int e = threadIdx.x; e <= E; e += THREADS) {
      if (e < E) p.counts[e] = all[e];
      else *p.routed = all[E];
      p.offsets[e] = starts[e];
    }
    return;
  }
  int64_t lo, hi, t1;
  token_range(p.tokens, (int64_t)p.blocks * WARPS, (int64_t)b * WARPS, lo, t1);
  token_range(p.tokens, (int64_t)p.blocks * WARPS, (int64_t)b * WARPS + WARPS - 1, t1, hi);
  for (int64_t i = lo * p.top + threadIdx.x; i < hi * p.top; i += THREADS) {
    const int e = p.chosen[i];
    if (e >= 0) p.slots[i] += starts[e] + before[e];
  }
}

// dz_i = [renormalised: w_i (dw_i - sum_j w_j dw_j) at the chosen] + p_i (g_i - sum p g),
// g_e = dloss E c_e / (C n) [+ dw_e at the chosen].  A warp takes one token at a time.
template <int V>
__global__ void __launch_bounds__(THREADS) route_grad_kernel(const __grid_constant__ RouteParams p) {
  const int E = p.experts, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int n = *p.routed, rows = p.offsets[E];
  const float dloss = p.dloss_scale * (p.dloss != nullptr ? *p.dloss : 1.0f);
  const float per_row = rows > 0 && n > 0 ? (float)((double)dloss * E / ((double)rows * (double)n)) : 0.0f;
  float share[V];
#pragma unroll
  for (int v = 0; v < V; ++v) share[v] = lane + 32 * v < E ? per_row * (float)p.counts[lane + 32 * v] : 0.0f;
  const int64_t warps = (int64_t)gridDim.x * WARPS;
  for (int64_t t = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); t < p.tokens; t += warps) {
    float z[V], e[V], g[V], direct[V];
    load_logits<V>(p, t, lane, z);
    int expert = -1;
    float w = 0.0f, dw = 0.0f;
    if (lane < p.top) {
      expert = p.chosen[t * p.top + lane];
      if (expert >= E) expert = -1;
      if (expert >= 0 && p.dweights != nullptr) {
        w = p.weights[t * p.top + lane];
        dw = p.dweights[t * p.top + lane];
      }
    }
    const bool any = __shfl_sync(0xffffffffu, expert, 0) >= 0;
    float m = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, z[v]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float inv = softmax<V>(z, m, e);
    // What a choice adds: to dz at once (renormalised), or to dL/dp.
    const float add = p.renormalize ? w * (dw - warp_sum(w * dw)) : dw;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      g[v] = share[v];
      direct[v] = 0.0f;
    }
    if (p.dweights != nullptr) {
      for (int j = 0; j < p.top; ++j) {
        const int x = __shfl_sync(0xffffffffu, expert, j);
        const float a = __shfl_sync(0xffffffffu, add, j);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (x == lane + 32 * v) direct[v] += a;
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      e[v] *= inv;
      if (!p.renormalize) {
        g[v] += direct[v];
        direct[v] = 0.0f;
      }
      s += lane + 32 * v < E ? e[v] * g[v] : 0.0f;
    }
    s = warp_sum(s);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 32 * v < E)
        store_float_as(p.dlogits, p.dtype, t * p.ldd + lane + 32 * v, any ? direct[v] + e[v] * (g[v] - s) : 0.0f);
  }
}

template <typename F>
cudaError_t with_values(int experts, F&& f) {
  if (experts <= 32) return f(TypeTag<1>{});
  if (experts <= 64) return f(TypeTag<2>{});
  if (experts <= 128) return f(TypeTag<4>{});
  if (experts <= 256) return f(TypeTag<8>{});
  if (experts <= 512) return f(TypeTag<16>{});
  return f(TypeTag<32>{});
}

template <typename... P>
cudaError_t launch_smem(void (*kernel)(P...), int grid, size_t smem, cudaStream_t stream, const RouteParams& p) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// CTAs that choose: one for up to 64 tokens (four per warp: one launch takes less than two),
// else one per SM as long as a warp has a token.
int route_blocks(int64_t tokens, int64_t experts, int sm_count) {
  (void)experts;
  if (tokens <= 4 * WARPS) return 1;
  return (int)std::min<int64_t>(sm_count, (tokens + WARPS - 1) / WARPS);
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  const size_t E = (size_t)p.experts;
  const cudaError_t e = with_values(p.experts, [&](auto v) {
    return launch_smem(route_choose_kernel<decltype(v)::value>, p.blocks, (2 * WARPS * E + 4 * E + 6) * 4, stream, p);
  });
  if (e != cudaSuccess || p.blocks == 1) return e;
  return launch_smem(route_place_kernel, p.blocks + 1, (5 * E + 6) * 4, stream, p);
}

cudaError_t launch_route_grad(const RouteParams& p, int sm_count, cudaStream_t stream) {
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(2 * (int64_t)sm_count, (p.tokens + WARPS - 1) / WARPS));
  return with_values(p.experts, [&](auto v) {
    return launch_smem(route_grad_kernel<decltype(v)::value>, grid, 0, stream, p);
  });
}

}  // namespace gemmlib
