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
// logits and one warp minimum of the index.  A lane keeps the sums of p of its own experts in
// registers over all tokens of its warp, which counts its experts' rows in shared memory, so
// a choice's number among its warp's rows is known when it is made.  Warps take tokens in
// order, CTAs too; a CTA adds up its warps' counts and leaves its own in scratch.  The second
// launch places: every CTA adds the counts of the CTAs before it (B x E integers, from L2) to
// its tokens' numbers, and one more CTA adds up the loss.  Nothing waits for another CTA and no atomics decide an order,
// so a routing is the same bits every time.  A batch that one CTA takes whole is one launch.
// Exponentials and quotients are the hardware's (2 steps of fp32, and |x| 2^-24 of an argument):
// every lane takes several per token, and beside fp32 sums over the experts they change little
// (weights and loss against 64 bits 3.4e-8 and 6.0e-8 of their norm in two cases, 3.3e-8 and 5.3e-8
// with accurate ones).
// Bound by latency and by the choice's instructions (400 per token and warp): the data are a few
// megabytes.  16384 tokens, top 6 of 64: 15.3 us, of which the choice takes 9; its gradient 6.1 us;
// 16 tokens, top 2 of 8: 3.8 us.
#include <atomic>

#include "layer.h"

namespace gemmlib {
namespace {

// Warps of a CTA: 32 where a lane's experts leave room in the registers.
__host__ __device__ constexpr int warps_of(int values) { return values <= 4 ? 32 : 16; }
constexpr int MAX_WARPS = 32;
constexpr int PLACE_THREADS = 512;
constexpr uint32_t LOWEST = 0x007fffffu;   // the key of -inf

// Orders like the float: -inf lowest, zeros alike, NaN highest.
__device__ __forceinline__ uint32_t key_of(float z) {
  if (z != z) return 0xffffffffu;
  const uint32_t b = __float_as_uint(z + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// exp(x) for x <= 0, by the hardware's power of two: off by 2 steps and |x| 2^-24.
__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(LOG2_E * x); }

// The tokens of warp `w`: in order, equal parts.
__device__ __forceinline__ void token_range(const RouteParams& p, int w, int64_t& lo, int64_t& hi) {
  lo = min(p.tokens, (int64_t)w * p.per_warp);
  hi = min(p.tokens, lo + p.per_warp);
}

// z of a token: lane's experts; -inf where there is none.
template <int V, int DT>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float (&z)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 32 * v;
    z[v] = e < p.experts ? load_as_float(p.logits, DT, t * p.ld + e) : -INFINITY;
  }
}

// exp(z - m) of a lane's experts and 1 / sum over the warp; m is the largest of them.
template <int V>
__device__ __forceinline__ float softmax(const float (&z)[V], float m, float (&e)[V]) {
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    e[v] = exp_fast(z[v] - m);
    s += e[v];
  }
  return rcp_fast(warp_sum(s));
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
__device__ __forceinline__ void write_loss(const RouteParams& p, const int* counts, const float* mass, int rows,
                                           int routed, int lane) {
  float s = 0.0f;
  if (rows > 0) {
    const float scale = (float)p.experts / (float)rows;
    for (int e = lane; e < p.experts; e += 32) s += (float)counts[e] * scale * (mass[e] / (float)routed);
  }
  s = warp_sum(s);
  if (lane == 0 && p.loss != nullptr) *p.loss = s;
}

// Chooses.  Dynamic shared memory: WARPS x E counts, then sums of p.
template <int V, int DT>
__global__ void __launch_bounds__(32 * warps_of(V)) route_choose_kernel(const __grid_constant__ RouteParams p) {
  constexpr int WARPS = warps_of(V), THREADS = 32 * WARPS;
  extern __shared__ int smem[];
  const int E = p.experts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* counts = smem;                                             // [WARPS][E]
  float* mass = reinterpret_cast<float*>(smem + WARPS * E);       // [WARPS][E]
  __shared__ int tokens_of[MAX_WARPS];
  pdl_launch_dependents();
  pdl_wait();
  int64_t lo, hi;
  token_range(p, (int)blockIdx.x * WARPS + warp, lo, hi);
  float sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sum[v] = 0.0f;
    if (lane + 32 * v < E) counts[warp * E + lane + 32 * v] = 0;
  }
  __syncwarp();
  int routed = 0;
  constexpr bool AHEAD = V <= 8;   // the next token's logits come in during this one's turns (registers allow it)
  float z[V], ahead[AHEAD ? V : 1];
  if constexpr (AHEAD) {
    if (lo < hi) load_logits<V, DT>(p, lo, lane, ahead);
  }
  auto masked = [&](int64_t t) { return p.mask != nullptr && p.mask[t] == 0; };
  bool mask_ahead = lo < hi && masked(lo);
  for (int64_t t = lo; t < hi; ++t) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = ahead[v];
      if (t + 1 < hi) load_logits<V, DT>(p, t + 1, lane, ahead);
    } else {
      load_logits<V, DT>(p, t, lane, z);
    }
    // Choice j is kept by lane j.
    int expert = -1, number = -1;
    uint32_t mine_key = LOWEST;
    const bool counts_in = !mask_ahead;
    mask_ahead = t + 1 < hi && masked(t + 1);
    uint32_t top_key = 0u;
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
        unsigned own = 0xffffffffu;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          if (key[v] == most) own = (unsigned)(lane + 32 * v);
        const unsigned e = __reduce_min_sync(0xffffffffu, own);
        if (own == e) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (e == (unsigned)(lane + 32 * v)) key[v] = 0u;
        }
        if (j == 0) top_key = most;
        if (lane == j) expert = (int)e, mine_key = most;
      }
      if (expert >= 0) number = counts[warp * E + expert]++;   // (a token's experts differ)
      __syncwarp();
    }
    const float first = value_of(top_key), value = value_of(mine_key);
    const bool any = __shfl_sync(0xffffffffu, expert, 0) >= 0;
    float w = 0.0f;
    if (any) {
      ++routed;
      float e[V];
      const float inv = softmax<V>(z, first, e);
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] += e[v] * inv;
      w = expert >= 0 ? exp_fast(value - first) : 0.0f;
      w *= p.renormalize ? rcp_fast(warp_sum(w)) : inv;
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
    if (e < E) mass[warp * E + e] = sum[v];
  }
  if (lane == 0) tokens_of[warp] = routed;
  __syncthreads();
  // The warps' counts become the numbers that their rows start at.
  const bool alone = gridDim.x == 1;
  int* starts = reinterpret_cast<int*>(mass + WARPS * E);   // alone: [E + 1]
  int* all = starts + E + 1;                                // alone: [E]
  float* total = reinterpret_cast<float*>(all + E);         // alone: [E]
  for (int e = threadIdx.x; e < E; e += THREADS) {
    int n = 0;
    float m = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const int c = counts[w * E + e];
      counts[w * E + e] = n;
      n += c;
      m += mass[w * E + e];
    }
    if (alone) {
      all[e] = n;
      total[e] = m;
      p.counts[e] = n;
    } else {
      p.hist[(int64_t)blockIdx.x * route_pitch(E) + e] = n;
      p.mass[(int64_t)blockIdx.x * route_pitch(E) + e] = m;
    }
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < WARPS; ++w) n += tokens_of[w];
    if (alone) *p.routed = n;
    else p.hist[(int64_t)blockIdx.x * route_pitch(E) + E] = n;
    tokens_of[0] = n;
  }
  __syncthreads();
  if (alone) {
    if (warp == 0) {
      scan_counts(all, starts, E, lane);
      __syncwarp();
      write_loss(p, all, total, starts[E], tokens_of[0], lane);
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += THREADS) p.offsets[e] = starts[e];
  }
  // The warp's own slots.
#pragma unroll 2
  for (int64_t i = lo * p.top + lane; i < hi * p.top; i += 32) {
    const int e = p.chosen[i], number = p.slots[i];
    if (e >= 0) p.slots[i] = number + counts[warp * E + e] + (alone ? starts[e] : 0);
  }
}

__host__ __device__ __forceinline__ int place_groups(int experts) {
  const int groups = PLACE_THREADS / (route_pitch(experts) / 4);
  return groups < 1 ? 1 : groups;
}

// Places.  CTA b < p.blocks adds what lies before its rows to its tokens' numbers; the last
// CTA writes the counts, offsets and the loss.  Dynamic shared memory: see place_smem.
__global__ void __launch_bounds__(PLACE_THREADS) route_place_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int smem[];
  const int E = p.experts, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x;
  const bool last = b == p.blocks;
  int* all = smem;             // [E + 1] all rows of an expert; tokens with any
  int* before = all + E + 1;   // [E] those of the CTAs before this one
  int* starts = before + E;    // [E + 1]
  float* mass = reinterpret_cast<float*>(starts + E + 1);   // last CTA: [groups][E]
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < 2 * E + 1; e += PLACE_THREADS) smem[e] = 0;
  __syncthreads();
  pdl_wait();
  // The table's rows are shared out over groups of threads, four experts to a thread.
  const int pitch = route_pitch(E), vecs = pitch / 4, groups = place_groups(E);
  const int g = (int)threadIdx.x / vecs;
  for (int v = (int)threadIdx.x - g * vecs; g < groups && v < vecs; v += PLACE_THREADS) {
    int sum[4] = {0, 0, 0, 0}, part[4] = {0, 0, 0, 0};
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int r0 = g; r0 < p.blocks; r0 += 8 * groups) {   // (eight loads under way)
      int4 n[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = r0 + u * groups;
        n[u] = make_int4(0, 0, 0, 0);
        if (r < p.blocks) n[u] = __ldcg(reinterpret_cast<const int4*>(p.hist + (int64_t)r * pitch) + v);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool mine = r0 + u * groups < b;
        sum[0] += n[u].x, sum[1] += n[u].y, sum[2] += n[u].z, sum[3] += n[u].w;
        if (mine) part[0] += n[u].x, part[1] += n[u].y, part[2] += n[u].z, part[3] += n[u].w;
      }
    }
    for (int r0 = g; last && r0 < p.blocks; r0 += 8 * groups) {
      float4 f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = r0 + u * groups;
        f[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < p.blocks) f[u] = __ldcg(reinterpret_cast<const float4*>(p.mass + (int64_t)r * pitch) + v);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) m[0] += f[u].x, m[1] += f[u].y, m[2] += f[u].z, m[3] += f[u].w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = 4 * v + k;
      if (c <= E) atomicAdd(&all[c], sum[k]);   // (integers: any order)
      if (c < E) {
        atomicAdd(&before[c], part[k]);
        if (last) mass[g * E + c] = m[k];
      }
    }
  }
  __syncthreads();
  if (last && (int)threadIdx.x < E) {
    for (int e = threadIdx.x; e < E; e += PLACE_THREADS)
      for (int h = 1; h < groups; ++h) mass[e] += mass[h * E + e];
  }
  if (warp == PLACE_THREADS / 32 - 1) scan_counts(all, starts, E, lane);
  __syncthreads();
  if (last) {
    if (warp == 0) write_loss(p, all, mass, starts[E], all[E], lane);
    for (int e = threadIdx.x; e <= E; e += PLACE_THREADS) {
      if (e < E) p.counts[e] = all[e];
      else *p.routed = all[E];
      p.offsets[e] = starts[e];
    }
    return;
  }
  int64_t lo, hi, t;
  token_range(p, b * p.warps, lo, t);
  token_range(p, b * p.warps + p.warps - 1, t, hi);
  for (int64_t i = lo * p.top + threadIdx.x; i < hi * p.top; i += PLACE_THREADS) {
    const int e = p.chosen[i];
    if (e >= 0) p.slots[i] += starts[e] + before[e];
  }
}

size_t place_smem(int experts) { return (size_t)(3 * experts + 2 + place_groups(experts) * experts) * sizeof(int); }

// dz_i = [renormalised: w_i (dw_i - sum_j w_j dw_j) at the chosen] + p_i (g_i - sum p g),
// g_e = dloss E c_e / (C n) [+ dw_e at the chosen].  A warp takes one token at a time.
template <int V, int DT>
__global__ void __launch_bounds__(512) route_grad_kernel(const __grid_constant__ RouteParams p) {
  constexpr int WARPS = 16;
  const int E = p.experts, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int n = *p.routed, rows = p.offsets[E];
  const float dloss = p.dloss_scale * (p.dloss != nullptr ? *p.dloss : 1.0f);
  const float per_row = rows > 0 && n > 0 ? dloss / (float)n * ((float)E / (float)rows) : 0.0f;
  float share[V];
#pragma unroll
  for (int v = 0; v < V; ++v) share[v] = lane + 32 * v < E ? per_row * (float)p.counts[lane + 32 * v] : 0.0f;
  const int64_t warps = (int64_t)gridDim.x * WARPS;
  for (int64_t t = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); t < p.tokens; t += warps) {
    float z[V], e[V], g[V], direct[V];
    load_logits<V, DT>(p, t, lane, z);
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
    uint32_t most = key_of(z[0]);
#pragma unroll
    for (int v = 1; v < V; ++v) most = max(most, key_of(z[v]));
    const float m = value_of(__reduce_max_sync(0xffffffffu, most));
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
        store_float_as(p.dlogits, DT, t * p.ldd + lane + 32 * v, any ? direct[v] + e[v] * (g[v] - s) : 0.0f);
  }
}

template <int DT, typename F>
cudaError_t with_values(int experts, F&& f) {
  if (experts <= 32) return f(TypeTag<1>{}, TypeTag<DT>{});
  if (experts <= 64) return f(TypeTag<2>{}, TypeTag<DT>{});
  if (experts <= 128) return f(TypeTag<4>{}, TypeTag<DT>{});
  if (experts <= 256) return f(TypeTag<8>{}, TypeTag<DT>{});
  if (experts <= 512) return f(TypeTag<16>{}, TypeTag<DT>{});
  return f(TypeTag<32>{}, TypeTag<DT>{});
}
template <typename F>
cudaError_t with_values(const RouteParams& p, F&& f) {
  if (p.dtype == GEMM_F32) return with_values<GEMM_F32>(p.experts, f);
  if (p.dtype == GEMM_F16) return with_values<GEMM_F16>(p.experts, f);
  return with_values<GEMM_BF16>(p.experts, f);
}

cudaError_t launch_routing(void (*kernel)(const RouteParams), int grid, int threads, size_t smem, cudaStream_t stream,
                           const RouteParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Bytes of shared memory of route_choose_kernel.
constexpr size_t choose_smem(int warps, size_t experts) { return (2 * (size_t)warps * experts + 3 * experts + 1) * sizeof(int); }

// The limit of shared memory is the function's on its device, not the launch's: threads that route
// over other numbers of experts at the same time share it, so it is set to the most that the
// instantiation can need and never to less.
template <int V, int DT>
cudaError_t launch_choose(const RouteParams& p, cudaStream_t stream) {
  constexpr int WARPS = warps_of(V);
  constexpr size_t MOST = choose_smem(WARPS, 32 * V);
  static_assert(MOST <= 232448, "shared memory budget");
  if constexpr (MOST > 48 * 1024) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> configured[64] = {};
    if (dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(route_choose_kernel<V, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MOST);
      if (e != cudaSuccess) return e;
      if (dev < 64) configured[dev].store(true, std::memory_order_release);
    }
  }
  return launch_routing(route_choose_kernel<V, DT>, p.blocks, 32 * WARPS, choose_smem(WARPS, (size_t)p.experts), stream, p);
}

}  // namespace

// CTAs that choose: one, and one launch, for up to two tokens per warp; else one per SM as long
// as a warp has a token.  One launch / two, us: 64 tokens, top 6 of 64 6.7 / 7.4, 128 tokens 10.0 / 7.5;
// 64 tokens, top 8 of 512 (half the warps) 23.1 / 12.3.
int route_warps(int64_t experts) { return warps_of(experts <= 32 ? 1 : experts <= 64 ? 2 : experts <= 128 ? 4 : 8); }
int route_blocks(int64_t tokens, int64_t experts, int sm_count) {
  const int warps = route_warps(experts);
  if (tokens <= 2 * warps) return 1;
  return (int)std::min<int64_t>(sm_count, (tokens + warps - 1) / warps);
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  const cudaError_t e = with_values(
      p, [&](auto v, auto dt) { return launch_choose<decltype(v)::value, decltype(dt)::value>(p, stream); });
  if (e != cudaSuccess || p.blocks == 1) return e;
  return launch_routing(route_place_kernel, p.blocks + 1, PLACE_THREADS, place_smem(p.experts), stream, p);
}

cudaError_t launch_route_grad(const RouteParams& p, int sm_count, cudaStream_t stream, int* ctas) {
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(4 * (int64_t)sm_count, (p.tokens + 15) / 16));
  *ctas = grid;
  return with_values(p, [&](auto v, auto dt) {
    return launch_routing(route_grad_kernel<decltype(v)::value, decltype(dt)::value>, grid, 512, 0, stream, p);
  });
}

}  // namespace gemmlib
