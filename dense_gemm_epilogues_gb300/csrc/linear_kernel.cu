// linear_kernel.cu -- fully connected layers where the product has few tiles, and the passes
// around their gradients.
//
// linear_split_kernel: D = act(x W + b) + R for few rows (a decoding step, a short prompt).
// Bound by memory: every weight is read once, so the weights have to stream at the chip's
// rate, but 128 columns of D per CTA are 32 CTAs for a width of 4096.  So a cluster of up to
// eight CTAs shares a tile's K: each streams its part of the depth with TMA through a ring
// into one tensor-memory accumulator (weights on the M side, rows on the N side: the MMA's N
// is the row count rounded up to 16), the partial sums go to shared memory, and after one
// cluster barrier every CTA adds an equal share of the tile from all of them, in the order of
// K, through distributed shared memory, and finishes it.  No scratch, no counters; two CTAs
// per SM, so that one's start and end hide behind the other's stream.
//
// Measured (graph replays, weights from HBM): 1 row, 4096 to 11008 17.4 us for 90 MB, of which
// 13.3 at the copy rate; the slope over larger widths is 7 TB/s, and 4.2 us go to the launch,
// the first loads' latency and the last sums. 4096 to 4096 9.5 us (four CTAs per tile; one
// 20), 7 rows of 11008 to 4096 18.4, 128 rows of 1024 to 1024 6.5.
//
// act_grad_kernel: dz = dy act'(z) in the operands' type, and its column sums (the bias's
// gradient) from the unrounded values: one pass at memory speed; a column's sums are added
// over row blocks by column_sums_kernel in one order.  4096 x 11008 with GELU: 46 us for both,
// 5.9 TB/s; with loads into registers instead of copies ahead 64.
// dz is rounded because it is an operand of two tensor-core products, which take 16 bits of
// the other operand's type: keeping what is rounded off would need a second half of dz, and
// with it each product twice (422 of 468 us at that size).  It costs half a step per term:
// against 64 bits, dx and dw in bf16 are off by 0.0023 of their norm instead of the 0.0017 that
// rounding the results alone leaves.
//
// Every wait is bounded, as in tc_kernel.cu.
#include "layer.h"

namespace gemmlib {
namespace {

constexpr int THREADS = 320;                       // producer warp, MMA warp, eight that read the accumulator
constexpr int A_BYTES = 128 * TC_BK * 2;           // 16 KiB: 128 columns of weights, 64 deep
constexpr uint32_t MN_BOX_BYTES = 64 * TC_BK * 2;  // MN-major box: 64 columns, 64 deep
constexpr int MAX_STAGES = 8;

// A limit below a microsecond, the step of the timer and less than the hardware may suspend a
// try for, gives a wait one look: these loads mostly land within a single try, which no limit
// would ever end.
constexpr uint64_t ONE_LOOK_NS = 1000;

__device__ __forceinline__ bool mbar_look(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
  uint32_t ok;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok != 0) return true;
  atomicCAS(wc.err, 0, (int32_t)GEMM_ERR_TIMEOUT);
  *wc.abort = 1;
  __threadfence_block();
  return false;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
  const bool ok = wc.timeout_ns >= ONE_LOOK_NS ? mbar_wait(bar, parity, wc) : mbar_look(bar, parity, wc);
  return __all_sync(0xffffffffu, ok) != 0;
}

__device__ __forceinline__ float4 lds_cluster(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// Four entries of a row (n of them exist) of a type.
template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, int n, bool vec, float (&x)[4]) {
  if (vec && n >= 4) {
    if constexpr (DT == GEMM_F32) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      const uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int h = 0; h < 2; ++h) unpack2<DT>(w[h], x[2 * h], x[2 * h + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = j < n ? load_as_float(p, DT, i + j) : 0.0f;
  }
}
template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, int n, bool vec, const float (&x)[4]) {
  if (vec && n >= 4) {
    if constexpr (DT == GEMM_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) w[h] = pack2<DT>(x[2 * h], x[2 * h + 1]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(w[0], w[1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) store_float_as(p, DT, i + j, x[j]);
  }
}

// Grid: (splits, column tiles, row tiles); a cluster is the splits of one tile.
template <bool A_MN>
__global__ void __launch_bounds__(THREADS) linear_split_kernel(const __grid_constant__ LinearSplitParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;   // the same offset in all CTAs of the cluster
  const uint32_t b_bytes = (uint32_t)(p.box_rows * TC_BK * 2), stage_bytes = A_BYTES + b_bytes;
  __shared__ uint64_t bars[2 * MAX_STAGES + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t abort_word;
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(MAX_STAGES + s); };
  const uint32_t done_bar = bar0 + 8u * (2 * MAX_STAGES);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int split = blockIdx.x, splits = gridDim.x;
  const int64_t m0 = (int64_t)blockIdx.y * 128;                 // first column of D
  const int64_t r0 = (int64_t)blockIdx.z * p.box_rows;          // first row
  const int rows = (int)min((int64_t)p.box_rows, p.rows - r0);
  const int n_mma = (rows + 15) & ~15;
  const uint32_t tmem_cols = n_mma <= 32 ? 32u : n_mma <= 64 ? 64u : 128u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(done_bar, 1);
    abort_word = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  const int num_kb = (int)((p.K + TC_BK - 1) / TC_BK);
  const int kb0 = (int)((int64_t)split * num_kb / splits), kb1 = (int)((int64_t)(split + 1) * num_kb / splits);
  pdl_launch_dependents();
  if (warp == 0 && elect_one()) {
    tma_prefetch_desc(&p.tmW);
    tma_prefetch_desc(&p.tmX);
  }
  __syncwarp();
  pdl_wait();
  const WaitCtx wc{&abort_word, p.err, p.timeout_ns};

  if (warp == 0) {
    const bool one = elect_one();
    int issued = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++issued) {
      const int s = issued % p.stages;
      if (!warp_wait(empty_bar(s), ((uint32_t)(issued / p.stages) & 1u) ^ 1u, wc)) break;
      if (one) {
        const uint32_t fb = full_bar(s), sa = base + (uint32_t)s * stage_bytes;
        mbar_expect_tx(fb, stage_bytes);
        if constexpr (A_MN) {
          tma_load_3d(sa, &p.tmW, (int)m0, kb * TC_BK, 0, fb);
          tma_load_3d(sa + MN_BOX_BYTES, &p.tmW, (int)m0 + 64, kb * TC_BK, 0, fb);
        } else {
          tma_load_3d(sa, &p.tmW, kb * TC_BK, (int)m0, 0, fb);
        }
        tma_load_3d(sa + A_BYTES, &p.tmX, kb * TC_BK, (int)r0, 0, fb);
      }
      __syncwarp();
    }
    // Every copy has landed before the ring is written below.
    if (one)
      for (int i = max(0, issued - p.stages); i < issued; ++i)
        drain_wait(full_bar(i % p.stages), (uint32_t)(i / p.stages) & 1u, p.timeout_ns);
    __syncwarp();
  } else if (warp == 1) {
    const bool one = elect_one();
    const uint32_t idesc = p.idesc | ((uint32_t)(n_mma >> 3) << 17);
    for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
      const int s = i % p.stages;
      if (!warp_wait(full_bar(s), (uint32_t)(i / p.stages) & 1u, wc)) break;
      tc_fence_after();
      if (one) {
        const uint32_t sa = base + (uint32_t)s * stage_bytes;
        const uint64_t ad = A_MN ? smem_desc_sw128(sa, MN_BOX_BYTES, 1024) : smem_desc_sw128(sa, 16, 1024);
        const uint64_t bd = smem_desc_sw128(sa + A_BYTES, 16, 1024);
#pragma unroll
        for (int q = 0; q < TC_BK / 16; ++q)   // (past K both operands read as zero)
          tc_mma_f16(tmem_base, ad + (A_MN ? q * 2048u >> 4 : q * 32u >> 4), bd + (q * 32u >> 4), idesc, i > 0 || q > 0 ? 1u : 0u);
        tc_commit(empty_bar(s));
      }
      __syncwarp();
    }
    if (one) {
      tc_commit(done_bar);
      drain_wait(done_bar, 0, p.timeout_ns);
    }
    __syncwarp();
  }
  // This CTA's share of the tile: four columns of a row at a time, a thread always the same
  // columns.  The bias and the first of the residual come in while the weights stream.
  const int items = rows * 32, lo = split * items / splits, hi = (split + 1) * items / splits;
  const int first = lo + (int)threadIdx.x, col = (first & 31) * 4;
  const int64_t d = m0 + col;
  const int n = (int)max((int64_t)0, min((int64_t)4, p.epi_n - d));
  with_type(p.epi.d_dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    constexpr int U = 2;   // items under way (four cost every call 0.6 us: more code to fetch)
    float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f}, res[U][4];
    if (p.epi.bias_mode == GEMM_BIAS_COL) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) bias[j] = load_as_float(p.epi.bias, p.epi.bias_dtype, d + j);
    }
    auto load_residual = [&](int i0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * THREADS;
        if (p.linear.residual != nullptr && i < hi) {
          load4<DT>(p.linear.residual, (r0 + (i >> 5)) * p.linear.ldr + d, n, p.vec, res[u]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) res[u][j] = 0.0f;
        }
      }
    };
    load_residual(first);
    // All MMAs are complete (warp 1 has waited for them), all copies have landed: the ring is free.
    __syncthreads();
    tc_fence_after();
    if (warp >= 2) {
      const int q = warp & 3;
      for (int c = (warp - 2) >> 2 << 5; c < n_mma; c += 64) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)c, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j < n_mma)   // [row][column of D]: a warp's lanes lie side by side
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + (uint32_t)(((c + j) * 128 + q * 32 + lane) * 4)), "r"(r[j]) : "memory");
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_sync();
    for (int i0 = first; i0 < hi; i0 += U * THREADS) {
      float x[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[u][j] = 0.0f;
      for (int s = 0; s < splits; ++s) {   // in the order of K
        const uint32_t from = mapa_shared(base, (uint32_t)s);
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i0 + u * THREADS < hi) v[u] = lds_cluster(from + (uint32_t)((((i0 + u * THREADS) >> 5) * 128 + col) * 4));
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i0 + u * THREADS < hi) x[u][0] += v[u].x, x[u][1] += v[u].y, x[u][2] += v[u].z, x[u][3] += v[u].w;
      }
      if (p.linear.pre != nullptr || p.epi.bias_mode == GEMM_BIAS_COL) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[u][j] += bias[j];
          const int i = i0 + u * THREADS;
          if (p.linear.pre != nullptr && i < hi) store4<DT>(p.linear.pre, (r0 + (i >> 5)) * p.linear.ldp + d, n, p.vec, x[u]);
        }
      }
      with_act(p.linear.act, [&](auto act) {
#pragma unroll
        for (int u = 0; u < U; ++u) activate<decltype(act)::value>(x[u]);
      });
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * THREADS;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[u][j] += res[u][j];
        if (i < hi) store4<DT>(p.epi.D, (r0 + (i >> 5)) * p.epi.ldd + d, n, p.vec, x[u]);
      }
      if (p.linear.residual != nullptr && i0 + U * THREADS < hi) load_residual(i0 + U * THREADS);
    }
  });
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // no CTA leaves while another may read its shared memory
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, tmem_cols);
}

// ------------------------- the gradient's elementwise pass -------------------------

constexpr int GRAD_THREADS = 256, GRAD_COLS = 256;   // a warp takes a row's 256 columns, eight per lane
constexpr int GRAD_WARPS = GRAD_THREADS / 32, GRAD_STAGES = 4;   // rows of a warp under way

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// At most N of the newest groups are still under way.
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// Eight entries of a row (n of them exist) as they lie in memory.
__device__ __forceinline__ uint4 load8_raw(const void* p, int64_t i, int n, bool vec) {
  const uint16_t* src = static_cast<const uint16_t*>(p) + i;
  if (vec && n >= 8) return *reinterpret_cast<const uint4*>(src);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j / 2] |= (uint32_t)src[j] << (16 * (j % 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT>
__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) unpack2<DT>(w[h], x[2 * h], x[2 * h + 1]);
}

// Grid: (256-column strips, row blocks).  A lane copies its pieces of four rows ahead into
// shared memory of its own (nobody else's, so no barrier): 32 warps per SM then have 128 KB
// under way, which registers do not hold beside the derivative's.
template <int DT>
__global__ void __launch_bounds__(GRAD_THREADS, 4) act_grad_kernel(const __grid_constant__ ActGradParams p) {
  __shared__ __align__(16) uint8_t ring[GRAD_STAGES][2][GRAD_THREADS * 16];
  __shared__ float sums[GRAD_WARPS][GRAD_COLS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t c = (int64_t)blockIdx.x * GRAD_COLS + lane * 8;
  const int n = (int)max((int64_t)0, min((int64_t)8, p.N - c));
  const int64_t lo = (int64_t)blockIdx.y * p.block_rows, hi = min(p.M, lo + p.block_rows);
  float sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
  with_act(p.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    const bool async = p.vec && n == 8;
    auto slot = [&](int stage, int which) { return smem_u32(&ring[stage][which][threadIdx.x * 16]); };
    auto copy = [&](int64_t r, int stage) {
      if (async && r < hi) {
        copy16_async(slot(stage, 0), static_cast<const uint16_t*>(p.dy) + r * p.ldy + c);
        if constexpr (ACT != ACT_NONE) copy16_async(slot(stage, 1), static_cast<const uint16_t*>(p.pre) + r * p.ldp + c);
      }
      copies_commit();
    };
    const int64_t first = n > 0 ? lo + warp : hi;
#pragma unroll
    for (int s = 0; s < GRAD_STAGES; ++s) copy(first + s * GRAD_WARPS, s);
    int stage = 0;
#pragma unroll 1
    for (int64_t r = first; r < hi; r += GRAD_WARPS) {
      copies_wait<GRAD_STAGES - 1>();
      float g[8];
      widen8<DT>(async ? lds16(slot(stage, 0)) : load8_raw(p.dy, r * p.ldy + c, n, p.vec), g);
      if constexpr (ACT != ACT_NONE) {
        float z[8];
        uint32_t w[4];
        widen8<DT>(async ? lds16(slot(stage, 1)) : load8_raw(p.pre, r * p.ldp + c, n, p.vec), z);
        copy(r + GRAD_STAGES * GRAD_WARPS, stage);
        activate_grad<ACT>(z, g);
#pragma unroll
        for (int h = 0; h < 4; ++h)   // (dz's rows are padded to whole pieces; what lies past N is 0)
          w[h] = pack2<DT>(g[2 * h], g[2 * h + 1]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dz) + r * p.ldz + c) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        copy(r + GRAD_STAGES * GRAD_WARPS, stage);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += g[j];
      stage = stage + 1 == GRAD_STAGES ? 0 : stage + 1;
    }
    copies_wait<0>();
  });
  if (p.partials == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[warp][lane * 8 + j] = sum[j];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * GRAD_COLS + threadIdx.x;
  if (col < p.N) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < GRAD_WARPS; ++w) s += sums[w][threadIdx.x];
    p.partials[(int64_t)blockIdx.y * p.N + col] = s;
  }
}

// out[c] = the sum of partials[b][c] over the row blocks, in one order: a CTA takes 32 columns,
// its warps equal parts of the blocks.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* partials, int blocks, int64_t N, float* out) {
  __shared__ float sums[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const int per = (blocks + 7) / 8, lo = warp * per, hi = min(blocks, lo + per);
  float s = 0.0f;
  for (int b = lo; b < hi; b += 8) {   // (eight loads under way)
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = b + u < hi && c < N ? partials[(int64_t)(b + u) * N + c] : 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < N) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][lane];
    out[c] = s;
  }
}

template <bool A_MN>
cudaError_t launch_split(const LinearSplitParams& p, int splits, cudaStream_t stream) {
  const size_t smem = 1024 + (size_t)p.stages * (size_t)(A_BYTES + p.box_rows * TC_BK * 2);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool configured[64] = {};
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(linear_split_kernel<A_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, SPLIT_SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)splits, (unsigned)((p.epi_n + 127) / 128), (unsigned)((p.rows + p.box_rows - 1) / p.box_rows));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_split_kernel<A_MN>, p);
}

}  // namespace

int split_stages(int box_rows) {
  return std::min(MAX_STAGES, (SPLIT_SMEM - 1024) / (A_BYTES + box_rows * TC_BK * 2));
}

cudaError_t launch_linear_split(const LinearSplitParams& p, bool a_mn, int splits, cudaStream_t stream) {
  return a_mn ? launch_split<true>(p, splits, stream) : launch_split<false>(p, splits, stream);
}

cudaError_t launch_act_grad(const ActGradParams& p, int dtype, int blocks, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.N + GRAD_COLS - 1) / GRAD_COLS), (unsigned)blocks);
  return dtype == GEMM_F16 ? launch_dependent(act_grad_kernel<GEMM_F16>, grid, GRAD_THREADS, stream, p)
                           : launch_dependent(act_grad_kernel<GEMM_BF16>, grid, GRAD_THREADS, stream, p);
}

cudaError_t launch_column_sums(const float* partials, int blocks, int64_t N, float* out, cudaStream_t stream) {
  return launch_dependent(column_sums_kernel, dim3((unsigned)((N + 31) / 32)), 256, stream, partials, blocks, N, out);
}

}  // namespace gemmlib
