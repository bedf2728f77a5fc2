// q4_kernel.cu -- products with 4-bit weights (one scale, and zero point, per output
// column and group of K):
//     D[r, n] = act(alpha * sum_k A[r, k] * s[n, k / G] * (q[n, k] - z[n, k / G]) + bias[n]).
//
// A few rows (a decoding step): q4_kernel reads every weight once per 8 * NT rows
// and is bound by that reading.  q - z is an integer of at most 15 in magnitude, exact
// in fp16 and bf16, and so is its product with a 16-bit x in fp32; the sums over one
// scale group therefore run on mma.sync (weights as the 16-row operand, rows of A as
// the 8-column one: a single row costs the same instructions as eight, about 1.6 per
// weight, where fp32 FMAs on converted weights cost 2 and more), and the scale
// multiplies the group's fp32 sum.  Nothing but the result is rounded to 16 bits.
//   - A CTA takes 16 * MT columns; its 8 warps take every eighth 128-deep chunk of K
//     and add up through shared memory at the end, in a fixed order.
//   - Each warp streams its chunks with cp.async into its own ring (no CTA barrier
//     in the loop).  The copies' 16-byte pieces (32 weights) are XOR-swizzled by row,
//     so that a lane's word -- 8 consecutive k of one row -- comes out without bank
//     conflicts, and all four lanes of a row stay inside one scale group.
//   - Nibbles i and i + 4 of a word become one 16-bit pair by a mask and an OR that
//     puts them into the low mantissa bits of a constant (1024 or, shifted by four,
//     64 * 16 in fp16; 128 in bf16), and one add or FMA that takes that constant and
//     the zero point away, exactly.  x is paired the same way.
//
// Many rows (a prompt): the weights are written once as 16-bit values s * (q - z)
// into scratch and the products run on the tensor cores (seg_kernel.cu).
#include "expert.h"

namespace gemmlib {
namespace {

constexpr int WARPS = 8;
constexpr int CHUNK = 128;   // k per chunk: 64 bytes of a row

template <int MT, int NT>
struct Q4Cfg {
  static constexpr int ROWS = 16 * MT;
  static constexpr int STAGES = MT == 4 ? 3 : 4;
  static constexpr int STAGE_BYTES = ROWS * 64;
  static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr int PITCH = ROWS + 1;                          // floats per row of the reduction
  static constexpr int RED = WARPS * 8 * NT * PITCH * 4;
  static constexpr int SMEM = RING > RED ? RING : RED;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The constants that take the magic numbers and the zero point away.
struct ZeroConst {
  uint32_t lo, hi;   // for nibbles in bits 0-3 and (fp16) in bits 4-7 of each half
};
template <bool BF16>
__device__ __forceinline__ ZeroConst zero_const(uint32_t z) {
  if constexpr (BF16) return {0xC300C300u + z * 0x00010001u, 0u};              // -(128 + z)
  else return {0xE400E400u + z * 0x00010001u, 0xD400D400u + z * 0x00100010u};   // -(1024 + z), -(64 + z)
}

// The eight weights of a word as pairs (k, k + 4), k = 0..3: q - z.
template <bool BF16>
__device__ __forceinline__ void unpack(uint32_t w, const ZeroConst& z, uint32_t (&h)[4]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
      asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(h[i]) : "r"(v), "r"(0x3F803F80u), "r"(z.lo));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = w >> (8 * i);
      const uint32_t a = (u & 0x000f000fu) | 0x64006400u, b = (u & 0x00f000f0u) | 0x64006400u;
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h[2 * i]) : "r"(a), "r"(z.lo));
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[2 * i + 1]) : "r"(b), "r"(0x2C002C00u), "r"(z.hi));   // * 1/16
    }
  }
}

// BPG: 32-deep blocks of a chunk that share a scale (G a multiple of 32 * BPG).
template <int MT, int NT, int BPG, bool BF16>
__global__ void __launch_bounds__(32 * WARPS, NT >= 4 ? 1 : 2) q4_kernel(const __grid_constant__ Q4Params p) {
  using Cfg = Q4Cfg<MT, NT>;
  constexpr int SPC = 4 / BPG;   // scales per chunk and row
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * Cfg::STAGES * Cfg::STAGE_BYTES);
  pdl_launch_dependents();
  pdl_wait();
  const int e = (int)blockIdx.y;
  int lo, hi;
  group_range(p.g, e, lo, hi);
  if (lo == hi) return;
  const int64_t n0 = (int64_t)blockIdx.x * Cfg::ROWS;
  const uint8_t* q = p.q + e * p.stride_q + n0 * p.ldq;
  const char* scales = static_cast<const char*>(p.scales) + e * p.stride_s * dtype_bytes(p.scale_dtype);
  const uint8_t* zeros = p.zeros ? p.zeros + e * p.stride_z : nullptr;
  const uint16_t* A = static_cast<const uint16_t*>(p.A);
  const int row_bytes = (p.K + 1) / 2, chunks = (p.K + CHUNK - 1) / CHUNK;
  const int mine = chunks > warp ? (chunks - warp + WARPS - 1) / WARPS : 0;
  const int rows_left = (int)min((int64_t)Cfg::ROWS, p.N - n0);

  // This warp's i-th chunk into its ring.
  auto fetch = [&](int i) {
    if (i < mine) {
      const int c = warp + WARPS * i;
      const uint32_t st = ring + (uint32_t)(i % Cfg::STAGES * Cfg::STAGE_BYTES);
#pragma unroll
      for (int j = 0; j < 2 * MT; ++j) {
        const int row = (lane >> 2) + 8 * j, pc = lane & 3, off = c * 64 + pc * 16;
        const int bytes = row < rows_left ? max(0, min(16, row_bytes - off)) : 0;
        const uint32_t dst = st + (uint32_t)(row * 64 + ((pc ^ ((row >> 1) & 3)) << 4));
        const uint8_t* src = bytes > 0 ? q + row * p.ldq + off : p.q;
        if (p.vec_q) {
          cp_async16(dst, src, bytes);
        } else {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int u = 0; u < 16; ++u)
            if (u < bytes) w[u >> 2] |= (uint32_t)src[u] << (8 * (u & 3));
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  for (int tok0 = lo; tok0 < hi; tok0 += 8 * NT) {
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.0f;
#pragma unroll
    for (int i = 0; i < Cfg::STAGES; ++i) fetch(i);
    for (int i = 0; i < mine; ++i) {
      const int k0 = (warp + WARPS * i) * CHUNK;
      // x: row tok0 + 8 n + g, this lane's 8 k of each block, paired (k, k + 4).
      uint32_t x[4][NT][4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int tok = tok0 + 8 * n + g, k = k0 + 32 * b + 8 * t;
          uint32_t v[4] = {0u, 0u, 0u, 0u};
          if (tok < hi) {
            const uint16_t* src = A + (int64_t)tok * p.lda + k;
            if (p.vec_a && k + 8 <= p.K) {
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(src));
              v[0] = u.x;
              v[1] = u.y;
              v[2] = u.z;
              v[3] = u.w;
            } else {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                if (k + u < p.K) v[u >> 1] |= (uint32_t)src[u] << (16 * (u & 1));
            }
          }
          x[b][n][0] = __byte_perm(v[0], v[2], 0x5410);
          x[b][n][1] = __byte_perm(v[0], v[2], 0x7632);
          x[b][n][2] = __byte_perm(v[1], v[3], 0x5410);
          x[b][n][3] = __byte_perm(v[1], v[3], 0x7632);
        }
      float s[MT][2][SPC];
      uint32_t z[MT][2][SPC];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < SPC; ++j) {
            const int row = 16 * m + 8 * h + g, k = k0 + 32 * BPG * j;
            const bool ok = row < rows_left && k < p.K;
            const int64_t gk = k / p.group;
            s[m][h][j] = ok ? load_as_float(scales, p.scale_dtype, (n0 + row) * p.lds + gk) : 0.0f;
            z[m][h][j] = zeros && ok ? zeros[(n0 + row) * p.ldz + gk] & 15u : 8u;
          }
      asm volatile("cp.async.wait_group %0;" ::"n"(Cfg::STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t st = ring + (uint32_t)(i % Cfg::STAGES * Cfg::STAGE_BYTES);
#pragma unroll
      for (int j = 0; j < SPC; ++j) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float blk[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) blk[n][0] = blk[n][1] = blk[n][2] = blk[n][3] = 0.0f;
          const ZeroConst z0 = zero_const<BF16>(z[m][0][j]), z1 = zero_const<BF16>(z[m][1][j]);
#pragma unroll
          for (int bb = 0; bb < BPG; ++bb) {
            const int b = j * BPG + bb, row = 16 * m + g;
            // Rows g and g + 8 have the same swizzle.
            const uint32_t a = st + (uint32_t)(row * 64 + ((b ^ ((row >> 1) & 3)) << 4) + t * 4);
            uint32_t w0, w1, h0[4], h1[4];
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w0) : "r"(a) : "memory");
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w1) : "r"(a + 512u) : "memory");
            unpack<BF16>(w0, z0, h0);
            unpack<BF16>(w1, z1, h1);
            const uint32_t f0[4] = {h0[0], h1[0], h0[1], h1[1]}, f1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<BF16>(blk[n], f0, x[b][n][0], x[b][n][1]);
              mma16816<BF16>(blk[n], f1, x[b][n][2], x[b][n][3]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[m][n][0] = fmaf(s[m][0][j], blk[n][0], acc[m][n][0]);
            acc[m][n][1] = fmaf(s[m][0][j], blk[n][1], acc[m][n][1]);
            acc[m][n][2] = fmaf(s[m][1][j], blk[n][2], acc[m][n][2]);
            acc[m][n][3] = fmaf(s[m][1][j], blk[n][3], acc[m][n][3]);
          }
        }
      }
      __syncwarp();   // the stage's readers are done
      fetch(i + Cfg::STAGES);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();   // every warp is done with its ring: the space holds the warps' sums
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          red[(warp * 8 * NT + 8 * n + 2 * t + (c & 1)) * Cfg::PITCH + 16 * m + 8 * (c >> 1) + g] = acc[m][n][c];
    __syncthreads();
    const char* bias = static_cast<const char*>(p.epi.bias) + e * p.epi.stride_bias * dtype_bytes(p.epi.bias_dtype);
    for (int i = threadIdx.x; i < 8 * NT * Cfg::ROWS; i += 32 * WARPS) {
      const int tok = i / Cfg::ROWS, row = i % Cfg::ROWS;
      if (tok0 + tok >= hi || row >= rows_left) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += red[(w * 8 * NT + tok) * Cfg::PITCH + row];
      v *= p.epi.alpha;
      if (p.epi.bias_mode == GEMM_BIAS_COL) v += load_as_float(bias, p.epi.bias_dtype, n0 + row);
      if (p.epi.relu) v = fmaxf(v, 0.0f);
      store_float_as(p.epi.D, p.epi.d_dtype, (int64_t)(tok0 + tok) * p.epi.ldd + n0 + row, v);
    }
    __syncthreads();   // the sums are read before the next rows' chunks land
  }
}

// Weights as 16-bit values s * (q - z), K-major with pitch ldw (zeros past K); groups
// without rows are skipped.  Eight weights (one word) per thread and step.
template <bool BF16>
__global__ void __launch_bounds__(256) q4_dequant_kernel(const __grid_constant__ Q4Params p, uint16_t* out, int64_t ldw,
                                                         int64_t stride_w) {
  const int e = (int)blockIdx.y;
  int lo, hi;
  group_range(p.g, e, lo, hi);
  if (lo == hi) return;
  const uint8_t* q = p.q + e * p.stride_q;
  const char* scales = static_cast<const char*>(p.scales) + e * p.stride_s * dtype_bytes(p.scale_dtype);
  const uint8_t* zeros = p.zeros ? p.zeros + e * p.stride_z : nullptr;
  out += e * stride_w;
  const int64_t per_row = ldw / 8, total = (int64_t)p.N * per_row;
  const int row_bytes = (p.K + 1) / 2;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t n = i / per_row;
    const int k = (int)(i - n * per_row) * 8;
    const uint8_t* src = q + n * p.ldq + k / 2;
    uint32_t w = 0;
    if (p.vec_q && k / 2 + 4 <= row_bytes) {
      w = *reinterpret_cast<const uint32_t*>(src);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k / 2 + u < row_bytes) w |= (uint32_t)src[u] << (8 * u);
    }
    float s = 0.0f;
    int z = 8;
    if (k < p.K) {
      const int64_t gk = k / p.group;
      s = load_as_float(scales, p.scale_dtype, n * p.lds + gk);
      if (zeros) z = zeros[n * p.ldz + gk] & 15;
    }
    uint32_t o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float a = k + 2 * u < p.K ? s * (float)((int)((w >> (8 * u)) & 15) - z) : 0.0f;
      const float b = k + 2 * u + 1 < p.K ? s * (float)((int)((w >> (8 * u + 4)) & 15) - z) : 0.0f;
      if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[u]) : "f"(b), "f"(a));
      else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[u]) : "f"(b), "f"(a));
    }
    *reinterpret_cast<uint4*>(out + n * ldw + k) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int MT, int NT, int BPG, bool BF16>
cudaError_t launch_q4_t(const Q4Params& p, cudaStream_t stream) {
  using Cfg = Q4Cfg<MT, NT>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  static bool configured[64] = {};
  if (dev >= 64 || !configured[dev]) {
    err = cudaFuncSetAttribute(q4_kernel<MT, NT, BPG, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (err != cudaSuccess) return err;
    if (dev < 64) configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.N + Cfg::ROWS - 1) / Cfg::ROWS), (unsigned)p.g.count, 1);
  cfg.blockDim = dim3(32 * WARPS, 1, 1);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_kernel<MT, NT, BPG, BF16>, p);
}

template <int MT, int NT>
cudaError_t launch_q4_tile(const Q4Params& p, cudaStream_t stream) {
  const bool bf16 = p.ab_dtype == GEMM_BF16;
  if (p.group % 128 == 0) return bf16 ? launch_q4_t<MT, NT, 4, true>(p, stream) : launch_q4_t<MT, NT, 4, false>(p, stream);
  if (p.group % 64 == 0) return bf16 ? launch_q4_t<MT, NT, 2, true>(p, stream) : launch_q4_t<MT, NT, 2, false>(p, stream);
  return bf16 ? launch_q4_t<MT, NT, 1, true>(p, stream) : launch_q4_t<MT, NT, 1, false>(p, stream);
}

}  // namespace

cudaError_t launch_q4(const Q4Params& p, int mt, int nt, cudaStream_t stream) {
  if (nt >= 4) return mt >= 2 ? launch_q4_tile<2, 4>(p, stream) : launch_q4_tile<1, 4>(p, stream);
  if (nt == 2) return mt >= 2 ? launch_q4_tile<2, 2>(p, stream) : launch_q4_tile<1, 2>(p, stream);
  return mt >= 4 ? launch_q4_tile<4, 1>(p, stream) : mt >= 2 ? launch_q4_tile<2, 1>(p, stream) : launch_q4_tile<1, 1>(p, stream);
}

cudaError_t launch_q4_dequant(const Q4Params& p, void* out, int64_t ldw, int64_t stride_w, cudaStream_t stream) {
  const int64_t per = ((int64_t)p.N * (ldw / 8) + 255) / 256;
  const dim3 grid((unsigned)std::min<int64_t>(per, std::max(152, 4864 / p.g.count)), (unsigned)p.g.count);
  if (p.ab_dtype == GEMM_BF16)
    q4_dequant_kernel<true><<<grid, 256, 0, stream>>>(p, static_cast<uint16_t*>(out), ldw, stride_w);
  else
    q4_dequant_kernel<false><<<grid, 256, 0, stream>>>(p, static_cast<uint16_t*>(out), ldw, stride_w);
  return cudaGetLastError();
}

}  // namespace gemmlib
