// q4_kernel.cu -- products with 4-bit weights (one scale, and zero point, per output
// column and group of K):
//     D[r, n] = act(alpha * sum_k A[r, k] * s[n, k / G] * (q[n, k] - z[n, k / G]) + bias[n]).
//
// A few rows (a decoding step): q4_kernel reads every weight once per 8 * NT rows.
// q - z is an integer of at most 15 in magnitude, exact in fp16 and bf16, and so is
// its product with a 16-bit x in fp32; the sums over one scale group therefore run on
// mma.sync (weights as the 16-row operand, rows of A as the 8-column one: a single
// row costs the same instructions as eight), and the scale multiplies the group's
// fp32 sum.  Nothing but the result is rounded to 16 bits.
// At 6.8 TB/s an SM takes 47 weights per clock, so about 2.7 lane instructions per
// weight are the most that keep up; the layout is made to save instructions:
//   - One TMA copy brings a warp's next chunk (128 k of the CTA's columns, 64-byte
//     rows with the 64-byte swizzle), two more the rows of A; each warp has its own
//     ring and barriers, and no CTA barrier stands in its loop.
//   - A lane's word is 8 consecutive k of one column, read without bank conflicts, and
//     all four lanes of a row stay inside one scale group.
//   - Nibbles i and i + 4 of a word become one 16-bit pair by one mask-and-or that
//     puts them into the low mantissa bits of a constant (1024 or, shifted by four,
//     64 * 16 in fp16; 128 in bf16) and one add or FMA that takes that constant and
//     the zero point away, exactly.  x is paired the same way, once for all columns.
// A CTA's 8 warps take every eighth chunk of K and add up through shared memory at
// the end, in a fixed order.
// Measured (graph replays): one row of 4096 to 4096 7.2 us, of 4096 to 11008 11.9 us (2 TB/s
// of packed weights); 16 rows 18.5, 32 rows 25 us; 24 rows over 16 experts, 2048 to 1408,
// 12.4 us.  Not bound by HBM (one row of 4096 to 11008 reads 1.5 TB/s): half of the issue
// slots are empty, so most of it is latency (launch, barriers, a warp's few chunks, the
// reduction), and the busy half is 5 to 7 lane instructions per weight.
//
// Many rows (a prompt): the weights are written once as 16-bit values s * (q - z)
// into scratch and the products run on the tensor cores (seg_kernel.cu).
#include "expert.h"

namespace gemmlib {
namespace {

constexpr int CHUNK = 128;   // k per chunk: 64 bytes of a column of weights, 256 bytes of a row of A

constexpr int WARPS = 8;

template <int MT, int NT>
struct Q4Cfg {
  static constexpr int W_BYTES = 16 * MT * 64, X_BYTES = 8 * NT * 256;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int CTAS = NT >= 4 ? 1 : 2;                    // resident per SM
  static constexpr int FIT = (227 * 1024 / CTAS - 2048) / (WARPS * STAGE_BYTES);
  static constexpr int STAGES = FIT >= 4 ? 4 : FIT;
  static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr int PITCH = 16 * MT + 1;                       // floats per row of the reduction
  static constexpr int RED = WARPS * 8 * NT * PITCH * 4;
  static constexpr int SMEM = 1024 + (RING > RED ? RING : RED);
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory budget");
};

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
// The same into a fresh accumulator.
template <bool BF16>
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
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

// Wait for a ring barrier, up to the plan's bound (then the error word is set and false
// returned); q4_drain waits at least a second and reports nothing.
__device__ __forceinline__ bool q4_wait(uint32_t bar, uint32_t parity, const Q4Params& p) {
  bool done = mbar_try_wait(bar, parity);
  if (!done) {
    const uint64_t t0 = globaltimer_ns();
    while (!(done = mbar_try_wait(bar, parity)))
      if (globaltimer_ns() - t0 > p.timeout_ns) break;
  }
  done = __all_sync(0xffffffffu, done) != 0;
  if (!done && (threadIdx.x & 31) == 0) atomicCAS(p.g.err, 0, (int32_t)GEMM_ERR_TIMEOUT);
  return done;
}
__device__ __forceinline__ void q4_drain(uint32_t bar, uint32_t parity, const Q4Params& p) {
  const uint64_t bound = p.timeout_ns > 1000000000ull ? p.timeout_ns : 1000000000ull, t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > bound) return;
}

// Eight consecutive x as pairs (k, k + 4), k = 0..3.
__device__ __forceinline__ void pair_up(const uint4& v, uint32_t (&x)[4]) {
  x[0] = __byte_perm(v.x, v.z, 0x5410);
  x[1] = __byte_perm(v.x, v.z, 0x7632);
  x[2] = __byte_perm(v.y, v.w, 0x5410);
  x[3] = __byte_perm(v.y, v.w, 0x7632);
}

// BPG: 32-deep blocks of a chunk that share a scale (G a multiple of 32 * BPG).  ZP: zero
// points (8 otherwise).  S32: scales of four bytes (16-bit ones otherwise).
template <int MT, int NT, int BPG, bool ZP, bool S32, bool BF16>
__global__ void __launch_bounds__(32 * WARPS, Q4Cfg<MT, NT>::CTAS) q4_kernel(const __grid_constant__ Q4Params p) {
  using Cfg = Q4Cfg<MT, NT>;
  constexpr int SPC = 4 / BPG;                        // scales per chunk and column
  constexpr int SW = S32 ? SPC : SPC == 4 ? 2 : 1;    // words that hold them
  constexpr int ES = S32 ? 4 : 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[WARPS * Cfg::STAGES];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);   // swizzle patterns start on 1024 bytes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * Cfg::STAGES * Cfg::STAGE_BYTES);
  const uint32_t bar0 = smem_u32(&bars[warp * Cfg::STAGES]);
  if (lane == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) mbar_init(bar0 + 8u * s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (warp == 0) {
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_x);
    }
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();
  const int e = (int)blockIdx.y, R = p.cta_rows;
  int lo, hi;
  group_range(p.g, e, lo, hi);
  if (lo == hi) return;
  // The last CTA's columns reach back so that every CTA has R of them (the shared ones
  // are written twice, with the same bits).
  const int n0 = min((int)blockIdx.x * R, p.N - R);
  const int chunks = (p.K + CHUNK - 1) / CHUNK;
  const int mine = chunks > warp ? (chunks - warp + WARPS - 1) / WARPS : 0;
  const char* s_base = static_cast<const char*>(p.scales) + (e * p.stride_s + n0 * p.lds) * ES;
  const uint8_t* z_base = ZP ? p.zeros + e * p.stride_z + n0 * p.ldz : nullptr;
  // All scales and zero points of this CTA's columns towards L2: the loop reads them a
  // chunk ahead, which covers L2's latency and not DRAM's.
  if (p.K > 0) {
    const int s_bytes = p.scale_cols * ES;
    for (int r = warp; r < R; r += WARPS) {
      for (int off = lane * 128; off < s_bytes + 128; off += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(s_base + r * p.lds * ES + min(off, s_bytes - ES)));
      if constexpr (ZP)
        for (int off = lane * 128; off < p.scale_cols + 128; off += 32 * 128)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(z_base + r * p.ldz + min(off, p.scale_cols - 1)));
    }
  }
  // This lane's columns: g and g + 8 of each tile of 16 (one past the CTA's reads the
  // last one's scales; its sums are not stored).
  int s_off[MT][2], z_off[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = min(16 * m + 8 * h + g, R - 1);
      s_off[m][h] = row * (int)p.lds * ES;
      z_off[m][h] = ZP ? row * (int)p.ldz : 0;
    }
  // A lane's 16-byte piece of block b of a column lies at piece b ^ ((row >> 1) & 3) of
  // the row (64-byte swizzle; the same for rows g, g + 8, ...), its 8 k of a row of A at
  // piece (4 b + t) % 8 ^ g of a 128-byte row (128-byte swizzle).
  uint32_t w_off[4], x_off[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    w_off[b] = (uint32_t)(g * 64 + ((b ^ ((g >> 1) & 3)) << 4) + t * 4);
    x_off[b] = (uint32_t)(Cfg::W_BYTES + (b >> 1) * (NT * 1024) + g * 128 + ((((b & 1) * 4 + t) ^ g) << 4));
  }

  bool ok = true;
  int issued = 0;   // chunks this warp has asked for since the kernel began
  for (int tok0 = lo; tok0 < hi; tok0 += 8 * NT) {
    const int first = issued;
    // This warp's i-th chunk into its ring.
    auto fetch = [&](int i) {
      if (i < mine && ok) {
        if (lane == 0) {
          const uint32_t st = (uint32_t)((first + i) % Cfg::STAGES), bar = bar0 + 8u * st, dst = ring + st * Cfg::STAGE_BYTES;
          const int c = warp + WARPS * i;
          mbar_expect_tx(bar, (uint32_t)(R * 64 + Cfg::X_BYTES));
          tma_load_3d(dst, &p.tm_q, c * 64, n0, p.q_batched ? e : 0, bar);
          tma_load_2d(dst + Cfg::W_BYTES, &p.tm_x, c * CHUNK, tok0, bar);
          tma_load_2d(dst + Cfg::W_BYTES + NT * 1024, &p.tm_x, c * CHUNK + 64, tok0, bar);
        }
        issued = first + i + 1;
      }
    };
    // A chunk's scales and zero points of this lane's columns, in one to four words each.
    uint32_t s_raw[MT][2][SW], z_raw[MT][2];
    auto fetch_scales = [&](int i) {
      const int c = warp + WARPS * i;
      const bool whole = SPC == 1 || (p.vec_s && c * CHUNK + CHUNK <= p.K);
      const int g0 = SPC > 1 ? c * SPC : p.group_shift >= 0 ? c >> p.group_shift : c / p.group_units;
      const char* sp = s_base + (int64_t)g0 * ES;
      const uint8_t* zp = ZP ? z_base + g0 : nullptr;
      if (whole) {   // a chunk's scales lie together (and aligned)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const char* a = sp + s_off[m][h];
            if constexpr (S32) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(a));
              s_raw[m][h][0] = v.x, s_raw[m][h][1 % SW] = v.y, s_raw[m][h][2 % SW] = v.z, s_raw[m][h][3 % SW] = v.w;
            } else if constexpr (SPC == 4) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(a));
              s_raw[m][h][0] = v.x, s_raw[m][h][1 % SW] = v.y;
            } else if constexpr (SPC == 2) {
              s_raw[m][h][0] = __ldg(reinterpret_cast<const uint32_t*>(a));
            } else {
              s_raw[m][h][0] = __ldg(reinterpret_cast<const uint16_t*>(a));
            }
            if constexpr (ZP) {
              const uint8_t* za = zp + z_off[m][h];
              z_raw[m][h] = SPC == 4 ? __ldg(reinterpret_cast<const uint32_t*>(za))
                            : SPC == 2 ? (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(za)) : (uint32_t)__ldg(za);
            }
          }
      } else {
#pragma unroll 1
        for (int j = 0; j < SPC; ++j) {
          const int unit = c * SPC + j;   // of 32 * BPG k
          const int gk = unit * 32 * BPG < p.K ? (p.group_shift >= 0 ? unit >> p.group_shift : unit / p.group_units) : 0;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const char* a = s_base + s_off[m][h] + (int64_t)gk * ES;
              const uint32_t v = S32 ? __ldg(reinterpret_cast<const uint32_t*>(a)) : (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(a));
#pragma unroll
              for (int u = 0; u < SW; ++u) {
                const uint32_t keep = j == 0 ? 0u : s_raw[m][h][u];
                s_raw[m][h][u] = (S32 ? j : j >> 1) == u ? (S32 || !(j & 1) ? v : keep | v << 16) : keep;
              }
              if constexpr (ZP) z_raw[m][h] = (j == 0 ? 0u : z_raw[m][h]) | (uint32_t)__ldg(z_base + z_off[m][h] + gk) << (8 * j);
            }
        }
      }
    };

    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][n][c] = 0.0f;
    for (int i = 0; i < Cfg::STAGES; ++i) fetch(i);
    if (mine > 0) fetch_scales(0);
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
      uint32_t s_cur[MT][2][SW], z_cur[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int u = 0; u < SW; ++u) s_cur[m][h][u] = s_raw[m][h][u];
          if constexpr (ZP) z_cur[m][h] = z_raw[m][h];
        }
      if (i + 1 < mine) fetch_scales(i + 1);
      const uint32_t si = (uint32_t)((first + i) % Cfg::STAGES), parity = (uint32_t)((first + i) / Cfg::STAGES) & 1u;
      if (!ok || !q4_wait(bar0 + 8u * si, parity, p)) {
        ok = false;
        break;
      }
      const uint32_t st = ring + si * Cfg::STAGE_BYTES;
      // x: row 8 n + g, this lane's 8 k of each block, paired (k, k + 4).
      uint32_t x[4][NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(st + x_off[b] + (uint32_t)(n * 1024)) : "memory");
          pair_up(v, x[b][n]);
        }
#pragma unroll
      for (int j = 0; j < SPC; ++j) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float s[2];
          ZeroConst zc[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (S32) {
              s[h] = __uint_as_float(s_cur[m][h][j % SW]);
            } else {
              const uint32_t w = s_cur[m][h][(j >> 1) % SW];
              s[h] = p.scale_dtype == GEMM_BF16 ? __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16)
                                                : __half2float(__ushort_as_half((uint16_t)(j & 1 ? w >> 16 : w)));
            }
            zc[h] = zero_const<BF16>(ZP ? (z_cur[m][h] >> (8 * j)) & 15u : 8u);
          }
          float blk[NT][4];
#pragma unroll
          for (int bb = 0; bb < BPG; ++bb) {
            const int b = j * BPG + bb;
            uint32_t w0, w1, h0[4], h1[4];
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w0) : "r"(st + w_off[b] + 1024u * m) : "memory");
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w1) : "r"(st + w_off[b] + 1024u * m + 512u) : "memory");
            unpack<BF16>(w0, zc[0], h0);
            unpack<BF16>(w1, zc[1], h1);
            const uint32_t f0[4] = {h0[0], h1[0], h0[1], h1[1]}, f1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (bb == 0) mma16816_first<BF16>(blk[n], f0, x[b][n][0], x[b][n][1]);
              else mma16816<BF16>(blk[n], f0, x[b][n][0], x[b][n][1]);
              mma16816<BF16>(blk[n], f1, x[b][n][2], x[b][n][3]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[m][n][0] = fmaf(s[0], blk[n][0], acc[m][n][0]);
            acc[m][n][1] = fmaf(s[0], blk[n][1], acc[m][n][1]);
            acc[m][n][2] = fmaf(s[1], blk[n][2], acc[m][n][2]);
            acc[m][n][3] = fmaf(s[1], blk[n][3], acc[m][n][3]);
          }
        }
      }
      __syncwarp();   // the stage's readers are done
      fetch(i + Cfg::STAGES);
    }
    if (!ok) {   // a wait ran out: let this warp's copies land before the CTA can leave
      for (int i = max(0, issued - Cfg::STAGES); i < issued; ++i)
        q4_drain(bar0 + 8u * (uint32_t)(i % Cfg::STAGES), (uint32_t)(i / Cfg::STAGES) & 1u, p);
    }
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
    const int row = threadIdx.x & 63, toks = min(8 * NT, hi - tok0);
    if (row < R) {
      float b = 0.0f;
      if (p.epi.bias_mode == GEMM_BIAS_COL) b = load_as_float(bias, p.epi.bias_dtype, n0 + row);
      for (int tok = threadIdx.x >> 6; tok < toks; tok += WARPS / 2) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += red[(w * 8 * NT + tok) * Cfg::PITCH + row];
        v = fmaf(v, p.epi.alpha, b);
        if (p.epi.relu) v = relu_keep_nan(v);
        store_float_as(p.epi.D, p.epi.d_dtype, (int64_t)(tok0 + tok) * p.epi.ldd + n0 + row, v);
      }
    }
    if (tok0 + 8 * NT < hi) {
      // The sums are read before the next rows' chunks land on them.
      fence_proxy_async_smem();
      __syncthreads();
    }
  }
}

// A word's weights as neighbours (2 k, 2 k + 1): its bytes and those of the word shifted
// by a nibble side by side.
template <bool BF16>
__device__ __forceinline__ void unpack_pairs(uint32_t w, uint32_t zero, uint32_t (&h)[4]) {
  const uint32_t odd = w >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = (__byte_perm(w, odd, 0x0400u + 0x0101u * (uint32_t)i) & 0x000f000fu) | (BF16 ? 0x43004300u : 0x64006400u);
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(h[i]) : "r"(v), "r"(0x3F803F80u), "r"(zero));
    else asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(v), "r"(zero));
  }
}

// Per column the power of two 2^(e - 11), 2^e <= its largest scale < 2^(e + 1): scales of a
// wider type than fp16 divided by it give weights below 15 * 2^12 < 65504 that are normal
// fp16 numbers down to 2^-25 of the column's largest, so decoding them into fp16 rounds each
// once, whatever the scales' size.  One warp per column; infinite and NaN scales are passed
// over (their weights are infinite or NaN in any case).
__global__ void __launch_bounds__(256) q4_range_kernel(const __grid_constant__ Q4Params p, float* out) {
  pdl_wait();
  const int e = (int)blockIdx.y, n = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
  int lo, hi;
  group_range(p.g, e, lo, hi);
  if (lo == hi || n >= p.N) return;
  const char* scales = static_cast<const char*>(p.scales) + e * p.stride_s * dtype_bytes(p.scale_dtype);
  float most = 0.0f;
  const int cols = (p.K + p.group - 1) / p.group;
  for (int c = lane; c < cols; c += 32) {
    const float s = fabsf(load_as_float(scales, p.scale_dtype, n * p.lds + c));
    if (s <= 3.402823466e38f) most = fmaxf(most, s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) {
    const int biased = (int)(__float_as_uint(most) >> 23) - 11;
    out[(int64_t)e * p.N + n] = most > 0.0f ? __uint_as_float((uint32_t)max(biased, 1) << 23) : 1.0f;
  }
}

// Weights as 16-bit values s * (q - z), K-major with pitch ldw (a multiple of 16; zeros
// past K); groups without rows are skipped.  Bound by memory (the store is four times the
// load): a thread takes 16 k of DQ_COLS columns, all of its loads before the first use and
// 32 bytes to a store: 4096 x 11008 in 17 us, 6.6 TB/s of loads and stores (with 1, 2 or 8
// columns a prompt of 2000 rows takes 11, 3.5 and 2.4 us longer).  With scales of A's own
// type the product s * (q - z) is one packed multiplication: its exact value is rounded
// once, as in fp32.
constexpr int DQ_COLS = 4;

template <bool BF16>
__global__ void __launch_bounds__(256) q4_dequant_kernel(const __grid_constant__ Q4Params p, uint16_t* out, int64_t ldw,
                                                         int64_t stride_w) {
  // (No early start for the products: their CTAs' registers would keep this kernel's out.)
  pdl_wait();
  const int e = (int)blockIdx.z;
  int lo, hi;
  group_range(p.g, e, lo, hi);
  if (lo == hi) return;
  const uint8_t* q = p.q + e * p.stride_q;
  const char* scales = static_cast<const char*>(p.scales) + e * p.stride_s * dtype_bytes(p.scale_dtype);
  const uint8_t* zeros = p.zeros ? p.zeros + e * p.stride_z : nullptr;
  out += e * stride_w;
  const int64_t k = (int64_t)(blockIdx.x * blockDim.x + threadIdx.x) * 16;
  if (k >= ldw) return;
  const int64_t gk = k < p.K ? k / p.group : 0, step = (int64_t)gridDim.y * blockDim.y * DQ_COLS;
  const bool packed = k + 16 <= p.K && p.scale_dtype == p.ab_dtype;
  for (int64_t n0 = (int64_t)(blockIdx.y * blockDim.y + threadIdx.y) * DQ_COLS; n0 < p.N; n0 += step) {
    if (packed) {
      uint2 w[DQ_COLS];
      uint32_t s[DQ_COLS], z[DQ_COLS];
#pragma unroll
      for (int i = 0; i < DQ_COLS; ++i) {
        const int64_t n = min(n0 + i, (int64_t)p.N - 1);
        w[i] = __ldg(reinterpret_cast<const uint2*>(q + n * p.ldq + k / 2));
        s[i] = __ldg(reinterpret_cast<const uint16_t*>(scales) + n * p.lds + gk);
        z[i] = zeros ? __ldg(zeros + n * p.ldz + gk) : 8u;
      }
#pragma unroll
      for (int i = 0; i < DQ_COLS; ++i) {
        const uint32_t zc = zero_const<BF16>(z[i] & 15u).lo, s2 = s[i] * 0x00010001u;
        uint32_t h[2][4], o[8];
        unpack_pairs<BF16>(w[i].x, zc, h[0]);
        unpack_pairs<BF16>(w[i].y, zc, h[1]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (BF16) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[j]) : "r"(h[j >> 2][j & 3]), "r"(s2));
          else asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o[j]) : "r"(h[j >> 2][j & 3]), "r"(s2));
        }
        if (n0 + i < p.N) st_row_32b(reinterpret_cast<char*>(out + (n0 + i) * ldw + k), o);
      }
    } else {
      for (int64_t n = n0; n < min(n0 + DQ_COLS, (int64_t)p.N); ++n) {
        float s = load_as_float(scales, p.scale_dtype, n * p.lds + gk);
        // (a power of two: its reciprocal has the mirrored exponent)
        if (p.col_scale != nullptr) s *= __uint_as_float((254u << 23) - __float_as_uint(p.col_scale[(int64_t)e * p.N + n]));
        const int z = zeros ? zeros[n * p.ldz + gk] & 15 : 8;
        uint32_t o[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t b = k + 2 * u < p.K ? q[n * p.ldq + k / 2 + u] : 0u;
          const float lo4 = k + 2 * u < p.K ? s * (float)((int)(b & 15) - z) : 0.0f;
          const float hi4 = k + 2 * u + 1 < p.K ? s * (float)((int)(b >> 4) - z) : 0.0f;
          if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[u]) : "f"(hi4), "f"(lo4));
          else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[u]) : "f"(hi4), "f"(lo4));
        }
        st_row_32b(reinterpret_cast<char*>(out + n * ldw + k), o);
      }
    }
  }
}

template <int MT, int NT, int BPG, bool ZP, bool S32, bool BF16>
cudaError_t launch_q4_t(const Q4Params& p, cudaStream_t stream) {
  using Cfg = Q4Cfg<MT, NT>;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  static bool configured[64] = {};
  if (dev >= 64 || !configured[dev]) {
    err = cudaFuncSetAttribute(q4_kernel<MT, NT, BPG, ZP, S32, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (err != cudaSuccess) return err;
    if (dev < 64) configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.N + p.cta_rows - 1) / p.cta_rows), (unsigned)p.g.count, 1);
  cfg.blockDim = dim3(32 * WARPS, 1, 1);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_kernel<MT, NT, BPG, ZP, S32, BF16>, p);
}

template <int MT, int NT, bool BF16>
cudaError_t launch_q4_tile(Q4Params p, cudaStream_t stream) {
  // A scale group in units of 32, 64 or 128 k, and its logarithm if that is whole.
  const int unit = p.scale_dtype == GEMM_F32 ? 32 : p.group % 128 == 0 ? 128 : p.group % 64 == 0 ? 64 : 32;
  p.scale_cols = (p.K + p.group - 1) / p.group;
  p.group_units = p.group / unit;
  p.group_shift = -1;
  for (int b = 0; b < 31; ++b)
    if (p.group_units == 1 << b) p.group_shift = b;
  const int per_chunk = CHUNK / unit, es = dtype_bytes(p.scale_dtype);
  auto aligned = [](const void* ptr, int64_t pitch, int64_t stride, int n) {
    return reinterpret_cast<uintptr_t>(ptr) % n == 0 && pitch % n == 0 && stride % n == 0;
  };
  p.vec_s = p.group_units == 1 && aligned(p.scales, p.lds * es, p.stride_s * es, per_chunk * es) &&
            (!p.zeros || aligned(p.zeros, p.ldz, p.stride_z, per_chunk)) ? 1 : 0;
  const bool zp = p.zeros != nullptr;
  if (p.scale_dtype == GEMM_F32)
    return zp ? launch_q4_t<MT, NT, 1, true, true, BF16>(p, stream) : launch_q4_t<MT, NT, 1, false, true, BF16>(p, stream);
  if (unit == 128)
    return zp ? launch_q4_t<MT, NT, 4, true, false, BF16>(p, stream) : launch_q4_t<MT, NT, 4, false, false, BF16>(p, stream);
  if (unit == 64)
    return zp ? launch_q4_t<MT, NT, 2, true, false, BF16>(p, stream) : launch_q4_t<MT, NT, 2, false, false, BF16>(p, stream);
  return zp ? launch_q4_t<MT, NT, 1, true, false, BF16>(p, stream) : launch_q4_t<MT, NT, 1, false, false, BF16>(p, stream);
}

template <bool BF16>
cudaError_t launch_q4_rows(const Q4Params& p, int nt, cudaStream_t stream) {
  if (nt == 4) return launch_q4_tile<2, 4, BF16>(p, stream);
  if (nt == 2) return launch_q4_tile<2, 2, BF16>(p, stream);
  if (p.cta_rows <= 16) return launch_q4_tile<1, 1, BF16>(p, stream);
  if (p.cta_rows <= 32) return launch_q4_tile<2, 1, BF16>(p, stream);
  return launch_q4_tile<3, 1, BF16>(p, stream);
}

}  // namespace

Q4Shape q4_shape(int64_t N, int64_t rows_per_group, int64_t groups_used, int sm_count) {
  Q4Shape s;
  s.nt = rows_per_group > 16 ? 4 : rows_per_group > 8 ? 2 : 1;
  // Columns per CTA: as many as give every resident CTA the same share in one wave
  // (not a multiple of 16: an MMA's spare rows cost less than a second, mostly empty
  // wave), in as few waves as the tile height allows.
  const int64_t most = s.nt == 1 ? 48 : 32, resident = (int64_t)sm_count * (s.nt == 4 ? 1 : 2);
  const int64_t columns = groups_used * N, waves = (columns + resident * most - 1) / (resident * most);
  const int64_t per_group = std::max<int64_t>(1, waves * resident / groups_used);   // CTAs of a group
  const int64_t rows = std::max<int64_t>(8, (N + per_group - 1) / per_group);
  s.cta_rows = (int)std::min(std::min(most, rows), N);
  return s;
}

cudaError_t launch_q4(const Q4Params& p, int nt, cudaStream_t stream) {
  return p.ab_dtype == GEMM_BF16 ? launch_q4_rows<true>(p, nt, stream) : launch_q4_rows<false>(p, nt, stream);
}

cudaError_t launch_q4_range(const Q4Params& p, float* out, cudaStream_t stream) {
  return launch_dependent(q4_range_kernel, dim3((unsigned)((p.N + 7) / 8), (unsigned)p.g.count), 256, stream, p, out);
}

cudaError_t launch_q4_dequant(const Q4Params& p, void* out, int64_t ldw, int64_t stride_w, cudaStream_t stream) {
  int tx = 1;   // threads along K
  while (tx < 256 && tx * 16 < ldw) tx *= 2;
  const int ty = 256 / tx;
  const int64_t per_cta = (int64_t)ty * DQ_COLS;
  const dim3 grid((unsigned)((ldw / 16 + tx - 1) / tx), (unsigned)std::min<int64_t>((p.N + per_cta - 1) / per_cta, 65535),
                  (unsigned)p.g.count);
  uint16_t* o = static_cast<uint16_t*>(out);
  const dim3 block((unsigned)tx, (unsigned)ty);
  return p.ab_dtype == GEMM_BF16 ? launch_dependent(q4_dequant_kernel<true>, grid, block, stream, p, o, ldw, stride_w)
                                 : launch_dependent(q4_dequant_kernel<false>, grid, block, stream, p, o, ldw, stride_w);
}

}  // namespace gemmlib
