// seg_kernel.cu -- tcgen05 products whose tiles are not one dense problem's:
//   TOKENS  D[r, :] = act(alpha * A[r, :] * op(B_g) + bias_g) for the rows r of each
//           group g (rows found on the device);
//   WGRAD   D_g = alpha * A_g' * B_g + beta * C_g, the sum over the rows of group g;
//   CHAIN   the products of the Newton-Schulz steps, all of them in one launch:
//           E = X X' - h I,  F = c E E' + b E,  X <- F X + a X  for every matrix of a batch
//           (in the last two steps F = c E E' + b E + a I,  X <- F X), X as a pair of fp16
//           halves, E and F as one half or, for results finer than bf16, as pairs too.
//
// One structure serves them all, on single CTAs (CG = 1, tiles of 128 x 128) and on
// CTA pairs (CG = 2, 256 x 256): a producer thread streams 64-deep slabs of both
// operands with TMA into a ring of 128-byte-swizzled stages (two slabs each), one
// thread issues tcgen05.mma into one of two tensor-memory accumulators, eight
// warps finish the other one.  Each CTA of a pair loads its own 128 rows of the
// M side and its half of the N side; the leader's MMAs read both.
//
// TOKENS puts the weights' columns on the M side and the group's rows on the N
// side.  The MMA's N is any multiple of 16, so a group of r rows costs r rounded
// up to 16 columns of MMA time (its tiles are of equal width), where rows on the
// M side would cost whole tiles of 128 or 256: a few hundred rows per expert lose a
// fifth to a third of the tensor time that way, and a decoding step's one or two
// rows nearly all of it.  The accumulator then holds D transposed; the epilogue
// turns each 32 x 32 chunk around through shared memory.
//
// WGRAD's K loop runs over a group's rows.  Its tensor maps are per group, with
// the group's first row as their base and its row count as their extent (built on
// the device by wgrad_maps_kernel): the last block's rows past the group read as
// zero, whatever other rows hold.
//
// CHAIN: E and F are symmetric, so only tiles on and below the diagonal are computed
// and each is stored twice, as it is and transposed.  The tiles of all phases form one
// list (step by step, product by product, matrix by matrix, the two halves of a batch a
// phase apart) that the workers take in turn.  A tile waits, per 256-row (CG = 1:
// 128-row) block of the matrices that it reads, for a counter of the finished tiles of
// that block row:
//   E(i, j) waits for rows i and j of X (the last step's F X tiles),
//   F(i, j) for rows i and j of E, and F X (i, n) for row i of F -- which has needed all
//   of E, and that all of X.
// The same order makes every buffer free when it is written again: whoever writes a
// tile of X, E or F has waited, through that chain, for every reader of its old value.
// Every wait is for earlier tiles of the list only, and all workers are resident (a
// cooperative launch), so the earliest unfinished tile can always run.  One launch in
// place of three per step saves the launches' fixed cost (6-8 us each, all of a small
// matrix's time) and lets the matrices of a batch fill each other's last waves.
//
// Measured (graph replays): 16384 rows over 64 experts, 2048 to 4096, bf16: 222 us, 5.7 TB/s
// of the operands' bytes, 85 % of a copy; over 32 experts, 4096 x 2048, input and weight
// gradient together: 399 us, 1.38 PFLOP/s, held by operand supply; 16 rows over 8 experts,
// 1024 to 2048: 9.0 us, the latency of a launch and eight stages.  Newton-Schulz, five
// steps, bf16 result: 4096 x 11008 2.19 ms with its input passes, 1.42 PFLOP/s (the symmetric
// products counted half), at the power cap; 16 x 768 x 2001 477 us (a tile of 768 k takes 6 us
// and more for 3.9 us of MMAs: L2 traffic; without X's second halves 384); 384 x 256 81 us,
// 15 dependent products of 5 us.  fp32 result, products of pairs: 5.95 ms, 885 and 114 us.
// Why three stages of two slabs, one producer, at the first case's 241 us of the time: six
// stages of one slab 257, stages as small as the tile 250, a second producer thread 242.
//
// Every wait is bounded, as in tc_kernel.cu.
#include "expert.h"

namespace gemmlib {
namespace {

constexpr int SLABS = 2;                             // 64-deep K blocks per stage
constexpr int STAGES = 3;
constexpr int SLAB_BYTES = 128 * TC_BK * 2;           // 16 KiB: 128 rows of one operand
constexpr int OPERAND_BYTES = SLABS * SLAB_BYTES;     // one operand of a stage
constexpr int STAGE_BYTES = 2 * OPERAND_BYTES;        // [M side][N side]
constexpr uint32_t MN_BOX_BYTES = 64 * 2 * SLABS * TC_BK;   // MN-major box: 64 wide, a stage deep
constexpr int EPI_WARPS = 8;                          // two per tensor-memory lane quarter
constexpr int TURN_BYTES = 2048;                      // an epilogue warp's turn-around buffer
constexpr int NUM_BARS = 2 * STAGES + 5;
constexpr size_t FIXED_SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + EPI_WARPS * TURN_BYTES + NUM_BARS * 8 + 16 + EPI_WARPS * 4;

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t user_timeout_ns) {
  const uint64_t timeout_ns = user_timeout_ns > 1000000000ull ? user_timeout_ns : 1000000000ull;
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > timeout_ns) return;
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& wc) {
  const bool ok = mbar_wait(bar, parity, wc);
  return __all_sync(0xffffffffu, ok) != 0;
}

// ------------------------------ output chunks -------------------------------

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t w;
  if constexpr (DT == GEMM_F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// 32 rows of 64 bytes (lane: its row's 16 words) of ES-byte elements at any alignment:
// turned around in the warp's buffer, whole rows per instruction; rows r < rows, columns
// j < cols.
template <int ES>
__device__ __forceinline__ void store_rows64(char* D, int64_t pitch, int rows, int cols, const uint32_t (&w)[16],
                                             uint32_t turn) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the buffer's last readers are done
#pragma unroll
  for (int q = 0; q < 4; ++q)
    sts128(turn + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  __syncwarp();
  constexpr int PER = 64 / ES, RPI = 32 / PER;   // elements per row, rows per instruction
  const int j = lane % PER;
#pragma unroll 8
  for (int r = lane / PER; r < 32; r += RPI) {
    const uint32_t a = turn + (uint32_t)(r * 64 + (((j * ES >> 4) ^ ((r >> 1) & 3)) << 4) + (j * ES & 15));
    if (r < rows && j < cols) {
      if constexpr (ES == 2) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
        *reinterpret_cast<uint16_t*>(D + r * pitch + j * 2) = v;
      } else {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
        *reinterpret_cast<uint32_t*>(D + r * pitch + j * 4) = v;
      }
    }
  }
}

// A warp's 32 x 32 chunk, lane r = row r, x = its columns: D[r][j], r < rows, j < cols.
// Aligned rows are stored straight from registers, 32 bytes (a whole sector) per lane:
// the MMAs' operand reads and the ring's writes leave little shared-memory bandwidth, and
// turning the chunk around there cost more than the wider pattern of the stores does.
template <int DT>
__device__ __forceinline__ void store_chunk(void* D, int64_t ldd, int64_t r0, int64_t c0, int rows, int cols,
                                            const float (&x)[32], uint32_t turn, bool vec) {
  constexpr int ES = DT == GEMM_F32 ? 4 : 2, PIECE = 32 / ES;   // columns of 32 bytes
  const int lane = threadIdx.x & 31;
  uint32_t w[32 * ES / 4];
  if constexpr (DT == GEMM_F32) {
#pragma unroll
    for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack2<DT>(x[2 * j], x[2 * j + 1]);
  }
  char* d = static_cast<char*>(D) + (r0 * ldd + c0) * ES;
  if (vec && cols % (16 / ES) == 0) {
    if (lane >= rows) return;
    d += lane * ldd * ES;
#pragma unroll
    for (int q = 0; q < 32 / PIECE; ++q) {
      if ((q + 1) * PIECE <= cols) st_row_32b(d + 32 * q, w + 8 * q);
      else if (q * PIECE < cols) *reinterpret_cast<uint4*>(d + 32 * q) = make_uint4(w[8 * q], w[8 * q + 1], w[8 * q + 2], w[8 * q + 3]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < ES / 2; ++h) {
      uint32_t u[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) u[j] = w[16 * h + j];
      store_rows64<ES>(d + h * 64, ldd * ES, rows, cols - h * 16, u, turn);
    }
  }
}

// The same chunk stored transposed: D[j][r], j < rows_out, r < cols_out.
template <int DT>
__device__ __forceinline__ void store_chunk_t(void* D, int64_t ldd, int64_t j0, int64_t r0, int rows_out, int cols_out,
                                              const float (&x)[32], uint32_t turn, bool vec) {
  const int lane = threadIdx.x & 31;
  const bool v = vec && cols_out % (DT == GEMM_F32 ? 4 : 8) == 0;
  if constexpr (DT == GEMM_F32) {
    float* d = static_cast<float*>(D) + j0 * ldd + r0;
    if (!v) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < rows_out && lane < cols_out) d[j * ldd + lane] = x[j];
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(turn + (uint32_t)(j * 128 + lane * 4)), "r"(__float_as_uint(x[16 * h + j])) : "memory");
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 4 * i + (lane >> 3);
        const uint4 q = lds128(turn + (uint32_t)(j * 128 + (lane & 7) * 16));
        if (16 * h + j < rows_out && (lane & 7) * 4 < cols_out)
          *reinterpret_cast<uint4*>(d + (16 * h + j) * ldd + (lane & 7) * 4) = q;
      }
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(D) + j0 * ldd + r0;
    if (!v) {
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const uint32_t w = pack2<DT>(x[j], x[j + 1]);
        if (lane < cols_out) {
          if (j < rows_out) d[j * ldd + lane] = (uint16_t)w;
          if (j + 1 < rows_out) d[(j + 1) * ldd + lane] = (uint16_t)(w >> 16);
        }
      }
      return;
    }
    // Row p of the buffer: output rows 2p and 2p + 1 as the halves of 32 words.
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 16; ++p)
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(turn + (uint32_t)(p * 128 + lane * 4)), "r"(pack2<DT>(x[2 * p], x[2 * p + 1])) : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int p = 8 * i + (lane >> 2), o = lane & 3, h = p & 1;
      // Odd rows read their two 16-byte pieces in the other order: no bank is hit twice.
      const uint4 a = lds128(turn + (uint32_t)(p * 128 + o * 32 + h * 16));
      const uint4 b = lds128(turn + (uint32_t)(p * 128 + o * 32 + (1 - h) * 16));
      const uint4 f = h ? b : a, s = h ? a : b;
      const uint4 lo = make_uint4(__byte_perm(f.x, f.y, 0x5410), __byte_perm(f.z, f.w, 0x5410),
                                  __byte_perm(s.x, s.y, 0x5410), __byte_perm(s.z, s.w, 0x5410));
      const uint4 hi = make_uint4(__byte_perm(f.x, f.y, 0x7632), __byte_perm(f.z, f.w, 0x7632),
                                  __byte_perm(s.x, s.y, 0x7632), __byte_perm(s.z, s.w, 0x7632));
      if (2 * p < rows_out && o * 8 < cols_out) *reinterpret_cast<uint4*>(d + (2 * p) * ldd + o * 8) = lo;
      if (2 * p + 1 < rows_out && o * 8 < cols_out) *reinterpret_cast<uint4*>(d + (2 * p + 1) * ldd + o * 8) = hi;
    }
  }
}

// beta * C of a chunk (lane r = row r), in two steps so that the loads run ahead of the
// accumulator: aligned rows of 16-bit C straight into registers, 32 bytes per load; other
// types and edges are read when they are added, by elements, whole rows per instruction.
// All coherent at L2: CHAIN's C was written by other SMs during the launch that reads it.
struct CChunk {
  uint32_t w[16];
  bool held;
};
__device__ __forceinline__ void ld_32b(const void* p, uint32_t* w) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("ld.relaxed.gpu.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p) + h);
      w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
    }
  }
}
__device__ __forceinline__ void load_c(const EpiParams& e, const void* C, int64_t r0, int64_t c0, int rows, int cols,
                                       CChunk& c) {
  const int lane = threadIdx.x & 31;
  c.held = e.vec_c && cols % 8 == 0 && e.c_dtype != GEMM_F32;
  if (!c.held) return;
  const uint16_t* src = static_cast<const uint16_t*>(C) + (r0 + lane) * e.ldc + c0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
#pragma unroll
    for (int u = 0; u < 8; ++u) c.w[8 * q + u] = 0u;
    if (lane >= rows) continue;
    if (16 * q + 16 <= cols) {
      ld_32b(src + 16 * q, c.w + 8 * q);
    } else if (16 * q < cols) {
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(src + 16 * q));
      c.w[8 * q] = v.x, c.w[8 * q + 1] = v.y, c.w[8 * q + 2] = v.z, c.w[8 * q + 3] = v.w;
    }
  }
}
// x += beta * 16 words of 16-bit C.
__device__ __forceinline__ void fma_c16(const EpiParams& e, float (&x)[32], const uint32_t* w, int j0, int n) {
#pragma unroll
  for (int h = 0; h < n; ++h) {
    float lo, hi;
    if (e.c_dtype == GEMM_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[h]));
      lo = f.x;
      hi = f.y;
    } else {
      lo = __uint_as_float(w[h] << 16);
      hi = __uint_as_float(w[h] & 0xffff0000u);
    }
    x[j0 + 2 * h] = fmaf(e.beta, lo, x[j0 + 2 * h]);
    x[j0 + 2 * h + 1] = fmaf(e.beta, hi, x[j0 + 2 * h + 1]);
  }
}
__device__ __forceinline__ void add_c(const EpiParams& e, const void* C, int64_t r0, int64_t c0, int rows, int cols,
                                      const CChunk& ch, float (&x)[32], uint32_t turn) {
  const int lane = threadIdx.x & 31;
  if (ch.held) {
    fma_c16(e, x, ch.w, 0, 16);
  } else if (e.c_dtype == GEMM_F32) {
    // 16 columns at a time: two rows per load instruction, turned around like 16-bit rows.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* src = static_cast<const float*>(C) + r0 * e.ldc + c0 + 16 * h;
      const int j = lane & 15;
      __syncwarp();
#pragma unroll 8
      for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        const float v = r < rows && 16 * h + j < cols ? __ldcg(src + r * e.ldc + j) : 0.0f;
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(turn + (uint32_t)(r * 64 + (((j >> 2) ^ ((r >> 1) & 3)) << 4) + (j & 3) * 4)), "f"(v) : "memory");
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 c = lds128(turn + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)));
        x[16 * h + 4 * q + 0] = fmaf(e.beta, __uint_as_float(c.x), x[16 * h + 4 * q + 0]);
        x[16 * h + 4 * q + 1] = fmaf(e.beta, __uint_as_float(c.y), x[16 * h + 4 * q + 1]);
        x[16 * h + 4 * q + 2] = fmaf(e.beta, __uint_as_float(c.z), x[16 * h + 4 * q + 2]);
        x[16 * h + 4 * q + 3] = fmaf(e.beta, __uint_as_float(c.w), x[16 * h + 4 * q + 3]);
      }
    }
  } else {
    const uint16_t* src = static_cast<const uint16_t*>(C) + r0 * e.ldc + c0 + lane;
    __syncwarp();
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      const uint16_t v = r < rows && lane < cols ? __ldcg(src + r * e.ldc) : (uint16_t)0;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(turn + (uint32_t)(r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2)), "h"(v) : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 c = lds128(turn + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)));
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      fma_c16(e, x, w, 8 * q, 4);
    }
  }
}

// ---------------------------------- tiles -----------------------------------

struct Tile {
  int e;          // group (TOKENS, WGRAD) or matrix of the batch (CHAIN)
  int m0, n0;     // first row of the M side and of the N side (TOKENS: the buffer's row)
  int n_valid;    // N-side rows that exist
  int n_mma;      // the MMA's N (a multiple of 16)
  int k;          // depth
  int step, product;   // CHAIN: the step, and 0: E, 1: F, 2: X
};

// Shared-memory tables: the groups' first rows and row counts (TOKENS, WGRAD) and first
// tiles (TOKENS).
struct GroupTable {
  int *lo, *cnt, *cum;
};

template <int MODE, int CG>
struct Tiles {
  static constexpr int BM = 128 * CG;
  static constexpr int BN = BM;   // TOKENS, WGRAD
  const SegParams& p;
  GroupTable g;
  int t, step, e;
  __device__ __forceinline__ Tiles(const SegParams& p_, const GroupTable& g_, int first, int step_)
      : p(p_), g(g_), t(first), step(step_), e(0) {}

  __device__ __forceinline__ bool next(Tile& o) {
    if constexpr (MODE == SEG_TOKENS) {
      if (t >= g.cum[p.groups.count]) return false;
      while (t >= g.cum[e + 1]) ++e;
      const int cnt = g.cnt[e], n_tiles = (cnt + BN - 1) / BN;
      // Equal widths: (n_tiles - 1) * per <= (n_tiles - 1) * BN < cnt, so none is empty.
      const int per = ((cnt + n_tiles - 1) / n_tiles + 15) & ~15;
      const int local = t - g.cum[e];
      // Bands of 8 tile rows; in a band the row runs fastest.
      const int band = local / (8 * n_tiles), first = band * 8, size = min(8, p.tiles_m - first);
      const int r = local - first * n_tiles;
      const int tn = r / size;
      o.e = e;
      o.m0 = (first + r - tn * size) * BM;
      o.n0 = g.lo[e] + tn * per;
      o.n_valid = min(per, cnt - tn * per);
      o.n_mma = (o.n_valid + 15) & ~15;
      o.k = p.K;
    } else if constexpr (MODE == SEG_WGRAD) {
      if (t >= p.num_tiles) return false;
      o.e = t / p.tiles_per_group;
      const int local = t - o.e * p.tiles_per_group;
      const int band = local / (8 * p.tiles_n), first = band * 8, size = min(8, p.tiles_m - first);
      const int r = local - first * p.tiles_n;
      const int tn = r / size;
      o.m0 = (first + r - tn * size) * BM;
      o.n0 = tn * BN;
      o.n_valid = min(BN, p.N - o.n0);
      o.n_mma = BN;
      o.k = g.cnt[o.e];
    } else {
      if (t >= p.num_tiles) return false;
      // Segments of one turn over the two halves A, B of the batch (B one phase and a half
      // behind): E_A, B's X of the step before, F_A, E_B, X_A, F_B.
      const int a = (p.batch + 1) / 2, b = p.batch - a, sym = p.tiles_per_group, dense = p.tiles_m * p.tiles_n;
      const int turn = p.batch * (2 * sym + dense);
      int local = t;
      if (local >= a * sym) local += b * dense;            // the first turn has no X_B,
      if (local >= p.steps * turn) local += a * sym;       // the one after the last nothing else
      o.step = local / turn;
      local -= o.step * turn;
      o.e = 0;
      if (local < a * sym) {
        o.product = 0;
      } else if ((local -= a * sym) < b * dense) {
        o.product = 2;
        o.e = a;
        --o.step;
      } else if ((local -= b * dense) < a * sym) {
        o.product = 1;
      } else if ((local -= a * sym) < b * sym) {
        o.product = 0;
        o.e = a;
      } else if ((local -= b * sym) < a * dense) {
        o.product = 2;
      } else {
        local -= a * dense;
        o.product = 1;
        o.e = a;
      }
      if (o.product < 2) {
        const int z = local / sym;
        o.e += z;
        local -= z * sym;
        // Block row tm has (tm + 1) * r tiles of bns columns, r to a block.
        const int r = BM / p.bns, q = local / r;
        int tm = (int)((sqrtf(8.0f * (float)q + 1.0f) - 1.0f) * 0.5f);
        while ((tm + 1) * (tm + 2) / 2 <= q) ++tm;
        while (tm * (tm + 1) / 2 > q) --tm;
        o.m0 = tm * BM;
        o.n0 = (local - tm * (tm + 1) / 2 * r) * p.bns;
        o.n_valid = max(0, (int)min((int64_t)p.bns, p.M - o.n0));
        o.n_mma = p.bns;
        o.k = o.product == 0 ? p.N : (int)p.M;
      } else {
        const int z = local / dense;
        o.e += z;
        local -= z * dense;
        // Bands of 8 tile rows; in a band the row runs fastest.
        const int band = local / (8 * p.tiles_n), first = band * 8, size = min(8, p.tiles_m - first);
        const int r = local - first * p.tiles_n, tn = r / size;
        o.m0 = (first + r - tn * size) * BM;
        o.n0 = tn * p.bn;
        o.n_valid = min(p.bn, p.N - o.n0);
        o.n_mma = p.bn;
        o.k = (int)p.M;
      }
    }
    t += step;
    return true;
  }
};

// CHAIN: the counter of the finished tiles of block row i of a product's result.
__device__ __forceinline__ int32_t* chain_counter(const SegParams& p, int step, int product, int e, int i) {
  return p.counters + (((int64_t)step * 3 + product) * p.batch + e) * p.tiles_m + i;
}

// Threads of a mode: producer warp, MMA warp, epilogue warps, and CHAIN's scout and publisher.
template <int MODE>
struct SegThreads {
  static constexpr int COUNT = 64 + 32 * EPI_WARPS + (MODE == SEG_CHAIN ? 64 : 0);
};

// Wait until block row i of a result is complete.  Bounded like mbar_wait.
__device__ __forceinline__ bool chain_wait(const int32_t* counter, int32_t target, const WaitCtx& wc) {
  if (ld_acquire_gpu(counter) >= target) return true;
  const uint64_t t0 = globaltimer_ns();
  while (ld_acquire_gpu(counter) < target) {
    if (*wc.abort) return false;
    if (globaltimer_ns() - t0 > wc.timeout_ns) {
      atomicCAS(wc.err, 0, (int32_t)GEMM_ERR_TIMEOUT);
      *wc.abort = 1;
      __threadfence_block();
      return false;
    }
  }
  return true;
}

// CHAIN: wait until the sequence number in shared memory has passed `tile`: the scout has
// found that tile's operands in place (its acquire and proxy fence, then this release and
// acquire, order the tile's loads after the stores that they read), or an epilogue warp
// has stored its part of the tile.
__device__ __forceinline__ bool chain_seen(const int32_t* seq, int tile, const WaitCtx& wc) {
  const uint32_t a = smem_u32(seq);
  for (;;) {
    int32_t v;
    asm volatile("ld.acquire.cta.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    if (v > tile) return true;
    if (*wc.abort) return false;   // (the waits of those who write it are bounded and set this)
    __nanosleep(20);
  }
}

// CHAIN: the operands of tile t in place (see the head of this file).
template <int CG>
__device__ __forceinline__ bool chain_ready(const SegParams& p, const Tile& t, const WaitCtx& wc) {
  constexpr int B = 128 * CG, PER_TILE = CG;   // every CTA of a tile counts once
  bool ok = true;
  if (t.product == 0) {
    if (t.step > 0) {
      const int32_t target = p.tiles_n * PER_TILE;   // X
      ok = chain_wait(chain_counter(p, t.step - 1, 2, t.e, t.m0 / B), target, wc) &&
           chain_wait(chain_counter(p, t.step - 1, 2, t.e, t.n0 / B), target, wc);
    }
  } else {
    const int32_t target = p.tiles_m * (B / p.bns) * PER_TILE;   // E, F
    ok = chain_wait(chain_counter(p, t.step, t.product - 1, t.e, t.m0 / B), target, wc);
    if (ok && t.product == 1) ok = chain_wait(chain_counter(p, t.step, 0, t.e, t.n0 / B), target, wc);
  }
  // The data was written by ordinary stores and is read by TMA: the proxy fence stands here,
  // once the stores are known to have happened.
  fence_proxy_async_smem();
  return ok;
}

template <int CG, bool A_MN, bool B_MN, int MODE>
__global__ void __launch_bounds__(SegThreads<MODE>::COUNT, 1) seg_kernel(const __grid_constant__ SegParams p) {
  constexpr int BN = 128 * CG, THREADS = SegThreads<MODE>::COUNT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;   // the same offset in both CTAs of a pair
  uint8_t* base_ptr = smem_raw + (base - raw);
  constexpr uint32_t TURN0 = STAGES * STAGE_BYTES, BAR0 = TURN0 + EPI_WARPS * TURN_BYTES;
  const uint32_t bar0 = base + BAR0;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + BAR0 + NUM_BARS * 8);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  int32_t* ready_seq = reinterpret_cast<int32_t*>(tmem_slot + 2);   // CHAIN: tiles whose operands are in place
  int32_t* stored_seq = reinterpret_cast<int32_t*>(tmem_slot + 4);  // CHAIN: tiles that each epilogue warp has stored
  int* table = reinterpret_cast<int*>(tmem_slot + 4 + EPI_WARPS);
  const GroupTable groups{table, table + p.groups.count, table + 2 * p.groups.count};

  auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 + b); };
  const uint32_t teardown_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 4);

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // (uniform)
  const uint32_t rank = CG == 2 ? (cluster_ctarank() & 1u) : 0u;
  const bool leader = rank == 0;
  const int worker = (int)blockIdx.x / CG, workers = (int)gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);     // the leader's expect_tx arrival + every CTA's bytes
      mbar_init(empty_bar(s), 1);    // the commit after the stage's MMAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), CG * EPI_WARPS);
    }
    mbar_init(teardown_bar, 1);
    *abort_flag = 0;
    *ready_seq = 0;
    for (int w = 0; w < EPI_WARPS; ++w) stored_seq[w] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if constexpr (CG == 2) {
    cluster_sync();
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 2 * BN);
  } else {
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 2 * BN);
  }
  // The prologue above touches no global data: overlap it with the previous kernel.
  if (MODE != SEG_CHAIN) pdl_launch_dependents();
  pdl_wait();
  if constexpr (MODE == SEG_TOKENS || MODE == SEG_WGRAD) {
    const int E = p.groups.count;
    for (int e = threadIdx.x; e < E; e += THREADS) {
      int lo, hi;
      group_range(p.groups, e, lo, hi);
      groups.lo[e] = lo;
      groups.cnt[e] = hi - lo;
    }
    if (MODE == SEG_TOKENS) __syncthreads();
    if (MODE == SEG_TOKENS && warp == 0) {
      // First tiles, saturated at MOST: offsets that decrease can give the same rows to many
      // groups, and a sum past 2^31 would wrap to tiles outside the buffers.  (What good
      // offsets give stays below 2^28, and a group's own tiles do in any case.)
      constexpr int MOST = 1 << 29;
      int sum = 0;
      for (int e0 = 0; e0 < E; e0 += 32) {
        int v = e0 + lane < E ? (groups.cnt[e0 + lane] + BN - 1) / BN * p.tiles_m : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v = min(v + u, MOST);
        }
        v = min(v + sum, MOST);
        if (e0 + lane < E) groups.cum[e0 + lane + 1] = v;
        sum = __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) groups.cum[0] = 0;
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtx wc{abort_flag, p.err, p.timeout_ns};

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    // (The whole warp walks the list and waits, one lane issues: see the MMA issuer.)
    const bool one = elect_one();
    int stage = 0, issued = 0;   // stages filled so far
    uint32_t phase = 0;
    bool ok = true;
    // WGRAD: a group's tensor maps are acquired and fetched a tile ahead of their use.
    int map_of = -1;
    auto acquire_maps = [&](const Tile& a) {
      if (a.k == 0 || a.e == map_of) return;
      map_of = a.e;
      if (one) {
        for (int i = 0; i < 2; ++i) {
          tensormap_acquire(p.group_maps + 2 * a.e + i);
          tma_prefetch_desc(p.group_maps + 2 * a.e + i);
        }
      }
      __syncwarp();
    };
    Tiles<MODE, CG> it(p, groups, worker, workers);
    int tile_no = 0;   // CHAIN
    Tile t, ahead;
    bool more = it.next(ahead);
    if (MODE == SEG_WGRAD && more) acquire_maps(ahead);
    while (ok && more) {
      t = ahead;
      more = it.next(ahead);
      const CUtensorMap *ma = &p.tmA, *mb = &p.tmB[0];
      int za = 0, zb = 0;
      const int m0 = t.m0 + (int)rank * 128, n0 = t.n0 + (int)rank * (t.n_mma / CG);
      uint32_t b_slab = (uint32_t)SLAB_BYTES;   // N-side bytes of one K-major slab
      if constexpr (MODE == SEG_TOKENS) {
        za = p.a_batched ? t.e : 0;
        int box = 0;                            // boxes of 128, 64, 32, 16, 8 rows: the smallest that holds the tile's
        while (box < 4 && (64 >> box) >= t.n_mma / CG) ++box;
        mb = &p.tmB[box];
        b_slab >>= box;
      } else if constexpr (MODE == SEG_WGRAD) {
        ma = p.group_maps + 2 * t.e;
        mb = ma + 1;
      } else {
        za = zb = t.e;
        const int cur = t.step & 1;
        ma = t.product == 0 ? &p.tmB[CHAIN_XK + cur] : t.product == 1 ? &p.tmA : &p.tmB[CHAIN_F];
        mb = t.product == 0 ? &p.tmB[CHAIN_XB + cur] : t.product == 1 ? &p.tmB[CHAIN_EB] : &p.tmB[CHAIN_XN + cur];
        b_slab = t.product == 2 ? (uint32_t)SLAB_BYTES : (uint32_t)(p.bns / CG * TC_BK * 2);
        if (!__all_sync(0xffffffffu, chain_seen(ready_seq, tile_no++, wc))) { ok = false; break; }
      }
      // CHAIN with pairs: three products into one accumulator, hi lo, lo hi, hi hi: the small
      // ones first, since every addition truncates at the running sum's size.
      const int parts = MODE == SEG_CHAIN && p.pairs ? 3 : 1;
      // N side contiguous along N (weights' gradients, X) rather than along K.
      const bool b_mn = MODE == SEG_CHAIN ? t.product == 2 : B_MN;
      const bool b_two = !(MODE == SEG_CHAIN && t.n_mma <= 64 * CG);   // MN-major: two boxes of 64 columns
      const uint32_t a_one = (uint32_t)(A_MN ? SLABS : 1) * (uint32_t)SLAB_BYTES;
      const uint32_t b_one = (uint32_t)(b_mn ? SLABS : 1) * (b_mn && !b_two ? b_slab / 2 : b_slab);
      const int num_kb = (t.k + TC_BK - 1) / TC_BK;
      for (int part = 0, kb = 0; part < parts; kb + SLABS < num_kb ? kb += SLABS : (kb = 0, ++part)) {
        if (num_kb == 0) break;
        if constexpr (MODE == SEG_CHAIN) {
          za = t.e + (parts == 3 && part == 1 ? p.batch : 0);
          zb = t.e + (parts == 3 && part == 0 ? p.batch : 0);
        }
        const bool two = kb + 1 < num_kb;   // K-major: two slabs
        if (!warp_wait(empty_bar(stage), phase ^ 1u, wc)) { ok = false; break; }
        if (one) {
          const uint32_t fb = leader ? full_bar(stage) : mapa_shared(full_bar(stage), 0);
          const uint32_t sa = base + (uint32_t)(stage * STAGE_BYTES), sb = sa + (uint32_t)OPERAND_BYTES;
          if (leader) mbar_expect_tx(full_bar(stage), (uint32_t)CG * ((A_MN || !two ? a_one : 2 * a_one) + (b_mn || !two ? b_one : 2 * b_one)));
          auto load = [&](uint32_t dst, const CUtensorMap* tm, int x, int y, int z) {
            if constexpr (CG == 2) tma_load_3d_pair(dst, tm, x, y, z, fb);
            else tma_load_3d(dst, tm, x, y, z, fb);
          };
          const int k0 = kb * TC_BK;
          if constexpr (A_MN) {
            load(sa, ma, m0, k0, za);
            load(sa + MN_BOX_BYTES, ma, m0 + 64, k0, za);
          } else {
            load(sa, ma, k0, m0, za);
            if (two) load(sa + SLAB_BYTES, ma, k0 + TC_BK, m0, za);
          }
          if (b_mn) {
            load(sb, mb, n0, k0, zb);
            if (b_two) load(sb + MN_BOX_BYTES, mb, n0 + 64, k0, zb);
          } else {
            load(sb, mb, k0, n0, zb);
            if (two) load(sb + SLAB_BYTES, mb, k0 + TC_BK, n0, zb);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        if (MODE == SEG_WGRAD && kb == 0 && more) acquire_maps(ahead);
      }
      if (MODE == SEG_WGRAD && t.k == 0 && more) acquire_maps(ahead);
    }
    // No copy is in flight when the CTA leaves (the peer of a pair waits at the last
    // cluster barrier: its copies complete on the leader's barriers).
    if (one && leader) {
      for (int i = max(0, issued - STAGES); i < issued; ++i)
        drain_wait(full_bar(i % STAGES), (uint32_t)(i / STAGES) & 1u, p.timeout_ns);
    } else if (one && !ok) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------ MMA issuer (the leader's) -----------------------
    // The whole warp walks the list and waits; one lane issues.  A stage's eight MMAs stand
    // in a row, their descriptors a constant apart: computed one by one, behind a test
    // each, they took 100 clocks apiece to issue, more than tiles of 64 columns take to run.
    if (leader) {
      const bool one = elect_one();
      int stage = 0;
      uint32_t phase = 0, acc_it = 0;
      bool ok = true;
      Tiles<MODE, CG> it(p, groups, worker, workers);
      Tile t;
      while (ok && it.next(t)) {
        if (t.k == 0) continue;
        const int buf = (int)(acc_it & 1u);
        if (!warp_wait(tempty_bar(buf), ((acc_it >> 1) & 1u) ^ 1u, wc)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * BN);
        const bool b_mn = MODE == SEG_CHAIN ? t.product == 2 : B_MN;
        const uint32_t idesc = p.idesc | ((uint32_t)(t.n_mma >> 3) << 17) |
                               ((MODE == SEG_CHAIN && b_mn ? 1u : 0u) << 16);   // bit 16: N side MN-major
        const int num_kb = (t.k + TC_BK - 1) / TC_BK, num_k16 = (t.k + 15) / 16;
        const int parts = MODE == SEG_CHAIN && p.pairs ? 3 : 1;
        for (int part = 0, kb = 0; part < parts; kb + SLABS < num_kb ? kb += SLABS : (kb = 0, ++part)) {
          if (!warp_wait(full_bar(stage), phase, wc)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = base + (uint32_t)(stage * STAGE_BYTES), sb = sa + (uint32_t)OPERAND_BYTES;
          auto issue = [&](auto mn, int count) {
            constexpr bool MN = decltype(mn)::value != 0;
            const uint64_t ad = A_MN ? smem_desc_sw128(sa, MN_BOX_BYTES, 1024) : smem_desc_sw128(sa, 16, 1024);
            const uint64_t bd = MN ? smem_desc_sw128(sb, MN_BOX_BYTES, 1024) : smem_desc_sw128(sb, 16, 1024);
            auto mma = [&](int q) {
              // Steps of 16 k: 2048 bytes of an MN-major operand; 32 bytes of a K-major slab's rows.
              const uint32_t km = (uint32_t)(q / (TC_BK / 16) * SLAB_BYTES + q % (TC_BK / 16) * 32) >> 4;
              const uint32_t mm = (uint32_t)q * 2048u >> 4;
              const uint32_t acc = q > 0 || kb > 0 || part > 0 ? 1u : 0u;
              if constexpr (CG == 2) tc_mma_f16_pair(d_tmem, ad + (A_MN ? mm : km), bd + (MN ? mm : km), idesc, acc);
              else tc_mma_f16(d_tmem, ad + (A_MN ? mm : km), bd + (MN ? mm : km), idesc, acc);
            };
            if (count >= SLABS * (TC_BK / 16)) {
#pragma unroll
              for (int q = 0; q < SLABS * (TC_BK / 16); ++q) mma(q);
            } else {
#pragma unroll 1
              for (int q = 0; q < count; ++q) mma(q);
            }
          };
          if (one) {
            const int count = num_k16 - kb * (TC_BK / 16);
            if (MODE == SEG_CHAIN ? b_mn : B_MN) issue(TypeTag<1>{}, count);
            else issue(TypeTag<0>{}, count);
            if constexpr (CG == 2) tc_commit_pair_mask(empty_bar(stage), 0x3);
            else tc_commit(empty_bar(stage));
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (one) {
          if constexpr (CG == 2) tc_commit_pair_mask(tfull_bar(buf), 0x3);
          else tc_commit(tfull_bar(buf));
        }
        __syncwarp();
        ++acc_it;
      }
      // Every MMA is complete before tensor memory is freed.
      if (one) {
        if constexpr (CG == 2) tc_commit_pair(teardown_bar);
        else tc_commit(teardown_bar);
        drain_wait(teardown_bar, 0, p.timeout_ns);
      }
      __syncwarp();
    }
  } else if (MODE == SEG_CHAIN && warp == 2 + EPI_WARPS) {
    // ---------------------------------- scout ----------------------------------
    // Walks the same list ahead of the others and waits for each tile's operands, so
    // that the producer's ring never stands still for a counter's round trip.
    if (lane == 0) {
      Tiles<MODE, CG> it(p, groups, worker, workers);
      Tile t;
      for (int n = 1; it.next(t); ++n) {
        if (!chain_ready<CG>(p, t, wc)) break;
        asm volatile("st.release.cta.shared.b32 [%0], %1;" ::"r"(smem_u32(ready_seq)), "r"(n) : "memory");
      }
    }
  } else if (MODE == SEG_CHAIN && warp == 3 + EPI_WARPS) {
    // -------------------------------- publisher --------------------------------
    // Waits until every epilogue warp has stored its part of a tile, then counts the tile
    // in on its block rows: the fence's wait for the stores delays no epilogue warp.
    Tiles<MODE, CG> it(p, groups, worker, workers);
    Tile t;
    for (int n = 1; it.next(t); ++n) {
      bool ok = true;
      if (lane < EPI_WARPS) ok = chain_seen(stored_seq + lane, n - 1, wc);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        __threadfence();
        atomicAdd(chain_counter(p, t.step, t.product, t.e, t.m0 / (128 * CG)), 1);
        if (t.product < 2 && t.n0 < t.m0) atomicAdd(chain_counter(p, t.step, t.product, t.e, t.n0 / (128 * CG)), 1);
      }
      __syncwarp();
    }
  } else {
    // -------------------------------- epilogue --------------------------------
    const int q = warp & 3;                 // this warp's tensor-memory lane quarter
    const int c_first = (warp - 2) >> 2;    // it takes every other 32-column chunk
    const uint32_t turn = base + TURN0 + (uint32_t)((warp - 2) * TURN_BYTES);
    uint32_t acc_it = 0;
    int tile_no = 0;   // CHAIN
    Tiles<MODE, CG> it(p, groups, worker, workers);
    Tile t;
    while (it.next(t)) {
      const int buf = (int)(acc_it & 1u);
      const int64_t m = (int64_t)t.m0 + rank * 128 + q * 32;   // this warp's first M-side row
      const int m_left = (int)max((int64_t)0, min((int64_t)32, p.M - m));
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN);
      EpiParams ep = p.epi;
      EpiPtrs ptr = epi_ptrs(p.epi, t.e);
      float shift = 0.0f;
      bool store_n = true, store_t = false;   // as it is, transposed
      bool scratch_d = MODE == SEG_CHAIN;     // D is scratch
      const __half* c_lo = nullptr;           // CHAIN: second halves of C and D, if any
      __half* d_lo = nullptr;
      auto ext = [](int cols) { return MODE == SEG_CHAIN ? min(32, (cols + 7) & ~7) : cols; };
      if constexpr (MODE == SEG_CHAIN) {
        const bool late = t.step >= p.steps - 2, last = t.step == p.steps - 1;
        const int64_t second = (int64_t)p.batch * p.chain.stride_e, at_e = t.e * p.chain.stride_e;
        const int64_t at_x = t.e * p.chain.stride_x;
        ep.ldc = p.chain.lde;
        ep.ldd = p.chain.lde;
        ep.d_dtype = GEMM_F16;
        ep.vec_d = 1;
        ptr.C = p.chain.e + at_e;
        if (t.product == 0) {
          ep.alpha = p.chain.inv_x * p.chain.inv_x * p.chain.scale_e;
          ep.read_c = 0;
          shift = late ? p.chain.scale_e : 0.0f;
          ptr.D = p.chain.e + at_e;
          if (p.pairs) d_lo = p.chain.e + at_e + second;
          store_t = t.n0 < t.m0;
        } else if (t.product == 1) {
          ep.alpha = p.chain.c * p.chain.inv_e;
          ep.beta = late ? p.chain.b[1] : p.chain.b[0];
          shift = late ? -p.chain.a[1] * p.chain.scale_e : 0.0f;
          ptr.D = p.chain.f + at_e;
          if (p.pairs) {
            c_lo = p.chain.e + at_e + second;
            d_lo = p.chain.f + at_e + second;
          }
          store_t = t.n0 < t.m0;
        } else {
          ep.alpha = p.chain.inv_e * (last ? p.chain.inv_x : 1.0f);
          // a X: early from both halves of X.  A direction that G lacks is in no other term, and
          // what is rounded there grows by a in every later step (a single fp16 X leaves 15 per
          // cent of the result's norm for a matrix of rank 1, the pair 0.3).  In the last two
          // steps it comes by F's diagonal, which holds a, and X is not read again (a fifth of the
          // L2 traffic of tiles 768 deep); from the start the rounding of a sum near 3.4 to fp16
          // would grow with the small singular values (272 x 5632: relative error of the
          // result 2.6e-3 instead of 2.2e-3).
          if (late) {
            ep.read_c = 0;
          } else {
            ep.beta = p.chain.a[0];
            ptr.C = p.chain.x[t.step & 1] + at_x;
            c_lo = p.chain.xlo[t.step & 1] + at_x;
            ep.ldc = p.chain.ldx;
          }
          ep.ldd = p.chain.ldx;
          ptr.D = p.chain.x[(t.step + 1) & 1] + at_x;
          if (p.pairs || t.step + 3 < p.steps) d_lo = p.chain.xlo[(t.step + 1) & 1] + at_x;
          if (last) {
            ep.ldd = p.epi.ldd;
            ep.d_dtype = p.epi.d_dtype;
            ep.vec_d = p.epi.vec_d;
            ptr.D = static_cast<char*>(p.epi.D) + t.e * p.epi.stride_d * dtype_bytes(p.epi.d_dtype);
            d_lo = nullptr;
            store_t = p.store_t != 0;
            store_n = !store_t;
            scratch_d = false;
          }
        }
      }
      CChunk cc, cl;
      cc.held = cl.held = false;
      // (one answer for the warp: lanes that saw the flag and lanes that saw an abort must not part)
      if (MODE == SEG_CHAIN && !__all_sync(0xffffffffu, chain_seen(ready_seq, tile_no++, wc))) break;
      if (MODE != SEG_TOKENS && ep.read_c)   // the first C chunk comes in during the MMAs
        load_c(ep, ptr.C, m, (int64_t)t.n0 + c_first * 32, m_left, ext(t.n_valid - c_first * 32), cc);
      if (MODE == SEG_CHAIN && c_lo != nullptr)
        load_c(ep, c_lo, m, (int64_t)t.n0 + c_first * 32, m_left, ext(t.n_valid - c_first * 32), cl);
      if (t.k > 0) {
        if (!warp_wait(tfull_bar(buf), (acc_it >> 1) & 1u, wc)) break;
        tc_fence_after();
      }
      // Chunk c of the accumulator into r (asynchronously: tmem_wait_ld before its use).
      uint32_t r[32];
      auto fetch = [&](int c) {
        if (t.k > 0) {
          tmem_ld_32x32b_x32(tb + (uint32_t)(c * 32), r);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0u;
        }
      };
      if (MODE == SEG_TOKENS && p.m_scale != nullptr && lane < m_left) ep.alpha *= p.m_scale[t.e * p.M + m + lane];
      auto take = [&](float (&x)[32]) {
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = ep.alpha * __uint_as_float(r[j]);
      };
      const int chunks = (t.n_valid + 31) / 32;
      // The accumulator is free for the next tile but one as soon as it is read.
      auto release = [&]() {
        if (t.k == 0) return;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(tempty_bar(buf));
          else mbar_arrive_cluster(mapa_shared(tempty_bar(buf), 0));
        }
        ++acc_it;
      };
      if (c_first < chunks) fetch(c_first);
      else release();
      if constexpr (MODE == SEG_TOKENS) {
        float bias = 0.0f;
        if (p.epi.bias_mode == GEMM_BIAS_COL && lane < m_left)
          bias = load_as_float(p.epi.bias, p.epi.bias_dtype, t.e * p.epi.stride_bias + m + lane);
        auto run = [&](auto dt) {
#pragma unroll 1
          for (int c = c_first; c < chunks; c += 2) {
            float x[32];
            take(x);
            if (c + 2 < chunks) fetch(c + 2);   // the next chunk while this one is stored
            else release();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              x[j] += bias;
              if (p.epi.relu) x[j] = relu_keep_nan(x[j]);
            }
            store_chunk_t<decltype(dt)::value>(p.epi.D, p.epi.ldd, (int64_t)t.n0 + c * 32, m, t.n_valid - c * 32, m_left,
                                               x, turn, p.epi.vec_d);
          }
        };
        with_type(p.epi.d_dtype, run);
      } else {
        auto run = [&](auto dt) {
          constexpr int DT = decltype(dt)::value;
#pragma unroll 1
          for (int c = c_first; c < chunks; c += 2) {
            const int64_t n = (int64_t)t.n0 + c * 32;
            // (CHAIN's scratch has rows of whole 16-byte pieces: their spare entries may be
            // read and written)
            const int n_left = t.n_valid - c * 32, n_ext = scratch_d ? ext(n_left) : n_left;
            float x[32];
            take(x);
            // The next chunk while this one is stored.  (CHAIN fetches it afterwards: with both
            // halves of C in registers the compiler would spill, which waits for the loads.)
            if (c + 2 >= chunks) release();
            else if (MODE != SEG_CHAIN) fetch(c + 2);
            if (ep.read_c) {
              add_c(ep, ptr.C, m, n, m_left, ext(n_left), cc, x, turn);
              if (c + 2 < chunks) load_c(ep, ptr.C, m, n + 64, m_left, ext(n_left - 64), cc);
            }
            if (MODE == SEG_CHAIN && c_lo != nullptr) {
              fma_c16(ep, x, cl.w, 0, 16);   // (scratch: always held)
              if (c + 2 < chunks) load_c(ep, c_lo, m, n + 64, m_left, ext(n_left - 64), cl);
            }
            if (MODE == SEG_CHAIN && shift != 0.0f) {
              const int64_t d = m + lane - n;   // the diagonal crosses this row of the chunk at column d
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == d) x[j] -= shift;
            }
            if (store_n) store_chunk<DT>(ptr.D, ep.ldd, m, n, m_left, n_ext, x, turn, ep.vec_d);
            if (MODE == SEG_CHAIN && store_t)
              store_chunk_t<DT>(ptr.D, ep.ldd, n, m, n_left, scratch_d ? ext(m_left) : m_left, x, turn, ep.vec_d);
            if (MODE == SEG_CHAIN && DT == GEMM_F16 && d_lo != nullptr) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] -= __half2float(__float2half_rn(x[j]));
              store_chunk<DT>(d_lo, ep.ldd, m, n, m_left, n_ext, x, turn, ep.vec_d);
              if (store_t) store_chunk_t<DT>(d_lo, ep.ldd, n, m, n_left, ext(m_left), x, turn, ep.vec_d);
            }
            if (MODE == SEG_CHAIN && c + 2 < chunks) fetch(c + 2);
          }
        };
        with_type(ep.d_dtype, run);
      }
      if constexpr (MODE == SEG_CHAIN) {
        // This warp's part of the tile is stored: tell the publisher.
        __syncwarp();
        if (lane == 0)
          asm volatile("st.release.cta.shared.b32 [%0], %1;" ::"r"(smem_u32(stored_seq + warp - 2)), "r"(tile_no) : "memory");
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();   // neither CTA leaves while the other may still signal it
  else __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (CG == 2) tmem_dealloc_pair(tmem_base, 2 * BN);
    else tmem_dealloc(tmem_base, 2 * BN);
  }
}

// Per group and operand a copy of the operand's tensor map with the group's first
// row as its base and the group's row count as its extent.  One warp per map.
__global__ void __launch_bounds__(32) wgrad_maps_kernel(const __grid_constant__ SegParams p, CUtensorMap* maps) {
  pdl_launch_dependents();   // the products' prologue may begin
  pdl_wait();
  const int e = (int)blockIdx.x >> 1, which = (int)blockIdx.x & 1, lane = threadIdx.x;
  int lo, hi;
  group_range(p.groups, e, lo, hi);
  if (hi == lo) return;   // never used
  CUtensorMap* out = maps + blockIdx.x;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(which ? &p.tmB[0] : &p.tmA);
  reinterpret_cast<uint32_t*>(out)[lane] = src[lane];
  __syncwarp();
  if (lane == 0) {
    const uint64_t addr = which ? p.b_base + (uint64_t)lo * p.b_pitch : p.a_base + (uint64_t)lo * p.a_pitch;
    asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(out), "l"(addr) : "memory");
    asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(out), "r"(hi - lo) : "memory");
    asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
    __threadfence();
  }
}

template <int CG, bool A_MN, bool B_MN, int MODE>
cudaError_t launch_mode(const SegParams& p, int workers, cudaStream_t stream) {
  constexpr bool GROUPED = MODE == SEG_TOKENS || MODE == SEG_WGRAD;
  const size_t smem = FIXED_SMEM + (GROUPED ? (3 * (size_t)p.groups.count + 1) * sizeof(int) : 0);
  constexpr size_t MOST = FIXED_SMEM + (GROUPED ? (3 * (size_t)kMaxGroups + 1) * sizeof(int) : 0);
  static_assert(MOST <= 232448, "shared memory budget");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static bool configured[64] = {};
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(seg_kernel<CG, A_MN, B_MN, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MOST);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(CG * workers), 1, 1);
  cfg.blockDim = dim3(SegThreads<MODE>::COUNT, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  if (MODE == SEG_CHAIN) {   // its CTAs wait for one another: all of them are resident, or none runs
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, seg_kernel<CG, A_MN, B_MN, MODE>, p);
}

template <int CG>
cudaError_t launch_cg(const SegParams& p, int mode, bool a_mn, int workers, cudaStream_t stream) {
  switch (mode) {
    case SEG_TOKENS:
      return a_mn ? launch_mode<CG, true, false, SEG_TOKENS>(p, workers, stream)
                  : launch_mode<CG, false, false, SEG_TOKENS>(p, workers, stream);
    case SEG_WGRAD: return launch_mode<CG, true, true, SEG_WGRAD>(p, workers, stream);
    default: return launch_mode<CG, false, false, SEG_CHAIN>(p, workers, stream);
  }
}

}  // namespace

cudaError_t launch_wgrad_maps(const SegParams& p, CUtensorMap* maps, cudaStream_t stream) {
  return launch_dependent(wgrad_maps_kernel, dim3(2u * (unsigned)p.groups.count), 32, stream, p, maps);
}

cudaError_t launch_seg(const SegParams& p, int mode, int cg, bool a_mn, int workers, cudaStream_t stream) {
  if (workers <= 0) return cudaErrorInvalidValue;
  return cg == 2 ? launch_cg<2>(p, mode, a_mn, workers, stream) : launch_cg<1>(p, mode, a_mn, workers, stream);
}

}  // namespace gemmlib
