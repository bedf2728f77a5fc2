// seg_kernel.cu -- tcgen05 products whose tiles are not one dense problem's:
//   TOKENS  D[r, :] = act(alpha * A[r, :] * op(B_g) + bias_g) for the rows r of each
//           group g (rows found on the device);
//   WGRAD   D_g = alpha * A_g' * B_g + beta * C_g, the sum over the rows of group g;
//   SYM     D = alpha * X * X' + beta * C - shift * I, symmetric: tiles on and below
//           the diagonal are computed, each also stored transposed;
//   DENSE   D = alpha * A * B + beta * C, optionally stored transposed.
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
// Every mbarrier wait is bounded, as in tc_kernel.cu.
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
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int TURN_BYTES = 2048;                      // an epilogue warp's turn-around buffer
constexpr int NUM_BARS = 2 * STAGES + 5;
constexpr size_t FIXED_SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + EPI_WARPS * TURN_BYTES + NUM_BARS * 8 + 16;

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t user_timeout_ns) {
  const uint64_t timeout_ns = user_timeout_ns > 1000000000ull ? user_timeout_ns : 1000000000ull;
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > timeout_ns) return;
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

// 32 rows of 64 bytes (lane: its row's 16 words) stored as whole sectors, 8 rows
// per instruction; `esize`-byte elements, rows r < rows, columns j < cols (64 /
// esize of them when `vec`, which needs 16-byte aligned rows).
template <int ES>
__device__ __forceinline__ void store_rows64(char* D, int64_t pitch, int rows, int cols, const uint32_t (&w)[16],
                                             uint32_t turn, bool vec) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the buffer's last readers are done
#pragma unroll
  for (int q = 0; q < 4; ++q)
    sts128(turn + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  __syncwarp();
  if (vec) {
    const int pl = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      const uint4 v = lds128(turn + (uint32_t)(r * 64 + ((pl ^ ((r >> 1) & 3)) << 4)));
      if (r < rows) *reinterpret_cast<uint4*>(D + r * pitch + pl * 16) = v;
    }
  } else {
    constexpr int PER = 64 / ES, RPI = 32 / PER;   // elements per row, rows per instruction
    const int j = lane % PER;
#pragma unroll 4
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
}

// A warp's 32 x 32 chunk, lane r = row r, x = its columns: D[r][j], r < rows, j < cols.
template <int DT>
__device__ __forceinline__ void store_chunk(void* D, int64_t ldd, int64_t r0, int64_t c0, int rows, int cols,
                                            const float (&x)[32], uint32_t turn, bool vec) {
  const bool v = vec && cols >= 32;
  uint32_t w[16];
  if constexpr (DT == GEMM_F32) {
    char* d = reinterpret_cast<char*>(static_cast<float*>(D) + r0 * ldd + c0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(x[16 * h + j]);
      store_rows64<4>(d + h * 64, ldd * 4, rows, cols - 16 * h, w, turn, v);
    }
  } else {
    char* d = reinterpret_cast<char*>(static_cast<uint16_t*>(D) + r0 * ldd + c0);
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack2<DT>(x[2 * j], x[2 * j + 1]);
    store_rows64<2>(d, ldd * 2, rows, cols, w, turn, v);
  }
}

// The same chunk stored transposed: D[j][r], j < rows_out, r < cols_out.
template <int DT>
__device__ __forceinline__ void store_chunk_t(void* D, int64_t ldd, int64_t j0, int64_t r0, int rows_out, int cols_out,
                                              const float (&x)[32], uint32_t turn, bool vec) {
  const int lane = threadIdx.x & 31;
  const bool v = vec && cols_out >= 32;
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
        if (16 * h + j < rows_out) *reinterpret_cast<uint4*>(d + (16 * h + j) * ldd + (lane & 7) * 4) = q;
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
      if (2 * p < rows_out) *reinterpret_cast<uint4*>(d + (2 * p) * ldd + o * 8) = lo;
      if (2 * p + 1 < rows_out) *reinterpret_cast<uint4*>(d + (2 * p + 1) * ldd + o * 8) = hi;
    }
  }
}

// x += beta * C for a chunk (lane r = row r): whole rows of 16-bit C turned around
// through the buffer, other types or edges element by element.
__device__ __forceinline__ void add_c(const EpiParams& e, const void* C, int64_t r0, int64_t c0, int rows, int cols,
                                      float (&x)[32], uint32_t turn) {
  const int lane = threadIdx.x & 31;
  if (e.vec_c && cols >= 32 && e.c_dtype != GEMM_F32) {
    const uint16_t* src = static_cast<const uint16_t*>(C) + r0 * e.ldc + c0;
    const int pl = lane & 3;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) v[i] = *reinterpret_cast<const uint4*>(src + r * e.ldc + pl * 8);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      sts128(turn + (uint32_t)(r * 64 + ((pl ^ ((r >> 1) & 3)) << 4)), v[i].x, v[i].y, v[i].z, v[i].w);
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 c = lds128(turn + (uint32_t)(lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)));
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float lo, hi;
        if (e.c_dtype == GEMM_F16) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[h]));
          lo = f.x;
          hi = f.y;
        } else {
          lo = __uint_as_float(w[h] << 16);
          hi = __uint_as_float(w[h] & 0xffff0000u);
        }
        x[8 * q + 2 * h] = fmaf(e.beta, lo, x[8 * q + 2 * h]);
        x[8 * q + 2 * h + 1] = fmaf(e.beta, hi, x[8 * q + 2 * h + 1]);
      }
    }
  } else if (lane < rows) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < cols) x[j] = fmaf(e.beta, load_as_float(C, e.c_dtype, (r0 + lane) * e.ldc + c0 + j), x[j]);
  }
}

// ---------------------------------- tiles -----------------------------------

struct Tile {
  int e;          // group (TOKENS, WGRAD) or matrix of the batch (SYM, DENSE)
  int m0, n0;     // first row of the M side and of the N side (TOKENS: the buffer's row)
  int n_valid;    // N-side rows that exist
  int n_mma;      // the MMA's N (a multiple of 16)
  int k;          // depth
};

// Shared-memory tables of TOKENS: the groups' first rows, row counts and first tiles.
struct GroupTable {
  int *lo, *cnt, *cum;
};

template <int MODE, int CG>
struct Tiles {
  static constexpr int BM = 128 * CG, BN = 128 * CG;
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
    } else {
      if (t >= p.num_tiles) return false;
      o.e = t / p.tiles_per_group;
      const int local = t - o.e * p.tiles_per_group;
      int tm, tn;
      if (MODE == SEG_SYM) {
        tm = (int)((sqrtf(8.0f * (float)local + 1.0f) - 1.0f) * 0.5f);
        while ((tm + 1) * (tm + 2) / 2 <= local) ++tm;
        while (tm * (tm + 1) / 2 > local) --tm;
        tn = local - tm * (tm + 1) / 2;
      } else {
        const int band = local / (8 * p.tiles_n), first = band * 8, size = min(8, p.tiles_m - first);
        const int r = local - first * p.tiles_n;
        tn = r / size;
        tm = first + r - tn * size;
      }
      o.m0 = tm * BM;
      o.n0 = tn * BN;
      o.n_valid = min(BN, p.N - o.n0);
      o.n_mma = BN;
      o.k = p.K;
      if constexpr (MODE == SEG_WGRAD) {
        int lo, hi;
        group_range(p.groups, o.e, lo, hi);
        o.k = hi - lo;
      }
    }
    t += step;
    return true;
  }
};

template <int CG, bool A_MN, bool B_MN, int MODE>
__global__ void __launch_bounds__(THREADS, 1) seg_kernel(const __grid_constant__ SegParams p) {
  constexpr int BN = 128 * CG;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;   // the same offset in both CTAs of a pair
  uint8_t* base_ptr = smem_raw + (base - raw);
  constexpr uint32_t TURN0 = STAGES * STAGE_BYTES, BAR0 = TURN0 + EPI_WARPS * TURN_BYTES;
  const uint32_t bar0 = base + BAR0;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + BAR0 + NUM_BARS * 8);
  volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
  int* table = reinterpret_cast<int*>(tmem_slot + 4);
  const GroupTable groups{table, table + p.groups.count, table + 2 * p.groups.count};

  auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * STAGES + 2 + b); };
  const uint32_t teardown_bar = bar0 + 8u * (uint32_t)(2 * STAGES + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  pdl_launch_dependents();
  pdl_wait();
  if constexpr (MODE == SEG_TOKENS) {
    const int E = p.groups.count;
    for (int e = threadIdx.x; e < E; e += THREADS) {
      int lo, hi;
      group_range(p.groups, e, lo, hi);
      groups.lo[e] = lo;
      groups.cnt[e] = hi - lo;
    }
    __syncthreads();
    if (warp == 0) {
      int sum = 0;
      for (int e0 = 0; e0 < E; e0 += 32) {
        int v = e0 + lane < E ? (groups.cnt[e0 + lane] + BN - 1) / BN * p.tiles_m : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += u;
        }
        if (e0 + lane < E) groups.cum[e0 + lane + 1] = sum + v;
        sum += __shfl_sync(0xffffffffu, v, 31);
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
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, last_parity = 0;
      bool ok = true;
      int map_of = -1;   // WGRAD: the group whose tensor maps were last acquired
      Tiles<MODE, CG> it(p, groups, worker, workers);
      Tile t;
      while (ok && it.next(t)) {
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
          if (map_of != t.e && t.k > 0) {
            tensormap_acquire(ma);
            tensormap_acquire(mb);
            map_of = t.e;
          }
        } else {
          za = zb = t.e;
        }
        const int num_kb = (t.k + TC_BK - 1) / TC_BK;
        for (int kb = 0; kb < num_kb; kb += SLABS) {
          const int nsl = min(SLABS, num_kb - kb);
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, wc)) { ok = false; break; }
          const uint32_t a_bytes = (uint32_t)(A_MN ? SLABS : nsl) * (uint32_t)SLAB_BYTES;
          const uint32_t b_bytes = (uint32_t)(B_MN ? SLABS : nsl) * b_slab;
          if (leader) mbar_expect_tx(full_bar(stage), (uint32_t)CG * (a_bytes + b_bytes));
          const uint32_t fb = leader ? full_bar(stage) : mapa_shared(full_bar(stage), 0);
          const uint32_t sa = base + (uint32_t)(stage * STAGE_BYTES), sb = sa + (uint32_t)OPERAND_BYTES;
          auto load = [&](uint32_t dst, const CUtensorMap* tm, int x, int y, int z) {
            if constexpr (CG == 2) tma_load_3d_pair(dst, tm, x, y, z, fb);
            else tma_load_3d(dst, tm, x, y, z, fb);
          };
          const int k0 = kb * TC_BK;
          if constexpr (A_MN) {
#pragma unroll
            for (int h = 0; h < 2; ++h) load(sa + h * MN_BOX_BYTES, ma, m0 + h * 64, k0, za);
          } else {
            for (int sl = 0; sl < nsl; ++sl) load(sa + sl * SLAB_BYTES, ma, k0 + sl * TC_BK, m0, za);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int h = 0; h < 2; ++h) load(sb + h * MN_BOX_BYTES, mb, n0 + h * 64, k0, zb);
          } else {
            for (int sl = 0; sl < nsl; ++sl) load(sb + sl * SLAB_BYTES, mb, k0 + sl * TC_BK, n0, zb);
          }
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // No copy is in flight when the CTA leaves (the peer of a pair waits at the last
      // cluster barrier: its copies complete on the leader's barriers).
      if (leader) {
        for (int s = 0; s < STAGES; ++s)
          if (issued & (1u << s)) drain_wait(full_bar(s), (last_parity >> s) & 1u, p.timeout_ns);
      } else if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------ MMA issuer (the leader's) -----------------------
    if (leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0, acc_it = 0;
      bool ok = true;
      Tiles<MODE, CG> it(p, groups, worker, workers);
      Tile t;
      while (ok && it.next(t)) {
        if (t.k == 0) continue;
        const int buf = (int)(acc_it & 1u);
        if (!mbar_wait(tempty_bar(buf), ((acc_it >> 1) & 1u) ^ 1u, wc)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(buf * BN);
        const uint32_t idesc = p.idesc | ((uint32_t)(t.n_mma >> 3) << 17);
        const int num_kb = (t.k + TC_BK - 1) / TC_BK, num_k16 = (t.k + 15) / 16;
        for (int kb = 0; kb < num_kb; kb += SLABS) {
          if (!mbar_wait(full_bar(stage), phase, wc)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = base + (uint32_t)(stage * STAGE_BYTES), sb = sa + (uint32_t)OPERAND_BYTES;
#pragma unroll
          for (int q = 0; q < SLABS * (TC_BK / 16); ++q) {
            const int sl = q / (TC_BK / 16), kk = q % (TC_BK / 16);
            if (kb * (TC_BK / 16) + q < num_k16) {
              const uint64_t ad = A_MN ? smem_desc_sw128(sa + q * 2048u, MN_BOX_BYTES, 1024)
                                       : smem_desc_sw128(sa + sl * SLAB_BYTES + kk * 32u, 16, 1024);
              const uint64_t bd = B_MN ? smem_desc_sw128(sb + q * 2048u, MN_BOX_BYTES, 1024)
                                       : smem_desc_sw128(sb + sl * SLAB_BYTES + kk * 32u, 16, 1024);
              if constexpr (CG == 2) tc_mma_f16_pair(d_tmem, ad, bd, idesc, (kb > 0 || q > 0) ? 1u : 0u);
              else tc_mma_f16(d_tmem, ad, bd, idesc, (kb > 0 || q > 0) ? 1u : 0u);
            }
          }
          if constexpr (CG == 2) tc_commit_pair_mask(empty_bar(stage), 0x3);
          else tc_commit(empty_bar(stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if constexpr (CG == 2) tc_commit_pair_mask(tfull_bar(buf), 0x3);
        else tc_commit(tfull_bar(buf));
        ++acc_it;
      }
      // Every MMA is complete before tensor memory is freed.
      if constexpr (CG == 2) tc_commit_pair(teardown_bar);
      else tc_commit(teardown_bar);
      drain_wait(teardown_bar, 0, p.timeout_ns);
    }
  } else {
    // -------------------------------- epilogue --------------------------------
    const int q = warp & 3;                 // this warp's tensor-memory lane quarter
    const int c_first = (warp - 2) >> 2;    // it takes every other 32-column chunk
    const uint32_t turn = base + TURN0 + (uint32_t)((warp - 2) * TURN_BYTES);
    uint32_t acc_it = 0;
    Tiles<MODE, CG> it(p, groups, worker, workers);
    Tile t;
    while (it.next(t)) {
      const int buf = (int)(acc_it & 1u);
      const int64_t m = (int64_t)t.m0 + rank * 128 + q * 32;   // this warp's first M-side row
      const int m_left = (int)max((int64_t)0, min((int64_t)32, p.M - m));
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN);
      if (t.k > 0) {
        if (!warp_wait(tfull_bar(buf), (acc_it >> 1) & 1u, wc)) break;
        tc_fence_after();
      }
      auto acc = [&](int c, float (&x)[32]) {
        if (t.k > 0) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tb + (uint32_t)(c * 32), r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = p.epi.alpha * __uint_as_float(r[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0.0f;
        }
      };
      const int chunks = (t.n_valid + 31) / 32;
      if constexpr (MODE == SEG_TOKENS) {
        float bias = 0.0f;
        if (p.epi.bias_mode == GEMM_BIAS_COL && lane < m_left)
          bias = load_as_float(p.epi.bias, p.epi.bias_dtype, t.e * p.epi.stride_bias + m + lane);
        auto run = [&](auto dt) {
#pragma unroll 1
          for (int c = c_first; c < chunks; c += 2) {
            float x[32];
            acc(c, x);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              x[j] += bias;
              if (p.epi.relu) x[j] = fmaxf(x[j], 0.0f);
            }
            store_chunk_t<decltype(dt)::value>(p.epi.D, p.epi.ldd, (int64_t)t.n0 + c * 32, m, t.n_valid - c * 32, m_left,
                                               x, turn, p.epi.vec_d);
          }
        };
        with_type(p.epi.d_dtype, run);
      } else {
        const EpiPtrs ptr = epi_ptrs(p.epi, t.e);
        auto run = [&](auto dt) {
          constexpr int DT = decltype(dt)::value;
#pragma unroll 1
          for (int c = c_first; c < chunks; c += 2) {
            const int64_t n = (int64_t)t.n0 + c * 32;
            const int n_left = t.n_valid - c * 32;
            float x[32];
            acc(c, x);
            if (p.epi.read_c) add_c(p.epi, ptr.C, m, n, m_left, n_left, x, turn);
            if (MODE == SEG_SYM && p.shift != 0.0f) {
              const int64_t d = m + lane - n;   // the diagonal crosses this row of the chunk at column d
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (j == d) x[j] -= p.shift;
            }
            if (MODE != SEG_DENSE || !p.store_t)
              store_chunk<DT>(ptr.D, p.epi.ldd, m, n, m_left, n_left, x, turn, p.epi.vec_d);
            if ((MODE == SEG_SYM && t.m0 != t.n0) || (MODE == SEG_DENSE && p.store_t))
              store_chunk_t<DT>(ptr.D, p.epi.ldd, n, m, n_left, m_left, x, turn, p.epi.vec_d);
          }
        };
        with_type(p.epi.d_dtype, run);
      }
      if (t.k > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(tempty_bar(buf));
          else mbar_arrive_cluster(mapa_shared(tempty_bar(buf), 0));
        }
        ++acc_it;
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
  const size_t smem = FIXED_SMEM + (MODE == SEG_TOKENS ? (3 * (size_t)p.groups.count + 1) * sizeof(int) : 0);
  constexpr size_t MOST = FIXED_SMEM + (MODE == SEG_TOKENS ? (3 * (size_t)kMaxGroups + 1) * sizeof(int) : 0);
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
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
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
    case SEG_SYM: return launch_mode<CG, false, false, SEG_SYM>(p, workers, stream);
    default: return launch_mode<CG, false, true, SEG_DENSE>(p, workers, stream);
  }
}

}  // namespace

cudaError_t launch_wgrad_maps(const SegParams& p, CUtensorMap* maps, cudaStream_t stream) {
  wgrad_maps_kernel<<<2 * p.groups.count, 32, 0, stream>>>(p, maps);
  return cudaGetLastError();
}

cudaError_t launch_seg(const SegParams& p, int mode, int cg, bool a_mn, int workers, cudaStream_t stream) {
  if (workers <= 0) return cudaErrorInvalidValue;
  return cg == 2 ? launch_cg<2>(p, mode, a_mn, workers, stream) : launch_cg<1>(p, mode, a_mn, workers, stream);
}

}  // namespace gemmlib
