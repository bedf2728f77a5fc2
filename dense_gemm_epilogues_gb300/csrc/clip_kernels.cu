// clip_kernels.cu -- the global norm of many tensors, and the tensors scaled to a bound:
//     n = sqrt(sum over all entries of g^2),   g' = g * min(1, max_norm / (n + eps)).
//
// Two passes over the list, each a launch (or one per 1024 tensors): the sums of squares,
// one fp64 number per CTA, then every CTA of the second pass adds those in one fixed order
// and scales its share, last entries first, since those are what the first pass left in L2.
// A CTA takes chunks of the tensors laid end to end (each tensor starts a chunk), so one
// long tensor and a thousand short ones occupy the chip alike.  Bound by memory: three
// trips over lists longer than L2, of which two are the floor.  369 million fp32 entries to
// bf16: 549 us, 6.7 TB/s over the three trips (2.2 GB are the floor's, 3.7 move); 2.1 million,
// fp32: 8.6 us.
//
// Squares are added in fp32 over eight entries at a time and over four such sums, then in
// fp64, in which only one warp of a CTA adds up and one thread takes the root: this chip adds
// two fp64 numbers per SM and clock (every thread taking the root itself cost 20 us).  Eight
// entries whose sum leaves the range that fp32 holds well (below 1e-30, above
// 1e37) are squared in fp64 instead, so entries of any size that fp32 holds count.
#include "layer.h"

namespace gemmlib {
namespace {

constexpr int THREADS = 512;
// Units of 8 entries that a thread has under way: 128 bytes where they are only read (beside the
// scaled values eight units would leave room for one CTA per SM).
__host__ __device__ constexpr int units_of(int dtype, bool scales) { return dtype == GEMM_F32 || scales ? 4 : 8; }

template <int CAP>
struct ClipList {
  const void* src[CAP];
  void* dst[CAP];
  int64_t count[CAP];
  int32_t first[CAP + 1];   // first chunks
  uint8_t types[CAP];       // src_type | dst_type << 4
  int32_t tensors;
};
static_assert(sizeof(ClipList<ClipTensors::LARGE>) + sizeof(ClipPass) + 16 <= 32764, "kernel parameters");

// The tensor of chunk c.
template <int CAP>
__device__ __forceinline__ int tensor_of(const ClipList<CAP>& l, int c) {
  int lo = 0, hi = l.tensors;   // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A tensor is cut into units of eight entries at its own alignment: the first unit starts
// `lead` entries before the tensor, where the memory is aligned to eight of them, so that
// all but the ends of a tensor moves 16 (fp32: 32) bytes at a time, wherever it starts.
__host__ __device__ __forceinline__ int lead_of(const void* p, int es) {
  return (int)((reinterpret_cast<uintptr_t>(p) & (uintptr_t)(8 * es - 1)) / (unsigned)es);
}

// Entries i .. i + 7 (zeros outside 0 .. n - 1) as they lie in memory: 16 bits take half the
// registers of their values while a thread's units are under way.
template <int DT>
struct Unit {
  static constexpr int WORDS = DT == GEMM_F32 ? 8 : 4;
  uint32_t w[WORDS];

  __device__ __forceinline__ void load(const void* p, int64_t i, int64_t n) {
    if (i >= 0 && i + 8 <= n) {
      if constexpr (DT == GEMM_F32) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(static_cast<const float*>(p) + i)
                     : "memory");
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < WORDS; ++k) w[k] = 0u;
    if (i >= n) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i + j < 0 || i + j >= n) continue;
      if constexpr (DT == GEMM_F32) w[j] = static_cast<const uint32_t*>(p)[i + j];
      else w[j / 2] |= (uint32_t) static_cast<const uint16_t*>(p)[i + j] << (16 * (j % 2));
    }
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if constexpr (DT == GEMM_F32) x[2 * h] = __uint_as_float(w[2 * h]), x[2 * h + 1] = __uint_as_float(w[2 * h + 1]);
      else unpack2<DT>(w[h], x[2 * h], x[2 * h + 1]);
    }
  }
};

// vec: the units are aligned in this tensor too.
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, int64_t n, bool vec, const float (&x)[8]) {
  if (vec && i >= 0 && i + 8 <= n) {
    uint32_t w[8];
    if constexpr (DT == GEMM_F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[j]);
      st_row_32b(static_cast<float*>(p) + i, w);
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) w[h] = pack2<DT>(x[2 * h], x[2 * h + 1]);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j >= 0 && i + j < n) store_float_as(p, DT, i + j, x[j]);
  }
}

// Where this thread's u-th unit of a step starts (a warp's units lie side by side).
__device__ __forceinline__ int64_t unit_at(int64_t base, int u) {
  return base + ((int64_t)u * THREADS + threadIdx.x) * 8;
}

// The sum of squares of eight entries: in fp32, or added to `wide` in fp64.
__device__ __forceinline__ float squares(const float (&x)[8], double& wide) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
  if (s >= 1e-30f && s <= 1e37f) return s;
  float most = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]));
  if (s == 0.0f && most == 0.0f) return 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) wide += (double)x[j] * (double)x[j];
  return 0.0f;
}

// The sum of n doubles in shared or global memory by one warp, in one order; valid in lane 0.
__device__ __forceinline__ double warp_total(const double* v, int n, int lane) {
  double s = 0.0;
  for (int i = lane; i < n; i += 32 * 10) {   // (ten loads under way: all of 304 CTAs')
    double x[10];
#pragma unroll
    for (int u = 0; u < 10; ++u) x[u] = i + 32 * u < n ? v[i + 32 * u] : 0.0;
#pragma unroll
    for (int u = 0; u < 10; ++u)
      if (i + 32 * u < n) s += x[u];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int CAP>
__global__ void __launch_bounds__(THREADS, 2) clip_norm_kernel(const __grid_constant__ ClipList<CAP> l,
                                                            const __grid_constant__ ClipPass p, int first_partial) {
  __shared__ double smem[THREADS];
  pdl_launch_dependents();
  pdl_wait();
  double wide = 0.0;
  const int chunks = l.first[l.tensors];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(l, c);
    const void* src = l.src[t];
    with_type(l.types[t] & 15, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      const int64_t lo = (int64_t)(c - l.first[t]) * p.chunk - lead_of(src, DT == GEMM_F32 ? 4 : 2);
      const int64_t hi = min(l.count[t], lo + p.chunk);
      constexpr int UNITS = units_of(DT, false);
      for (int64_t at = lo; at < hi; at += 8 * THREADS * UNITS) {
        Unit<DT> v[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) v[u].load(src, unit_at(at, u), hi);
#pragma unroll
        for (int h = 0; h < UNITS; h += 4) {
          float s = 0.0f;
#pragma unroll
          for (int u = h; u < h + 4; ++u) {
            float x[8];
            v[u].get(x);
            if (unit_at(at, u) < hi) s += squares(x, wide);
          }
          if (s != 0.0f) wide += (double)s;
        }
      }
    });
  }
  smem[threadIdx.x] = wide;
  __syncthreads();
  if (threadIdx.x < 32) {
    const double sum = warp_total(smem, THREADS, (int)threadIdx.x);
    if (threadIdx.x == 0) p.partials[first_partial + blockIdx.x] = sum;
  }
}

template <int CAP>
__global__ void __launch_bounds__(THREADS, 2) clip_scale_kernel(const __grid_constant__ ClipList<CAP> l,
                                                             const __grid_constant__ ClipPass p, int write_norm) {
  __shared__ float factor;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x < 32) {
    const double sum = warp_total(p.partials, p.num_partials, (int)threadIdx.x);
    if (threadIdx.x == 0) {
      const double n = sqrt(sum);
      const float norm = (float)n;
      if (write_norm && blockIdx.x == 0) *p.norm = norm;
      factor = isfinite(norm) ? fminf(1.0f, (float)((double)p.max_norm / (n + (double)p.eps))) : 1.0f;
    }
  }
  __syncthreads();
  const float scale = factor;
  const int chunks = p.scales ? l.first[l.tensors] : 0;
  for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
    const int c = chunks - 1 - i, t = tensor_of(l, c);
    const void* src = l.src[t];
    void* dst = l.dst[t];
    if (dst == nullptr || (dst == src && scale == 1.0f)) continue;
    with_type(l.types[t] & 15, [&](auto st) {
      constexpr int ST = decltype(st)::value;
      with_type(l.types[t] >> 4, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const int lead = lead_of(src, ST == GEMM_F32 ? 4 : 2);
        const int64_t lo = (int64_t)(c - l.first[t]) * p.chunk - lead, hi = min(l.count[t], lo + p.chunk);
        const uintptr_t from = reinterpret_cast<uintptr_t>(dst) - (uintptr_t)(lead * (DT == GEMM_F32 ? 4 : 2));
        const bool vec = (from & 15) == 0;
        constexpr int UNITS = units_of(ST, true);
        for (int64_t at = lo; at < hi; at += 8 * THREADS * UNITS) {
          Unit<ST> v[UNITS];
#pragma unroll
          for (int u = 0; u < UNITS; ++u) v[u].load(src, unit_at(at, u), hi);
#pragma unroll
          for (int u = 0; u < UNITS; ++u) {
            float x[8];
            v[u].get(x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= scale;
            if (unit_at(at, u) < hi) store8<DT>(dst, unit_at(at, u), hi, vec, x);
          }
        }
      });
    });
  }
}

int64_t chunks_of(const ClipTensor& t, int64_t chunk) {
  return t.count == 0 ? 0 : (t.count + lead_of(t.src, dtype_bytes(t.src_type)) + chunk - 1) / chunk;
}

template <int CAP>
ClipList<CAP> list_of(const ClipTensor* t, int count, int64_t chunk) {
  ClipList<CAP> l;
  l.first[0] = 0;
  for (int i = 0; i < count; ++i) {
    l.src[i] = t[i].src;
    l.dst[i] = t[i].dst;
    l.count[i] = t[i].count;
    l.first[i + 1] = l.first[i] + (int32_t)chunks_of(t[i], chunk);
    l.types[i] = (uint8_t)(t[i].src_type | t[i].dst_type << 4);
  }
  l.tensors = count;
  return l;
}

}  // namespace

// Up to 32768 entries, so that finding a chunk's tensor costs nothing beside it, and as many
// that all resident CTAs (two per SM) take equally many: 10.5 million bf16 entries 17 us, with
// chunks of 8192 22.
int64_t clip_chunk(int64_t total, int sm_count) {
  const int64_t ctas = 2 * (int64_t)sm_count;
  const int64_t rounds = std::max<int64_t>(1, (total + ctas * 32768 - 1) / (ctas * 32768));
  int64_t chunk = std::max<int64_t>(1, (total + ctas * rounds - 1) / (ctas * rounds) + 4095) / 4096 * 4096;
  chunk = std::max<int64_t>(4096, chunk);
  while (total / chunk >= (int64_t(1) << 30)) chunk *= 2;   // (chunk numbers are 32-bit)
  return chunk;
}

int clip_blocks(const ClipTensor* t, int count, int64_t chunk, int sm_count) {
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) chunks += chunks_of(t[i], chunk);
  return (int)std::max<int64_t>(1, std::min<int64_t>(chunks, 2 * (int64_t)sm_count));
}

cudaError_t launch_clip_norm(const ClipTensor* t, int count, const ClipPass& p, int first_partial, int blocks,
                             cudaStream_t stream) {
  if (count <= ClipTensors::SMALL)
    return launch_dependent(clip_norm_kernel<ClipTensors::SMALL>, dim3(blocks), THREADS, stream,
                            list_of<ClipTensors::SMALL>(t, count, p.chunk), p, first_partial);
  return launch_dependent(clip_norm_kernel<ClipTensors::LARGE>, dim3(blocks), THREADS, stream,
                          list_of<ClipTensors::LARGE>(t, count, p.chunk), p, first_partial);
}

cudaError_t launch_clip_scale(const ClipTensor* t, int count, const ClipPass& p, bool first, int blocks,
                              cudaStream_t stream) {
  const int write = first ? 1 : 0;
  if (count <= ClipTensors::SMALL)
    return launch_dependent(clip_scale_kernel<ClipTensors::SMALL>, dim3(blocks), THREADS, stream,
                            list_of<ClipTensors::SMALL>(t, count, p.chunk), p, write);
  return launch_dependent(clip_scale_kernel<ClipTensors::LARGE>, dim3(blocks), THREADS, stream,
                          list_of<ClipTensors::LARGE>(t, count, p.chunk), p, write);
}

}  // namespace gemmlib
