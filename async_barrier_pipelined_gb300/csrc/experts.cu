// Rows of layers of experts: tokens sorted by expert (experts_maps), their
// rows in that order (experts_gather), and the experts' rows brought back with
// weights (experts_combine) with the gradients (experts_combine_gradient).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm_f8.h"
#include "host.h"
#include "ptx.cuh"

using namespace gf16;
using namespace gf16::host;

namespace {

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_ENTRIES = 1 << 26;
constexpr int MAX_SIZE = 0x7fffffff - 1023;

// ------------------------------------------------------------------ the sort
//
// A counting sort that keeps the entries' order, in one launch: one cluster of
// up to eight CTAs of 32 warps, each warp with its own run of entries and its
// own counts in shared memory, so that nothing is added atomically.  Twice over
// the entries: first each warp counts (lanes with the same expert found by
// match_any, their first one adds), then sums over warps, CTAs (read from the
// others' shared memory) and experts turn the counts into first rows, and the
// second time each entry's row is its warp's next one for that expert.
//
// Bound by latency: 32 entries a step and warp, 16 steps in all for 65,536
// entries over eight CTAs, and three rounds of barriers between.

constexpr int MAP_THREADS = 1024, MAP_WARPS = 32;
constexpr int MAP_CLUSTER = 8;
constexpr int ONE_CTA = 4096;     // entries up to which one CTA is as fast as a cluster

struct MapParams {
  int entries, experts, align, max_rows;
  const void* picks;
  int32_t *starts, *rows, *source;
  int* status;
};

template <typename I>
__global__ void __launch_bounds__(MAP_THREADS) experts_maps_kernel(const MapParams p) {
  extern __shared__ int32_t counts[];             // [32][experts]
  __shared__ int32_t total[MAX_EXPERTS];          // this CTA's entries of each expert
  __shared__ int32_t first[MAX_EXPERTS + 1];      // first row
  __shared__ int32_t next[MAX_EXPERTS];           // first row of this CTA's entries
  __shared__ int32_t ends[MAX_EXPERTS];           // end of an expert's entries
  __shared__ int32_t sums[MAP_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)ptx::cluster_ctarank(), ctas = (int)ptx::cluster_nctarank();
  const I* picks = static_cast<const I*>(p.picks);
  int32_t* mine = counts + warp * p.experts;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int e = threadIdx.x; e < MAP_WARPS * p.experts; e += MAP_THREADS) counts[e] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();

  const int runs = ctas * MAP_WARPS;
  const int run = ((p.entries + runs - 1) / runs + 31) / 32 * 32;
  const int64_t begin = (int64_t)(rank * MAP_WARPS + warp) * run;
  const int64_t end = min((int64_t)p.entries, begin + run);
  const auto expert_at = [&](int64_t i) {
    if (i >= end) return -1;
    const I e = picks[i];
    return e < 0 || e >= (I)p.experts ? -1 : (int)e;
  };
  for (int64_t i = begin; i < end; i += 32) {
    if (i + lane < end && picks[i + lane] >= (I)p.experts)
      *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
    const int e = expert_at(i + lane);
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += MAP_THREADS) {
    int sum = 0;
    for (int w = 0; w < MAP_WARPS; ++w) {
      const int c = counts[w * p.experts + e];
      counts[w * p.experts + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  __syncthreads();
  if (ctas > 1) ptx::cluster_sync();
  int before = 0, all = 0;
  const int e = threadIdx.x;
  if (e < p.experts) {
    for (int c = 0; c < ctas; ++c) {
      int t;
      if (ctas == 1) {
        t = total[e];
      } else {
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(t)
                     : "r"(ptx::map_to_cta(ptx::smem_u32(&total[e]), (uint32_t)c))
                     : "memory");
      }
      if (c < rank) before += t;
      all += t;
    }
  }
  if (ctas > 1) ptx::cluster_sync();   // none of the others reads `total` any more
  const int filled = (all + p.align - 1) / p.align * p.align;
  int sum = filled;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 31) sums[warp] = sum;
  __syncthreads();
  int base = sum - filled;
  for (int w = 0; w < warp; ++w) base += sums[w];
  if (e < p.experts) {
    first[e] = base;
    next[e] = base + before;
    ends[e] = base + all;
    if (e == p.experts - 1) first[p.experts] = base + filled;
    if (rank == 0) {
      p.starts[e] = base;
      if (e == p.experts - 1) p.starts[p.experts] = base + filled;
    }
  }
  __syncthreads();
  for (int64_t i = begin; i < end; i += 32) {
    const int x = expert_at(i + lane);
    const unsigned same = __match_any_sync(0xffffffffu, x);
    int row = -1;
    if (x >= 0) row = next[x] + mine[x] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (x >= 0 && lane == __ffs(same) - 1) mine[x] += __popc(same);
    __syncwarp();
    if (i + lane < end) {
      p.rows[i + lane] = row;
      if (row >= 0) p.source[row] = (int)(i + lane);
    }
  }
  // Rows that fill an expert's up, and those past the last expert.
  for (int x = rank * MAP_WARPS + warp; x < p.experts; x += runs)
    for (int r = ends[x] + lane; r < first[x + 1]; r += 32) p.source[r] = -1;
  for (int64_t r = (int64_t)first[p.experts] + rank * MAP_THREADS + threadIdx.x; r < p.max_rows;
       r += (int64_t)ctas * MAP_THREADS)
    p.source[r] = -1;
}

// ------------------------------------------------------------------ rows
//
// All three are bound by the memory.  A warp takes 512 bytes at a time (16 a
// lane) where rows start on 16-byte boundaries, else a number a lane.

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// V numbers of a row that move together: 16 bytes, or one number.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* at) {
  Vec<T, V> x;
  if constexpr (V > 1) *reinterpret_cast<uint4*>(x.v) = *reinterpret_cast<const uint4*>(at);
  else x.v[0] = *at;
  return x;
}
// `once`: read (written) and not wanted in the cache again.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_once(const T* at) {
  Vec<T, V> x;
  if constexpr (V > 1) *reinterpret_cast<uint4*>(x.v) = __ldcs(reinterpret_cast<const uint4*>(at));
  else x.v[0] = *at;
  return x;
}
template <typename T, int V>
__device__ __forceinline__ void store(T* at, const Vec<T, V>& x, bool once = false) {
  if constexpr (V > 1) {
    const uint4 v = *reinterpret_cast<const uint4*>(x.v);
    if (once) __stcs(reinterpret_cast<uint4*>(at), v);
    else *reinterpret_cast<uint4*>(at) = v;
  } else {
    *at = x.v[0];
  }
}

constexpr int ROW_THREADS = 256, ROW_WARPS = 8;

// Sorted rows of more bytes than this are written past the cache, which keeps
// the tokens' rows for the other choices: 8192 tokens of 4096 16-bit numbers to
// four experts each, there 75 -> 70 us (169 -> 138 MB read of the memory).
constexpr int64_t CACHE_BYTES = 48 << 20;
constexpr int COMBINE_LOADS = 8;

struct RowParams {
  int64_t rows;             // of the output
  int cols, choices;
  int64_t entries;
  const void* X;            // gather: X; combine: S; gradient: S
  int64_t ldx;
  int x_rows;
  const void* dY;
  int64_t lddy;
  const int32_t *map, *source;
  const void* w;
  void* Y;
  int64_t ldy;
  void* dw;
  int once;                 // the sorted rows are too many for the cache to keep
  int* status;
};

__device__ __forceinline__ void report(const RowParams& p) {
  *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
}

constexpr int GATHER_STEPS = 4;   // a warp's piece of a row: 4 x 32 units

template <typename T, int V>
__global__ void __launch_bounds__(ROW_THREADS) experts_gather_kernel(const RowParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int units = p.cols / V, pieces = (units + 32 * GATHER_STEPS - 1) / (32 * GATHER_STEPS);
  const int64_t work = p.rows * pieces, step = (int64_t)gridDim.x * ROW_WARPS;
  for (int64_t at = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); at < work; at += step) {
    const int64_t r = at / pieces;
    const int u0 = (int)(at - r * pieces) * 32 * GATHER_STEPS + lane;
    const int s = p.source[r];
    const bool real = s >= 0 && s / p.choices < p.x_rows;
    if (!real && s != -1) report(p);
    const T* x = static_cast<const T*>(p.X) + (real ? (int64_t)(s / p.choices) * p.ldx : 0);
    T* y = static_cast<T*>(p.Y) + r * p.ldy;
    Vec<T, V> v[GATHER_STEPS];
#pragma unroll
    for (int i = 0; i < GATHER_STEPS; ++i) {
      const int u = u0 + 32 * i;
      if (real && u < units) {
        v[i] = load<T, V>(x + (int64_t)u * V);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) v[i].v[k] = from_float<T>(0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < GATHER_STEPS; ++i)
      if (u0 + 32 * i < units) store<T, V>(y + (int64_t)(u0 + 32 * i) * V, v[i], p.once);
  }
}

// A warp takes a piece of a token, UNITS units a lane, and adds its choices in
// their order, AT_ONCE of them on their way at a time, eight loads a lane in all:
// 89 -> 71 us for 8192 tokens of 4096 numbers from four rows each, against a unit
// a thread.
template <typename T, typename W, int V, int AT_ONCE>
__global__ void __launch_bounds__(ROW_THREADS) experts_combine_kernel(const RowParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int UNITS = COMBINE_LOADS / AT_ONCE;
  const int lane = threadIdx.x & 31;
  const int units = p.cols / V, pieces = (units + 32 * UNITS - 1) / (32 * UNITS);
  const int64_t work = p.rows * pieces, step = (int64_t)gridDim.x * ROW_WARPS;
  for (int64_t at = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); at < work; at += step) {
    const int64_t t = at / pieces;
    const int u0 = (int)(at - t * pieces) * 32 * UNITS + lane;
    float sum[UNITS][V];
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) sum[i][k] = 0.f;
    for (int j0 = 0; j0 < p.choices; j0 += AT_ONCE) {
      Vec<T, V> x[AT_ONCE][UNITS];
      int r[AT_ONCE];
      float w[AT_ONCE];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        const int64_t n = t * p.choices + j0 + j;
        r[j] = j0 + j < p.choices ? p.map[n] : -1;
        w[j] = p.w && j0 + j < p.choices ? to_float<W>(static_cast<const W*>(p.w)[n]) : 1.f;
      }
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        if (r[j] != -1 && (r[j] < 0 || r[j] >= p.x_rows)) {
          report(p);
          r[j] = -1;
        }
        const T* row = static_cast<const T*>(p.X) + (int64_t)r[j] * p.ldx;
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
          if (r[j] >= 0 && u0 + 32 * i < units)
            x[j][i] = load_once<T, V>(row + (int64_t)(u0 + 32 * i) * V);
      }
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        if (r[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k)
            sum[i][k] = fmaf(w[j], to_float<T>(x[j][i].v[k]), sum[i][k]);
      }
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      if (u0 + 32 * i >= units) continue;
      Vec<T, V> y;
#pragma unroll
      for (int k = 0; k < V; ++k) y.v[k] = from_float<T>(sum[i][k]);
      store<T, V>(static_cast<T*>(p.Y) + t * p.ldy + (int64_t)(u0 + 32 * i) * V, y);
    }
  }
}

// A warp takes a row of S: its part of dw is a sum over the lanes in a fixed
// order, and dS's row comes from the same reading of dY.
template <typename T, typename W, int V>
__global__ void __launch_bounds__(ROW_THREADS) experts_combine_gradient_kernel(const RowParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int AT_ONCE = 2;
  const int lane = threadIdx.x & 31, units = p.cols / V;
  const int64_t step = (int64_t)gridDim.x * ROW_WARPS;
  for (int64_t r = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5); r < p.rows; r += step) {
    const int s = p.source[r];
    const bool real = s >= 0 && s < p.entries;
    if (!real && s != -1) report(p);
    T* ds = static_cast<T*>(p.Y) + r * p.ldy;
    if (!real) {
      if (p.Y) {
        Vec<T, V> zero;
#pragma unroll
        for (int k = 0; k < V; ++k) zero.v[k] = from_float<T>(0.f);
        for (int u = lane; u < units; u += 32) store<T, V>(ds + (int64_t)u * V, zero, p.once);
      }
      continue;
    }
    const T* dy = static_cast<const T*>(p.dY) + (int64_t)(s / p.choices) * p.lddy;
    const T* x = static_cast<const T*>(p.X) + r * p.ldx;
    const float w = p.w ? to_float<W>(static_cast<const W*>(p.w)[s]) : 1.f;
    float dot = 0.f;
    for (int u0 = lane; u0 < units; u0 += 32 * AT_ONCE) {
      Vec<T, V> g[AT_ONCE], v[AT_ONCE];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int u = u0 + 32 * i;
        if (u < units) {
          g[i] = load<T, V>(dy + (int64_t)u * V);
          if (p.dw) v[i] = load_once<T, V>(x + (int64_t)u * V);
        }
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int u = u0 + 32 * i;
        if (u < units) {
          Vec<T, V> o;
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float f = to_float<T>(g[i].v[k]);
            if (p.dw) dot = fmaf(f, to_float<T>(v[i].v[k]), dot);
            o.v[k] = from_float<T>(w * f);
          }
          if (p.Y) store<T, V>(ds + (int64_t)u * V, o, p.once);
        }
      }
    }
    if (p.dw) {
#pragma unroll
      for (int d = 16; d > 0; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
      if (lane == 0) static_cast<W*>(p.dw)[s] = from_float<W>(dot);
    }
  }
  if (p.dw)   // choices that have no row
    for (int64_t i = (int64_t)blockIdx.x * ROW_THREADS + threadIdx.x; i < p.entries;
         i += (int64_t)gridDim.x * ROW_THREADS)
      if (p.map[i] < 0) static_cast<W*>(p.dw)[i] = from_float<W>(0.f);
}

using RowKernel = void (*)(const RowParams);

enum Which { COMBINE, COMBINE_FEW, GRADIENT };   // FEW: up to two choices

template <typename T, typename W, int V>
RowKernel pick_row(Which which) {
  return which == COMBINE       ? experts_combine_kernel<T, W, V, 4>
         : which == COMBINE_FEW ? experts_combine_kernel<T, W, V, 2>
                                : experts_combine_gradient_kernel<T, W, V>;
}
template <typename T>
RowKernel pick_row(Which which, bool f32_weights, bool vec) {
  constexpr int V = 16 / sizeof(T);
  if (f32_weights) return vec ? pick_row<T, float, V>(which) : pick_row<T, float, 1>(which);
  return vec ? pick_row<T, T, V>(which) : pick_row<T, T, 1>(which);
}
RowKernel pick_row(Which which, int type, bool f32_weights, bool vec) {
  return type == GEMM_F8_F16    ? pick_row<__half>(which, f32_weights, vec)
         : type == GEMM_F8_BF16 ? pick_row<__nv_bfloat16>(which, f32_weights, vec)
                                : pick_row<float>(which, f32_weights, vec);
}

bool off(const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) != 0; }
int size_of(int type) { return type == GEMM_F8_F32 ? 4 : 2; }

// Whether rows of X start on 16-byte boundaries.
bool vec_rows(const void* X, int64_t ld, int64_t rows, int size) {
  return !off(X, 15) && (rows <= 1 || ld * size % 16 == 0);
}

// A matrix of `rows` x cols numbers, where it is used.
int check_rows(const void* X, int64_t ld, int64_t rows, int cols, int size) {
  if (rows == 0) return GEMM_F16_OK;
  if (!X || (rows > 1 && (ld < cols || ld >= ((int64_t)1 << 38)))) return GEMM_F16_ERR_INVALID_ARG;
  return off(X, size - 1) ? GEMM_F16_ERR_MISALIGNED : GEMM_F16_OK;
}

int launch_rows(gemm_f16_plan_s* p, RowKernel k, int64_t ctas, cudaStream_t st, const RowParams& prm,
                const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)p->num_sms * 64)), 1, 1);
  cfg.blockDim = dim3(ROW_THREADS, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  GF16_CUDA(cudaLaunchKernelEx(&cfg, k, prm), what);
  return GEMM_F16_OK;
}

}  // namespace

namespace gf16 {
namespace host {

int experts_plan_init(gemm_f16_plan_s*, const cudaDeviceProp&) {
  const int most = MAP_WARPS * MAX_EXPERTS * 4;
  GF16_CUDA(cudaFuncSetAttribute(experts_maps_kernel<int32_t>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, most),
            "cudaFuncSetAttribute(experts' maps smem)");
  GF16_CUDA(cudaFuncSetAttribute(experts_maps_kernel<int64_t>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, most),
            "cudaFuncSetAttribute(experts' maps smem)");
  return GEMM_F16_OK;
}

}  // namespace host
}  // namespace gf16

extern "C" {

int64_t experts_max_rows(int entries, int num_experts, int align) {
  if (entries < 0 || entries > MAX_ENTRIES || num_experts < 1 || num_experts > MAX_EXPERTS ||
      align < 1 || align > 1024)
    return GEMM_F16_ERR_INVALID_ARG;
  const int64_t most = entries + (int64_t)std::min(num_experts, entries) * (align - 1);
  return ceil_div(most, align) * align;
}

int experts_maps_validate(int entries, const void* experts, int wide, int num_experts, int align,
                          int max_rows, const int32_t* starts, const int32_t* rows,
                          const int32_t* source) {
  const int64_t most = experts_max_rows(entries, num_experts, align);
  if (most < 0 || max_rows < most || max_rows > MAX_SIZE || (wide & ~1) || !starts)
    return GEMM_F16_ERR_INVALID_ARG;
  if (entries > 0 && (!experts || !rows)) return GEMM_F16_ERR_INVALID_ARG;
  if (max_rows > 0 && !source) return GEMM_F16_ERR_INVALID_ARG;
  if (off(experts, wide ? 7 : 3) || off(starts, 3) || off(rows, 3) || off(source, 3))
    return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

int experts_maps(gemm_f16_plan_t p, int entries, const void* experts, int wide, int num_experts,
                 int align, int max_rows, int32_t* starts, int32_t* rows, int32_t* source,
                 gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  const int rc = experts_maps_validate(entries, experts, wide, num_experts, align, max_rows, starts,
                                       rows, source);
  if (rc) return rc;
  DeviceGuard g(p->device);
  const MapParams prm = {entries, num_experts, align, max_rows, experts, starts, rows, source,
                         p->status_dev};
  const int ctas = entries <= ONE_CTA ? 1 : MAP_CLUSTER;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(MAP_THREADS, 1, 1);
  cfg.dynamicSmemBytes = (size_t)MAP_WARPS * num_experts * 4;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  GF16_CUDA(cudaLaunchKernelEx(&cfg, wide ? experts_maps_kernel<int64_t> : experts_maps_kernel<int32_t>,
                               prm),
            "launch experts_maps_kernel");
  return GEMM_F16_OK;
}

int experts_gather_validate(int type, int rows, int cols, const void* X, int64_t ldx, int x_rows,
                            int choices, const int32_t* source, const void* Y, int64_t ldy) {
  if (type < GEMM_F8_F16 || type > GEMM_F8_F32 || rows < 0 || rows > MAX_SIZE || cols < 1 ||
      cols > MAX_SIZE || x_rows < 0 || choices < 1)
    return GEMM_F16_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_F16_OK;
  if (!source) return GEMM_F16_ERR_INVALID_ARG;
  int rc = check_rows(X, ldx, x_rows, cols, size_of(type));
  if (!rc) rc = check_rows(Y, ldy, rows, cols, size_of(type));
  if (!rc && off(source, 3)) rc = GEMM_F16_ERR_MISALIGNED;
  return rc;
}

int experts_gather(gemm_f16_plan_t p, int type, int rows, int cols, const void* X, int64_t ldx,
                   int x_rows, int choices, const int32_t* source, void* Y, int64_t ldy,
                   gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  const int rc = experts_gather_validate(type, rows, cols, X, ldx, x_rows, choices, source, Y, ldy);
  if (rc || rows == 0) return rc;
  DeviceGuard g(p->device);
  const int size = size_of(type), v = 16 / size;
  const bool vec = cols % v == 0 && vec_rows(X, ldx, x_rows, size) && vec_rows(Y, ldy, rows, size);
  RowParams prm = {};
  prm.rows = rows;
  prm.cols = cols;
  prm.choices = choices;
  prm.X = X;
  prm.ldx = ldx;
  prm.x_rows = x_rows;
  prm.source = source;
  prm.Y = Y;
  prm.ldy = ldy;
  prm.once = (int64_t)rows * cols * size > CACHE_BYTES;
  prm.status = p->status_dev;
  const int64_t pieces = ceil_div(cols / (vec ? v : 1), 32 * GATHER_STEPS);
  const RowKernel k = type == GEMM_F8_F32
                          ? (vec ? experts_gather_kernel<float, 4> : experts_gather_kernel<float, 1>)
                          // a copy: both 16-bit types alike
                          : (vec ? experts_gather_kernel<__half, 8> : experts_gather_kernel<__half, 1>);
  return launch_rows(p, k, ceil_div(rows * pieces, ROW_WARPS), (cudaStream_t)stream, prm,
                     "launch experts_gather_kernel");
}

int experts_combine_validate(int type, int tokens, int choices, int cols, const void* S,
                             int64_t lds, int s_rows, const int32_t* rows, const void* weights,
                             int weights_type, const void* Y, int64_t ldy) {
  if (type < GEMM_F8_F16 || type > GEMM_F8_F32 || tokens < 0 || choices < 1 || cols < 1 ||
      cols > MAX_SIZE || s_rows < 0 || s_rows > MAX_SIZE || (int64_t)tokens * choices > MAX_ENTRIES ||
      (weights_type != GEMM_F8_F32 && weights_type != type))
    return GEMM_F16_ERR_INVALID_ARG;
  if (tokens == 0) return GEMM_F16_OK;
  if (!rows) return GEMM_F16_ERR_INVALID_ARG;
  int rc = check_rows(S, lds, s_rows, cols, size_of(type));
  if (!rc) rc = check_rows(Y, ldy, tokens, cols, size_of(type));
  if (!rc && (off(rows, 3) || off(weights, size_of(weights_type) - 1))) rc = GEMM_F16_ERR_MISALIGNED;
  return rc;
}

int experts_combine(gemm_f16_plan_t p, int type, int tokens, int choices, int cols, const void* S,
                    int64_t lds, int s_rows, const int32_t* rows, const void* weights,
                    int weights_type, void* Y, int64_t ldy, gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  const int rc = experts_combine_validate(type, tokens, choices, cols, S, lds, s_rows, rows, weights,
                                          weights_type, Y, ldy);
  if (rc || tokens == 0) return rc;
  DeviceGuard g(p->device);
  const int size = size_of(type), v = 16 / size;
  const bool vec = cols % v == 0 && vec_rows(S, lds, s_rows, size) && vec_rows(Y, ldy, tokens, size);
  RowParams prm = {};
  prm.rows = tokens;
  prm.cols = cols;
  prm.choices = choices;
  prm.X = S;
  prm.ldx = lds;
  prm.x_rows = s_rows;
  prm.map = rows;
  prm.w = weights;
  prm.Y = Y;
  prm.ldy = ldy;
  prm.status = p->status_dev;
  const bool few = choices <= 2;
  const int64_t pieces = ceil_div(cols / (vec ? v : 1), 32 * COMBINE_LOADS / (few ? 2 : 4));
  return launch_rows(p, pick_row(few ? COMBINE_FEW : COMBINE, type, weights_type == GEMM_F8_F32, vec),
                     ceil_div(tokens * pieces, ROW_WARPS), (cudaStream_t)stream, prm,
                     "launch experts_combine_kernel");
}

int experts_combine_gradient_validate(int type, int tokens, int choices, int cols, const void* dY,
                                      int64_t lddy, const void* S, int64_t lds, int s_rows,
                                      const int32_t* rows, const int32_t* source,
                                      const void* weights, int weights_type, const void* dS,
                                      int64_t ldds, const void* dw) {
  if (type < GEMM_F8_F16 || type > GEMM_F8_F32 || tokens < 0 || choices < 1 || cols < 1 ||
      cols > MAX_SIZE || s_rows < 0 || s_rows > MAX_SIZE || (int64_t)tokens * choices > MAX_ENTRIES ||
      (weights_type != GEMM_F8_F32 && weights_type != type))
    return GEMM_F16_ERR_INVALID_ARG;
  if (!dS && !dw) return GEMM_F16_OK;
  const int size = size_of(type);
  int rc = check_rows(dY, lddy, tokens, cols, size);
  if (!rc && dw) rc = check_rows(S, lds, s_rows, cols, size);
  if (!rc && dS) rc = check_rows(dS, ldds, s_rows, cols, size);
  if (rc) return rc;
  if ((s_rows > 0 && !source) || (dw && tokens > 0 && !rows)) return GEMM_F16_ERR_INVALID_ARG;
  if (off(rows, 3) || off(source, 3) || off(weights, size_of(weights_type) - 1) ||
      off(dw, size_of(weights_type) - 1))
    return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

int experts_combine_gradient(gemm_f16_plan_t p, int type, int tokens, int choices, int cols,
                             const void* dY, int64_t lddy, const void* S, int64_t lds, int s_rows,
                             const int32_t* rows, const int32_t* source, const void* weights,
                             int weights_type, void* dS, int64_t ldds, void* dw,
                             gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  const int rc = experts_combine_gradient_validate(type, tokens, choices, cols, dY, lddy, S, lds,
                                                   s_rows, rows, source, weights, weights_type, dS,
                                                   ldds, dw);
  if (rc || (!dS && !dw) || (s_rows == 0 && tokens == 0)) return rc;
  DeviceGuard g(p->device);
  const int size = size_of(type), v = 16 / size;
  const bool vec = cols % v == 0 && vec_rows(dY, lddy, tokens, size) &&
                   (!dw || vec_rows(S, lds, s_rows, size)) &&
                   (!dS || vec_rows(dS, ldds, s_rows, size));
  RowParams prm = {};
  prm.rows = s_rows;
  prm.cols = cols;
  prm.choices = choices;
  prm.entries = (int64_t)tokens * choices;
  prm.X = S;
  prm.ldx = lds;
  prm.x_rows = s_rows;
  prm.dY = dY;
  prm.lddy = lddy;
  prm.map = rows;
  prm.source = source;
  prm.w = weights;
  prm.Y = dS;
  prm.ldy = ldds;
  prm.dw = dw;
  prm.once = (int64_t)s_rows * cols * size > CACHE_BYTES;
  prm.status = p->status_dev;
  const int64_t ctas = std::max(ceil_div(s_rows, ROW_WARPS), ceil_div(prm.entries, ROW_THREADS));
  return launch_rows(p, pick_row(GRADIENT, type, weights_type == GEMM_F8_F32, vec), ctas,
                     (cudaStream_t)stream, prm, "launch experts_combine_gradient_kernel");
}

}  // extern "C"
