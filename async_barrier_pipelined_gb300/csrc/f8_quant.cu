// Quantisation to 8-bit codes with a scale for each block of 128
// (gemm_f8_quantize).
//
// For a block with largest finite magnitude a (at least 2^-100) and the
// format's largest number L: scale = fl(a / L), code = round(fl(x * fl(L / a))).
// Two divisions a block and one multiplication a number, all IEEE, so that the
// codes are the same bits however a block is spread over threads; the
// conversion rounds to nearest even and clamps the one number whose product
// may pass L by FP32's rounding.
//
// Bound by the memory: each number is read once and written once (or twice,
// for both directions).  ROWS: eight lanes a block, 16 numbers each, so that
// a lane stores 16 bytes; nothing but shuffles.  The others: a CTA takes a tile
// of 128 x 128 into registers (64 numbers a thread), reduces it along the rows
// by shuffles and along the columns through 4 KB of shared memory, and writes
// the codes of one or both directions from the same registers.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm_f8.h"
#include "host.h"

using namespace gf16;
using namespace gf16::host;

namespace {

constexpr float FLOOR = 7.8886090522101181e-31f;   // 2^-100
constexpr int MAX_SIZE = 0x7fffffff - 1023;

struct Params {
  int rows, cols, batch;
  const void* X;
  int64_t ldx, x_batch;
  const int32_t* source;
  int choices, x_rows;
  uint8_t* Q;
  int64_t ldq, q_batch;
  float* S;
  uint8_t* Q2;
  float* S2;
  int blk_cols, blk_rows;   // blocks along a row, along a column
  int* status;
};

// Sixteen numbers of a lane, kept in their own type.
template <typename T>
struct Pack;
template <>
struct alignas(16) Pack<float> {
  float v[16];
  __device__ float get(int i) const { return v[i]; }
};
template <>
struct alignas(16) Pack<__half> {
  __half2 v[8];
  __device__ float get(int i) const { return i & 1 ? __high2float(v[i / 2]) : __low2float(v[i / 2]); }
};
template <>
struct alignas(16) Pack<__nv_bfloat16> {
  __nv_bfloat162 v[8];
  __device__ float get(int i) const { return i & 1 ? __high2float(v[i / 2]) : __low2float(v[i / 2]); }
};

// Numbers col .. col + 15 of a row (0 past `cols`, and everywhere for a null
// row).  VEC: rows start on 16-byte boundaries.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(Pack<T>& x, const T* row, int col, int cols) {
  constexpr int V = 16 / sizeof(T);
  T* out = reinterpret_cast<T*>(x.v);
  if (VEC && row && col + 16 <= cols) {
#pragma unroll
    for (int i = 0; i < 16 / V; ++i)
      reinterpret_cast<uint4*>(out)[i] = __ldg(reinterpret_cast<const uint4*>(row + col) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = row && col + i < cols ? row[col + i] : T(0.f);
  }
}

// Largest magnitude, NaN left out (infinity if there is one).
template <typename T>
__device__ __forceinline__ float largest(const Pack<T>& x) {
  if constexpr (sizeof(T) == 4) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x.v[i]));
    return a;
  } else {
    auto a = __habs2(x.v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) a = __hmax2(a, __habs2(x.v[i]));
    const float lo = __low2float(a), hi = __high2float(a);
    return fmaxf(fmaxf(lo, hi), 0.f);     // fmaxf leaves a NaN out
  }
}
// The same of the finite ones, for blocks that hold an infinity.
template <typename T>
__device__ __forceinline__ float largest_finite(const Pack<T>& x) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = fabsf(x.get(i));
    a = fmaxf(a, v < INFINITY ? v : 0.f);
  }
  return a;
}

// Four codes, the first in the lowest byte.
template <int FORMAT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  if constexpr (FORMAT == GEMM_F8_E4M3) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  } else {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  }
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// An infinity times the block's factor would be clamped: it becomes NaN.
__device__ __forceinline__ float scaled(float x, float f) {
  const float y = __fmul_rn(x, f);
  return fabsf(y) < INFINITY ? y : NAN;
}

template <int FORMAT>
constexpr float LARGEST = FORMAT == GEMM_F8_E4M3 ? 448.f : 57344.f;

__device__ __forceinline__ void store_codes(uint8_t* row, int col, int cols, const uint32_t (&w)[4]) {
  if (col + 16 <= cols) {
    *reinterpret_cast<uint4*>(row + col) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (col + i < cols) row[col + i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
  }
}

template <typename T>
__device__ __forceinline__ const T* row_of(const Params& p, int b, int r) {
  const T* X = static_cast<const T*>(p.X);
  if (!p.source) return X + (int64_t)b * p.x_batch + (int64_t)r * p.ldx;
  const int s = p.source[r];
  if (s == -1) return nullptr;
  if (s < 0 || s / p.choices >= p.x_rows) {
    *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
    return nullptr;
  }
  return X + (int64_t)(s / p.choices) * p.ldx;
}

constexpr int ROW_THREADS = 256;
constexpr int PER_WARP = 4;      // blocks of 128 that a warp takes at once

template <typename T, int FORMAT, bool VEC>
__global__ void __launch_bounds__(ROW_THREADS) quantize_rows_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, part = lane & 7;
  const int64_t per_matrix = (int64_t)p.rows * p.blk_cols, blocks = per_matrix * p.batch;
  const int64_t step = (int64_t)gridDim.x * (ROW_THREADS / 32) * PER_WARP;
  for (int64_t at = ((int64_t)blockIdx.x * (ROW_THREADS / 32) + (threadIdx.x >> 5)) * PER_WARP;
       at < blocks; at += step) {
    const int64_t blk = at + (lane >> 3);
    const bool real = blk < blocks;
    const int b = real && p.batch > 1 ? (int)(blk / per_matrix) : 0;
    const int64_t in = real ? blk - (int64_t)b * per_matrix : 0;
    const int r = p.batch * per_matrix <= 0x7fffffff ? (int)((uint32_t)in / (uint32_t)p.blk_cols)
                                                     : (int)(in / p.blk_cols);
    const int cb = (int)(in - (int64_t)r * p.blk_cols), col = cb * 128 + part * 16;
    Pack<T> x;
    load16<T, VEC>(x, real ? row_of<T>(p, b, r) : nullptr, col, p.cols);
    float a = largest(x);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    const bool inf = !(a < INFINITY);
    if (__any_sync(0xffffffffu, inf)) {
      float f = largest_finite(x);
#pragma unroll
      for (int d = 1; d < 8; d *= 2) f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, d));
      a = f;
    }
    a = fmaxf(a, FLOOR);
    const float f = __fdiv_rn(LARGEST<FORMAT>, a);
    if (!real) continue;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = codes4<FORMAT>(scaled(x.get(4 * i), f), scaled(x.get(4 * i + 1), f),
                            scaled(x.get(4 * i + 2), f), scaled(x.get(4 * i + 3), f));
    if (col < p.cols)
      store_codes(p.Q + (int64_t)b * p.q_batch + (int64_t)r * p.ldq, col, p.cols, w);
    if (part == 0) p.S[blk] = __fdiv_rn(a, LARGEST<FORMAT>);
  }
}

constexpr int TILE_THREADS = 256;

// BLOCKS: GEMM_F8_COLUMNS, _TILES or _BOTH.  Thread (warp w, lane l): rows
// 16 w + 4 i + l / 8 for i < 4, columns 16 (l % 8) .. + 15.
template <typename T, int FORMAT, int BLOCKS, bool VEC>
__global__ void __launch_bounds__(TILE_THREADS) quantize_tile_kernel(const Params p) {
  __shared__ float top[8][128];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane & 7;
  const int tile = (int)blockIdx.x;
  const int rb = tile / p.blk_cols, cb = tile - rb * p.blk_cols, b = (int)blockIdx.y;
  const int row0 = rb * 128 + warp * 16 + (lane >> 3), col = cb * 128 + part * 16;
  Pack<T> x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + 4 * i;
    load16<T, VEC>(x[i], r < p.rows ? row_of<T>(p, b, r) : nullptr, col, p.cols);
  }
  uint8_t* Q = p.Q + (int64_t)b * p.q_batch;
  if constexpr (BLOCKS == GEMM_F8_BOTH) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = largest(x[i]);
#pragma unroll
      for (int d = 1; d < 8; d *= 2) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      if (__any_sync(0xffffffffu, !(a < INFINITY))) {
        a = largest_finite(x[i]);
#pragma unroll
        for (int d = 1; d < 8; d *= 2) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      }
      a = fmaxf(a, FLOOR);
      const float f = __fdiv_rn(LARGEST<FORMAT>, a);
      const int r = row0 + 4 * i;
      if (r < p.rows) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = codes4<FORMAT>(scaled(x[i].get(4 * k), f), scaled(x[i].get(4 * k + 1), f),
                                scaled(x[i].get(4 * k + 2), f), scaled(x[i].get(4 * k + 3), f));
        if (col < p.cols) store_codes(Q + (int64_t)r * p.ldq, col, p.cols, w);
        if (part == 0) p.S[(int64_t)r * p.blk_cols + cb] = __fdiv_rn(a, LARGEST<FORMAT>);
      }
    }
  }
  if constexpr (BLOCKS == GEMM_F8_TILES) {
    float a = fmaxf(fmaxf(largest(x[0]), largest(x[1])), fmaxf(largest(x[2]), largest(x[3])));
    if (__syncthreads_or(!(a < INFINITY)))
      a = fmaxf(fmaxf(largest_finite(x[0]), largest_finite(x[1])),
                fmaxf(largest_finite(x[2]), largest_finite(x[3])));
#pragma unroll
    for (int d = 1; d < 32; d *= 2) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    if (lane == 0) top[0][warp] = a;
    __syncthreads();
    a = FLOOR;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, top[0][i]);
    const float f = __fdiv_rn(LARGEST<FORMAT>, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 4 * i;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = codes4<FORMAT>(scaled(x[i].get(4 * k), f), scaled(x[i].get(4 * k + 1), f),
                              scaled(x[i].get(4 * k + 2), f), scaled(x[i].get(4 * k + 3), f));
      if (r < p.rows && col < p.cols) store_codes(Q + (int64_t)r * p.ldq, col, p.cols, w);
    }
    if (threadIdx.x == 0)
      p.S[((int64_t)b * p.blk_rows + rb) * p.blk_cols + cb] = __fdiv_rn(a, LARGEST<FORMAT>);
  } else {
    // Columns: each thread's four rows, the warp's sixteen, the CTA's 128.
    float a[16];
    bool inf = false;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      a[k] = fmaxf(fmaxf(fabsf(x[0].get(k)), fabsf(x[1].get(k))),
                   fmaxf(fabsf(x[2].get(k)), fabsf(x[3].get(k))));
      inf = inf || !(a[k] < INFINITY);   // a NaN in all four, or an infinity
    }
    if (__any_sync(0xffffffffu, inf)) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        a[k] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = fabsf(x[i].get(k));
          a[k] = fmaxf(a[k], v < INFINITY ? v : 0.f);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      a[k] = fmaxf(a[k], __shfl_xor_sync(0xffffffffu, a[k], 8));
      a[k] = fmaxf(a[k], __shfl_xor_sync(0xffffffffu, a[k], 16));
    }
    if (lane < 8) {
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        *reinterpret_cast<float4*>(&top[warp][part * 16 + k]) =
            make_float4(a[k], a[k + 1], a[k + 2], a[k + 3]);
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      float m = FLOOR;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, top[i][threadIdx.x]);
      top[0][threadIdx.x] = __fdiv_rn(LARGEST<FORMAT>, m);
      float* S = BLOCKS == GEMM_F8_BOTH ? p.S2 : p.S;
      const int c = cb * 128 + (int)threadIdx.x;
      if (c < p.cols)
        S[((int64_t)b * p.blk_rows + rb) * p.cols + c] = __fdiv_rn(m, LARGEST<FORMAT>);
    }
    __syncthreads();
    float f[16];
#pragma unroll
    for (int k = 0; k < 16; k += 4)
      *reinterpret_cast<float4*>(&f[k]) = *reinterpret_cast<const float4*>(&top[0][part * 16 + k]);
    if (BLOCKS == GEMM_F8_BOTH) Q = p.Q2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 4 * i;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = codes4<FORMAT>(scaled(x[i].get(4 * k), f[4 * k]), scaled(x[i].get(4 * k + 1), f[4 * k + 1]),
                              scaled(x[i].get(4 * k + 2), f[4 * k + 2]),
                              scaled(x[i].get(4 * k + 3), f[4 * k + 3]));
      if (r < p.rows && col < p.cols) store_codes(Q + (int64_t)r * p.ldq, col, p.cols, w);
    }
  }
}

using Kernel = void (*)(const Params);

template <typename T, int FORMAT, bool VEC>
Kernel pick(int blocks) {
  switch (blocks) {
    case GEMM_F8_ROWS: return quantize_rows_kernel<T, FORMAT, VEC>;
    case GEMM_F8_COLUMNS: return quantize_tile_kernel<T, FORMAT, GEMM_F8_COLUMNS, VEC>;
    case GEMM_F8_TILES: return quantize_tile_kernel<T, FORMAT, GEMM_F8_TILES, VEC>;
    default: return quantize_tile_kernel<T, FORMAT, GEMM_F8_BOTH, VEC>;
  }
}
template <typename T>
Kernel pick(int blocks, int format, bool vec) {
  if (format == GEMM_F8_E4M3)
    return vec ? pick<T, GEMM_F8_E4M3, true>(blocks) : pick<T, GEMM_F8_E4M3, false>(blocks);
  return vec ? pick<T, GEMM_F8_E5M2, true>(blocks) : pick<T, GEMM_F8_E5M2, false>(blocks);
}

bool off(const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) != 0; }

}  // namespace

extern "C" {

int gemm_f8_quantize_validate(int blocks, int format, int type, int batch, int rows, int cols,
                              const void* X, int64_t ldx, int64_t x_batch, const int32_t* source,
                              int choices, int x_rows, const void* Q, int64_t ldq,
                              int64_t q_batch, const float* S, const void* Q2, const float* S2) {
  if (blocks < GEMM_F8_ROWS || blocks > GEMM_F8_BOTH || type < GEMM_F8_F16 || type > GEMM_F8_F32 ||
      (format != GEMM_F8_E4M3 && format != GEMM_F8_E5M2))
    return GEMM_F16_ERR_INVALID_ARG;
  if (batch < 0 || batch > 65535 || rows < 0 || rows > MAX_SIZE || cols < 1 || cols > MAX_SIZE)
    return GEMM_F16_ERR_INVALID_ARG;
  if (source && (batch > 1 || choices < 1 || x_rows < 0)) return GEMM_F16_ERR_INVALID_ARG;
  if (batch == 0 || rows == 0) return GEMM_F16_OK;
  if (ceil_div(rows, 128) * ceil_div(cols, 128) > MAX_SIZE) return GEMM_F16_ERR_INVALID_ARG;
  if ((!X && !(source && x_rows == 0)) || !Q || !S) return GEMM_F16_ERR_INVALID_ARG;
  if (blocks == GEMM_F8_BOTH && (!Q2 || !S2 || batch > 1)) return GEMM_F16_ERR_INVALID_ARG;
  const int size = type == GEMM_F8_F32 ? 4 : 2;
  const int lines = source ? x_rows : rows;
  if ((lines > 1 && ldx < cols) || (batch > 1 && (x_batch < 0 || q_batch < 0)) ||
      (rows > 1 && ldq < cols))
    return GEMM_F16_ERR_INVALID_ARG;
  if (off(X, size - 1) || off(source, 3) || off(S, 3) || off(Q, 15) || (rows > 1 && (ldq & 15)) ||
      (batch > 1 && (q_batch & 15)))
    return GEMM_F16_ERR_MISALIGNED;
  if (blocks == GEMM_F8_BOTH && (off(Q2, 15) || off(S2, 3))) return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

int gemm_f8_quantize(gemm_f16_plan_t p, int blocks, int format, int type, int batch, int rows,
                     int cols, const void* X, int64_t ldx, int64_t x_batch,
                     const int32_t* source, int choices, int x_rows, void* Q, int64_t ldq,
                     int64_t q_batch, float* S, void* Q2, float* S2, gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  const int rc = gemm_f8_quantize_validate(blocks, format, type, batch, rows, cols, X, ldx, x_batch,
                                           source, choices, x_rows, Q, ldq, q_batch, S, Q2, S2);
  if (rc) return rc;
  if (batch == 0 || rows == 0) return GEMM_F16_OK;
  DeviceGuard g(p->device);
  const int size = type == GEMM_F8_F32 ? 4 : 2;
  Params prm = {};
  prm.rows = rows;
  prm.cols = cols;
  prm.batch = batch;
  prm.X = X;
  prm.ldx = ldx;
  prm.x_batch = x_batch;
  prm.source = source;
  prm.choices = choices;
  prm.x_rows = x_rows;
  prm.Q = static_cast<uint8_t*>(Q);
  prm.ldq = ldq;
  prm.q_batch = q_batch;
  prm.S = S;
  prm.Q2 = static_cast<uint8_t*>(Q2);
  prm.S2 = S2;
  prm.blk_cols = (int)ceil_div(cols, 128);
  prm.blk_rows = (int)ceil_div(rows, 128);
  prm.status = p->status_dev;
  const int lines = source ? x_rows : rows;
  const bool vec = !off(X, 15) && (lines <= 1 || ldx * size % 16 == 0) &&
                   (batch == 1 || x_batch * size % 16 == 0);
  const Kernel k = type == GEMM_F8_F16    ? pick<__half>(blocks, format, vec)
                   : type == GEMM_F8_BF16 ? pick<__nv_bfloat16>(blocks, format, vec)
                                          : pick<float>(blocks, format, vec);
  cudaLaunchConfig_t cfg = {};
  if (blocks == GEMM_F8_ROWS) {
    const int64_t warps = ceil_div((int64_t)batch * rows * prm.blk_cols, PER_WARP);
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(ceil_div(warps, ROW_THREADS / 32),
                                                   (int64_t)p->num_sms * 64), 1, 1);
    cfg.blockDim = dim3(ROW_THREADS, 1, 1);
  } else {
    cfg.gridDim = dim3((unsigned)((int64_t)prm.blk_rows * prm.blk_cols), (unsigned)batch, 1);
    cfg.blockDim = dim3(TILE_THREADS, 1, 1);
  }
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  GF16_CUDA(cudaLaunchKernelEx(&cfg, k, prm), "launch quantize kernel");
  return GEMM_F16_OK;
}

}  // extern "C"
