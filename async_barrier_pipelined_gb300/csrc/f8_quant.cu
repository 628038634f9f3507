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
// ROWS is bound by the memory: eight lanes a block, 16 numbers each, so that a
// lane stores 16 bytes; nothing but shuffles (16001 x 4104 bf16: 34 us, 5.8 TB/s).
// The others: a CTA takes a tile of 128 x 128 into registers (32 numbers a
// thread), reduces it along the rows by shuffles and along the columns through
// 8 KB of shared memory, and writes the codes of one or both directions from the
// same registers, so that X is read once.  Maxima are taken of pairs in the
// numbers' own type, divisions spread over the lanes.  Tiles take 43 us (4.6
// TB/s), columns 54 and both directions 73 (3.6 TB/s).  What bounds them is too
// little overlap: at 64 registers two CTAs of 512 threads an SM load, wait at two
// barriers and store in turn, and neither the memory (38 % of its time in both
// directions) nor the issue slots (51 %) are busy; the bf16 form of both
// directions also spills a few registers.  Tried: four columns of eight rows
// a lane (stores of four bytes; tiles 55, both 73), CTAs that stay and fetch the
// next tile early (82), two FP32 products at once (the pairs' moves cost more).

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
  using Pair = float2;      // two magnitudes
  __device__ Pair size(int i) const { return make_float2(fabsf(v[2 * i]), fabsf(v[2 * i + 1])); }
};
template <>
struct alignas(16) Pack<__half> {
  __half2 v[8];
  __device__ float get(int i) const { return i & 1 ? __high2float(v[i / 2]) : __low2float(v[i / 2]); }
  using Pair = __half2;
  __device__ Pair size(int i) const { return __habs2(v[i]); }
};
template <>
struct alignas(16) Pack<__nv_bfloat16> {
  uint32_t v[8];            // by their bits: FP32's upper half, and a sign
  __device__ float get(int i) const {
    return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
  }
  using Pair = __nv_bfloat162;
  __device__ Pair size(int i) const {
    const uint32_t m = v[i] & 0x7fff7fffu;
    return *reinterpret_cast<const __nv_bfloat162*>(&m);
  }
};
// Larger of two magnitudes; a NaN is left out beside a number.
__device__ __forceinline__ float2 larger(float2 a, float2 b) {
  return make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y));
}
__device__ __forceinline__ __half2 larger(__half2 a, __half2 b) { return __hmax2(a, b); }
__device__ __forceinline__ __nv_bfloat162 larger(__nv_bfloat162 a, __nv_bfloat162 b) {
  return __hmax2(a, b);
}
__device__ __forceinline__ float2 floats(float2 a) { return a; }
__device__ __forceinline__ float2 floats(__half2 a) { return __half22float2(a); }
__device__ __forceinline__ float2 floats(__nv_bfloat162 a) { return __bfloat1622float2(a); }
__device__ __forceinline__ float2 other_lane(float2 a, int d) {
  return make_float2(__shfl_xor_sync(0xffffffffu, a.x, d), __shfl_xor_sync(0xffffffffu, a.y, d));
}
template <typename P>
__device__ __forceinline__ P other_lane(P a, int d) {
  return __shfl_xor_sync(0xffffffffu, a, d);
}

// Numbers col .. col + 15 of a row (0 past `cols`, and everywhere for a null
// row).  VEC: rows start on 16-byte boundaries.
template <typename T, bool VEC>
__device__ __forceinline__ void load16(Pack<T>& x, const T* row, int col, int cols) {
  constexpr int V = 16 / sizeof(T);
  T* out = reinterpret_cast<T*>(x.v);
  if (VEC && row && col + 16 <= cols) {
#pragma unroll
    for (int i = 0; i < 16 / V; ++i)
      reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(row + col)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = row && col + i < cols ? row[col + i] : T(0.f);
  }
}

// Largest magnitude, NaN left out (infinity if there is one).
template <typename T>
__device__ __forceinline__ float largest(const Pack<T>& x) {
  auto a = x.size(0);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = larger(a, x.size(i));
  const float2 f = floats(a);
  return fmaxf(fmaxf(f.x, f.y), 0.f);     // fmaxf leaves a NaN out
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
// Sixteen codes; f(i): the factor of number i.  `inf`, the same in
// the whole warp: there are infinities, which the conversion would clamp and
// which become NaN.
template <int FORMAT, typename T, typename F>
__device__ __forceinline__ void codes16(uint32_t (&w)[4], const Pack<T>& x, bool inf, const F& f) {
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(x.get(i), f(i));
  if (inf) {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = fabsf(y[i]) < INFINITY ? y[i] : NAN;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = codes4<FORMAT>(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
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
    const bool inf = __any_sync(0xffffffffu, !(a < INFINITY));
    if (inf) {
      a = largest_finite(x);
#pragma unroll
      for (int d = 1; d < 8; d *= 2) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    }
    a = fmaxf(a, FLOOR);
    // One division a lane: the factor by a block's even lanes, the scale by the odd.
    const bool odd = part & 1;
    const float q = __fdiv_rn(odd ? a : LARGEST<FORMAT>, odd ? LARGEST<FORMAT> : a);
    const float f = __shfl_sync(0xffffffffu, q, lane & ~1);
    if (!real) continue;
    uint32_t w[4];
    codes16<FORMAT>(w, x, inf, [&](int) { return f; });
    if (col < p.cols)
      store_codes(p.Q + (int64_t)b * p.q_batch + (int64_t)r * p.ldq, col, p.cols, w);
    if (part == 1) p.S[blk] = q;
  }
}

constexpr int TILE_THREADS = 512, TILE_WARPS = TILE_THREADS / 32;
constexpr int LINES = 1024 / TILE_THREADS;      // rows of a thread

// BLOCKS: GEMM_F8_COLUMNS, _TILES or _BOTH.  Thread (warp w, lane l): rows
// 4 LINES w + 4 i + l / 8 for i < LINES, columns 16 (l % 8) .. + 15.
template <typename T, int FORMAT, int BLOCKS, bool VEC>
__global__ void __launch_bounds__(TILE_THREADS, 2) quantize_tile_kernel(const Params p) {
  __shared__ __align__(16) float top[TILE_WARPS][128];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane & 7;
  const int tile = (int)blockIdx.x;
  const int rb = tile / p.blk_cols, cb = tile - rb * p.blk_cols, b = (int)blockIdx.y;
  const int row0 = rb * 128 + warp * 4 * LINES + (lane >> 3), col = cb * 128 + part * 16;
  Pack<T> x[LINES];
#pragma unroll
  for (int i = 0; i < LINES; ++i) {
    const int r = row0 + 4 * i;
    load16<T, VEC>(x[i], r < p.rows ? row_of<T>(p, b, r) : nullptr, col, p.cols);
  }
  uint8_t* Q = p.Q + (int64_t)b * p.q_batch;
  if constexpr (BLOCKS == GEMM_F8_BOTH) {
    float a[LINES];
    bool inf = false;
#pragma unroll
    for (int i = 0; i < LINES; ++i) {
      a[i] = largest(x[i]);
#pragma unroll
      for (int d = 1; d < 8; d *= 2) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], d));
      inf = inf || !(a[i] < INFINITY);
    }
    inf = __any_sync(0xffffffffu, inf);
    if (inf) {
#pragma unroll
      for (int i = 0; i < LINES; ++i) {
        a[i] = largest_finite(x[i]);
#pragma unroll
        for (int d = 1; d < 8; d *= 2) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], d));
      }
    }
    // One division a lane: the first of a row's eight lanes have its lines'
    // factors, the next ones their scales.
    const bool upper = part >= LINES && part < 2 * LINES;
    const int mine = part % LINES;
    float m = a[0];
#pragma unroll
    for (int i = 1; i < LINES; ++i) m = mine == i ? a[i] : m;
    m = fmaxf(m, FLOOR);
    const float q = __fdiv_rn(upper ? m : LARGEST<FORMAT>, upper ? LARGEST<FORMAT> : m);
    if (upper && row0 + 4 * mine < p.rows) p.S[(int64_t)(row0 + 4 * mine) * p.blk_cols + cb] = q;
#pragma unroll
    for (int i = 0; i < LINES; ++i) {
      const float f = __shfl_sync(0xffffffffu, q, (lane & 24) + i);
      const int r = row0 + 4 * i;
      uint32_t w[4];
      codes16<FORMAT>(w, x[i], inf, [&](int) { return f; });
      if (r < p.rows && col < p.cols) store_codes(Q + (int64_t)r * p.ldq, col, p.cols, w);
    }
  }
  if constexpr (BLOCKS == GEMM_F8_TILES) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < LINES; ++i) a = fmaxf(a, largest(x[i]));
    const bool inf = __syncthreads_or(!(a < INFINITY));
    if (inf) {
      a = 0.f;
#pragma unroll
      for (int i = 0; i < LINES; ++i) a = fmaxf(a, largest_finite(x[i]));
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    if (lane == 0) top[0][warp] = a;
    __syncthreads();
    a = FLOOR;
#pragma unroll
    for (int i = 0; i < TILE_WARPS; ++i) a = fmaxf(a, top[0][i]);
    const float f = __fdiv_rn(LARGEST<FORMAT>, a);
#pragma unroll
    for (int i = 0; i < LINES; ++i) {
      const int r = row0 + 4 * i;
      uint32_t w[4];
      codes16<FORMAT>(w, x[i], inf, [&](int) { return f; });
      if (r < p.rows && col < p.cols) store_codes(Q + (int64_t)r * p.ldq, col, p.cols, w);
    }
    if (threadIdx.x == 0)
      p.S[((int64_t)b * p.blk_rows + rb) * p.blk_cols + cb] = __fdiv_rn(a, LARGEST<FORMAT>);
  } else {
    // Columns: each thread's lines, the warp's, the CTA's 128 rows.
    // A NaN that no number of its column replaces falls out at the end, where the
    // floor does.
    typename Pack<T>::Pair top2[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      top2[k] = x[0].size(k);
#pragma unroll
      for (int i = 1; i < LINES; ++i) top2[k] = larger(top2[k], x[i].size(k));
    }
    typename Pack<T>::Pair all = top2[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) all = larger(all, top2[k]);
    const float2 of_all = floats(all);
    const bool inf = __any_sync(0xffffffffu, of_all.x == INFINITY || of_all.y == INFINITY);
    float a[16];
    if (inf) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        a[k] = 0.f;
#pragma unroll
        for (int i = 0; i < LINES; ++i) {
          const float v = fabsf(x[i].get(k));
          a[k] = fmaxf(a[k], v < INFINITY ? v : 0.f);
        }
        a[k] = fmaxf(a[k], __shfl_xor_sync(0xffffffffu, a[k], 8));
        a[k] = fmaxf(a[k], __shfl_xor_sync(0xffffffffu, a[k], 16));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        top2[k] = larger(top2[k], other_lane(top2[k], 8));
        top2[k] = larger(top2[k], other_lane(top2[k], 16));
        const float2 f = floats(top2[k]);
        a[2 * k] = f.x;
        a[2 * k + 1] = f.y;
      }
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
      for (int i = 0; i < TILE_WARPS; ++i) m = fmaxf(m, top[i][threadIdx.x]);
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
    for (int i = 0; i < LINES; ++i) {
      const int r = row0 + 4 * i;
      uint32_t w[4];
      codes16<FORMAT>(w, x[i], inf, [&](int k) { return f[k]; });
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
