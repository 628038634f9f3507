// Shared by the two kernels of 8-bit products with block scales (f8_large.cuh,
// f8_small.cuh): parameters, bounded waits, the table of the experts' rows and
// the typed stores.
//
// Mathematics.  C[m,n] = sum_b sa[m,b] sb[b,n] T_b[m,n], T_b the product over
// the 128 inner numbers of block b.  The tensor core computes each T_b from
// zero into tensor memory (FP32; products of 4-bit by 4-bit significands are
// exact) and the promotion warps add it, scaled, to FP32 registers: the scales
// change from block to block, so a tile's sum cannot stay in tensor memory.
//
// Loads.  Every kernel here starts beside the end of the one before it
// (griddepcontrol) and its inputs may be written after it has started: they are
// read by ordinary loads after the wait, never as data that stay the same while
// the kernel runs (__ldg, ld.global.nc).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "gemm_f8.h"
#include "ptx.cuh"
#include "schedule.h"

namespace gf16 {
namespace f8 {

constexpr int BLOCK = 128;          // inner numbers with one scale = one K block
constexpr int MMA_K = 32;           // inner numbers of one kind::f8f6f4 MMA
constexpr int MAX_EXPERTS = 1024;

// Instruction descriptor of tcgen05.mma kind::f8f6f4: D FP32 (bits 4-5 = 1),
// A format at bits 7-9 and B format at 10-12 (0 e4m3, 1 e5m2), A / B
// MN-major at bits 15 / 16, N >> 3 at 17-22, M >> 4 at 24-28.
__host__ __device__ constexpr uint32_t idesc_f8(int fa, int fb, bool a_mn, bool b_mn, int m, int n) {
  return (1u << 4) | ((uint32_t)fa << 7) | ((uint32_t)fb << 10) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Both operand layouts are one box of 128 rows of 128 bytes with the 128-byte
// swizzle and 1024 bytes between groups of eight rows.  K-major: a row is one
// of M (N), and a step of 32 inner numbers is 32 bytes further along the rows.
// MN-major: a row is one inner number, and a step is 32 rows further.
constexpr uint32_t DESC_LBO = 16, DESC_SBO = 1024;
constexpr uint32_t K_STEP = 32, MN_STEP = 32 * 128;

struct Params {
  int form;                  // GEMM_F8_DENSE, _BY_ROWS, _BY_INNER
  int M, N, K;
  int experts;
  const int* starts;
  int a_mn, b_mn;            // operand's outer dimension is contiguous
  uint32_t idesc;
  const float* sa;           // scales: strides along the outer dimension (after >> shift)
  int64_t sa_outer, sa_inner;
  const float* sb;
  int64_t sb_outer, sb_inner, sb_batch;
  int sa_shift, sb_shift;    // 7: one scale for 128 rows (columns)
  void* C;
  int64_t ldc, c_batch;
  int type, accumulate, vec; // vec: C's rows start on 16-byte boundaries
  int tiles_m, tiles_n;      // DENSE: tiles of M; always: tiles of N
  int kblocks;               // DENSE
  int units;                 // DENSE, BY_INNER; BY_ROWS knows them on the device
  int full_units, cut_units, parts;   // large kernel, DENSE: see there
  int join_pieces;           // pieces of 32 rows x 128 columns of all cut tiles
  float* ws;
  int* status;
  unsigned long long timeout_ns;
  int fault_unit;
};

__device__ __forceinline__ bool wait_loop(uint32_t bar, uint32_t parity, const Params& p,
                                          volatile int* abort_flag, bool cluster) {
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (cluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity))
      return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      *abort_flag = 1;
      *(volatile int*)p.status = (int)GEMM_F16_ERR_TIMEOUT;
      __threadfence_system();
      return false;
    }
  }
}

__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, const Params& p,
                                       volatile int* abort_flag, bool cluster) {
  return wait_loop(bar, parity, p, abort_flag, cluster);
}

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const Params& p,
                                           volatile int* abort_flag) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, p, abort_flag, false);
}

// Without a call: the promotion warps' registers are all in use, and a call
// would have to save some of them.
__device__ __forceinline__ bool wait_phase_inline(uint32_t bar, uint32_t parity, const Params& p,
                                                  volatile int* abort_flag) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_loop(bar, parity, p, abort_flag, false);
}

// For barriers on which other CTAs' data was announced.
__device__ __forceinline__ bool wait_phase_cluster(uint32_t bar, uint32_t parity, const Params& p,
                                                   volatile int* abort_flag) {
  if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
  return wait_slow(bar, parity, p, abort_flag, true);
}

__device__ __forceinline__ void report_bad_index(const Params& p) {
  *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
}

// The experts' segments in shared memory: lo[e], first row of expert e; len[e],
// its rows, or -1 where its starts are bad (no tiles and no K blocks then);
// tiles[e], the tiles of `rows` rows of the experts before it (BY_ROWS),
// tiles[experts] of all.  Called by the whole CTA, which synchronises
// afterwards; the scan is warp 0's.
struct Segments {
  int* lo;       // [MAX_EXPERTS]
  int* len;      // [MAX_EXPERTS]
  int* tiles;    // [MAX_EXPERTS + 1]
};
constexpr uint32_t SEGMENT_BYTES = (3 * MAX_EXPERTS + 4) * 4;

__device__ __forceinline__ Segments segments_at(void* smem) {
  int* i = static_cast<int*>(smem);
  return Segments{i, i + MAX_EXPERTS, i + 2 * MAX_EXPERTS};
}

// Where starts decrease, segments may hold the same rows, which two experts
// would then store in a race: those that begin before the end of an earlier
// one are bad too.  Warp 0's; experts e0 .. e1 - 1 are this lane's.  Returns
// their tiles.
__device__ __noinline__ int drop_overlaps(const Segments s, int e0, int e1, int rows) {
  int before = 0;
  for (int e = e0; e < e1; ++e)
    if (s.len[e] >= 0) before = max(before, s.lo[e] + s.len[e]);
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, before, d);
    if ((int)threadIdx.x >= d) before = max(before, up);
  }
  before = __shfl_up_sync(0xffffffffu, before, 1);
  if (threadIdx.x == 0) before = 0;
  int tiles = 0;
  for (int e = e0; e < e1; ++e) {
    if (s.len[e] < 0) continue;
    const int lo = s.lo[e], end = lo + s.len[e];
    if (lo < before) s.len[e] = -1;
    else tiles += (s.len[e] + rows - 1) / rows;
    before = max(before, end);
  }
  return tiles;
}

__device__ __forceinline__ void load_segments(const Params& p, const Segments& s, int rows,
                                              int threads) {
  const int room = p.form == GEMM_F8_BY_INNER ? p.K : p.M;
  for (int e = threadIdx.x; e < p.experts; e += threads) {
    const int lo = p.starts[e], hi = p.starts[e + 1];
    bool bad = lo < 0 || hi < lo || hi > room;
    if (p.form == GEMM_F8_BY_INNER)
      bad = bad || (lo & (BLOCK - 1)) || ((hi & (BLOCK - 1)) && hi != room);
    if (bad) report_bad_index(p);
    s.lo[e] = bad ? 0 : lo;
    s.len[e] = bad ? -1 : hi - lo;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int per = (p.experts + 31) / 32, e0 = (int)threadIdx.x * per;
    int sum = 0;
    bool bad = false;
    for (int e = e0; e < min(e0 + per, p.experts); ++e) {
      sum += (s.len[e] + rows - 1) / rows;      // 0 for -1
      bad = bad || s.len[e] < 0;
    }
    // Starts that never decrease make segments without common rows.
    if (__any_sync(0xffffffffu, bad) && p.form == GEMM_F8_BY_ROWS)
      sum = drop_overlaps(s, e0, min(e0 + per, p.experts), rows);
    int before = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, before, d);
      if ((int)threadIdx.x >= d) before += up;
    }
    before -= sum;
    for (int e = e0; e < min(e0 + per, p.experts); ++e) {
      s.tiles[e] = before;
      before += (s.len[e] + rows - 1) / rows;
    }
    if (threadIdx.x == 31) s.tiles[p.experts] = before;   // e0 + per >= experts here
  }
}

// The expert whose tiles hold tile t: the last with tiles[e] <= t (experts
// without rows share the next one's number and come before it).
__device__ __forceinline__ int expert_of_tile(const Segments& s, int experts, int t) {
  int lo = 0, hi = experts - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.tiles[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A row of C, by a warp: every 16 bits those of `bits`.
__device__ __forceinline__ void fill_row(uint8_t* row, int64_t bytes, uint32_t bits, bool vec,
                                         uint32_t lane) {
  int64_t at = 0;
  if (vec) {
    for (int64_t i = (int64_t)lane * 16; i + 16 <= bytes; i += 512)
      *reinterpret_cast<uint4*>(row + i) = make_uint4(bits, bits, bits, bits);
    at = bytes & ~(int64_t)15;
  }
  for (int64_t i = at + (int64_t)lane * 2; i < bytes; i += 64)
    *reinterpret_cast<uint16_t*>(row + i) = (uint16_t)bits;
}

// What no tile stores, by warp `w` of `warps`.  BY_ROWS: rows of C past the last
// expert's are 0 (by the segments that were found good: starts[experts] may be a
// bad one, below rows that others store).  BY_INNER: the matrix of an expert
// whose starts are bad is NaN, for zeros would pass for a gradient.
__device__ __forceinline__ void fill_rest(const Params& p, const Segments& s, int w, int warps,
                                          uint32_t lane) {
  if (p.form == GEMM_F8_DENSE) return;
  const int size = p.type == GEMM_F8_F32 ? 4 : 2;
  const int64_t bytes = (int64_t)p.N * size;
  uint8_t* C = static_cast<uint8_t*>(p.C);
  if (p.form == GEMM_F8_BY_INNER) {
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
      const int mine = e0 + (int)lane;
      for (uint32_t bad = __ballot_sync(0xffffffffu, mine < p.experts && s.len[mine] < 0); bad != 0;
           bad &= bad - 1) {
        const int64_t e = e0 + __ffs(bad) - 1;
        for (int64_t r = w; r < p.M; r += warps)
          fill_row(C + (e * p.c_batch + r * p.ldc) * size, bytes, 0xffffffffu, p.vec, lane);
      }
    }
    return;
  }
  if (p.accumulate) return;
  int last = p.experts - 1;
  while (last >= 0 && s.len[last] < 0) --last;
  if (last < 0) return;
  const int end = s.lo[last] + s.len[last];
  for (int64_t r = (int64_t)end + w; r < p.M; r += warps)
    fill_row(C + r * p.ldc * size, bytes, 0, p.vec, lane);
}

template <typename T>
__device__ __forceinline__ T to_type(float x);
template <>
__device__ __forceinline__ float to_type<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half to_type<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 to_type<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Two numbers of a 16-bit type in one word.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_b64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

}  // namespace f8
}  // namespace gf16
