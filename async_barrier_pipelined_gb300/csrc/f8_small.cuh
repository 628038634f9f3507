// 8-bit products with block scales: the kernel for few rows.
//
// With few rows of A the time is that of reading B.  The operands change
// places: 128 columns of C (rows of B's transpose) are the MMA's 128 rows and
// NT (16, 32 or 64) rows of A its columns, so that no tensor-core work is
// spent on more rows than there are.  A cluster of `split` CTAs (1, 2, 4 or 8)
// shares a tile's K blocks, so that all SMs read B even where it has few
// tiles; each CTA sums its blocks in registers (one column of C and NT rows a
// thread), and at the end the CTAs of the cluster read one another's sums from
// shared memory, each a share of the rows, add them in the order of the ranks
// and store.  No workspace, one launch, the same bits every time.
//
// What bounds it: B's bytes at the rate of the memory.  A stage holds 16 KB of
// B; with three to five stages in two CTAs per SM, 96 to 160 KB are on their way
// per SM, twice to three times what 6.8 TB/s need at a latency of a microsecond.
//
// Work units: tiles of 128 columns x NT rows, those of the same columns side by
// side (they read the same part of B); clusters walk them.  BY_ROWS: NT rows
// within an expert's segment.
#pragma once

#include "f8.cuh"

namespace gf16 {
namespace f8 {
namespace small {

constexpr int CN = 128;              // columns of C in a tile
constexpr int NUM_THREADS = 192;
constexpr int PROMOTE_WARP0 = 2, PROMOTE_WARPS = 4;
constexpr int MAX_SPLIT = 8;
constexpr uint32_t B_STAGE = CN * BLOCK;   // 16 KB

template <int NT>
struct Cfg {
  static constexpr int STAGES = NT == 64 ? 3 : NT == 32 ? 4 : 5;
  static constexpr int CTAS = 2;                         // per SM
  static constexpr int RED = NT < 32 ? NT : 32;          // rows of A summed across the cluster at a time
  static constexpr uint32_t A_STAGE = NT * BLOCK;
  static constexpr uint32_t STAGE = A_STAGE + B_STAGE;
  static constexpr uint32_t TMEM_COLS = 2 * NT < 32 ? 32 : 2 * NT;
  static constexpr uint32_t OFF_RED = STAGES * STAGE;
  static constexpr uint32_t OFF_SA = OFF_RED + RED * CN * 4;   // a warp's scales of A's rows, twice
  // BY_ROWS only: a product without experts is launched without it
  static constexpr uint32_t OFF_BAR = OFF_SA + PROMOTE_WARPS * 2 * NT * 4;
  static constexpr uint32_t NUM_BARS = 2 * STAGES + 2 + 2 + 1 + 2;
  static constexpr uint32_t OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr uint32_t OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr uint32_t OFF_SEG = (OFF_ABORT + 4 + 15) / 16 * 16;
  static constexpr uint32_t SMEM = OFF_SEG + 1024;
  static constexpr uint32_t SMEM_EXPERTS = SMEM + SEGMENT_BYTES;
  static_assert(STAGE % 1024 == 0 && OFF_BAR % 8 == 0 && OFF_SA % 16 == 0, "alignment");
  static_assert(CTAS * (SMEM_EXPERTS + 1024) <= 233472, "shared memory of an SM");
};

struct Bars {
  uint32_t full, empty, tfull, tempty, mma_done, red_full, red_empty;
};

struct Unit {
  int m0, m_end, n0, expert;
};

template <int NT>
__device__ __forceinline__ int total_units(const Params& p, const Segments& s) {
  return p.form == GEMM_F8_BY_ROWS ? s.tiles[p.experts] * p.tiles_n : p.units;
}

template <int NT>
__device__ __forceinline__ Unit unit_at(const Params& p, const Segments& s, int u) {
  Unit g;
  if (p.form == GEMM_F8_BY_ROWS) {
    const int e = expert_of_tile(s, p.experts, u / p.tiles_n);
    const int r = u - s.tiles[e] * p.tiles_n, count = s.tiles[e + 1] - s.tiles[e];
    const int tn = r / count;
    g.expert = e;
    g.m0 = s.lo[e] + (r - tn * count) * NT;
    g.m_end = s.lo[e] + s.len[e];
    g.n0 = tn * CN;
  } else {
    const int tn = u / p.tiles_m;
    g.expert = 0;
    g.m0 = (u - tn * p.tiles_m) * NT;
    g.m_end = p.M;
    g.n0 = tn * CN;
  }
  return g;
}

template <int NT>
__device__ __forceinline__ uint32_t producer_role(const CUtensorMap* tmA, const CUtensorMap* tmB,
                                                  const Params& p, const Segments& s,
                                                  uint32_t base, int kb0, int kb1, int cluster,
                                                  int clusters, const Bars& b,
                                                  volatile int* abort_flag) {
  using C = Cfg<NT>;
  RingPos pos{0, 0};
  uint32_t issued = 0;
  const int units = total_units<NT>(p, s);
  for (int u = cluster; u < units; u += clusters) {
    const Unit g = unit_at<NT>(p, s, u);
    for (int i = kb0; i < kb1; ++i) {
      if (!wait_phase(b.empty + 8 * pos.stage, producer_wait_parity(pos), p, abort_flag))
        return issued;
      const uint32_t bar = b.full + 8 * pos.stage, at = base + pos.stage * C::STAGE;
      ptx::mbar_arrive_expect_tx_relaxed(bar, C::STAGE);
      ++issued;
      if (u != p.fault_unit || i != kb0) {
        if (p.b_mn) ptx::tma_load_3d(at, tmB, bar, g.n0, i * BLOCK, g.expert);
        else ptx::tma_load_3d(at, tmB, bar, i * BLOCK, g.n0, g.expert);
        ptx::tma_load_3d(at + B_STAGE, tmA, bar, i * BLOCK, g.m0, 0);
      }
      ring_advance(pos, C::STAGES);
    }
  }
  return issued;
}

template <int NT>
__device__ __forceinline__ void mma_role(const Params& p, const Segments& s, uint32_t base,
                                         uint32_t tmem_base, int kb0, int kb1, int cluster,
                                         int clusters, const Bars& b, volatile int* abort_flag) {
  using C = Cfg<NT>;
  RingPos pos{0, 0};
  uint32_t done = 0;
  const uint32_t b_step = (p.b_mn ? MN_STEP : K_STEP) >> 4;
  const int units = total_units<NT>(p, s);
  bool ok = true;
  for (int u = cluster; u < units && ok; u += clusters) {
    for (int i = kb0; i < kb1; ++i, ++done) {
      const uint32_t half = done & 1u;
      if (!wait_phase(b.tempty + 8 * half, ((done >> 1) & 1u) ^ 1u, p, abort_flag) ||
          !wait_phase(b.full + 8 * pos.stage, consumer_wait_parity(pos), p, abort_flag)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t at = base + pos.stage * C::STAGE;
      const uint64_t rows = smem_desc_sw128(at, DESC_LBO, DESC_SBO);
      const uint64_t cols = smem_desc_sw128(at + B_STAGE, DESC_LBO, DESC_SBO);
#pragma unroll
      for (uint32_t k = 0; k < BLOCK / MMA_K; ++k)
        ptx::mma_f8(tmem_base + half * NT, rows + k * b_step, cols + k * (K_STEP >> 4), p.idesc,
                    k != 0);
      ptx::mma_commit(b.empty + 8 * pos.stage);
      ptx::mma_commit(b.tfull + 8 * half);
      ring_advance(pos, C::STAGES);
    }
  }
  ptx::mma_commit(b.mma_done);
  wait_drain(b.mma_done, 0, p.timeout_ns);
}

// One number of C, row m and column n.
template <typename T>
__device__ __forceinline__ void store_one(const Params& p, T* C, int m, int n, float v) {
  T* at = C + (int64_t)m * p.ldc + n;
  if constexpr (sizeof(T) == 4) *at = p.accumulate ? *at + v : v;
  else *at = to_type<T>(v);
}
__device__ __forceinline__ void store_any(const Params& p, int m, int n, float v) {
  if (p.type == GEMM_F8_F16) store_one(p, static_cast<__half*>(p.C), m, n, v);
  else if (p.type == GEMM_F8_BF16) store_one(p, static_cast<__nv_bfloat16*>(p.C), m, n, v);
  else store_one(p, static_cast<float*>(p.C), m, n, v);
}

template <int NT>
__device__ __forceinline__ void promote_role(const Params& p, const Segments& s, uint32_t base,
                                             uint32_t tmem_base, uint32_t rank, uint32_t split,
                                             int kb0, int kb1, int cluster, int clusters,
                                             const Bars& b, uint32_t warp, uint32_t lane,
                                             volatile int* abort_flag) {
  using C = Cfg<NT>;
  constexpr int PER = NT < 32 ? 1 : NT / 32;      // scales of A's rows a lane fetches
  constexpr int LD = NT < 32 ? NT : 32;           // columns of a tensor-memory load
  const uint32_t quarter = warp & 3u, me = quarter * 32u + lane;
  const uint32_t sa_buf = base + C::OFF_SA + (warp - PROMOTE_WARP0) * 2 * NT * 4;
  const uint32_t t_row = tmem_base + ((quarter * 32u) << 16);
  uint32_t done = 0, reds = 0;
  const int units = total_units<NT>(p, s);
  for (int u = cluster; u < units; u += clusters) {
    const Unit g = unit_at<NT>(p, s, u);
    const int n = g.n0 + (int)me;
    const float* pb = p.sb + (p.form == GEMM_F8_BY_ROWS ? g.expert * p.sb_batch : 0) +
                      (int64_t)(min(n, p.N - 1) >> p.sb_shift) * p.sb_outer + (int64_t)kb0 * p.sb_inner;
    const float* pa[PER];
    float na[PER], nb = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      pa[i] = p.sa + (int64_t)(min(g.m0 + (int)lane + 32 * i, g.m_end - 1) >> p.sa_shift) * p.sa_outer +
              (int64_t)kb0 * p.sa_inner;
    if (kb0 < kb1) {
      nb = *pb;
#pragma unroll
      for (int i = 0; i < PER; ++i) na[i] = *pa[i];
    }
    uint64_t acc[NT / 2];
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) acc[i] = 0;
    for (int i = kb0; i < kb1; ++i, ++done) {
      const uint32_t half = done & 1u, abuf = sa_buf + half * NT * 4;
      const float sb = nb;
#pragma unroll
      for (int c = 0; c < PER; ++c)
        if (NT >= 32 || (int)lane < NT) st_shared_f32(abuf + (lane + 32u * c) * 4u, na[c]);
      if (i + 1 < kb1) {
        pb += p.sb_inner;
        nb = *pb;
#pragma unroll
        for (int c = 0; c < PER; ++c) {
          pa[c] += p.sa_inner;
          na[c] = *pa[c];
        }
      }
      const bool got = wait_phase(b.tfull + 8 * half, (done >> 1) & 1u, p, abort_flag);
      if (!__all_sync(0xffffffffu, got)) return;
      __syncwarp();     // the warp's scales are in shared memory
      ptx::tc_fence_after();
      const uint64_t sb2 = ptx::pack_f2(sb, sb);
#pragma unroll
      for (int c = 0; c < NT / LD; ++c) {
        uint32_t r[LD];
        if constexpr (LD == 16) ptx::tmem_ld_32x32b_x16(t_row + half * NT, r);
        else ptx::tmem_ld_32x32b_x32(t_row + half * NT + 32u * c, r);
        ptx::tmem_ld_wait();
        ptx::reg_fence(r);
        if (c == NT / LD - 1) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(b.tempty + 8 * half);
        }
#pragma unroll
        for (int j = 0; j < LD / 4; ++j) {
          const uint4 q = ld_shared_v4(abuf + (LD * c + 4u * j) * 4u);
          const uint64_t x0 = ptx::pack_f2(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]));
          const uint64_t x1 = ptx::pack_f2(__uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
          const uint64_t q0 = ptx::pack_f2(__uint_as_float(q.x), __uint_as_float(q.y));
          const uint64_t q1 = ptx::pack_f2(__uint_as_float(q.z), __uint_as_float(q.w));
          uint64_t* a = acc + (LD * c) / 2 + 2 * j;
          a[0] = ptx::fma_f2(ptx::mul_f2(x0, q0), sb2, a[0]);
          a[1] = ptx::fma_f2(ptx::mul_f2(x1, q1), sb2, a[1]);
        }
      }
    }
    if (split == 1) {
      if (n < p.N) {
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
          float v0, v1;
          ptx::unpack_f2(acc[i], v0, v1);
          if (g.m0 + 2 * i < g.m_end) store_any(p, g.m0 + 2 * i, n, v0);
          if (g.m0 + 2 * i + 1 < g.m_end) store_any(p, g.m0 + 2 * i + 1, n, v1);
        }
      }
      continue;
    }
    // The cluster's sums, RED rows of A at a time.
    const uint32_t share = C::RED / split;     // rows of them that this CTA adds and stores
    const uint32_t shift = 31 - __clz(split);  // split is 2, 4 or 8
    const uint32_t mine = base + C::OFF_RED + me * 4u;
#pragma unroll
    for (int c = 0; c < NT / C::RED; ++c) {
      if (g.m0 + c * C::RED >= g.m_end) break;   // the same in all CTAs of the cluster
      bool got = wait_phase_cluster(b.red_empty, (reds & 1u) ^ 1u, p, abort_flag);
      if (!__all_sync(0xffffffffu, got)) return;
#pragma unroll
      for (int i = 0; i < C::RED / 2; ++i) {
        float v0, v1;
        ptx::unpack_f2(acc[(c * C::RED) / 2 + i], v0, v1);
        st_shared_f32(mine + (2 * i) * CN * 4, v0);
        st_shared_f32(mine + (2 * i + 1) * CN * 4, v1);
      }
      __syncwarp();
      if (lane < split) ptx::mbar_arrive_cluster(ptx::map_to_cta(b.red_full, lane));
      got = wait_phase_cluster(b.red_full, reds & 1u, p, abort_flag);
      if (!__all_sync(0xffffffffu, got)) return;
      // Sixteen remote numbers on their way at a time, of one row after another
      // (7 x 12288 x 4096: 13.6 us with one at a time, 12.6).
      for (uint32_t i0 = 0; i0 < (uint32_t)C::RED; i0 += 16) {
        float v[16];
#pragma unroll
        for (uint32_t k = 0; k < 16; ++k) {
          const uint32_t i = i0 + k, row = rank * share + (i >> shift);
          v[k] = ptx::ld_cluster_f32(ptx::map_to_cta(mine + row * CN * 4, i & (split - 1)));
        }
        float sum = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < 16; ++k) {
          const uint32_t i = i0 + k, q = i & (split - 1);
          sum = (q == 0 ? 0.f : sum) + v[k];
          const int m = g.m0 + c * C::RED + (int)(rank * share + (i >> shift));
          if (q == split - 1 && n < p.N && m < g.m_end) store_any(p, m, n, sum);
        }
      }
      // The loads have been used, all but those of columns that are not stored:
      // nothing to wait for before the others may write again.
      __syncwarp();
      if (lane < split) ptx::mbar_arrive_cluster_relaxed(ptx::map_to_cta(b.red_empty, lane));
      ++reds;
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(NUM_THREADS, Cfg<NT>::CTAS)
    f8_small_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Params p) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = ptx::cluster_ctarank(), split = ptx::cluster_nctarank();
  const int cluster = (int)(blockIdx.x / split), clusters = (int)(gridDim.x / split);
  const Segments seg = segments_at(smem + C::OFF_SEG);
  int kb0, kb1;
  split_range(p.kblocks, (int)split, (int)rank, &kb0, &kb1);

  Bars b;
  b.full = base + C::OFF_BAR;
  b.empty = b.full + 8 * C::STAGES;
  b.tfull = b.empty + 8 * C::STAGES;
  b.tempty = b.tfull + 16;
  b.mma_done = b.tempty + 16;
  b.red_full = b.mma_done + 8;
  b.red_empty = b.red_full + 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);

  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(b.full + 8 * s, 1);
      ptx::mbar_init(b.empty + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(b.tfull + 8 * a, 1);
      ptx::mbar_init(b.tempty + 8 * a, PROMOTE_WARPS);
    }
    ptx::mbar_init(b.mma_done, 1);
    ptx::mbar_init(b.red_full, PROMOTE_WARPS * split);
    ptx::mbar_init(b.red_empty, PROMOTE_WARPS * split);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(base + C::OFF_TMEM_SLOT, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ptx::tc_fence_before();
  __syncthreads();
  if (split > 1) ptx::cluster_sync();   // the others' barriers exist
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM_SLOT);
  // All of this beside the end of the kernel before; its results from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.form != GEMM_F8_DENSE) {
    load_segments(p, seg, NT, NUM_THREADS);
    __syncthreads();
  }

  uint32_t issued = 0;
  if (warp == 0) {
    if (lane == 0)
      issued = producer_role<NT>(&tmA, &tmB, p, seg, base, kb0, kb1, cluster, clusters, b,
                                 abort_flag);
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0)
      mma_role<NT>(p, seg, base, tmem_base, kb0, kb1, cluster, clusters, b, abort_flag);
    __syncwarp();
  } else {
    promote_role<NT>(p, seg, base, tmem_base, rank, split, kb0, kb1, cluster, clusters, b, warp,
                     lane, abort_flag);
    __syncwarp();
    fill_rest(p, seg, (int)blockIdx.x * PROMOTE_WARPS + (int)warp - PROMOTE_WARP0,
              (int)gridDim.x * PROMOTE_WARPS, lane);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (split > 1) ptx::cluster_sync();   // none of the others reads our sums any more
  if (warp == 0 && lane == 0 && *abort_flag) {
    // Until the copies that were issued have landed (a bounded wait each: the
    // fill that an abort waited for in vain may never complete).
    const uint32_t lo = issued > (uint32_t)C::STAGES ? issued - C::STAGES : 0u;
    for (uint32_t j = lo; j < issued; ++j)
      wait_drain(b.full + 8 * (j % C::STAGES), (j / C::STAGES) & 1u, p.timeout_ns);
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace small
}  // namespace f8
}  // namespace gf16
