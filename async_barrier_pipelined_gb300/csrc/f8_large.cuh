// 8-bit products with block scales: the kernel for many rows.
//
// A cluster of two CTAs (tcgen05 cta_group::2) computes tiles of 256 x 256:
// each CTA holds 128 rows of A and 128 columns of B (16 KB each per K block of
// 128, one swizzled copy each, K-major or MN-major), the even CTA issues four
// 256 x 256 x 32 MMAs per K block, and each block's products go to one half of
// tensor memory (256 of 512 columns) while eight promotion warps per CTA take
// the block before out of the other half and add it, scaled, to FP32
// registers: a thread holds one row and 128 columns.
//
// What bounds it: an SM's tensor core takes 512 cycles for a K block (128 x
// 256 x 128 products at 8192 a cycle), its four FP32 pipes 256 for one fused
// multiply-add per product (scales per tile of B: sa * sb is one number for a
// thread's 128 columns) or 512 for two operations (a scale per column of B).
// So the accumulation hides behind the tensor core, just so in the second
// case.
//
// DENSE: pairs walk the tiles in bands of eight tile rows.  A last wave of
// `rem` tiles with rem <= pairs / 2 is cut into `parts` ranges of K blocks, so
// that no pair idles: each writes FP32 sums to the workspace, and whichever warp finds itself the last of
// its rows and columns (a counter, one for each warp's piece of a tile) adds
// the parts in their order and stores C.  BY_ROWS: tiles of 256 rows within
// an expert's segment, those of one column of tiles side by side.  BY_INNER:
// all tiles of each expert, with that expert's K blocks.
//
// Barriers (as in gemm_pair.cuh): full[s] leader only, 1 arrival and both
// CTAs' bytes; empty[s] both CTAs, multicast commit; tfull[a] both CTAs,
// multicast commit after a K block; tempty[a] leader only, 16 arrivals (8
// promotion warps per CTA); mma_done leader only.  Waits are bounded; after an
// abort the leader completes the phases of copies that were issued.
#pragma once

#include "f8.cuh"

namespace gf16 {
namespace f8 {
namespace large {

constexpr int PM = 256, PN = 256, CM = 128;
constexpr int STAGES = 5;
constexpr int NUM_THREADS = 384;
constexpr int PROMOTE_WARP0 = 4, PROMOTE_WARPS = 8;
constexpr int BAND = 8;              // tile rows of a band

constexpr uint32_t A_STAGE = CM * BLOCK;      // 16 KB
constexpr uint32_t B_STAGE = (PN / 2) * BLOCK;
constexpr uint32_t CTA_STAGE_TX = A_STAGE + B_STAGE;
constexpr uint32_t EPI_BUF = 32 * 128;        // 32 rows of 128 bytes
constexpr uint32_t TMEM_COLS = 512;

constexpr uint32_t OFF_A = 0;
constexpr uint32_t OFF_B = OFF_A + STAGES * A_STAGE;
constexpr uint32_t OFF_EPI = OFF_B + STAGES * B_STAGE;
constexpr uint32_t OFF_SB = OFF_EPI + PROMOTE_WARPS * EPI_BUF;     // a warp's column scales, twice
constexpr uint32_t OFF_SEG = OFF_SB + PROMOTE_WARPS * 2 * 128 * 4;
constexpr uint32_t OFF_BAR = OFF_SEG + SEGMENT_BYTES;
constexpr uint32_t NUM_BARS = 2 * STAGES + 2 + 2 + 1;
constexpr uint32_t OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr uint32_t OFF_PEER_ISSUED = OFF_ABORT + 4;
constexpr uint32_t SMEM_BYTES = OFF_PEER_ISSUED + 4 + 1024;
static_assert(SMEM_BYTES <= 232448, "over the 227 KB shared-memory limit per CTA");
static_assert(OFF_BAR % 8 == 0 && OFF_EPI % 128 == 0 && OFF_SB % 16 == 0, "alignment");

// Registers: 384 threads launch with 168 each (64,512); the four other warps
// give up 112 each and the promotion warps take 56 more (128 * 56 + 256 * 224).
constexpr int IO_REGS = 56, PROMOTE_REGS = 224;
static_assert(128 * IO_REGS + 256 * PROMOTE_REGS <= 384 * 168, "register split");

// FP32 numbers of a cut tile's part, and the counters of a cut tile.
constexpr int PART_FLOATS = PM * PN;
constexpr int TILE_COUNTERS = 2 * PROMOTE_WARPS;

struct Bars {
  uint32_t full, empty, tfull, tempty, mma_done;
};

struct Unit {
  int m0, m_end;     // first row of the tile, end of its rows
  int n0;
  int expert;        // B's matrix (BY_ROWS), C's (BY_INNER), else 0
  int k0, blk0;      // first inner number and first block
  int nkb;           // K blocks
  int tail, part;    // cut tile and part, or -1
};

__device__ __forceinline__ void band_tile(int t, int tiles_m, int tiles_n, int* tm, int* tn) {
  const int per = BAND * tiles_n, band = t / per, r = t - band * per;
  const int h = min(BAND, tiles_m - band * BAND);
  *tn = r / h;
  *tm = band * BAND + r - *tn * h;
}

__device__ __forceinline__ int total_units(const Params& p, const Segments& s) {
  return p.form == GEMM_F8_BY_ROWS ? s.tiles[p.experts] * p.tiles_n : p.units;
}

__device__ __forceinline__ Unit unit_at(const Params& p, const Segments& s, int u) {
  Unit g;
  g.tail = -1;
  g.part = 0;
  g.expert = 0;
  g.k0 = 0;
  g.blk0 = 0;
  g.nkb = p.kblocks;
  g.m_end = p.M;
  int tm, tn;
  if (p.form == GEMM_F8_BY_ROWS) {
    const int e = expert_of_tile(s, p.experts, u / p.tiles_n);
    const int r = u - s.tiles[e] * p.tiles_n, count = s.tiles[e + 1] - s.tiles[e];
    tn = r / count;
    tm = r - tn * count;
    g.expert = e;
    g.m0 = s.lo[e] + tm * PM;
    g.m_end = s.lo[e] + s.len[e];
    g.n0 = tn * PN;
    return g;
  }
  if (p.form == GEMM_F8_BY_INNER) {
    const int per = p.tiles_m * p.tiles_n;
    g.expert = u / per;
    g.k0 = s.lo[g.expert];
    g.blk0 = g.k0 / BLOCK;
    g.nkb = (s.len[g.expert] + BLOCK - 1) / BLOCK;
    band_tile(u - g.expert * per, p.tiles_m, p.tiles_n, &tm, &tn);
  } else {
    int t = u;
    if (u >= p.full_units) {
      const int v = u - p.full_units;
      g.tail = v / p.parts;
      g.part = v - g.tail * p.parts;
      int end;
      split_range(p.kblocks, p.parts, g.part, &g.blk0, &end);
      g.nkb = end - g.blk0;
      g.k0 = g.blk0 * BLOCK;
      t = p.full_units + g.tail;
    }
    band_tile(t, p.tiles_m, p.tiles_n, &tm, &tn);
  }
  g.m0 = tm * PM;
  g.n0 = tn * PN;
  return g;
}

__device__ __forceinline__ uint32_t producer_role(const CUtensorMap* tmA, const CUtensorMap* tmB,
                                                  const Params& p, const Segments& s,
                                                  uint32_t base, uint32_t rank, int pair,
                                                  int npairs, const Bars& b,
                                                  volatile int* abort_flag) {
  const uint32_t leader_full = ptx::map_to_cta(b.full, 0);
  RingPos pos{0, 0};
  uint32_t issued = 0;
  const int units = total_units(p, s);
  for (int u = pair; u < units; u += npairs) {
    const Unit g = unit_at(p, s, u);
    const int m0 = g.m0 + (int)rank * CM, n0 = g.n0 + (int)rank * (PN / 2);
    const int zb = p.form == GEMM_F8_BY_ROWS ? g.expert : 0;
    const int skip = (u == p.fault_unit && rank == 0) ? 0 : -1;
    for (int i = 0; i < g.nkb; ++i) {
      if (!wait_phase(b.empty + 8 * pos.stage, producer_wait_parity(pos), p, abort_flag))
        return issued;
      if (rank == 0) ptx::mbar_arrive_expect_tx_relaxed(b.full + 8 * pos.stage, 2 * CTA_STAGE_TX);
      if (i != skip) {
        const uint32_t fb = leader_full + 8 * pos.stage;
        const int k = g.k0 + i * BLOCK;
        const uint32_t sa = base + OFF_A + pos.stage * A_STAGE;
        const uint32_t sb = base + OFF_B + pos.stage * B_STAGE;
        if (p.a_mn) ptx::tma_load_3d_pair(sa, tmA, fb, m0, k, 0);
        else ptx::tma_load_3d_pair(sa, tmA, fb, k, m0, 0);
        if (p.b_mn) ptx::tma_load_3d_pair(sb, tmB, fb, n0, k, zb);
        else ptx::tma_load_3d_pair(sb, tmB, fb, k, n0, zb);
      }
      ++issued;
      ring_advance(pos, STAGES);
    }
  }
  return issued;
}

__device__ __forceinline__ void mma_role(const Params& p, const Segments& s, uint32_t base,
                                         uint32_t tmem_base, int pair, int npairs, const Bars& b,
                                         volatile int* abort_flag) {
  RingPos pos{0, 0};
  uint32_t done = 0;    // K blocks so far: block i uses half i & 1
  const uint32_t a_step = (p.a_mn ? MN_STEP : K_STEP) >> 4;
  const uint32_t b_step = (p.b_mn ? MN_STEP : K_STEP) >> 4;
  const int units = total_units(p, s);
  bool ok = true;
  for (int u = pair; u < units && ok; u += npairs) {
    const int nkb = unit_at(p, s, u).nkb;
    for (int i = 0; i < nkb; ++i, ++done) {
      const uint32_t half = done & 1u;
      if (!wait_phase(b.tempty + 8 * half, ((done >> 1) & 1u) ^ 1u, p, abort_flag) ||
          !wait_phase(b.full + 8 * pos.stage, consumer_wait_parity(pos), p, abort_flag)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint64_t a = smem_desc_sw128(base + OFF_A + pos.stage * A_STAGE, DESC_LBO, DESC_SBO);
      const uint64_t bd = smem_desc_sw128(base + OFF_B + pos.stage * B_STAGE, DESC_LBO, DESC_SBO);
#pragma unroll
      for (uint32_t k = 0; k < BLOCK / MMA_K; ++k)
        ptx::mma_f8_pair(tmem_base + half * PN, a + k * a_step, bd + k * b_step, p.idesc, k != 0);
      ptx::mma_commit_pair(b.empty + 8 * pos.stage, 0x3);
      ptx::mma_commit_pair(b.tfull + 8 * half, 0x3);
      ring_advance(pos, STAGES);
    }
  }
  ptx::mma_commit_pair(b.mma_done, 0x1);
  wait_drain(b.mma_done, 0, p.timeout_ns);
}

// A warp's 32 rows x 128 columns (acc: this lane's row) to C through a staging
// buffer of 32 rows x 128 bytes, so that a store instruction writes four whole
// lines of 128 bytes and not 16 bytes of each of 32 rows.
template <typename T>
__device__ __forceinline__ void store_rows(const Params& p, T* C, const uint64_t (&acc)[64],
                                           uint32_t stage, int row0, int row_end, int col0,
                                           uint32_t lane) {
  constexpr int V = 16 / sizeof(T);        // numbers of a 16-byte unit
  constexpr int COLS = 128 / sizeof(T);    // columns of a staging buffer
#pragma unroll
  for (int c = 0; c < 128 / COLS; ++c) {
    if (col0 + c * COLS >= p.N) break;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      float v[V];
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        ptx::unpack_f2(acc[(c * COLS + (int)j * V) / 2 + i], v[2 * i], v[2 * i + 1]);
      uint32_t w[4];
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
      }
      ptx::st_shared_v4(stage + lane * 128u + ((j ^ (lane & 7u)) << 4), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t r = i * 4 + (lane >> 3), j = lane & 7u;
      uint4 v = ld_shared_v4(stage + r * 128u + ((j ^ (r & 7u)) << 4));
      const int row = row0 + (int)r, col = col0 + c * COLS + (int)j * V;
      if (row >= row_end || col >= p.N) continue;
      T* at = C + (int64_t)row * p.ldc + col;
      if (p.vec && col + V <= p.N) {
        if constexpr (sizeof(T) == 4) {
          if (p.accumulate) {
            const float4 old = *reinterpret_cast<const float4*>(at);
            v.x = __float_as_uint(old.x + __uint_as_float(v.x));
            v.y = __float_as_uint(old.y + __uint_as_float(v.y));
            v.z = __float_as_uint(old.z + __uint_as_float(v.z));
            v.w = __float_as_uint(old.w + __uint_as_float(v.w));
          }
        }
        *reinterpret_cast<uint4*>(at) = v;
      } else {
        const T* x = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (col + k < p.N) {
            if constexpr (sizeof(T) == 4) at[k] = p.accumulate ? at[k] + x[k] : x[k];
            else at[k] = x[k];
          }
        }
      }
    }
    __syncwarp();
  }
}

// This warp's piece of a cut tile: its part to the workspace; true for the
// warp that finds all others' there, with their sum (in the parts' order) in
// acc.
__device__ __forceinline__ bool join_parts(const Params& p, const Unit& g, uint32_t rank,
                                           uint32_t w, uint32_t lane, uint64_t (&acc)[64]) {
  // part -> [rank][warp][pair of float2][lane], 16 bytes a lane
  const int64_t stride = PART_FLOATS / 4;
  ulonglong2* base = reinterpret_cast<ulonglong2*>(p.ws) + (int64_t)g.tail * p.parts * stride +
                     (rank * PROMOTE_WARPS + w) * 32 * 32 + lane;
  ulonglong2* mine = base + g.part * stride;
#pragma unroll
  for (int j = 0; j < 32; ++j) __stcg(mine + j * 32, make_ulonglong2(acc[2 * j], acc[2 * j + 1]));
  __threadfence();
  __syncwarp();
  unsigned before = 0;
  if (lane == 0)
    before = atomicAdd(p.counters + g.tail * TILE_COUNTERS + rank * PROMOTE_WARPS + w, 1u);
  before = __shfl_sync(0xffffffffu, before, 0);
  if (before != (unsigned)p.parts - 1) return false;
  __threadfence();
  const uint64_t one = ptx::pack_f2(1.f, 1.f);
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    ulonglong2 sum = __ldcg(base + j * 32);
    for (int i = 1; i < p.parts; ++i) {
      const ulonglong2 x = __ldcg(base + i * stride + j * 32);
      sum.x = ptx::fma_f2(x.x, one, sum.x);
      sum.y = ptx::fma_f2(x.y, one, sum.y);
    }
    acc[2 * j] = sum.x;
    acc[2 * j + 1] = sum.y;
  }
  return true;
}

// COLS: B has a scale for each column (else one for a thread's 128 columns).
template <bool COLS>
__device__ __forceinline__ void promote_role(const Params& p, const Segments& s, uint32_t base,
                                             uint32_t tmem_base, uint32_t rank, int pair,
                                             int npairs, const Bars& b, uint32_t warp,
                                             uint32_t lane, volatile int* abort_flag) {
  const uint32_t w = warp - PROMOTE_WARP0, quarter = warp & 3u, right = w >> 2;
  const uint32_t stage = base + OFF_EPI + w * EPI_BUF;
  const uint32_t sb_buf = base + OFF_SB + w * 2 * 128 * 4;
  const uint32_t t_row = tmem_base + ((quarter * 32u) << 16) + right * 128u;
  const uint32_t leader_tempty = ptx::map_to_cta(b.tempty, 0);
  uint32_t done = 0;
  const int units = total_units(p, s);
  for (int u = pair; u < units; u += npairs) {
    const Unit g = unit_at(p, s, u);
    const int row0 = g.m0 + (int)(rank * CM + quarter * 32);
    const int col0 = g.n0 + (int)right * 128;
    const int row = min(row0 + (int)lane, g.m_end - 1);
    const float* pa = p.sa + (int64_t)(row >> p.sa_shift) * p.sa_outer + (int64_t)g.blk0 * p.sa_inner;
    const float* pb = p.sb + (int64_t)g.blk0 * p.sb_inner +
                      (p.form == GEMM_F8_BY_ROWS ? g.expert * p.sb_batch : 0);
    if constexpr (!COLS) pb += (int64_t)(min(col0, p.N - 1) >> 7) * p.sb_outer;
    // This lane's column scales of a K block (COLS), or the one of all columns.
    const auto column_scales = [&](float(&v)[COLS ? 4 : 1]) {
      if constexpr (COLS) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = __ldg(pb + (int64_t)min(col0 + (int)lane + 32 * i, p.N - 1) * p.sb_outer);
      } else {
        v[0] = __ldg(pb);
      }
    };
    uint64_t acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0;
    float na = 0.f, nb[COLS ? 4 : 1];
    if (g.nkb > 0) {
      na = __ldg(pa);
      column_scales(nb);
    }
    for (int i = 0; i < g.nkb; ++i, ++done) {
      const uint32_t half = done & 1u;
      const float sa = na;
      float sb = nb[0];
      const uint32_t sbuf = sb_buf + half * 512u;
      if constexpr (COLS) {
#pragma unroll
        for (int c = 0; c < 4; ++c) st_shared_f32(sbuf + (lane + 32u * c) * 4u, nb[c]);
      }
      if (i + 1 < g.nkb) {     // the next block's scales, on their way during this one
        pa += p.sa_inner;
        na = __ldg(pa);
        pb += p.sb_inner;
        column_scales(nb);
      }
      // sa * sb is one number, unless it leaves FP32's normal range where the
      // product with the block's sum may not: then one after the other.
      const float sab = sa * sb;
      const bool split = !COLS && __any_sync(0xffffffffu, !(fabsf(sab) >= 1.17549435e-38f &&
                                                             fabsf(sab) <= 3.4e38f));
      const uint64_t s1 = ptx::pack_f2(sab, sab), sb2 = ptx::pack_f2(sb, sb),
                     sa2 = ptx::pack_f2(sa, sa);
      const bool got = wait_phase_inline(b.tfull + 8 * half, (done >> 1) & 1u, p, abort_flag);
      if (!__all_sync(0xffffffffu, got)) return;
      ptx::tc_fence_after();
      const uint32_t t = t_row + half * PN;
      // Two loads of 32 columns on their way at a time: a load's latency is
      // waited for twice a block.
      uint32_t r[2][32];
      ptx::tmem_ld_32x32b_x32(t, r[0]);
      ptx::tmem_ld_32x32b_x32(t + 32u, r[1]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if ((c & 1) == 0) {
          ptx::tmem_ld_wait();
          ptx::reg_fence(r[0]);
          ptx::reg_fence(r[1]);
          if (c == 2) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_cluster_relaxed(leader_tempty + 8 * half);
          }
        }
        const uint32_t(&x)[32] = r[c & 1];
        if constexpr (COLS) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 q = ld_shared_v4(sbuf + (32u * c + 4u * j) * 4u);
            const uint64_t q0 = ptx::pack_f2(__uint_as_float(q.x), __uint_as_float(q.y));
            const uint64_t q1 = ptx::pack_f2(__uint_as_float(q.z), __uint_as_float(q.w));
            const uint64_t x0 = ptx::pack_f2(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1]));
            const uint64_t x1 = ptx::pack_f2(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3]));
            acc[16 * c + 2 * j] = ptx::fma_f2(ptx::mul_f2(x0, q0), sa2, acc[16 * c + 2 * j]);
            acc[16 * c + 2 * j + 1] = ptx::fma_f2(ptx::mul_f2(x1, q1), sa2, acc[16 * c + 2 * j + 1]);
            asm volatile("" : "+l"(acc[16 * c + 2 * j]), "+l"(acc[16 * c + 2 * j + 1]));
          }
        } else if (!split) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[16 * c + j] = ptx::fma_f2(
                ptx::pack_f2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), s1,
                acc[16 * c + j]);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[16 * c + j] = ptx::fma_f2(
                ptx::mul_f2(ptx::pack_f2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])),
                            sb2), sa2, acc[16 * c + j]);
        }
        if (c < 2) ptx::tmem_ld_32x32b_x32(t + 64u + 32u * c, r[c]);
      }
    }
    if (row0 >= g.m_end && g.tail < 0) continue;
    if (g.tail >= 0 && !join_parts(p, g, rank, w, lane, acc)) continue;
    const int64_t off = p.form == GEMM_F8_BY_INNER ? g.expert * p.c_batch : 0;
    if (p.type == GEMM_F8_F16)
      store_rows<__half>(p, static_cast<__half*>(p.C) + off, acc, stage, row0, g.m_end, col0, lane);
    else if (p.type == GEMM_F8_BF16)
      store_rows<__nv_bfloat16>(p, static_cast<__nv_bfloat16*>(p.C) + off, acc, stage, row0,
                                g.m_end, col0, lane);
    else
      store_rows<float>(p, static_cast<float*>(p.C) + off, acc, stage, row0, g.m_end, col0, lane);
  }
}

// As pair::leader_drain: completes the phases that a producer opened, after an
// abort, so that no copy is in flight when the CTAs exit.
__device__ __noinline__ void leader_drain(const Bars& b, uint32_t mine, uint32_t peer,
                                          uint64_t limit_ns) {
  const uint32_t hi = mine > peer ? mine : peer;
  const uint32_t lo = hi > (uint32_t)STAGES ? hi - (uint32_t)STAGES : 0u;
  for (uint32_t j = lo; j < hi; ++j) {
    const uint32_t bar = b.full + 8 * (j % STAGES);
    if (j >= mine) ptx::mbar_arrive_expect_tx_relaxed(bar, CTA_STAGE_TX);
    if (j >= peer) ptx::mbar_complete_tx(bar, CTA_STAGE_TX);
    wait_drain(bar, (j / STAGES) & 1u, limit_ns);
  }
}

template <bool COLS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    f8_large_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = ptx::cluster_ctarank();
  const int pair = (int)(blockIdx.x >> 1), npairs = (int)(gridDim.x >> 1);
  const Segments seg = segments_at(smem + OFF_SEG);

  Bars b;
  b.full = base + OFF_BAR;
  b.empty = b.full + 8 * STAGES;
  b.tfull = b.empty + 8 * STAGES;
  b.tempty = b.tfull + 16;
  b.mma_done = b.tempty + 16;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);

  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(b.full + 8 * s, 1);
      ptx::mbar_init(b.empty + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(b.tfull + 8 * a, 1);
      ptx::mbar_init(b.tempty + 8 * a, 2 * PROMOTE_WARPS);
    }
    ptx::mbar_init(b.mma_done, 1);
    *abort_flag = 0;
    *reinterpret_cast<volatile uint32_t*>(smem + OFF_PEER_ISSUED) = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(base + OFF_TMEM_SLOT, TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.form != GEMM_F8_DENSE) load_segments(p, seg, PM, NUM_THREADS);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers exist before anyone signals them
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);

  uint32_t issued = 0;
  if (warp >= PROMOTE_WARP0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PROMOTE_REGS));
    promote_role<COLS>(p, seg, base, tmem_base, rank, pair, npairs, b, warp, lane, abort_flag);
    __syncwarp();
    zero_rest(p, (int)blockIdx.x * PROMOTE_WARPS + (int)warp - PROMOTE_WARP0,
              (int)gridDim.x * PROMOTE_WARPS, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(IO_REGS));
    if (warp == 0 && lane == 0)
      issued = producer_role(&tmA, &tmB, p, seg, base, rank, pair, npairs, b, abort_flag);
    if (warp == 1 && lane == 0 && rank == 0)
      mma_role(p, seg, base, tmem_base, pair, npairs, b, abort_flag);
    __syncwarp();
  }

  if (warp == 0 && lane == 0 && rank == 1)
    ptx::st_cluster_u32(ptx::map_to_cta(base + OFF_PEER_ISSUED, 0), issued);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs have stopped issuing
  if (warp == 0 && lane == 0 && rank == 0) {
    const uint32_t peer = *reinterpret_cast<volatile uint32_t*>(smem + OFF_PEER_ISSUED);
    leader_drain(b, issued, peer, p.timeout_ns);
  }
  ptx::cluster_sync();  // no copy into either CTA is still in flight
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace large
}  // namespace f8
}  // namespace gf16
