// 8-bit products with block scales: the kernel for many rows.
//
// A cluster of two CTAs (tcgen05 cta_group::2) computes tiles of 256 x 256:
// each CTA holds 128 rows of A and 128 columns of B (16 KB each per K block of
// 128, one swizzled copy each, K-major or MN-major), the even CTA issues four
// 256 x 256 x 32 MMAs per K block, and each block's products go to one half of
// tensor memory (256 of 512 columns) while eight promotion warps per CTA take
// the block before out of the other half and add it, scaled, to FP32
// registers: 128 sums a thread.
//
// What bounds it: an SM's tensor core takes 512 cycles for a K block (128 x
// 256 x 128 products at 8192 a cycle), its four FP32 pipes 256 for one fused
// multiply-add per product (scales per tile of B: sa * sb is one number for a
// thread's 128 columns) or 512 for two operations (a scale per column of B).
// Measured at 4864 x 4096 x 8192: 405 ns a block with a scale per tile (3.1
// PFLOP/s while blocks follow one another), 650 with one per column (2.0), 350
// (3.6) for the copies and the tensor core alone; the start and the end of a tile
// come on top, about 3 us.  MMAs of 128 columns, which would give tensor memory four slots
// and the promotion warps more time for each, took 600.
//
// DENSE: pairs walk the tiles in bands of eight tile rows.  The `rem` tiles of
// an incomplete wave, at most half as many as pairs, are cut into `parts`
// ranges of K blocks, so that no pair idles.  These come first: the pairs that
// had one are then out of step with the others, and the tiles' stores of some
// run beside the products of the others.  Each writes FP32 sums to the workspace,
// and a second kernel adds a tile's parts in their order and stores C (129 x 4096
// x 4096: 16.5 us; with the last warp to arrive adding them, 40).  BY_ROWS: tiles
// of 256 rows within an expert's segment, those of one column of tiles side by
// side.  BY_INNER: all tiles of each expert, with that expert's K blocks.
//
// Barriers (as in gemm_pair.cuh): full[s] leader only, 1 arrival and both
// CTAs' bytes; empty[s] both CTAs, multicast commit; tfull[a] both CTAs,
// multicast commit after a K block; tempty[a] leader only, 16 arrivals (8
// promotion warps per CTA); sfull[s], sempty[s] each CTA (COLS), 64 copying
// threads and 8 promotion warps; mma_done leader only.  Waits are bounded; after an
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
// Ring of scales (COLS): those of the CTA's 128 rows, then of the tile's 256
// columns, four K blocks at a time; eight words between the blocks' banks, so
// that the copies of a warp, eight rows by four blocks, do not collide.
constexpr int CHUNK = 4, CHUNKS = 3;
constexpr uint32_t SCALE_BLOCK = (CM + PN + 8) * 4, SCALE_CHUNK = CHUNK * SCALE_BLOCK;
constexpr int SCALE_WARP0 = 2, SCALE_THREADS = 64;

constexpr uint32_t OFF_A = 0;
constexpr uint32_t OFF_B = OFF_A + STAGES * A_STAGE;
constexpr uint32_t OFF_EPI = OFF_B + STAGES * B_STAGE;
constexpr uint32_t OFF_SCALE = OFF_EPI + PROMOTE_WARPS * EPI_BUF;
constexpr uint32_t OFF_SEG = OFF_SCALE + CHUNKS * SCALE_CHUNK;
constexpr uint32_t OFF_BAR = OFF_SEG + SEGMENT_BYTES;
constexpr uint32_t NUM_BARS = 2 * STAGES + 2 * CHUNKS + 2 + 2 + 1;
constexpr uint32_t OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr uint32_t OFF_PEER_ISSUED = OFF_ABORT + 4;
constexpr uint32_t SMEM_BYTES = OFF_PEER_ISSUED + 4 + 1024;
static_assert(SMEM_BYTES <= 232448, "over the 227 KB shared-memory limit per CTA");
static_assert(OFF_BAR % 8 == 0 && OFF_EPI % 128 == 0 && OFF_SCALE % 16 == 0, "alignment");

// Registers: 384 threads launch with 168 each (64,512); the four other warps
// give up 112 each and the promotion warps take 56 more (128 * 56 + 256 * 224).
constexpr int IO_REGS = 56, PROMOTE_REGS = 224;
static_assert(128 * IO_REGS + 256 * PROMOTE_REGS <= 384 * 168, "register split");

// FP32 numbers of a cut tile's part.
constexpr int PART_FLOATS = PM * PN;
constexpr int MAX_PARTS = 8;

struct Bars {
  uint32_t full, empty, tfull, tempty, sfull, sempty, mma_done;
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
    const int len = s.len[g.expert];
    g.nkb = (len + BLOCK - 1) / BLOCK;
    if (len < 0) g.m_end = 0;     // no rows to store: fill_rest's
    band_tile(u - g.expert * per, p.tiles_m, p.tiles_n, &tm, &tn);
  } else {
    int t = u - p.cut_units;
    if (t < 0) {
      g.tail = u / p.parts;
      g.part = u - g.tail * p.parts;
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

// A warp's 32 rows x 128 columns (acc: as in promote_role) to C through a staging
// buffer of 32 rows x 128 bytes, so that a store instruction writes four whole
// lines of 128 bytes and not 16 bytes of each of 32 rows.
template <typename T, bool COLS>
__device__ __forceinline__ void store_rows(const Params& p, T* C, const uint64_t (&acc)[64],
                                           uint32_t stage, int row0, int row_end, int col0,
                                           uint32_t lane) {
  constexpr int V = 16 / sizeof(T);        // numbers of a 16-byte unit
  constexpr int WIDE = 128 / sizeof(T);    // columns of a staging buffer
  constexpr int COLS_N = WIDE / 8;
#pragma unroll
  for (int c = 0; c < 128 / WIDE; ++c) {
    if (col0 + c * WIDE >= p.N) break;
    if constexpr (COLS) {
#pragma unroll
      for (int n = 0; n < COLS_N; ++n) {
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
          const uint32_t row = (lane >> 2) + 8 * q, col = 8 * n + 2 * (lane & 3u);
          const uint32_t byte = col * sizeof(T);
          const uint32_t at = stage + row * 128u + (((byte >> 4) ^ (row & 7u)) << 4) + (byte & 15u);
          const uint64_t v = acc[(c * COLS_N + n) * 4 + q];
          if constexpr (sizeof(T) == 4) {
            st_shared_b64(at, v);
          } else {
            float lo, hi;
            ptx::unpack_f2(v, lo, hi);
            st_shared_b32(at, pack2<T>(lo, hi));
          }
        }
      }
    } else {
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) {
        float v[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
          ptx::unpack_f2(acc[(c * WIDE + (int)j * V) / 2 + i], v[2 * i], v[2 * i + 1]);
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
    }
    __syncwarp();
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t r = i * 4 + (lane >> 3), j = lane & 7u;
      uint4 v = ld_shared_v4(stage + r * 128u + ((j ^ (r & 7u)) << 4));
      const int row = row0 + (int)r, col = col0 + c * WIDE + (int)j * V;
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

// This warp's piece of a cut tile's part to the workspace, as its lanes hold it:
// [part][rank][warp][32][lane], 16 bytes a lane.
__device__ __forceinline__ void store_part(const Params& p, const Unit& g, uint32_t rank, uint32_t w,
                                           uint32_t lane, const uint64_t (&acc)[64]) {
  ulonglong2* mine = reinterpret_cast<ulonglong2*>(p.ws) +
                     ((int64_t)g.tail * p.parts + g.part) * (PART_FLOATS / 4) +
                     (rank * PROMOTE_WARPS + w) * 32 * 32 + lane;
#pragma unroll
  for (int j = 0; j < 32; ++j) __stcg(mine + j * 32, make_ulonglong2(acc[2 * j], acc[2 * j + 1]));
}

// Columns of B lie in the ring in the order in which the promotion warps' lanes
// hold them (see promote_role).
__device__ __forceinline__ uint32_t column_at(uint32_t j) {
  return (j & ~15u) | ((j & 6u) << 1) | ((j & 8u) >> 2) | (j & 1u);
}

// `blocks` blocks' scales of OUTER rows (columns) of which `real` exist, by 64
// threads: four blocks of a row side by side where the inner dimension is
// contiguous, else rows side by side, so that a warp's copies share their
// sectors.  Those past `real` belong to results that are not stored.
template <int OUTER>
__device__ __forceinline__ void copy_scales(uint32_t dst, const float* src, int64_t s_outer,
                                            int64_t s_inner, int real, int blocks, uint32_t t) {
  if (s_inner == 1) {
    const uint32_t k = t % CHUNK, o = t / CHUNK;
    constexpr int STEP = SCALE_THREADS / CHUNK;
    if ((int)k >= blocks) return;
    dst += k * SCALE_BLOCK + (OUTER == PN ? column_at(o) : o) * 4u;
    src += k + o * s_outer;
#pragma unroll 8
    for (int i = 0; i < OUTER / STEP; ++i) {
      if ((int)o + i * STEP < real) ptx::cp_async_4(dst + i * STEP * 4u, src);
      src += STEP * s_outer;
    }
  } else {
    dst += (OUTER == PN ? column_at(t) : t) * 4u;
    src += t * s_outer;
#pragma unroll
    for (int i = 0; i < OUTER / SCALE_THREADS; ++i) {
      if ((int)t + i * SCALE_THREADS >= real) return;
      const float* at = src;
#pragma unroll
      for (int k = 0; k < CHUNK; ++k) {
        if (k < blocks) ptx::cp_async_4(dst + k * SCALE_BLOCK + i * SCALE_THREADS * 4u, at);
        at += s_inner;
      }
      src += SCALE_THREADS * s_outer;
    }
  }
}

// The scales of each K block into the ring, by asynchronous copies: the
// promotion warps read them blocks later, when they have long arrived.  (Loaded
// by those warps one block ahead, column scales were waited for: 890 ns a block
// where they lie side by side, 1,530 where they do not, and 587 without them.)
__device__ __forceinline__ void scale_role(const Params& p, const Segments& s, uint32_t base,
                                           uint32_t rank, int pair, int npairs, const Bars& b,
                                           uint32_t t, volatile int* abort_flag) {
  RingPos pos{0, 0};
  const int units = total_units(p, s);
  bool ok = true;
  for (int u = pair; u < units && ok; u += npairs) {
    const Unit g = unit_at(p, s, u);
    const int m0 = g.m0 + (int)rank * CM;
    const float* pa = p.sa + (p.sa_shift ? 0 : m0 * p.sa_outer) + g.blk0 * p.sa_inner;
    const float* pb = p.sb + g.n0 * p.sb_outer + g.blk0 * p.sb_inner +
                      (p.form == GEMM_F8_BY_ROWS ? g.expert * p.sb_batch : 0);
    for (int k = 0; k < g.nkb; k += CHUNK) {
      const uint32_t dst = base + OFF_SCALE + pos.stage * SCALE_CHUNK;
      if (!wait_phase(b.sempty + 8 * pos.stage, producer_wait_parity(pos), p, abort_flag)) {
        ok = false;
        break;
      }
      const int blocks = min(CHUNK, g.nkb - k);
      copy_scales<PN>(dst + CM * 4u, pb, p.sb_outer, p.sb_inner, p.N - g.n0, blocks, t);
      if (p.sa_shift == 0) {
        copy_scales<CM>(dst, pa, p.sa_outer, p.sa_inner, g.m_end - m0, blocks, t);
      } else {     // a scale for 128 rows of A
        for (int i = (int)t; i < CM; i += SCALE_THREADS)
          for (int j = 0; j < blocks && m0 + i < g.m_end; ++j)
            ptx::cp_async_4(dst + j * SCALE_BLOCK + i * 4u,
                            pa + ((m0 + i) >> p.sa_shift) * p.sa_outer + j * p.sa_inner);
      }
      ptx::cp_async_arrive(b.sfull + 8 * pos.stage);
      ring_advance(pos, CHUNKS);
      pa += CHUNK * p.sa_inner;
      pb += CHUNK * p.sb_inner;
    }
  }
  ptx::cp_async_wait_all();   // nothing in flight when the CTA exits
}

// COLS: B has a scale for each column (else one for a thread's 128 columns).
// Without, a lane holds one row and 128 columns; with, four rows (lane / 4 and
// every eighth after it) and 32 columns (2 (lane % 4) and the next, of every
// eight), so that it reads 32 column scales a block from shared memory, not
// 128, which the tensor core's operands and their copies need.
template <bool COLS>
__device__ __forceinline__ void promote_role(const Params& p, const Segments& s, uint32_t base,
                                             uint32_t tmem_base, uint32_t rank, int pair,
                                             int npairs, const Bars& b, uint32_t warp,
                                             uint32_t lane, volatile int* abort_flag) {
  const uint32_t w = warp - PROMOTE_WARP0, quarter = warp & 3u, right = w >> 2;
  const uint32_t stage = base + OFF_EPI + w * EPI_BUF;
  const uint32_t row_scale = base + OFF_SCALE + (quarter * 32u + (lane >> 2)) * 4u;
  const uint32_t col_scale = base + OFF_SCALE + (CM + right * 128u + (lane & 3u) * 4u) * 4u;
  const uint32_t t_row = tmem_base + ((quarter * 32u) << 16) + right * 128u;
  const uint32_t leader_tempty = ptx::map_to_cta(b.tempty, 0);
  uint32_t done = 0;    // K blocks so far: block i uses half i & 1
  RingPos pos{0, 0};    // chunk of scales
  const int units = total_units(p, s);
  // A unit's K blocks and, without COLS, its first scales.
  int nkb = 0;
  const float *pa = nullptr, *pb = nullptr;
  float na = 0.f, nb = 0.f;
  const auto begin = [&](int u) {
    const Unit g = unit_at(p, s, u);
    nkb = g.nkb;
    if (COLS || nkb == 0) return;
    const int row = min(g.m0 + (int)(rank * CM + quarter * 32 + lane), g.m_end - 1);
    const int col = min(g.n0 + (int)right * 128, p.N - 1);
    pa = p.sa + (int64_t)(row >> p.sa_shift) * p.sa_outer + (int64_t)g.blk0 * p.sa_inner;
    pb = p.sb + (int64_t)(col >> 7) * p.sb_outer + (int64_t)g.blk0 * p.sb_inner +
         (p.form == GEMM_F8_BY_ROWS ? g.expert * p.sb_batch : 0);
    na = *pa;
    nb = *pb;
  };
  if (pair < units) begin(pair);
  for (int u = pair; u < units; u += npairs) {
    uint64_t acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0;
    for (int i = 0; i < nkb; ++i, ++done) {
      const uint32_t half = done & 1u;
      const float sa = na, sb = nb;
      bool got = true;
      if constexpr (COLS) {
        if (i % CHUNK == 0)
          got = wait_phase_inline(b.sfull + 8 * pos.stage, consumer_wait_parity(pos), p, abort_flag);
      } else if (i + 1 < nkb) {     // the next block's scales, on their way during this one
        pa += p.sa_inner;
        na = *pa;
        pb += p.sb_inner;
        nb = *pb;
      }
      got = wait_phase_inline(b.tfull + 8 * half, (done >> 1) & 1u, p, abort_flag) && got;
      if (!__all_sync(0xffffffffu, got)) return;
      ptx::tc_fence_after();
      const uint32_t t = t_row + half * PN;
      // Loads of 2 x 32 columns on their way at a time: a load's latency is
      // waited for twice a block.
      const auto release = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_relaxed(leader_tempty + 8 * half);
      };
      if constexpr (COLS) {
        const uint32_t in_ring = pos.stage * SCALE_CHUNK + (i % CHUNK) * SCALE_BLOCK;
        const uint32_t cols = col_scale + in_ring;
        uint32_t lo[2][16], hi[2][16];     // rows 0-15 and 16-31
        const auto load = [&](int c) {
          ptx::tmem_ld_16x256b_x4(t + 32u * c, lo[c & 1]);
          ptx::tmem_ld_16x256b_x4(t + 32u * c + (16u << 16), hi[c & 1]);
        };
        load(0);
        load(1);
        uint4 ahead = ld_shared_v4(cols);     // each group's scales one group ahead
        uint64_t s4[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
          const float v = ld_shared_f32(row_scale + in_ring + 32u * q);
          s4[q] = ptx::pack_f2(v, v);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if ((c & 1) == 0) {
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              ptx::reg_fence(lo[k]);
              ptx::reg_fence(hi[k]);
            }
            if (c == 2) release();
          }
          const uint32_t(&xl)[16] = lo[c & 1], (&xh)[16] = hi[c & 1];
#pragma unroll
          for (int m = 0; m < 2; ++m) {     // two groups of eight columns
            const uint4 w4 = ahead;
            if (2 * c + m < 7) ahead = ld_shared_v4(cols + (2 * c + m + 1) * 64u);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint64_t q = n ? ptx::pack_f2(__uint_as_float(w4.z), __uint_as_float(w4.w))
                                   : ptx::pack_f2(__uint_as_float(w4.x), __uint_as_float(w4.y));
              uint64_t* a = acc + 16 * c + (2 * m + n) * 4;
              const int j = (2 * m + n) * 4;
              const auto add = [&](uint64_t& sum, uint32_t x0, uint32_t x1, uint64_t row) {
                const uint64_t x = ptx::pack_f2(__uint_as_float(x0), __uint_as_float(x1));
                sum = ptx::fma_f2(ptx::mul_f2(x, q), row, sum);
              };
              add(a[0], xl[j], xl[j + 1], s4[0]);
              add(a[1], xl[j + 2], xl[j + 3], s4[1]);
              add(a[2], xh[j], xh[j + 1], s4[2]);
              add(a[3], xh[j + 2], xh[j + 3], s4[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) asm volatile("" : "+l"(a[k]));
            }
          }
          if (c < 2) load(c + 2);
        }
        if (i % CHUNK == CHUNK - 1 || i == nkb - 1) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(b.sempty + 8 * pos.stage);
          ring_advance(pos, CHUNKS);
        }
      } else {
        // sa * sb is one number, unless it leaves FP32's normal range where the
        // product with the block's sum may not: then one after the other.
        const float sab = sa * sb;
        const bool split = __any_sync(0xffffffffu, !(fabsf(sab) >= 1.17549435e-38f &&
                                                      fabsf(sab) <= 3.4e38f));
        const uint64_t s1 = ptx::pack_f2(sab, sab);
        uint32_t r[2][32];
        ptx::tmem_ld_32x32b_x32(t, r[0]);
        ptx::tmem_ld_32x32b_x32(t + 32u, r[1]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if ((c & 1) == 0) {
            ptx::tmem_ld_wait();
            ptx::reg_fence(r[0]);
            ptx::reg_fence(r[1]);
            if (c == 2) release();
          }
          const uint32_t(&x)[32] = r[c & 1];
          if (!split) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              acc[16 * c + j] = ptx::fma_f2(
                  ptx::pack_f2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), s1,
                  acc[16 * c + j]);
          } else {
            const uint64_t sa2 = ptx::pack_f2(sa, sa), sb2 = ptx::pack_f2(sb, sb);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              acc[16 * c + j] = ptx::fma_f2(
                  ptx::mul_f2(
                      ptx::pack_f2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), sb2),
                  sa2, acc[16 * c + j]);
          }
          if (c < 2) ptx::tmem_ld_32x32b_x32(t + 64u + 32u * c, r[c]);
        }
      }
    }
    // The unit again, so that the loop's registers are the sums' alone.
    int same = u;
    asm volatile("" : "+r"(same));
    const Unit g = unit_at(p, s, same);
    if (u + npairs < units) begin(u + npairs);   // on their way during the stores
    const int row0 = g.m0 + (int)(rank * CM + quarter * 32), col0 = g.n0 + (int)right * 128;
    if (row0 >= g.m_end) continue;
    if (g.tail >= 0) {
      store_part(p, g, rank, w, lane, acc);
      continue;
    }
    const int64_t off = p.form == GEMM_F8_BY_INNER ? g.expert * p.c_batch : 0;
    if (p.type == GEMM_F8_F16)
      store_rows<__half, COLS>(p, static_cast<__half*>(p.C) + off, acc, stage, row0, g.m_end, col0, lane);
    else if (p.type == GEMM_F8_BF16)
      store_rows<__nv_bfloat16, COLS>(p, static_cast<__nv_bfloat16*>(p.C) + off, acc, stage, row0,
                                g.m_end, col0, lane);
    else
      store_rows<float, COLS>(p, static_cast<float*>(p.C) + off, acc, stage, row0, g.m_end, col0, lane);
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
  b.sfull = b.tempty + 16;
  b.sempty = b.sfull + 8 * CHUNKS;
  b.mma_done = b.sempty + 8 * CHUNKS;
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
    for (int s = 0; s < CHUNKS; ++s) {
      ptx::mbar_init(b.sfull + 8 * s, SCALE_THREADS);
      ptx::mbar_init(b.sempty + 8 * s, PROMOTE_WARPS);
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
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers exist before anyone signals them
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);
  // All of this beside the end of the kernel before; its results from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.form != GEMM_F8_DENSE) {
    load_segments(p, seg, PM, NUM_THREADS);
    __syncthreads();
  }

  uint32_t issued = 0;
  if (warp >= PROMOTE_WARP0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PROMOTE_REGS));
    promote_role<COLS>(p, seg, base, tmem_base, rank, pair, npairs, b, warp, lane, abort_flag);
    __syncwarp();
    fill_rest(p, seg, (int)blockIdx.x * PROMOTE_WARPS + (int)warp - PROMOTE_WARP0,
              (int)gridDim.x * PROMOTE_WARPS, lane);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(IO_REGS));
    if (warp == 0 && lane == 0)
      issued = producer_role(&tmA, &tmB, p, seg, base, rank, pair, npairs, b, abort_flag);
    if (warp == 1 && lane == 0 && rank == 0)
      mma_role(p, seg, base, tmem_base, pair, npairs, b, abort_flag);
    if (COLS && warp >= SCALE_WARP0)
      scale_role(p, seg, base, rank, pair, npairs, b, (warp - SCALE_WARP0) * 32 + lane,
                 abort_flag);
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

// The sums of cut tiles' parts, in their order, to C.  A CTA takes a warp's piece
// (32 rows x 128 columns) of a tile at a time; there are as many CTAs as pieces
// unless fewer SMs may be used.  Bound by latency and the cache: all parts' loads
// are on their way together.
constexpr int JOIN_THREADS = 256;

template <typename T>
__device__ __forceinline__ void store_joined(const Params& p, const float (&x)[32][132], int row0,
                                             int col0) {
  constexpr int V = 16 / sizeof(T), UNITS = 128 / V;
  T* C = static_cast<T*>(p.C);
#pragma unroll
  for (int i = 0; i < 32 * UNITS / JOIN_THREADS; ++i) {
    const int at = (int)threadIdx.x + i * JOIN_THREADS, r = at / UNITS, c = at % UNITS * V;
    const int row = row0 + r, col = col0 + c;
    if (row >= p.M || col >= p.N) continue;
    T* to = C + (int64_t)row * p.ldc + col;
    alignas(16) T y[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if constexpr (sizeof(T) == 4) y[k] = p.accumulate && col + k < p.N ? to[k] + x[r][c + k] : x[r][c + k];
      else y[k] = to_type<T>(x[r][c + k]);
    }
    if (p.vec && col + V <= p.N) {
      *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(y);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (col + k < p.N) to[k] = y[k];
    }
  }
}

template <bool COLS>
__global__ void __launch_bounds__(JOIN_THREADS) f8_join_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) float x[32][132];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int at_piece = (int)blockIdx.x; at_piece < p.join_pieces; at_piece += (int)gridDim.x) {
    const int tail = at_piece / (2 * PROMOTE_WARPS), piece = at_piece % (2 * PROMOTE_WARPS);
    const int rank = piece / PROMOTE_WARPS, w = piece % PROMOTE_WARPS;
    int tm, tn;
    band_tile(p.full_units + tail, p.tiles_m, p.tiles_n, &tm, &tn);
    const int row0 = tm * PM + rank * CM + (w & 3) * 32, col0 = tn * PN + (w >> 2) * 128;
    if (row0 >= p.M || col0 >= p.N) continue;      // the same in the whole CTA
    const float4* base = reinterpret_cast<const float4*>(p.ws) +
                         (int64_t)tail * p.parts * (PART_FLOATS / 4) + piece * 32 * 32;
#pragma unroll
    for (int u = 0; u < 1024 / JOIN_THREADS; ++u) {
      const int at = (int)threadIdx.x + u * JOIN_THREADS, j = at >> 5, lane = at & 31;
      float4 v[MAX_PARTS];
#pragma unroll
      for (int i = 0; i < MAX_PARTS; ++i)
        if (i < p.parts) v[i] = __ldcg(base + i * (PART_FLOATS / 4) + at);
      float4 sum = v[0];
#pragma unroll
      for (int i = 1; i < MAX_PARTS; ++i) {
        if (i < p.parts) {
          sum.x += v[i].x;
          sum.y += v[i].y;
          sum.z += v[i].z;
          sum.w += v[i].w;
        }
      }
      if constexpr (COLS) {      // two columns of two rows (see promote_role)
        const int r = (lane >> 2) + 16 * (j & 1), c = 8 * (j >> 1) + 2 * (lane & 3);
        *reinterpret_cast<float2*>(&x[r][c]) = make_float2(sum.x, sum.y);
        *reinterpret_cast<float2*>(&x[r + 8][c]) = make_float2(sum.z, sum.w);
      } else {
        *reinterpret_cast<float4*>(&x[lane][4 * j]) = sum;
      }
    }
    __syncthreads();
    if (p.type == GEMM_F8_F16) store_joined<__half>(p, x, row0, col0);
    else if (p.type == GEMM_F8_BF16) store_joined<__nv_bfloat16>(p, x, row0, col0);
    else store_joined<float>(p, x, row0, col0);
    __syncthreads();      // x is free again
  }
}

}  // namespace large
}  // namespace f8
}  // namespace gf16
