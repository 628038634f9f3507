// Attention over a paged cache for requests with few new tokens (token
// generation, drafted tokens): at most N rows (new tokens x the query heads
// of one key/value head) per request.
//
// Bound by reading the cache, so each key and value is read once for all N
// rows, and the products are turned around to fit: keys are the rows of the
// tensor core's operand A,
//   S^T = K Q^T    128 keys x N, K = 256   (A: key block as it lies, K-major)
//   O^T += V^T P^T  2 x 128 numbers x N    (A: value block as it lies, MN-major)
// so the copies feed the tensor core without a pass through registers, an MMA
// has no padding rows to read, and a softmax thread owns one key (its row of
// S^T) for all N queries: the work of a block is spread over 128 threads even
// for a single query.  128 keys x 512 bytes twice take ~2.9 us at an SM's
// share of the memory rate; the MMAs of a block take ~0.55 us.
//
// One CTA per SM; the step's key blocks are dealt out evenly (paged_schedule.h),
// whatever the lengths.  Warp 0 copies (lanes take the pages of a block side
// by side), one lane of warp 1 issues the MMAs, and each 16 rows of the tile
// have four softmax warps, one key per thread, that share nothing with the
// others (a thread that held all 64 rows of the widest tile spilled its
// registers and took 13 us for a block).  Per block the threads only agree on
// whether some score passed the exponent offset in use by more than
// OVER_LOG2 (one barrier with an OR); only then do they take the block's
// maximum, move the offset and rescale O.  Row sums stay one per thread and
// row until a tile ends.
//
// A tile that is cut between CTAs: each writes its unnormalised FP32 O with
// its offsets and sums, and a second kernel merges the parts in their order.
// (A merge by the last CTA to finish, found with a counter, took 5 to 17 us at
// the end of the kernel, where one CTA reads what all the others wrote; the
// second launch takes 3 and spreads the rows over the GPU.)
//
// Barriers: q_full / q_empty, full[s] / empty[s] (ring of 32 KB slots, 128 keys
// by 128 numbers each: a block's keys take two, then its values two), s_full[2],
// p_full[2], o_done[2] (the O products of a block).  Every wait is bounded;
// after an abort the roles stop issuing and the copies in flight are waited for.
#pragma once

namespace gf16 {
namespace paged {

constexpr int HD = 256;
// Weights are 2^(score - offset), in FP32 for the row sum and rounded to binary16
// for the product with V.  A new offset lies TAIL_LOG2 below the largest score
// and stays until a score passes it by OVER_LOG2, so the row's largest weight is
// 2^7 .. 2^15 (binary16 ends at 2^16) and a weight disappears from the product
// only below 2^-25 / 2^7 = 2^-32 of it.  (With the offset at the largest score
// the limit was 2^-25: a key that scores 2^25.5 times above 100,000 others took
// half to all of their 0.2 % from O.)
constexpr float TAIL_LOG2 = 7.f, OVER_LOG2 = 15.f;
constexpr float NO_OFFSET = -3.0e38f;   // offset of a row without a finite score

// The tile whose blocks go on past a worker's share, having begun in it: what
// the merge kernel needs (last < 0: there is none).
struct CutTile {
  int last;      // last worker with a part of it
  int first;     // slot of its first part; worker c's is 2c after that
  int token;     // row in O of its first token
  int tokens;
  int head;      // key/value head
  int pad[3];
};

// What the kernels get.
struct Params {
  int batch, total_q, max_q, q_heads, kv_heads, group;   // group: query heads per key/value head
  int num_pages, page_size, max_pages;
  int rows;                       // keys per copy group (paged_schedule.h)
  const int32_t *table, *starts, *kv_lens;
  int64_t table_stride;
  __half* O;
  int64_t o_tok, o_head;
  float scale_log2;
  Masks masks;
  int tile_tokens;                // tokens that a tile (small kernel: a request) can hold
  int skip_tokens;                // large kernel: requests with at most this many are not its own
  int zero_rows;                  // whether this launch writes the rows past the last request's
  float* part;                    // partial O, FP32, a slot's rows together
  float2* part_ml;                // their offsets and sums [slot][row]
  CutTile* cut;                   // [worker]
  int* status;
  unsigned long long timeout_ns;
  int fault_unit;                 // test only: CTA whose first ring fill gets no copy
};

__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, const Params& p,
                                          volatile int* abort_flag) {
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      *abort_flag = 1;
      *(volatile int*)p.status = (int)GEMM_F16_ERR_TIMEOUT;
      __threadfence_system();
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const Params& p,
                                           volatile int* abort_flag) {
  if (ptx::mbar_try_wait_poll(bar, parity)) return true;
  return wait_slow(bar, parity, p, abort_flag);
}

__device__ __forceinline__ Request load_request(const Params& p, int b) {
  return read_request(p.starts[b], p.starts[b + 1], p.kv_lens[b], p.total_q, p.max_q,
                      (int64_t)p.max_pages * p.page_size);
}

// Rows past the last request's are zero: all warps of the grid, a head each.
__device__ __forceinline__ void zero_tail(const Params& p, int worker, int workers) {
  const int lane = threadIdx.x & 31;
  const int64_t from = imin(imax(p.starts[p.batch], 0), p.total_q);
  const int64_t todo = (p.total_q - from) * p.q_heads;
  for (int64_t i = worker; i < todo; i += workers) {
    const int64_t t = from + i / p.q_heads, h = i % p.q_heads;
    *reinterpret_cast<uint4*>(p.O + t * p.o_tok + h * p.o_head + lane * 8) = make_uint4(0, 0, 0, 0);
  }
}

// Shared-memory matrix descriptors (common.cuh, smem_desc_sw128) as two words:
// within a tile only the address in the low word moves, by a constant per MMA.
// Built from scratch each time, 24 pairs of them were half of the MMA thread's
// time for a block.
constexpr uint32_t DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t low) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "r"(DESC_HIGH));
  return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// The page of key group `g` (of `rows` keys) of key block `blk` as the block
// table has it, or num_pages for a group that is not needed ...
__device__ __forceinline__ int group_page(const Params& p, const Span& s, int b, int blk, int g) {
  const int k0 = blk * BLOCK_KEYS + g * p.rows;
  if (!key_group(s, k0, p.rows, p.masks).need) return p.num_pages;
  return p.table[(int64_t)b * p.table_stride + k0 / p.page_size];
}
// ... and the page and row where the group's copy starts: past the last page,
// where it reads as zeros, if the group is not needed or the table's entry
// is out of range (reported).
__device__ __forceinline__ int2 group_source(const Params& p, const Span& s, int blk, int g,
                                             int page) {
  const int k0 = blk * BLOCK_KEYS + g * p.rows;
  const Group grp = key_group(s, k0, p.rows, p.masks);
  if (!grp.need) return make_int2(p.num_pages, 0);
  if (page < 0 || page >= p.num_pages) {
    *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
    return make_int2(p.num_pages, 0);
  }
  return make_int2(page, k0 % p.page_size - grp.shift);
}

// 3-D tiled load global -> shared, crediting `bar` with the box bytes.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint32_t bar, int32_t x,
                                            int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

namespace small {

constexpr int WIN = 192;                // requests kept in shared memory
constexpr int COLS = 16;                // rows of the tile (columns of S^T) per softmax group
constexpr uint32_t CHUNK = 128 * 128;   // 128 keys x 64 numbers: 16 KB
constexpr uint32_t SLOT = 2 * CHUNK;

template <int N>
struct Cfg {
  static constexpr int GROUPS = N / COLS;                 // softmax groups of four warps
  static constexpr int THREADS = 64 + 128 * GROUPS;
  static constexpr int WARPS = THREADS / 32;
  static constexpr int RING = N == 16 ? 6 : (N == 32 ? 5 : 4);
  static constexpr uint32_t Q_CHUNK = N * 128;
  static constexpr uint32_t Q_BYTES = 4 * Q_CHUNK;
  static constexpr uint32_t P_CHUNK = N * 128;            // 64 keys
  static constexpr uint32_t P_BYTES = 2 * P_CHUNK;
  static constexpr uint32_t OFF_RING = 0;
  static constexpr uint32_t OFF_Q = OFF_RING + RING * SLOT;
  static constexpr uint32_t OFF_P = OFF_Q + Q_BYTES;
  static constexpr uint32_t OFF_RED = OFF_P + 2 * P_BYTES;          // [4][N] floats
  static constexpr uint32_t OFF_REQ = OFF_RED + 4 * N * 4;          // WIN x (start, n, len)
  static constexpr uint32_t OFF_SCHED = OFF_REQ + WIN * 12;         // see Sched
  static constexpr uint32_t OFF_BAR = (OFF_SCHED + 64 + 7) / 8 * 8;
  static constexpr uint32_t NUM_BARS = 2 + 2 * RING + 6 + 1;
  static constexpr uint32_t OFF_TMEM = OFF_BAR + NUM_BARS * 8;
  static constexpr uint32_t SMEM = OFF_TMEM + 16 + 1024;
  static_assert(SMEM <= 232448, "over the 227 KB shared-memory limit per CTA");
  // Tensor memory: two S buffers, then O (two halves of 128 numbers).
  static constexpr uint32_t S_COL = 0, O_COL = 2 * N;
  static constexpr uint32_t TMEM_COLS = N == 64 ? 256 : (N == 32 ? 128 : 64);
  // kind::f16, FP32 accumulate, M = 128: S^T with both operands K-major;
  // O^T with A (V^T) MN-major (bit 15) and B (P) K-major.
  static constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
  static constexpr uint32_t IDESC_O = IDESC_S | (1u << 15);
};

struct Sched {
  long long w0, w1, per;    // this CTA's blocks on the line, blocks per CTA
  int b, head, j;           // where w0 lies
  int base;                 // first request in shared memory
};

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[COLS]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  ptx::tmem_ld_wait();
  ptx::reg_fence(r);
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[COLS]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Barrier of the 128 threads of a softmax group (named barrier 1 + group);
// the first returns the OR of `pred`.
__device__ __forceinline__ bool group_or(int grp, bool pred) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)pred), "r"(1 + grp)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int grp) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + grp) : "memory");
}

// Warp maximum of floats (no NaN needed): as ordered integers.
__device__ __forceinline__ float warp_max(float x) {
  int i = __float_as_int(x);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(0xffffffffu, i);
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// A request of this kernel: some new tokens, no more rows than N.
__device__ __forceinline__ bool own_request(const Params& p, const Request& r) {
  return r.n > 0 && r.n <= p.tile_tokens;
}
__device__ __forceinline__ int request_blocks(const Params& p, const Request& r) {
  return own_request(p, r) ? tile_span(r, 0, r.n - 1, p.masks).nb : 0;
}

// A walk over this CTA's share of the line, tile by tile; every role runs
// its own.
struct Walk {
  const Params& p;
  const int* req;           // WIN x 3 in shared memory
  long long w, w1;
  int b, head, j, base;
  Request r;
  Span s;
  int j0, j1;               // blocks of the current tile that are this CTA's
  __device__ __forceinline__ Walk(const Params& p_, const Sched& sc, const int* req_)
      : p(p_), req(req_), w(sc.w0), w1(sc.w1), b(sc.b), head(sc.head), j(sc.j), base(sc.base) {
    if (w < w1) fetch();
  }
  __device__ __forceinline__ void fetch() {
    const int k = b - base;
    if (k < WIN) {
      r.start = req[3 * k];
      r.n = req[3 * k + 1];
      r.len = req[3 * k + 2];
    } else {
      r = load_request(p, b);
    }
    if (own_request(p, r)) s = tile_span(r, 0, r.n - 1, p.masks);
  }
  // The next tile, or false.
  __device__ __forceinline__ bool next() {
    if (w >= w1) return false;
    if (head == p.kv_heads) {
      head = 0;
      do {
        ++b;
        fetch();
      } while (!own_request(p, r));
    }
    j0 = j;
    j1 = (int)lmin(s.nb, (long long)j0 + (w1 - w));
    w += j1 - j0;
    j = 0;
    ++head;                 // the current tile's head is head - 1
    return true;
  }
  __device__ __forceinline__ long long line() const { return w - j1; }   // of the tile's block 0
};

template <int N>
__device__ __forceinline__ void schedule(const Params& p, uint8_t* smem, int cta, int ctas) {
  using C = Cfg<N>;
  int* req = reinterpret_cast<int*>(smem + C::OFF_REQ);
  Sched* sc = reinterpret_cast<Sched*>(smem + C::OFF_SCHED);
  __shared__ long long warp_sum[C::WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // First pass: all blocks of the step.  The second finds the request that
  // holds the CTA's first block; a step of up to WIN requests needs one.
  const bool one = p.batch <= WIN;
  long long total = 0;
  if (!one) {
    long long sum = 0;
    for (int b = tid; b < p.batch; b += C::THREADS) {
      const Request r = load_request(p, b);
      if (r.bad) *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
      sum += (long long)request_blocks(p, r) * p.kv_heads;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    for (int k = 0; k < C::WARPS; ++k) total += warp_sum[k];
    __syncthreads();
  }
  if (tid == 0) {
    sc->w0 = sc->w1 = 0;
    sc->per = 1;
  }
  long long before = 0;
  for (int b0 = 0; b0 < p.batch; b0 += WIN) {
    const int b = b0 + tid;
    Request r{0, 0, 0, false};
    if (tid < WIN) {
      if (b < p.batch) r = load_request(p, b);
      if (one && r.bad) *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
      req[3 * tid] = r.start;
      req[3 * tid + 1] = r.n;
      req[3 * tid + 2] = r.len;
    }
    const int nb = request_blocks(p, r);
    const long long mine = (long long)nb * p.kv_heads;
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    long long all = 0, base = before;
    for (int k = 0; k < C::WARPS; ++k) {
      if (k < warp) base += warp_sum[k];
      all += warp_sum[k];
    }
    inc += base;
    if (one) total = all;
    const long long per = per_worker(total, ctas), w0 = per * cta;
    const bool found = w0 < total && w0 < before + all;
    if (mine > 0 && w0 >= inc - mine && w0 < inc) {
      const long long at = w0 - (inc - mine);
      sc->per = per;
      sc->w0 = w0;
      sc->w1 = lmin(w0 + per, total);
      sc->b = b;
      sc->head = (int)(at / nb);
      sc->j = (int)(at % nb);
      sc->base = b0;
    }
    before += all;
    __syncthreads();
    if (found || w0 >= total) break;   // the same for all threads
  }
}

template <int N>
__global__ void __launch_bounds__(Cfg<N>::THREADS, 1)
    paged_small_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Cfg<N>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const uint32_t lane = threadIdx.x & 31u;
  const int cta = (int)blockIdx.x, ctas = (int)gridDim.x;

  const uint32_t q_full = base + C::OFF_BAR, q_empty = q_full + 8, full = q_empty + 8,
                 empty = full + 8 * C::RING, s_full = empty + 8 * C::RING, p_full = s_full + 16,
                 o_done = p_full + 16, mma_done = o_done + 16;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_TMEM + 4);

  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(q_empty, 1);
    for (int s = 0; s < C::RING; ++s) {
      ptx::mbar_init(full + 8 * s, 1);
      ptx::mbar_init(empty + 8 * s, 1);
    }
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(s_full + 8 * k, 1);
      ptx::mbar_init(p_full + 8 * k, 4 * C::GROUPS);
      ptx::mbar_init(o_done + 8 * k, 1);
    }
    ptx::mbar_init(mma_done, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(base + C::OFF_TMEM, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  // Rows of Q that no copy fills must be numbers (their results are dropped).
  for (uint32_t i = threadIdx.x; i < C::Q_BYTES / 16; i += C::THREADS)
    ptx::st_shared_v4(base + C::OFF_Q + 16 * i, 0, 0, 0, 0);
  ptx::fence_proxy_async_smem();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  schedule<N>(p, smem, cta, ctas);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TMEM);
  const Sched sc = *reinterpret_cast<const Sched*>(smem + C::OFF_SCHED);
  Walk walk(p, sc, reinterpret_cast<const int*>(smem + C::OFF_REQ));

  uint32_t fills = 0, qloads = 0;
  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    RingPos pos{0, 0};
    bool ok = true;
    const int groups = BLOCK_KEYS / p.rows;
    const uint32_t q_bytes = 4u * 128u * (uint32_t)(p.tile_tokens * p.group);
    while (ok && walk.next()) {
      const int head = walk.head - 1;
      if (qloads > 0)
        ok = __all_sync(0xffffffffu, wait_phase(q_empty, (qloads - 1) & 1u, p, abort_flag));
      if (!ok) break;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx_relaxed(q_full, q_bytes);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tma_load_3d(base + C::OFF_Q + c * C::Q_CHUNK, &tmQ, q_full, 64 * c, head * p.group,
                      walk.r.start);
      }
      ++qloads;
      // One slot: 128 keys by 128 numbers, as 64-number chunks of page groups.
      auto fill = [&](const CUtensorMap* tm, int2 src, int half) -> bool {
        if (!__all_sync(0xffffffffu, wait_phase(empty + 8 * pos.stage, producer_wait_parity(pos),
                                                p, abort_flag)))
          return false;
        const uint32_t fb = full + 8 * pos.stage;
        if (lane == 0) ptx::mbar_arrive_expect_tx_relaxed(fb, SLOT);
        __syncwarp();
        // Lane l copies chunk l / 16 of group l % 16.
        const int g = (int)lane & 15, c = (int)lane >> 4;
        if (g < groups && !(fills == 0 && cta == p.fault_unit))
          ptx::tma_load_4d(base + C::OFF_RING + pos.stage * SLOT + c * CHUNK +
                               (uint32_t)(g * p.rows) * 128u,
                           tm, fb, 128 * half + 64 * c, src.y, head, src.x);
        ++fills;
        ring_advance(pos, C::RING);
        return true;
      };
      // Table entries are loaded a block before they are used.
      const int g = imin((int)lane & 15, groups - 1);
      auto page_of = [&](int j) {
        return j < walk.j1 ? group_page(p, walk.s, walk.b, span_block(walk.s, j), g) : 0;
      };
      auto source = [&](int j, int page) {
        return group_source(p, walk.s, span_block(walk.s, j), g, page);
      };
      int page0 = page_of(walk.j0), page1 = page_of(walk.j0 + 1);
      int2 src = source(walk.j0, page0), nxt = src;
      ok = fill(&tmK, src, 0) && fill(&tmK, src, 1);
      for (int j = walk.j0; ok && j < walk.j1; ++j) {
        const int page2 = page_of(j + 2);
        if (j + 1 < walk.j1) {
          nxt = source(j + 1, page1);
          ok = fill(&tmK, nxt, 0) && fill(&tmK, nxt, 1);
        }
        ok = ok && fill(&tmV, src, 0) && fill(&tmV, src, 1);
        src = nxt;
        page1 = page2;
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    if (lane == 0) {
      RingPos pos{0, 0};
      bool ok = true;
      uint32_t g0 = 0, tiles = 0;     // blocks and tiles done
      const uint32_t ring_low = desc_low(base + C::OFF_RING, 0);
      while (ok && walk.next()) {
        const uint32_t nb = (uint32_t)(walk.j1 - walk.j0);
        ok = wait_phase(q_full, tiles & 1u, p, abort_flag);
        auto issue_s = [&](uint32_t gs, bool last) -> bool {
          for (int half = 0; half < 2; ++half) {
            if (!wait_phase(full + 8 * pos.stage, consumer_wait_parity(pos), p, abort_flag))
              return false;
            ptx::tc_fence_after();
            const uint32_t k_low = ring_low + pos.stage * (SLOT >> 4) + (1u << 16);   // LBO 16
            const uint32_t q_low =
                desc_low(base + C::OFF_Q + (uint32_t)half * 2u * C::Q_CHUNK, 16);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              ptx::mma_f16(tmem + C::S_COL + (gs & 1u) * N,
                           desc(k_low + ((kk >> 2) * CHUNK + (kk & 3) * 32u) / 16),
                           desc(q_low + ((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32u) / 16),
                           C::IDESC_S, (half > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(empty + 8 * pos.stage);
            ring_advance(pos, C::RING);
          }
          ptx::mma_commit(s_full + 8 * (gs & 1u));
          if (last) ptx::mma_commit(q_empty);
          return true;
        };
        ok = ok && issue_s(g0, nb == 1);
        for (uint32_t j = 0; ok && j < nb; ++j) {
          const uint32_t gj = g0 + j, pb = gj & 1u;
          if (j + 1 < nb && !(ok = issue_s(gj + 1, j + 2 == nb))) break;
          ok = wait_phase(p_full + 8 * pb, (gj >> 1) & 1u, p, abort_flag);
          for (int half = 0; ok && half < 2; ++half) {
            ok = wait_phase(full + 8 * pos.stage, consumer_wait_parity(pos), p, abort_flag);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t v_low = ring_low + pos.stage * (SLOT >> 4) + ((CHUNK >> 4) << 16);
            const uint32_t p_low = desc_low(base + C::OFF_P + pb * C::P_BYTES, 16);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)   // 16 keys each
              ptx::mma_f16(tmem + C::O_COL + (uint32_t)half * N,
                           desc(v_low + (uint32_t)kk * 128u),
                           desc(p_low + ((kk >> 2) * C::P_CHUNK + (kk & 3) * 32u) / 16),
                           C::IDESC_O, (j > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(empty + 8 * pos.stage);
            ring_advance(pos, C::RING);
          }
          if (ok) ptx::mma_commit(o_done + 8 * pb);
        }
        g0 += nb;
        ++tiles;
      }
      // Every MMA issued must be finished before the memory is given back.
      ptx::mma_commit(mma_done);
      wait_drain(mma_done, 0, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax
    // Group grp works on rows col0 .. col0 + 15 of the tile; its threads'
    // keys are rows of S^T.
    const uint32_t quarter = warp & 3u;
    const int grp = (int)(warp - 2) >> 2, col0 = grp * COLS;
    const uint32_t t_lane = ((quarter * 32u) << 16) + (uint32_t)col0;
    const int key_row = (int)(quarter * 32u + lane);
    float* red = reinterpret_cast<float*>(smem + C::OFF_RED) + 4 * col0;    // [4][COLS]
    const uint32_t p_off = base + C::OFF_P + (uint32_t)(key_row >> 6) * C::P_CHUNK +
                           (uint32_t)col0 * 128u + (uint32_t)(key_row & 7) * 2u;
    const uint32_t p_col = (uint32_t)(key_row & 63) >> 3;   // 16-byte column, swizzled by row
    const float sl2 = p.scale_log2;
    if (p.zero_rows)
      zero_tail(p, cta * 4 * C::GROUPS + (int)warp - 2, ctas * 4 * C::GROUPS);
    if (warp == 2 && lane == 0) p.cut[cta].last = -1;
    uint32_t g = 0;
    bool ok = true;
    while (walk.next()) {
      const int head = walk.head - 1;
      const int rows = imin(imax(walk.r.n * p.group - col0, 0), COLS);   // of this group
      const int pos0 = walk.r.len - walk.r.n;               // position of the first new token
      float m[COLS], l[COLS];
#pragma unroll
      for (int n = 0; n < COLS; ++n) {
        m[n] = NO_OFFSET;
        l[n] = 0.f;
      }
      for (int j = walk.j0; j < walk.j1; ++j, ++g) {
        const uint32_t sb = g & 1u;
        const int blk = span_block(walk.s, j);
        const bool full_block = block_is_full(pos0, pos0 + walk.r.n - 1, blk, p.masks);
        int lo = 0, hi = N;
        if (!full_block)
          rows_that_see(walk.s, blk, key_row, p.rows, pos0, p.group, p.masks, N, &lo, &hi);
        lo -= col0;
        hi -= col0;
        const bool got = wait_phase(s_full + 8 * sb, (g >> 1) & 1u, p, abort_flag);
        // The four warps go on or stop together: the barriers below need all.
        if (group_or(grp, !(ok && got))) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (rows > 0) {
          uint32_t s[COLS];
          tmem_ld(tmem + t_lane + C::S_COL + sb * N, s);
          bool over = false;
#pragma unroll
          for (int n = 0; n < COLS; ++n) {
            float x = __uint_as_float(s[n]) * sl2;
            if (!full_block) x = (n >= lo && n < hi) ? x : -INFINITY;
            s[n] = __float_as_uint(x);
            over |= x > m[n] + OVER_LOG2;
          }
          // P buffer sb was last read by the O products of block g - 2.
          if (g >= 2 && !__all_sync(0xffffffffu, wait_phase(o_done + 8 * sb, ((g - 2) >> 1) & 1u, p,
                                                           abort_flag)))
            ok = false;
          if (group_or(grp, over)) {
#pragma unroll
            for (int n = 0; n < COLS; ++n) {
              const float wm = warp_max(__uint_as_float(s[n]));
              if (lane == 0) red[quarter * COLS + n] = wm;
            }
            group_sync(grp);
            if (j > walk.j0 &&
                !__all_sync(0xffffffffu, wait_phase(o_done + 8 * ((g - 1) & 1u),
                                                    ((g - 1) >> 1) & 1u, p, abort_flag)))
              ok = false;
            ptx::tc_fence_after();
            float alpha[COLS];
#pragma unroll
            for (int n = 0; n < COLS; ++n) {
              const float mx = fmaxf(fmaxf(red[n], red[COLS + n]),
                                     fmaxf(red[2 * COLS + n], red[3 * COLS + n]));
              const float mn = mx > m[n] + OVER_LOG2 ? mx - TAIL_LOG2 : m[n];
              alpha[n] = ptx::ex2_approx(m[n] - mn);
              l[n] *= alpha[n];
              m[n] = mn;
            }
            if (j > walk.j0) {
#pragma unroll 1
              for (int half = 0; half < 2; ++half) {
                uint32_t o[COLS];
                const uint32_t ta = tmem + t_lane + C::O_COL + (uint32_t)half * N;
                tmem_ld(ta, o);
#pragma unroll
                for (int n = 0; n < COLS; ++n)
                  o[n] = __float_as_uint(__uint_as_float(o[n]) * alpha[n]);
                tmem_st(ta, o);
              }
              ptx::tmem_st_wait();
            }
            group_sync(grp);   // `red` is read
          }
          const uint32_t p_buf = p_off + sb * C::P_BYTES;
#pragma unroll
          for (int n = 0; n < COLS; ++n) {
            const float w = ptx::ex2_approx(__uint_as_float(s[n]) - m[n]);
            l[n] += w;
            // The product with V takes binary16 weights: half a step each, 2^-11 of
            // the weight or 2^-25 below the normal range (see TAIL_LOG2).
            const unsigned short h = __half_as_ushort(__float2half_rn(w));
            asm volatile(
                "st.shared.u16 [%0], %1;" ::"r"(p_buf + n * 128u + ((p_col ^ (n & 7)) << 4)), "h"(h)
                : "memory");
          }
          ptx::fence_proxy_async_smem();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full + 8 * sb);
      }
      // The tile ends: sums over the 128 keys' threads, then O.
      if (group_or(grp, !ok)) ok = false;
      if (rows > 0) {
#pragma unroll
        for (int n = 0; n < COLS; ++n) {
          float v = l[n];
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
          if (lane == 0) red[quarter * COLS + n] = v;
        }
        group_sync(grp);
#pragma unroll
        for (int n = 0; n < COLS; ++n)
          l[n] = (red[n] + red[COLS + n]) + (red[2 * COLS + n] + red[3 * COLS + n]);
      }
      if (ok && !__all_sync(0xffffffffu, wait_phase(o_done + 8 * ((g - 1) & 1u),
                                                    ((g - 1) >> 1) & 1u, p, abort_flag)))
        ok = false;
      group_sync(grp);       // `red` is read
      const bool whole = walk.j0 == 0 && walk.j1 == walk.s.nb;
      const long long L = walk.line();
      const int slot = part_slot(L, sc.per, cta);
      if (ok && rows > 0) {
        ptx::tc_fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t o[COLS];
          tmem_ld(tmem + t_lane + C::O_COL + (uint32_t)half * N, o);
          const int d = half * 128 + key_row;
          if (whole) {
            int tok = col0 / p.group, in_group = col0 - tok * p.group;
            __half* dst = p.O + (int64_t)(walk.r.start + tok) * p.o_tok +
                          (int64_t)(head * p.group + in_group) * p.o_head + d;
#pragma unroll
            for (int n = 0; n < COLS; ++n) {
              if (n < rows) {
                const float inv = l[n] > 0.f ? 1.f / l[n] : 0.f;
                *dst = __float2half_rn(__uint_as_float(o[n]) * inv);
                dst += p.o_head;
                if (++in_group == p.group) {
                  in_group = 0;
                  dst += p.o_tok - (int64_t)p.group * p.o_head;
                }
              }
            }
          } else {
            float* dst = p.part + ((int64_t)slot * N + col0) * HD + d;
#pragma unroll
            for (int n = 0; n < COLS; ++n)
              if (n < rows) __stcg(dst + n * HD, __uint_as_float(o[n]));
          }
        }
        if (!whole && key_row == 0) {
#pragma unroll
          for (int n = 0; n < COLS; ++n)
            if (n < rows)
              __stcg(p.part_ml + (int64_t)slot * N + col0 + n, make_float2(m[n], l[n]));
        }
      }
      if (ok && warp == 2 && lane == 0 && L >= sc.w0 && walk.j1 < walk.s.nb) {
        CutTile t = {};
        t.last = (int)((L + walk.s.nb - 1) / sc.per);
        t.first = slot;
        t.token = walk.r.start;
        t.tokens = walk.r.n;
        t.head = head;
        p.cut[cta] = t;
      }
      // The next tile's first O product overwrites O; it follows this
      // thread's next arrival on p_full.
      ptx::tc_fence_before();
    }
  }

  // After an abort the copies issued must have landed before the shared
  // memory is given back (otherwise their data has been waited for).
  __syncthreads();
  if (*abort_flag && warp == 0 && lane == 0) {
    for (uint32_t f = fills > (uint32_t)C::RING ? fills - C::RING : 0; f < fills; ++f)
      wait_drain(full + 8 * (f % C::RING), (f / C::RING) & 1u, p.timeout_ns);
    if (qloads > 0) wait_drain(q_full, (qloads - 1) & 1u, p.timeout_ns);
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Merges the cut tiles: block (w, y) rows ROWS * y .. ROWS * y + ROWS - 1 of
// the tile that worker w began and others ended.  16 / ROWS warps per row share
// its parts; a lane has eight numbers.  Launched behind the kernel above, whose
// end it waits for.
constexpr int MERGE_WARPS = 16, MERGE_THREADS = 32 * MERGE_WARPS;
// Rows of a block.  Where a tile has few parts, four warps a row are enough and
// fewer blocks are better (40 drafts under a window: 45.4 us; 49.0 with two
// rows a block).  With fewer than a tile for every four workers the parts are
// many, and the time is the reading of them by few SMs (one token over 100,000
// keys of one head: 38.3 -> 34.7 us with two rows, 4 x 20,000 keys 26.2 -> 25.0).
constexpr int merge_rows(int64_t tiles, int workers) { return tiles * 4 <= workers ? 2 : 4; }

template <int N, int ROWS>
__global__ void __launch_bounds__(MERGE_THREADS) paged_small_merge_kernel(const Params p) {
  constexpr int SHARE = MERGE_WARPS / ROWS;
  __shared__ float part_sum[SHARE][ROWS][32][9];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = (int)blockIdx.x, lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  const int in = warp % ROWS, share = warp / ROWS;
  const int n = (int)blockIdx.y * ROWS + in;       // row of the tile
  const CutTile t = p.cut[w];
  const int rows = t.tokens * p.group;
  if (t.last < 0 || (int)blockIdx.y * ROWS >= rows) return;   // all of the block
  auto slot = [&](int c) { return (int64_t)(c == w ? t.first : 2 * c); };
  float acc[8] = {}, sum = 0.f;
  if (n < rows) {
    float mx = NO_OFFSET;
    for (int c = w + lane; c <= t.last; c += 32)
      mx = fmaxf(mx, __ldcg(p.part_ml + slot(c) * N + n).x);
    mx = warp_max(mx);
#pragma unroll 4
    for (int c = w + share; c <= t.last; c += SHARE) {
      const float2 ml = __ldcg(p.part_ml + slot(c) * N + n);
      const float4* src = reinterpret_cast<const float4*>(p.part + (slot(c) * N + n) * HD) + lane * 2;
      const float4 a = __ldcg(src), b = __ldcg(src + 1);
      const float wgt = ptx::ex2_approx(ml.x - mx);
      sum = fmaf(wgt, ml.y, sum);
      acc[0] = fmaf(wgt, a.x, acc[0]);
      acc[1] = fmaf(wgt, a.y, acc[1]);
      acc[2] = fmaf(wgt, a.z, acc[2]);
      acc[3] = fmaf(wgt, a.w, acc[3]);
      acc[4] = fmaf(wgt, b.x, acc[4]);
      acc[5] = fmaf(wgt, b.y, acc[5]);
      acc[6] = fmaf(wgt, b.z, acc[6]);
      acc[7] = fmaf(wgt, b.w, acc[7]);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) part_sum[share][in][lane][k] = acc[k];
  part_sum[share][in][lane][8] = sum;
  __syncthreads();
  if (share != 0 || n >= rows) return;
#pragma unroll
  for (int o = 1; o < SHARE; ++o) {
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] += part_sum[o][in][lane][k];
    sum += part_sum[o][in][lane][8];
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int tok = n / p.group;
  uint4 out;
  out.x = pack_half2(acc[0] * inv, acc[1] * inv);
  out.y = pack_half2(acc[2] * inv, acc[3] * inv);
  out.z = pack_half2(acc[4] * inv, acc[5] * inv);
  out.w = pack_half2(acc[6] * inv, acc[7] * inv);
  *(reinterpret_cast<uint4*>(p.O + (int64_t)(t.token + tok) * p.o_tok +
                             (int64_t)(t.head * p.group + n - tok * p.group) * p.o_head) + lane) =
      out;
}

}  // namespace small
}  // namespace paged
}  // namespace gf16
