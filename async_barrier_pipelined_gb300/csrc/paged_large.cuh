// Attention over a paged cache for requests with many new tokens (prompts and
// chunks of them): tiles of up to 256 rows, a row being one new token's query
// under one of the query heads that share a key/value head.
//
// Bound by the tensor cores.  The same CTA pair as the dense attention kernel
// (attn_pair.cuh): S = Q K^T and O += P V as 256-row MMAs over two SMs, P and O
// in tensor memory, the softmax of a block beside the products of its
// neighbours, O written while the next tile runs.  What is different:
//   rows     CTA r holds tokens T*r .. T*(r+1) - 1 of the tile, T = 128 / group,
//            times the `group` query heads: a tile reads each key once for
//            all of them, and Q lands in row order by one 3-D copy per chunk.
//   keys     come page by page: lane l of the copy warp takes one group of
//            rows (at most 64) of one 64-number chunk; the pages of the next
//            block are looked up a block ahead.  Groups that no query of the
//            tile sees, and rows past its last key, read as zeros without
//            touching memory (paged_schedule.h).
//   masks    only in blocks that the causal edge, the window's edge or the
//            sinks cut; there each softmax thread builds the 128 bits of the
//            keys that its row sees.
//   dealing  the pairs get equal shares of the step's key blocks, whatever
//            the lengths (causal tiles differ in cost); a tile that is cut
//            leaves FP32 partials that a second kernel merges.  Where there are
//            many long tiles, whole ones are dealt out in turn first (`Deal`).
// Barriers and signals are those of attn_pair.cuh.
#pragma once

namespace gf16 {
namespace paged {
namespace large {

constexpr int CQ = 128;                 // rows per CTA
constexpr int BKV = BLOCK_KEYS;
constexpr int MAX_ROWS = 64;            // most keys per copy group (a CTA's half of a key block)
constexpr int RING = 2;                 // key tiles, and value tiles, in flight
constexpr int SLOTS = 2 * RING;         // keys in slots 0 .. RING - 1, values in the others
constexpr int SM_WARPS = 4;             // softmax warps 0..3
constexpr int EP_WARPS = 4;             // epilogue warps 4..7
constexpr int COPY_K_WARP = 8, COPY_V_WARP = 9, MMA_WARP = 10;
constexpr int NUM_THREADS = 384;        // three warpgroups (the last warp is idle)
// Registers per thread: 168 at launch, then more for the softmax, whose
// threads hold a row of 128 scores, and the epilogue (64 numbers of O and of a
// part), less for copies and MMAs.
constexpr int SM_REGS = 208, EP_REGS = 176, IO_REGS = 120;
static_assert(SM_REGS + EP_REGS + IO_REGS <= 3 * 168, "the launch's registers");
constexpr int NUM_WARPS = NUM_THREADS / 32;
constexpr int WIN = 320;                // requests kept in shared memory

constexpr uint32_t CHUNK_Q = CQ * 128;
constexpr uint32_t Q_BYTES = 4 * CHUNK_Q;
constexpr uint32_t K_CHUNK = (BKV / 2) * 128;
constexpr uint32_t V_CHUNK = BKV * 128;
constexpr uint32_t SLOT_BYTES = 32768;
constexpr uint32_t BOX = 32 * 128;      // 32 rows by 128 bytes of O
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_RING = OFF_Q + Q_BYTES;
constexpr uint32_t OFF_STAGE = OFF_RING + SLOTS * SLOT_BYTES;  // one box per epilogue warp
constexpr uint32_t OFF_L = OFF_STAGE + EP_WARPS * BOX;         // row sums and offsets
constexpr uint32_t OFF_REQ = OFF_L + 2 * CQ * 4;               // WIN x (start, n, len, blocks)
constexpr uint32_t OFF_SCHED = OFF_REQ + WIN * 16;
constexpr int MAX_CLUSTERS = 128;
constexpr uint32_t DEAL_BYTES = 4 * (MAX_CLUSTERS + 1 + MAX_CLUSTERS + WIN + 1);
constexpr uint32_t OFF_DEAL = OFF_SCHED + 64;
constexpr uint32_t OFF_BAR = (OFF_DEAL + DEAL_BYTES + 7) / 8 * 8;
constexpr uint32_t NUM_BARS = 2 + 2 * SLOTS + 2 + 2 + 2 + 3 + 1;
constexpr uint32_t OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr uint32_t OFF_PEER = OFF_ABORT + 4;                   // see Issued
constexpr uint32_t OFF_MINE = OFF_PEER + 12;
constexpr uint32_t OFF_NOTE = OFF_MINE + 12;                   // the tile's blocks, for the MMAs
constexpr uint32_t OFF_SIG = (OFF_NOTE + 4 + 15) / 16 * 16;
constexpr uint32_t SIG_BYTES = 16;
constexpr uint32_t SIG_P = 0;
constexpr uint32_t SIG_S = SIG_P + SM_WARPS * SIG_BYTES;
constexpr uint32_t SIG_O = SIG_S + SM_WARPS * SIG_BYTES;
constexpr uint32_t SIG_SRC = SIG_O + EP_WARPS * SIG_BYTES;
constexpr uint32_t SMEM_BYTES = OFF_SIG + SIG_SRC + (SM_WARPS + EP_WARPS) * SIG_BYTES + 1024;
static_assert(SMEM_BYTES <= 232448, "over the 227 KB shared-memory limit per CTA");
static_assert(OFF_RING % 1024 == 0 && OFF_STAGE % 1024 == 0, "swizzled buffers");

constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL = 0;     // S: columns 0 .. 127 (FP32)
constexpr uint32_t P_COL = 128;   // two P buffers of 64 columns (FP16 pairs)
constexpr uint32_t O_COL = 256;   // O: columns 256 .. 511
constexpr uint32_t IDESC_QK = (1u << 4) | ((uint32_t)(BKV >> 3) << 17) | ((uint32_t)(2 * CQ >> 4) << 24);
constexpr uint32_t IDESC_PV =
    (1u << 4) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((uint32_t)(2 * CQ >> 4) << 24);

// Rows of a pair's partial.
constexpr int PART_ROWS = 2 * CQ;

struct Bars {
  uint32_t q_full, q_empty, full, empty, s_full, s_free, p_full, o_done, o_free, l_ready, l_free,
      mma_done;
};

// This cluster's share of the line, and the tile that it begins in.  With whole
// tiles dealt out first (whole > 0, their number) per is 0 and the shares are
// those of Deal.
struct Sched {
  long long w0, w1, per;
  int b, head, tile, j;
  int base, whole;
};
static_assert(sizeof(Sched) <= 64, "room for the schedule");

// Tiles dealt out whole: tile i of the line's first `whole` to cluster
// i % clusters, so that the clusters work on tiles of the same head at the same
// time and read its keys and values from memory but once between them.  The
// blocks of the last one to two rounds of tiles make up for the differences.
// With equal shares a cluster takes neighbouring tiles one after another, and
// the head's keys have left L2 from one to the next.  Measured, equal shares ->
// whole tiles, in us (floor): a mixed step of 50 requests 418 -> 374 (160), four
// prompts of 4000 tokens 384 -> 357 (269).  Short tiles stay with equal shares
// (their keys have not left L2, and the prologue is longer): 32 prompts of 200
// (1.5 blocks a tile) 68 -> 74 (19), eight of 2000 (8.5) 234 -> 231 (134), one of
// 4001 with a window (10) 86 -> 90 (35); and so do fewer tiles than two for each
// cluster.
struct Deal {
  int start[MAX_CLUSTERS + 1];   // where each cluster's share of the rest begins
  int load[MAX_CLUSTERS];        // blocks of its whole tiles
  int tiles[WIN];                // tiles before each request
  int count;                     // tiles in all
};
static_assert(sizeof(Deal) <= DEAL_BYTES, "room for the deal");
constexpr int LONG_TILE = 12;    // mean blocks of a tile from which whole tiles are dealt

__device__ __forceinline__ bool own_request(const Params& p, const Request& r) {
  return r.n > p.skip_tokens;
}
__device__ __forceinline__ Span span_of(const Params& p, const Request& r, int tile) {
  const int i0 = tile * p.tile_tokens;
  return tile_span(r, i0, imin(i0 + p.tile_tokens, r.n) - 1, p.masks);
}
__device__ __forceinline__ int tiles_of(const Params& p, const Request& r) {
  return (r.n + p.tile_tokens - 1) / p.tile_tokens;
}

// (Deal lies behind Sched.)
__device__ __forceinline__ const Deal& deal_of(const Sched& sc) {
  return *reinterpret_cast<const Deal*>(reinterpret_cast<const uint8_t*>(&sc) + (OFF_DEAL - OFF_SCHED));
}

struct Walk {
  const Params& p;
  const Sched& sc;
  const int4* req;
  int next_whole;           // the cluster's next whole tile; -1: none are dealt, or left
  long long w, w1;
  int b, head, tile, j, base, tiles;
  Request r;
  Span s;
  int j0, j1;
  int cur_head, i0, cnt;    // of the current tile: head, first token, tokens
  __device__ __forceinline__ Walk(const Params& p_, const Sched& sc_, const int4* req_, int cluster)
      : p(p_), sc(sc_), req(req_), next_whole(-1), w(sc_.w0), w1(sc_.w1), b(sc_.b), head(sc_.head),
        tile(sc_.tile), j(sc_.j), base(sc_.base), tiles(0) {
    if (sc.whole > 0) {
      next_whole = cluster;
      b = 0;
    } else if (w < w1) {
      fetch();
    }
  }
  __device__ __forceinline__ void fetch() {
    const int k = b - base;
    if (k < WIN) {
      const int4 v = req[k];
      r.start = v.x;
      r.n = v.y;
      r.len = v.z;
    } else {
      r = load_request(p, b);
    }
    tiles = tiles_of(p, r);
  }
  // (Whole tiles leave w alone: every share of the rest holds a block.)
  __device__ __forceinline__ bool next() {
    if (w >= w1) return false;
    if (next_whole >= 0) {
      if (next_whole < sc.whole) {
        const int* before = deal_of(sc).tiles;
        while (b + 1 < p.batch && before[b + 1] <= next_whole) ++b;
        fetch();
        const int of = next_whole - before[b];
        next_whole += (int)(gridDim.x >> 1);
        cur_head = of / tiles;
        take(of - cur_head * tiles);
        j0 = 0;
        j1 = s.nb;
        return true;
      }
      next_whole = -1;
      b = sc.b;
      fetch();
    }
    if (tile == tiles) {
      tile = 0;
      ++head;
    }
    if (head == p.kv_heads) {
      head = 0;
      do {
        ++b;
        fetch();
      } while (!own_request(p, r));
    }
    take(tile);
    cur_head = head;
    j0 = j;
    j1 = (int)lmin(s.nb, (long long)j0 + (w1 - w));
    w += j1 - j0;
    j = 0;
    ++tile;
    return true;
  }
  __device__ __forceinline__ void take(int t) {
    s = span_of(p, r, t);
    i0 = t * p.tile_tokens;
    cnt = imin(p.tile_tokens, r.n - i0);
  }
  __device__ __forceinline__ bool more() const { return w < w1; }
  __device__ __forceinline__ long long line() const { return w - j1; }
};

// Key blocks of one head of a request, by a whole warp.
__device__ __forceinline__ long long head_blocks(const Params& p, const Request& r, int lane) {
  long long sum = 0;
  if (own_request(p, r)) {
    const int tiles = tiles_of(p, r);
    for (int t = lane; t < tiles; t += 32) sum += span_of(p, r, t).nb;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// Deals out the first `whole` tiles (at least as many are left as there are
// workers) and sets where the workers' shares of the other `rest` blocks begin:
// each brings its worker to a common level, and holds a block at least.
__device__ __forceinline__ void deal_tiles(const Params& p, const int4* req, Deal* deal, int whole,
                                           int workers, int total, int* warp_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Tiles before each request.
  int mine = 0;
  if (tid < p.batch) {
    const int4 v = req[tid];
    if (v.w > 0) mine = tiles_of(p, Request{v.x, v.y, v.z, false}) * p.kv_heads;
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sum[warp] = inc;
  if (tid < workers) deal->load[tid] = 0;
  __syncthreads();
  for (int k = 0; k < warp; ++k) inc += warp_sum[k];
  if (tid < p.batch) deal->tiles[tid] = inc - mine;
  __syncthreads();
  for (int i = tid; i < whole; i += NUM_THREADS) {
    int lo = 0, hi = p.batch;        // the last request with no more than i tiles before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (deal->tiles[mid] <= i) lo = mid; else hi = mid;
    }
    const int4 v = req[lo];
    const Request r{v.x, v.y, v.z, false};
    atomicAdd(&deal->load[i % workers], span_of(p, r, (i - deal->tiles[lo]) % tiles_of(p, r)).nb);
  }
  __syncthreads();
  if (warp == 0) {                   // four workers a lane
    constexpr int EACH = MAX_CLUSTERS / 32;
    int load[EACH], sum = 0, least = 2147483647, most = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int c = lane * EACH + k;
      load[k] = c < workers ? deal->load[c] : 0;
      if (c < workers) {
        sum += load[k];
        least = imin(least, load[k]);
        most = imax(most, load[k]);
      }
    }
    const int dealt = __reduce_add_sync(0xffffffffu, sum), rest = total - dealt;
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    auto shares = [&](int level) {           // of the lane's workers
      int n = 0;
#pragma unroll
      for (int k = 0; k < EACH; ++k)
        if (lane * EACH + k < workers) n += deal_share(level, load[k]);
      return n;
    };
    const int level = deal_level(least, most, rest, workers, [&](int at_level) {
      return __reduce_add_sync(0xffffffffu, shares(at_level));
    });
    sum = shares(level);
    int at = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, at, d);
      if (lane >= d) at += o;
    }
    at -= sum;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int c = lane * EACH + k;
      if (c < workers) {
        deal->start[c] = dealt + deal_start(at, rest, workers, c);
        at += deal_share(level, load[k]);
      }
    }
    if (lane == 0) deal->start[workers] = total;
  }
  __syncthreads();
}

__device__ __forceinline__ void schedule(const Params& p, uint8_t* smem, int worker, int workers,
                                         long long* warp_sum) {
  int4* req = reinterpret_cast<int4*>(smem + OFF_REQ);
  Sched* sc = reinterpret_cast<Sched*>(smem + OFF_SCHED);
  Deal* deal = reinterpret_cast<Deal*>(smem + OFF_DEAL);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sc->w0 = sc->w1 = 0;
    sc->per = 1;
    sc->whole = 0;
    deal->count = 0;
  }
  long long total = 0, w0 = 0, w1 = 0, per = 1, before = 0;
  // First pass: all blocks of the step (request counts up to WIN stay in
  // shared memory).  The second finds the worker's first tile.
  const bool one = p.batch <= WIN;
  for (int pass = 0; pass < 2; ++pass) {
    before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += WIN) {
      if (pass == 0 || !one) {
        __syncthreads();
        const int b = b0 + tid;
        if (tid < WIN) {
          Request r{0, 0, 0, false};
          if (b < p.batch) r = load_request(p, b);
          if (pass == 0 && r.bad) *(volatile int*)p.status = (int)GEMM_F16_ERR_BAD_INDEX;
          req[tid] = make_int4(r.start, r.n, r.len, 0);
        }
        __syncthreads();
        const int left = imin(WIN, p.batch - b0);
        for (int k = warp; k < left; k += NUM_WARPS) {
          const int4 v = req[k];
          const long long hb = head_blocks(p, Request{v.x, v.y, v.z, false}, lane);
          // (at most 2^31 / 128 blocks per tile, 2^31 tokens: a request that
          // does not fit 32 bits would not end in a century)
          if (lane == 0) {
            req[k].w = (int)lmin(hb, 2147483647);
            if (one && hb > 0)
              atomicAdd(&deal->count, (int)lmin((int64_t)tiles_of(p, Request{v.x, v.y, v.z, false}) *
                                                    p.kv_heads, MOST_TILES + 1));
          }
        }
        __syncthreads();
      }
      const long long mine = tid < WIN ? (long long)req[tid].w * p.kv_heads : 0;
      long long inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (lane == 31) warp_sum[warp] = inc;
      __syncthreads();
      long long all = 0, basis = before;
      for (int k = 0; k < NUM_WARPS; ++k) {
        if (k < warp) basis += warp_sum[k];
        all += warp_sum[k];
      }
      inc += basis;
      if (pass == 1 && mine > 0 && w0 >= inc - mine && w0 < inc) {
        const long long at = w0 - (inc - mine), hb = req[tid].w;
        sc->w0 = w0;
        sc->w1 = w1;
        sc->per = per;
        sc->b = b0 + tid;
        sc->head = (int)(at / hb);
        sc->tile = 0;
        sc->j = (int)(at % hb);   // for now: blocks into the head
        sc->base = b0;
      }
      before += all;
      __syncthreads();
      if (pass == 1 && w0 < before) break;   // found: req holds its part of the batch
    }
    if (pass == 0) {
      total = before;
      const int tiles = one ? deal->count : 0, whole = whole_tiles(tiles, workers);
      if (whole > 0 && total < (1 << 30) && total >= (long long)tiles * LONG_TILE) {
        deal_tiles(p, req, deal, whole, workers, (int)total, reinterpret_cast<int*>(warp_sum));
        per = 0;
        w0 = deal->start[worker];
        w1 = deal->start[worker + 1];
        if (tid == 0) sc->whole = whole;
      } else {
        per = per_worker(total, workers);
        w0 = per * worker;
        w1 = lmin(w0 + per, total);
        if (w0 >= total) return;
      }
    }
  }
  // The tile within the head, 32 at a time.
  if (warp == 0) {
    const int4 v = req[sc->b - sc->base];
    const Request r{v.x, v.y, v.z, false};
    const int tiles = tiles_of(p, r);
    int at = sc->j;
    for (int t0 = 0; t0 < tiles; t0 += 32) {
      const int t = t0 + lane;
      const int nb = t < tiles ? span_of(p, r, t).nb : 0;
      int inc = nb;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      const int all = __shfl_sync(0xffffffffu, inc, 31);
      if (at < all) {
        if (at >= inc - nb && at < inc) {
          sc->tile = t;
          sc->j = at - (inc - nb);
        }
        break;
      }
      at -= all;
    }
  }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Params& p,
                                          volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, p, abort_flag));
}

// The epilogue warps wait most of a tile: they sleep between polls.
__device__ __noinline__ bool wait_sleepy(uint32_t bar, uint32_t parity, const Params& p,
                                         volatile int* abort_flag) {
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (ptx::mbar_try_wait_poll(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      *abort_flag = 1;
      *(volatile int*)p.status = (int)GEMM_F16_ERR_TIMEOUT;
      __threadfence_system();
      return false;
    }
    __nanosleep(256);
  }
}
__device__ __forceinline__ bool wait_suspend(uint32_t bar, uint32_t parity, const Params& p,
                                             volatile int* abort_flag) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, p, abort_flag);
}

// The same wait by one lane for its warp: 32 lanes polling a barrier slow the
// copies that complete it.
__device__ __forceinline__ bool lane_wait(uint32_t bar, uint32_t parity, uint32_t lane,
                                          const Params& p, volatile int* abort_flag) {
  bool ok = true;
  if (lane == 0) ok = wait_suspend(bar, parity, p, abort_flag);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// One arrival per warp on a leader barrier (see attn_pair.cuh).
__device__ __forceinline__ void signal_leader(uint32_t rank, uint32_t lane, uint32_t local_bar,
                                              uint32_t leader_bar, uint32_t dst, uint32_t src) {
  ptx::tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    if (rank == 0)
      ptx::mbar_arrive_expect_tx(local_bar, SIG_BYTES);
    else
      ptx::bulk_copy_to_cluster(dst, src, SIG_BYTES, leader_bar);
  }
}

// Copies that a CTA has issued: key tiles, value tiles, Q tiles.
struct Issued {
  uint32_t keys, values, queries;
};

// The note that goes with a tile's Q.
constexpr uint32_t NOTE_MORE = 1u << 31;
__device__ __forceinline__ uint32_t blocks_note(int blocks, bool more) {
  return (uint32_t)blocks | (more ? NOTE_MORE : 0u);
}

// ------------------------------------------------------------------ copies
// Keys and values each have a warp and a ring of their own: with pages of 16
// rows a tile is 16 copies of 2 KB and one warp that issues both kinds falls
// behind the MMAs (4096 tokens over 8192 in pages of 16, when this was split:
// 598 us with one warp, 518 with two).
// Both CTAs fill their halves, crediting the leader's barriers; the leader
// also arrives (expect_tx) for the pair.
template <bool KEYS>
__device__ __forceinline__ uint32_t fill_ring(const CUtensorMap* tmQ, const CUtensorMap* tm,
                                              const Params& p, Walk& walk, uint32_t base,
                                              const Bars& b, uint32_t rank, uint32_t lane,
                                              int cluster, uint32_t* queries,
                                              volatile uint32_t* note,
                                              volatile int* abort_flag) {
  const uint32_t leader_q = ptx::map_to_cta(b.q_full, 0);
  const uint32_t bar0 = KEYS ? 0u : 8u * RING;          // of this ring among full / empty
  const uint32_t leader_full = ptx::map_to_cta(b.full + bar0, 0);
  const int cta_tokens = p.tile_tokens / 2;
  const uint32_t q_bytes = 4u * 128u * (uint32_t)(cta_tokens * p.group);
  // Keys: this CTA's 64 of the block, lane = chunk * 8 + group of rows (4 x 1 .. 8).
  // Values: all 128, this CTA's 128 numbers, lane = chunk * 16 + group (2 x 2 .. 16).
  const int half_groups = MAX_ROWS / p.rows;
  const int groups = KEYS ? half_groups : 2 * half_groups;
  const int chunk = (int)lane / (KEYS ? 8 : 16), in = (int)lane % (KEYS ? 8 : 16);
  const int group = (KEYS ? (int)rank * half_groups : 0) + imin(in, groups - 1);
  const int col = KEYS ? 64 * chunk : (int)rank * 128 + 64 * chunk;
  const uint32_t to = base + OFF_RING + (KEYS ? 0u : RING * SLOT_BYTES) +
                      (uint32_t)chunk * (KEYS ? K_CHUNK : V_CHUNK) + (uint32_t)(in * p.rows) * 128u;
  RingPos pos{0, 0};
  uint32_t fills = 0, loads = 0;
  bool ok = true;
  while (ok && walk.next()) {
    auto load_queries = [&] {
      if (lane == 0) {
        if (rank == 0) {
          *note = blocks_note(walk.j1 - walk.j0, walk.more());
          ptx::mbar_arrive_expect_tx(b.q_full, 2 * q_bytes);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          ptx::tma_load_3d_pair(base + OFF_Q + c * CHUNK_Q, tmQ, leader_q, 64 * c,
                                walk.cur_head * p.group,
                                walk.r.start + walk.i0 + (int)rank * cta_tokens);
      }
      ++loads;
    };
    bool asked = !KEYS || loads == 0;    // (a worker's first Q waits for nothing)
    if (KEYS && asked) load_queries();
    // Table entries are looked up two blocks ahead.
    auto page_of = [&](int j) {
      return j < walk.j1 ? group_page(p, walk.s, walk.b, span_block(walk.s, j), group) : 0;
    };
    int page = page_of(walk.j0), page1 = page_of(walk.j0 + 1);
    for (int j = walk.j0; j < walk.j1; ++j) {
      const int page2 = page_of(j + 2);
      const int2 src = group_source(p, walk.s, span_block(walk.s, j), group, page);
      page = page1;
      page1 = page2;
      ok = lane_wait(b.empty + bar0 + 8 * pos.stage, producer_wait_parity(pos), lane, p, abort_flag);
      if (!ok) break;
      if (rank == 0 && lane == 0)
        ptx::mbar_arrive_expect_tx_relaxed(b.full + bar0 + 8 * pos.stage, 2 * SLOT_BYTES);
      __syncwarp();
      if (in < groups && !(KEYS && fills == 0 && cluster == p.fault_unit && rank == 0))
        ptx::tma_load_4d_pair(to + pos.stage * SLOT_BYTES, tm, leader_full + 8 * pos.stage, col,
                              src.y, walk.cur_head, src.x);
      ++fills;
      ring_advance(pos, RING);
      // The next tile's first keys do not wait for the last one's Q to go (68.4 ->
      // 67.4 us where 100 tokens look at 30,000 keys).
      if (KEYS && !asked) {
        ok = lane_wait(b.q_empty, (loads - 1) & 1u, lane, p, abort_flag);
        if (!ok) break;
        load_queries();
        asked = true;
      }
    }
  }
  *queries = loads;
  return fills;
}

// ------------------------------------------------------------------ MMAs (leader)
// Does not walk: the key warp's note beside each tile's Q says how many blocks
// the tile has and whether another follows (`more`: whether there is any tile).
// A walk in this thread costs its loop over blocks registers: a mixed step of 50
// requests 383 -> 415 us, a prompt of 4001 with a window 87 -> 94.
__device__ __forceinline__ void mma_role(const Params& p, bool more, const volatile uint32_t* note,
                                         uint32_t base, uint32_t tmem_base, const Bars& b,
                                         volatile int* abort_flag) {
  RingPos kpos{0, 0}, vpos{0, 0};
  const uint32_t q_low = desc_low(base + OFF_Q, 16);
  const uint32_t k_ring = desc_low(base + OFF_RING, 16);
  const uint32_t v_ring = desc_low(base + OFF_RING + RING * SLOT_BYTES, V_CHUNK);
  const uint32_t o_tmem = tmem_base + O_COL;
  auto issue_qk = [&](uint32_t gs, bool last_of_tile) -> bool {
    if (gs > 0) {
      if (!wait_suspend(b.s_free, (gs - 1) & 1u, p, abort_flag)) return false;
    }
    if (!wait_suspend(b.full + 8 * kpos.stage, consumer_wait_parity(kpos), p, abort_flag))
      return false;
    ptx::tc_fence_after();
    const uint32_t k_low = k_ring + kpos.stage * (SLOT_BYTES >> 4);
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const uint32_t off_q = (uint32_t)(kk >> 2) * CHUNK_Q + (uint32_t)(kk & 3) * 32u;
      const uint32_t off_k = (uint32_t)(kk >> 2) * K_CHUNK + (uint32_t)(kk & 3) * 32u;
      ptx::mma_f16_pair(tmem_base + S_COL, desc(q_low + off_q / 16), desc(k_low + off_k / 16),
                        IDESC_QK, kk > 0 ? 1u : 0u);
    }
    ptx::mma_commit_pair(b.empty + 8 * kpos.stage, 0x3);
    ptx::mma_commit_pair(b.s_full, 0x3);
    if (last_of_tile) ptx::mma_commit_pair(b.q_empty, 0x3);
    ring_advance(kpos, RING);
    return true;
  };
  uint32_t g0 = 0, ki = 0;
  bool ok = true;
  while (ok && more) {
    if (!wait_suspend(b.q_full, ki & 1u, p, abort_flag)) break;
    ptx::tc_fence_after();
    const uint32_t of_tile = *note;
    const int nb = (int)(of_tile & ~NOTE_MORE);
    more = (of_tile & NOTE_MORE) != 0;
    ok = issue_qk(g0, nb == 1);
    for (int j = 0; j < nb && ok; ++j) {
      const uint32_t gj = g0 + (uint32_t)j;
      if (j + 1 < nb && !issue_qk(gj + 1, j + 2 == nb)) {
        ok = false;
        break;
      }
      const uint32_t pb = gj & 1u;
      if (!wait_suspend(b.p_full + 8 * pb, (gj >> 1) & 1u, p, abort_flag) ||
          !wait_suspend(b.full + 8 * (RING + vpos.stage), consumer_wait_parity(vpos), p, abort_flag)) {
        ok = false;
        break;
      }
      if (j == 0 && ki > 0 && !wait_suspend(b.o_free, (ki - 1) & 1u, p, abort_flag)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t v_low = v_ring + vpos.stage * (SLOT_BYTES >> 4);
      const uint32_t p_tmem = tmem_base + P_COL + pb * (BKV / 2);
#pragma unroll
      for (int kk = 0; kk < BKV / 16; ++kk)
        ptx::mma_f16_pair_tmem_a(o_tmem, p_tmem + (uint32_t)kk * 8u,
                                 desc(v_low + (uint32_t)kk * 128u),
                                 IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
      ptx::mma_commit_pair(b.empty + 8 * (RING + vpos.stage), 0x3);
      ptx::mma_commit_pair(b.o_done + 8 * pb, 0x3);
      ring_advance(vpos, RING);
    }
    g0 += (uint32_t)nb;
    ++ki;
  }
}

// ------------------------------------------------------------------ softmax
// New exponent offset of one row for a key block (base-2 units): it moves, to
// TAIL_LOG2 below the block's maximum, only when that passes it by more than
// OVER_LOG2.
__device__ __forceinline__ float block_offset(const uint32_t (&s)[BKV], float sl2, float m,
                                              float* alpha) {
  float r8[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) r8[k] = __uint_as_float(s[k]);
  if (sl2 > 0.f) {
#pragma unroll
    for (int c = 8; c < BKV; ++c) r8[c & 7] = fmaxf(r8[c & 7], __uint_as_float(s[c]));
#pragma unroll
    for (int k = 1; k < 8; ++k) r8[0] = fmaxf(r8[0], r8[k]);
  } else {
#pragma unroll
    for (int c = 8; c < BKV; ++c) r8[c & 7] = fminf(r8[c & 7], __uint_as_float(s[c]));
#pragma unroll
    for (int k = 1; k < 8; ++k) r8[0] = fminf(r8[0], r8[k]);
  }
  const float to = fmaf(r8[0], sl2, -TAIL_LOG2);
  const float m_new = (to > m + (OVER_LOG2 - TAIL_LOG2)) ? to : m;
  *alpha = (m_new == m) ? 1.f : ptx::ex2_approx(m - m_new);
  return m_new;
}

// Weights 2^(sl2 s - m) as binary16 pairs (the product with V takes binary16;
// half a step each: 2^-11 of the weight, or 2^-25 below the normal range, which
// TAIL_LOG2 keeps 2^-32 below the row's largest), and their FP32 sum before that
// rounding.
__device__ __forceinline__ float block_weights(const uint32_t (&s)[BKV], float sl2, float neg_m,
                                               uint32_t (&pk)[BKV / 2]) {
  float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < BKV / 2; ++c) {
    const float p0 = ptx::ex2_approx(fmaf(__uint_as_float(s[2 * c]), sl2, neg_m));
    const float p1 = ptx::ex2_approx(fmaf(__uint_as_float(s[2 * c + 1]), sl2, neg_m));
    pk[c] = pack_half2(p0, p1);
    l4[c & 3] += p0 + p1;
  }
  return (l4[0] + l4[1]) + (l4[2] + l4[3]);
}

__device__ __forceinline__ void softmax_role(const Params& p, Walk& walk, uint32_t base,
                                             uint32_t tmem_base, const Bars& b, float* l_rows,
                                             uint32_t rank, uint32_t warp, uint32_t lane,
                                             volatile int* abort_flag) {
  const uint32_t quarter = warp & 3u;
  const uint32_t t_lane = (quarter * 32u) << 16;
  const uint32_t row = quarter * 32u + lane;
  const uint32_t leader_p_full = ptx::map_to_cta(b.p_full, 0);
  const uint32_t leader_s_free = ptx::map_to_cta(b.s_free, 0);
  const uint32_t sig_p = ptx::map_to_cta(base + OFF_SIG + SIG_P + warp * SIG_BYTES, 0);
  const uint32_t sig_s = ptx::map_to_cta(base + OFF_SIG + SIG_S + warp * SIG_BYTES, 0);
  const uint32_t sig_src = base + OFF_SIG + SIG_SRC + warp * SIG_BYTES;
  const float sl2 = p.scale_log2;
  const int my_tok = (int)rank * (p.tile_tokens / 2) + (int)row / p.group;   // in the tile
  uint32_t g = 0, ki = 0;
  bool ok = true;
  while (ok && walk.next()) {
    const int p0 = walk.r.len - walk.r.n + walk.i0;      // positions of the tile's tokens
    const int p1 = p0 + walk.cnt - 1, pos = p0 + my_tok;
    float m = NO_OFFSET, l = 0.f;
    for (int j = walk.j0; j < walk.j1; ++j, ++g) {
      const int blk = span_block(walk.s, j);
      const bool full_block = block_is_full(p0, p1, blk, p.masks);
      uint32_t see[4];
      if (!full_block) seen_words(walk.s, blk, p.rows, pos, p.masks, see);
      if (!warp_wait(b.s_full, g & 1u, p, abort_flag)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      uint32_t s[BKV];
#pragma unroll
      for (int c = 0; c < BKV / 32; ++c)
        ptx::tmem_ld_32x32b_x32(tmem_base + t_lane + S_COL + 32u * c,
                                *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
      ptx::tmem_ld_wait();
      ptx::reg_fence(s);
      if (j + 1 < walk.j1 || walk.more())
        signal_leader(rank, lane, b.s_free, leader_s_free, sig_s, sig_src);
      float alpha;
      uint32_t pk[BKV / 2];
      if (!full_block) {
        // A hidden key's score becomes the infinity whose weight is 0.
        const uint32_t fill = __float_as_uint(sl2 > 0.f ? -INFINITY : INFINITY);
#pragma unroll
        for (int c = 0; c < BKV; ++c) s[c] = (see[c >> 5] >> (c & 31)) & 1u ? s[c] : fill;
      }
      const float m_new = block_offset(s, sl2, m, &alpha);
      const float lsum = block_weights(s, sl2, -m_new, pk);
      const uint32_t pb = g & 1u;
      if (g >= 2) {
        if (!warp_wait(b.o_done + 8 * pb, ((g - 2) >> 1) & 1u, p, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
      }
      const uint32_t p_tmem = tmem_base + t_lane + P_COL + pb * (BKV / 2);
      ptx::tmem_st_32x32b_x32(p_tmem, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
      ptx::tmem_st_32x32b_x32(p_tmem + 32u, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
      if (j > walk.j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        const uint32_t ob = (g - 1) & 1u;
        if (!warp_wait(b.o_done + 8 * ob, ((g - 1) >> 1) & 1u, p, abort_flag)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          const uint32_t ta = tmem_base + t_lane + O_COL + (uint32_t)c * 32u;
          ptx::tmem_ld_32x32b_x32(ta, o);
          ptx::tmem_ld_wait();
          ptx::reg_fence(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          ptx::tmem_st_32x32b_x32(ta, o);
        }
      }
      ptx::tmem_st_wait();
      signal_leader(rank, lane, b.p_full + 8 * pb, leader_p_full + 8 * pb, sig_p, sig_src);
      l = l * alpha + lsum;
      m = m_new;
    }
    if (!ok) break;
    if (ki > 0 && !warp_wait(b.l_free, (ki - 1) & 1u, p, abort_flag)) break;
    l_rows[row] = l;
    l_rows[CQ + row] = m;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(b.l_ready);
    ++ki;
  }
}

// ------------------------------------------------------------------ epilogue
// 64 numbers of each of a warp's 32 rows (one row per thread, FP32, times
// `factor`) to O: through a box in shared memory, so that each row's 128 bytes
// go out together.
__device__ __forceinline__ void store_rows(const float (&f)[64], float factor,
                                           uint32_t box, const uint4* box_rows, uint32_t lane,
                                           const int64_t (&row_off)[8], int rows, __half* dst0,
                                           int cc) {
  const uint32_t lsw = lane & 7u;
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i)
    ptx::st_shared_v4(box + lane * 128u + ((i ^ lsw) << 4),
                      pack_half2(f[8 * i] * factor, f[8 * i + 1] * factor),
                      pack_half2(f[8 * i + 2] * factor, f[8 * i + 3] * factor),
                      pack_half2(f[8 * i + 4] * factor, f[8 * i + 5] * factor),
                      pack_half2(f[8 * i + 6] * factor, f[8 * i + 7] * factor));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (int)(lane >> 3);
    const uint4 v = box_rows[r * 8 + (int)((lane & 7u) ^ (uint32_t)(r & 7))];
    if (r < rows) {
      *reinterpret_cast<uint4*>(dst0 + row_off[i] + cc * 64) = v;
    }
  }
  __syncwarp();
}

// Per tile, each warp its 32 rows, a row per thread.  A tile that is the
// cluster's alone: O out of tensor memory, normalised, to O.  A part of a tile
// that is cut: to the workspace, unnormalised, as [number / 4][row][4], so
// that the threads of a warp write (and the merge reads) 512 bytes together.
__device__ __forceinline__ void epilogue_role(const Params& p, const Sched& sc, Walk& walk,
                                              uint8_t* smem, uint32_t base, uint32_t tmem_base,
                                              const Bars& b, const float* l_rows, uint32_t rank,
                                              uint32_t warp, uint32_t lane, int cluster,
                                              volatile int* abort_flag) {
  const uint32_t quarter = warp & 3u;
  const uint32_t o_addr = tmem_base + ((quarter * 32u) << 16) + O_COL;
  const uint32_t e = warp - SM_WARPS;
  const uint32_t leader_o_free = ptx::map_to_cta(b.o_free, 0);
  const uint32_t sig_o = ptx::map_to_cta(base + OFF_SIG + SIG_O + e * SIG_BYTES, 0);
  const uint32_t sig_src = base + OFF_SIG + SIG_SRC + (SM_WARPS + e) * SIG_BYTES;
  const uint32_t box = base + OFF_STAGE + e * BOX;
  const uint4* box_rows = reinterpret_cast<const uint4*>(smem + OFF_STAGE + e * BOX);
  const int cta_tokens = p.tile_tokens / 2;
  const int sub = (int)rank * EP_WARPS + (int)quarter;      // these 32 rows among the pair's
  // The rows that this thread writes (store_rows), and its 16 bytes of them.
  int64_t row_off[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rr = (int)(quarter * 32u + i * 4 + (lane >> 3)), tok = rr / p.group;
    row_off[i] = tok * p.o_tok + (int64_t)(rr - tok * p.group) * p.o_head + (lane & 7u) * 8;
  }
  uint32_t ki = 0, g_end = 0;
  bool ok = true;
  // 64 numbers of this thread's row of O; after the last ones O may be overwritten.
  auto load_o = [&](int cc, bool more, float (&f)[64]) {
    uint32_t o[64];
    ptx::tmem_ld_32x32b_x32(o_addr + (uint32_t)cc * 64u,
                            *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
    ptx::tmem_ld_32x32b_x32(o_addr + (uint32_t)cc * 64u + 32u,
                            *reinterpret_cast<uint32_t(*)[32]>(&o[32]));
    ptx::tmem_ld_wait();
    ptx::reg_fence(o);
    if (cc == HD / 64 - 1 && more)
      signal_leader(rank, lane, b.o_free, leader_o_free, sig_o, sig_src);
#pragma unroll
    for (int i = 0; i < 64; ++i) f[i] = __uint_as_float(o[i]);
  };
  if (sub == 0 && lane == 0) p.cut[cluster].last = -1;
  while (walk.next()) {
    const int head = walk.cur_head;
    const bool more = walk.more();
    const bool whole = walk.j0 == 0 && walk.j1 == walk.s.nb;
    g_end += (uint32_t)(walk.j1 - walk.j0);
    const uint32_t g_last = g_end - 1;
    // Tokens of this CTA that exist; where its rows go.
    const int tokens = imin(imax(walk.cnt - (int)rank * cta_tokens, 0), cta_tokens);
    const int rows = imin(imax(tokens * p.group - (int)quarter * 32, 0), 32);
    __half* const dst0 = p.O + (int64_t)(walk.r.start + walk.i0 + (int)rank * cta_tokens) * p.o_tok +
                         (int64_t)(head * p.group) * p.o_head;
    float l = 0.f, m = NO_OFFSET;
    ok = ok && __all_sync(0xffffffffu, wait_sleepy(b.l_ready, ki & 1u, p, abort_flag));
    if (ok) {
      l = l_rows[quarter * 32u + lane];
      m = l_rows[CQ + quarter * 32u + lane];
      __syncwarp();
      if (more && lane == 0) ptx::mbar_arrive(b.l_free);
      ok = warp_wait(b.o_done + 8 * (g_last & 1u), (g_last >> 1) & 1u, p, abort_flag);
      ptx::tc_fence_after();
    }
    ++ki;
    if (whole) {
      if (!ok) continue;
      const float inv_l = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
      for (int cc = 0; cc < HD / 64; ++cc) {
        float f[64];
        load_o(cc, more, f);
        store_rows(f, inv_l, box, box_rows, lane, row_off, rows, dst0, cc);
      }
      continue;
    }
    if (!ok) continue;
    // A share has at most two parts: of a tile that others began, of its own.
    const int own = 2 * cluster + (walk.j0 == 0 ? 1 : 0);
    __stcg(p.part_ml + (int64_t)own * PART_ROWS + sub * 32 + lane, make_float2(m, l));
#pragma unroll 1
    for (int cc = 0; cc < HD / 64; ++cc) {
      float f[64];
      load_o(cc, more, f);
      float4* dst = reinterpret_cast<float4*>(p.part + ((int64_t)own * PART_ROWS + sub * 32) * HD) +
                    cc * 16 * 32 + lane;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        __stcg(dst + i * 32, make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]));
    }
    if (sub == 0 && lane == 0 && walk.j0 == 0) {
      CutTile t = {};
      const long long end = walk.line() + walk.s.nb;
      if (sc.per > 0) {
        t.last = (int)((end - 1) / sc.per);
      } else {
        const int* start = deal_of(sc).start;
        for (t.last = cluster; start[t.last + 1] < end;) ++t.last;
      }
      t.first = own;
      t.token = walk.r.start + walk.i0;
      t.tokens = walk.cnt;
      t.head = head;
      p.cut[cluster] = t;
    }
  }
}

// Merges the cut tiles: block (w, y) rows 32y .. 32y + 31 of the pair's tile
// that worker w began and others ended; a lane a row, a warp sixteen numbers of
// each.  Launched behind the kernel below, whose end it waits for.
constexpr int MERGE_THREADS = 512;
__global__ void __launch_bounds__(MERGE_THREADS) paged_large_merge_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = (int)blockIdx.x, sub = (int)blockIdx.y;
  const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
  const CutTile t = p.cut[w];
  const int cta_tokens = p.tile_tokens / 2, rank = sub / EP_WARPS;
  const int tokens = imin(imax(t.tokens - rank * cta_tokens, 0), cta_tokens);
  const int rr = (sub % EP_WARPS) * 32 + lane;            // row within the CTA's 128
  if (t.last < 0 || (sub % EP_WARPS) * 32 >= tokens * p.group) return;
  auto row0 = [&](int c) { return (int64_t)(c == w ? t.first : 2 * c) * PART_ROWS + sub * 32; };
  float mx = NO_OFFSET;
#pragma unroll 4
  for (int c = w; c <= t.last; ++c) mx = fmaxf(mx, __ldcg(p.part_ml + row0(c) + lane).x);
  float acc[16] = {}, sum = 0.f;
#pragma unroll 4
  for (int c = w; c <= t.last; ++c) {
    const float2 ml = __ldcg(p.part_ml + row0(c) + lane);
    const float4* src = reinterpret_cast<const float4*>(p.part + row0(c) * HD) + warp * 4 * 32 + lane;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __ldcg(src + i * 32);
    const float wgt = ptx::ex2_approx(ml.x - mx);
    sum = fmaf(wgt, ml.y, sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[4 * i] = fmaf(wgt, v[i].x, acc[4 * i]);
      acc[4 * i + 1] = fmaf(wgt, v[i].y, acc[4 * i + 1]);
      acc[4 * i + 2] = fmaf(wgt, v[i].z, acc[4 * i + 2]);
      acc[4 * i + 3] = fmaf(wgt, v[i].w, acc[4 * i + 3]);
    }
  }
  if (rr >= tokens * p.group) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int tok = rr / p.group;
  uint4* dst = reinterpret_cast<uint4*>(
      p.O + (int64_t)(t.token + rank * cta_tokens + tok) * p.o_tok +
      (int64_t)(t.head * p.group + rr - tok * p.group) * p.o_head + warp * 16);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    dst[i] = make_uint4(pack_half2(acc[8 * i] * inv, acc[8 * i + 1] * inv),
                        pack_half2(acc[8 * i + 2] * inv, acc[8 * i + 3] * inv),
                        pack_half2(acc[8 * i + 4] * inv, acc[8 * i + 5] * inv),
                        pack_half2(acc[8 * i + 6] * inv, acc[8 * i + 7] * inv));
}

// See attn_pair.cuh: completes every phase a copy warp opened and waits
// (bounded) for the copies that were issued.  Fill f of a ring used slot
// f % RING in phase parity (f / RING) & 1.
__device__ __forceinline__ void drain_ring(uint32_t bar0, uint32_t mine, uint32_t peer,
                                           uint32_t slots, uint32_t bytes, uint64_t limit_ns) {
  const uint32_t hi = mine > peer ? mine : peer;
  for (uint32_t f = hi > slots ? hi - slots : 0u; f < hi; ++f) {
    const uint32_t bar = bar0 + 8 * (f % slots);
    if (f >= mine) ptx::mbar_arrive_expect_tx_relaxed(bar, bytes);
    if (f >= peer) ptx::mbar_complete_tx(bar, bytes);
    wait_drain(bar, (f / slots) & 1u, limit_ns);
  }
}
__device__ __noinline__ void leader_drain(const Bars& b, Issued mine, Issued peer, uint32_t q_bytes,
                                          uint64_t limit_ns) {
  drain_ring(b.full, mine.keys, peer.keys, RING, SLOT_BYTES, limit_ns);
  drain_ring(b.full + 8 * RING, mine.values, peer.values, RING, SLOT_BYTES, limit_ns);
  drain_ring(b.q_full, mine.queries, peer.queries, 1, q_bytes, limit_ns);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    paged_large_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long warp_sum[NUM_WARPS];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t rank = ptx::cluster_ctarank();
  const int cluster = (int)(blockIdx.x >> 1);
  const int nclusters = (int)(gridDim.x >> 1);
  float* l_rows = reinterpret_cast<float*>(smem + OFF_L);

  Bars b;
  b.q_full = base + OFF_BAR;
  b.q_empty = b.q_full + 8;
  b.full = b.q_empty + 8;
  b.empty = b.full + 8 * SLOTS;
  b.s_full = b.empty + 8 * SLOTS;
  b.s_free = b.s_full + 8;
  b.p_full = b.s_free + 8;
  b.o_done = b.p_full + 16;
  b.o_free = b.o_done + 16;
  b.l_ready = b.o_free + 8;
  b.l_free = b.l_ready + 8;
  b.mma_done = b.l_free + 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
  volatile uint32_t* note = reinterpret_cast<volatile uint32_t*>(smem + OFF_NOTE);

  if (warp == COPY_K_WARP && lane == 0) {
    ptx::prefetch_tmap(&tmQ);
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
    ptx::mbar_init(b.q_full, 1);
    ptx::mbar_init(b.q_empty, 1);
    for (int s = 0; s < SLOTS; ++s) {
      ptx::mbar_init(b.full + 8 * s, 1);
      ptx::mbar_init(b.empty + 8 * s, 1);
    }
    ptx::mbar_init(b.s_full, 1);
    ptx::mbar_init(b.s_free, SM_WARPS);  // leader warps (+ the peer's bytes)
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(b.p_full + 8 * k, SM_WARPS);
      ptx::mbar_init(b.o_done + 8 * k, 1);
    }
    ptx::mbar_init(b.o_free, EP_WARPS);
    ptx::mbar_init(b.l_ready, SM_WARPS);
    ptx::mbar_init(b.l_free, EP_WARPS);
    ptx::mbar_init(b.mma_done, 1);
    *abort_flag = 0;
    for (int k = 0; k < 6; ++k)
      *reinterpret_cast<volatile uint32_t*>(smem + OFF_PEER + 4 * k) = 0;
    ptx::fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    ptx::tmem_alloc_pair(base + OFF_TMEM_SLOT, TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  // Rows of Q past group * tokens are never copied: numbers whose results are dropped.
  for (uint32_t i = threadIdx.x; i < Q_BYTES / 16; i += NUM_THREADS)
    ptx::st_shared_v4(base + OFF_Q + 16 * i, 0, 0, 0, 0);
  ptx::fence_proxy_async_smem();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  schedule(p, smem, cluster, nclusters, warp_sum);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers exist before anyone signals them
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);
  const Sched& sc = *reinterpret_cast<const Sched*>(smem + OFF_SCHED);
  const int4* req = reinterpret_cast<const int4*>(smem + OFF_REQ);

  if (warp < SM_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SM_REGS));
    Walk walk(p, sc, req, cluster);
    softmax_role(p, walk, base, tmem_base, b, l_rows, rank, warp, lane, abort_flag);
  } else if (warp < SM_WARPS + EP_WARPS) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EP_REGS));
    if (p.zero_rows)
      zero_tail(p, (int)blockIdx.x * EP_WARPS + (int)warp - SM_WARPS, (int)gridDim.x * EP_WARPS);
    Walk walk(p, sc, req, cluster);
    epilogue_role(p, sc, walk, smem, base, tmem_base, b, l_rows, rank, warp, lane, cluster,
                  abort_flag);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(IO_REGS));
    if (warp == COPY_K_WARP || warp == COPY_V_WARP) {
      Walk walk(p, sc, req, cluster);
      uint32_t queries, fills;
      if (warp == COPY_K_WARP)
        fills = fill_ring<true>(&tmQ, &tmK, p, walk, base, b, rank, lane, cluster, &queries, note,
                                abort_flag);
      else
        fills = fill_ring<false>(&tmQ, &tmV, p, walk, base, b, rank, lane, cluster, &queries, note,
                                 abort_flag);
      // What each CTA issued, for the leader's drain: its own beside the peer's.
      if (lane == 0) {
        const uint32_t at = base + (rank == 0 ? OFF_MINE : OFF_PEER);
        if (warp == COPY_K_WARP) {
          ptx::st_cluster_u32(ptx::map_to_cta(at, 0), fills);
          ptx::st_cluster_u32(ptx::map_to_cta(at + 8, 0), queries);
        } else {
          ptx::st_cluster_u32(ptx::map_to_cta(at + 4, 0), fills);
        }
      }
    } else if (warp == MMA_WARP) {
      if (lane == 0 && rank == 0) {
        mma_role(p, sc.w0 < sc.w1, note, base, tmem_base, b, abort_flag);
        ptx::mma_commit_pair(b.mma_done, 0x1);
        wait_drain(b.mma_done, 0, p.timeout_ns);
      }
      __syncwarp();
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs have stopped issuing
  if (warp == COPY_K_WARP && lane == 0 && rank == 0) {
    const volatile uint32_t* mine = reinterpret_cast<volatile uint32_t*>(smem + OFF_MINE);
    const volatile uint32_t* peer = reinterpret_cast<volatile uint32_t*>(smem + OFF_PEER);
    leader_drain(b, Issued{mine[0], mine[1], mine[2]}, Issued{peer[0], peer[1], peer[2]},
                 4u * 128u * (uint32_t)(p.tile_tokens / 2 * p.group), p.timeout_ns);
  }
  ptx::cluster_sync();  // no copy into either CTA is still in flight
  if (warp == MMA_WARP) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace large
}  // namespace paged
}  // namespace gf16
