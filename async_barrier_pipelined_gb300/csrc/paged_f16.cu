// The maps of a serving step over a paged key/value cache
// (attn_f16_paged_maps) and rotary positions with the write of new keys and
// values into their slots (attn_f16_rope): kernels and entry points.

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "host.h"

using namespace gf16;
using namespace gf16::host;

namespace {

constexpr int HEAD_DIM = 256;

__device__ __forceinline__ void report(int* status, int code) {
  *(volatile int*)status = code;
}

// ------------------------------------------------------------------ maps

constexpr int MAP_THREADS = 256;
constexpr int MAP_EACH = 4;                          // requests (and tokens) per thread
constexpr int MAP_CHUNK = MAP_THREADS * MAP_EACH;    // requests scanned at a time

struct MapsParams {
  int batch;
  const int32_t *cached, *added;
  int32_t* table;
  int64_t table_stride;
  int64_t rows;                 // max_pages * page_size: the most tokens a request can have
  const int32_t* free_pages;
  int num_free;
  const int32_t* free_head;
  int page_size, max_tokens;
  int32_t *starts, *kv_lens, *positions, *slots, *free_head_out;
  int* status;
};

// Running sums that stop at a limit: min(a + b, limit) is associative for
// values in [0, limit], so a block scan may group it freely, and no sum
// leaves 32 bits.
__device__ __forceinline__ uint32_t add_to(uint32_t a, uint32_t b, uint32_t limit) {
  return min(a + b, limit);
}

// Exclusive block scan of one value per thread; *total receives the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t limit, uint32_t* warp_sums,
                                               uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc = add_to(inc, o, limit);
  }
  uint32_t before = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) before = 0;
  __syncthreads();  // warp_sums of the last scan are read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < MAP_THREADS / 32; ++w) {
    if (w == warp) base = all;
    all = add_to(all, warp_sums[w], limit);
  }
  *total = all;
  return add_to(base, before, limit);
}

// One block per MAP_CHUNK new tokens.  Every block scans the lengths itself
// (8 bytes per request, from L2 after the first block), so the whole step is
// one launch and no block waits for another; each thread then finds the
// requests of its four consecutive tokens by bisection in shared memory.
// The token that is first in a page that the request did not have yet also
// writes that page's table entry: a new page's first row always belongs to
// a new token.
__global__ void __launch_bounds__(MAP_THREADS) paged_maps_kernel(const MapsParams p) {
  __shared__ uint32_t s_start[MAP_CHUNK + 1];  // first new token of each request of the chunk
  __shared__ int32_t s_cached[MAP_CHUNK];
  __shared__ uint32_t s_page[MAP_CHUNK];       // free-list offset of the request's first new page
  __shared__ uint32_t warp_sums[MAP_THREADS / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t most = (uint32_t)p.max_tokens;
  const uint32_t page_limit = 0x7fffffffu;
  const uint32_t ps = (uint32_t)p.page_size;
  const int64_t t0 = ((int64_t)blockIdx.x * MAP_THREADS + threadIdx.x) * MAP_EACH;
  const int64_t block_end = ((int64_t)blockIdx.x + 1) * MAP_CHUNK;
  int32_t head = *p.free_head;
  bool bad = head < 0 || head > p.num_free;
  head = head < 0 ? p.num_free : min(head, p.num_free);
  const bool writer0 = blockIdx.x == 0;
  uint32_t tok0 = 0, page0 = 0;                // sums before the chunk
  int32_t pos4[MAP_EACH] = {0, 0, 0, 0}, slot4[MAP_EACH] = {-1, -1, -1, -1};

  for (int b0 = 0, chunk = 0; b0 < p.batch; b0 += MAP_CHUNK, ++chunk) {
    // The next chunk, from this one on, whose starts and lengths this block writes.
    const int64_t ahead = ((int64_t)blockIdx.x + gridDim.x - chunk % (int)gridDim.x) % gridDim.x;
    if (!writer0 && (int64_t)tok0 >= block_end && b0 + ahead * MAP_CHUNK >= p.batch)
      break;  // no later chunk has work for this block
    uint32_t c[MAP_EACH], n[MAP_EACH];
#pragma unroll
    for (int i = 0; i < MAP_EACH; ++i) {
      const int b = b0 + (int)threadIdx.x * MAP_EACH + i;
      int32_t ci = 0, ni = 0;
      if (b < p.batch) {
        ci = p.cached[b];
        ni = p.added[b];
      }
      int64_t room = p.rows - max(ci, 0);
      bad |= ci < 0 || ni < 0 || room < max(ni, 0);
      ci = (int32_t)min((int64_t)max(ci, 0), p.rows);
      room = p.rows - ci;
      // kv_lens is a 32-bit number
      room = min(room, (int64_t)INT32_MAX - ci);
      bad |= room < max(ni, 0);
      c[i] = (uint32_t)ci;
      n[i] = (uint32_t)min((int64_t)max(ni, 0), room);
      bad |= n[i] > most;
      n[i] = min(n[i], most);
    }
    // Tokens: thread sums, block scan, then each request's first token.
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < MAP_EACH; ++i) sum = add_to(sum, n[i], most);
    uint32_t tok_all, page_all;
    uint32_t at = add_to(tok0, block_scan(sum, most, warp_sums, &tok_all), most);
    uint32_t need[MAP_EACH], pages = 0, st[MAP_EACH];
#pragma unroll
    for (int i = 0; i < MAP_EACH; ++i) {
      st[i] = at;
      const uint32_t next = add_to(at, n[i], most);
      bad |= next - at < n[i];
      n[i] = next - at;                        // what max_tokens leaves of it
      at = next;
      const uint32_t first = (c[i] + ps - 1) / ps, last = (c[i] + n[i] + ps - 1) / ps;
      need[i] = last - first;
      pages = add_to(pages, need[i], page_limit);
    }
    uint32_t pg = add_to(page0, block_scan(pages, page_limit, warp_sums, &page_all), page_limit);
#pragma unroll
    for (int i = 0; i < MAP_EACH; ++i) {
      const int k = (int)threadIdx.x * MAP_EACH + i, b = b0 + k;
      s_start[k] = st[i];
      s_cached[k] = (int32_t)c[i];
      s_page[k] = pg;
      pg = add_to(pg, need[i], page_limit);
      if (ahead == 0 && b < p.batch) {
        p.starts[b] = (int32_t)st[i];
        p.kv_lens[b] = (int32_t)(c[i] + n[i]);
        if (b == p.batch - 1) p.starts[p.batch] = (int32_t)(st[i] + n[i]);
      }
    }
    if (threadIdx.x == MAP_THREADS - 1) s_start[MAP_CHUNK] = at;
    __syncthreads();
    tok0 = add_to(tok0, tok_all, most);
    page0 = add_to(page0, page_all, page_limit);

    // This thread's tokens that belong to the chunk's requests.
    const uint32_t lo_tok = s_start[0], hi_tok = s_start[MAP_CHUNK];
    int k = -1;
#pragma unroll
    for (int i = 0; i < MAP_EACH; ++i) {
      const int64_t t64 = t0 + i;
      if (t64 < (int64_t)lo_tok || t64 >= (int64_t)hi_tok) continue;
      const uint32_t t = (uint32_t)t64;
      if (k < 0) {
        // The last request with s_start <= t: the largest k in [0, MAP_CHUNK)
        // (requests without tokens share a start, so the last one is the owner).
        int lo = 0, hi = MAP_CHUNK;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_start[mid] <= t) lo = mid; else hi = mid;
        }
        k = lo;
      } else {
        while (s_start[k + 1] <= t) ++k;
      }
      const uint32_t cached = (uint32_t)s_cached[k];
      const uint32_t pos = cached + (t - s_start[k]);
      const uint32_t pi = pos / ps, row = pos - pi * ps;
      const uint32_t first = (cached + ps - 1) / ps;
      int32_t* entry = p.table + (int64_t)(b0 + k) * p.table_stride + pi;
      int32_t page;
      if (pi < first) {
        page = *entry;
        bad |= page < 0;
      } else {
        const int64_t f = (int64_t)head + s_page[k] + (pi - first);
        page = f < (int64_t)p.num_free ? p.free_pages[f] : -1;
        bad |= page < 0;
        if (row == 0) *entry = page < 0 ? -1 : page;
      }
      const int64_t slot = (int64_t)page * ps + row;
      bad |= slot > INT32_MAX;
      pos4[i] = (int32_t)pos;
      slot4[i] = page < 0 || slot > INT32_MAX ? -1 : (int32_t)slot;
    }
    __syncthreads();  // the chunk's arrays are read
  }

  if (t0 + MAP_EACH <= p.max_tokens && (((uintptr_t)p.positions | (uintptr_t)p.slots) & 15) == 0) {
    *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos4[0], pos4[1], pos4[2], pos4[3]);
    *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot4[0], slot4[1], slot4[2], slot4[3]);
  } else {
#pragma unroll
    for (int i = 0; i < MAP_EACH; ++i) {
      if (t0 + i < p.max_tokens) {
        p.positions[t0 + i] = pos4[i];
        p.slots[t0 + i] = slot4[i];
      }
    }
  }
  if (writer0 && threadIdx.x == 0)
    *p.free_head_out = (int32_t)min((int64_t)head + page0, (int64_t)p.num_free);
  if (bad) report(p.status, GEMM_F16_ERR_BAD_INDEX);
}

// ------------------------------------------------------------------ rope

constexpr int ROPE_THREADS = 128;
constexpr int ROPE_LANES = 16;                              // threads per head
constexpr int ROPE_HEADS = ROPE_THREADS / ROPE_LANES;       // heads in flight per block ...
constexpr int ROPE_EACH = 4;                                // ... and per thread
constexpr int ROPE_BLOCK_HEADS = ROPE_HEADS * ROPE_EACH;

struct RopeParams {
  int q_heads, kv_heads, rot_dim, layout, inverse;
  float factor;
  const uint64_t* turns;
  const int32_t *positions, *slots;
  const __half *Q, *K, *V;
  __half *Qo, *Kc, *Vc;
  int64_t q_st[2], qo_st[2], k_st[2], v_st[2], kc_st[3], vc_st[3];
  int page_size;
  int64_t num_slots;
  int* status;
};

__device__ __forceinline__ uint32_t rotate_pair(uint32_t lo_hi_a, uint32_t lo_hi_b, float2 cs0,
                                                float2 cs1, uint32_t* out_b) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo_hi_a));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&lo_hi_b));
  __half2 ra = __floats2half2_rn(a.x * cs0.x - b.x * cs0.y, a.y * cs1.x - b.y * cs1.y);
  __half2 rb = __floats2half2_rn(b.x * cs0.x + a.x * cs0.y, b.y * cs1.x + a.y * cs1.y);
  *out_b = *reinterpret_cast<uint32_t*>(&rb);
  return *reinterpret_cast<uint32_t*>(&ra);
}

// y0 = x0 c - x1 s, y1 = x1 c + x0 s for neighbouring numbers.
__device__ __forceinline__ uint32_t rotate_neighbours(uint32_t x01, float2 cs) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&x01));
  __half2 y = __floats2half2_rn(x.x * cs.x - x.y * cs.y, x.y * cs.x + x.x * cs.y);
  return *reinterpret_cast<uint32_t*>(&y);
}

// One block per token and 32 of its heads (queries, keys, values in that
// order); 16 threads per head, 16 numbers each as two 16-byte vectors, so a
// rotated pair never leaves its thread: in the half layout thread i < rot/16
// holds vectors i and i + rot/16 (pairs 8i .. 8i+7) and the others the rest of
// the head, in the interleaved one vectors i and i + 16 (four pairs each);
// either way the threads of a head touch 256 bytes side by side at a time
// (two neighbouring vectors per thread wrote half sectors: 27.2 us on 2999
// interleaved tokens of 48 heads, now 24.7).  The angle of pair i at position p is
// p * turns[i] modulo 2^64, in units of 2^-64 turns: an integer product, so no
// position loses bits; each thread computes one pair's cosine and sine for
// the block, while the loads of its heads are in flight.
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeParams p) {
  __shared__ float2 cs[HEAD_DIM / 2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = blockIdx.x;
  const int sub = (int)threadIdx.x / ROPE_LANES, i = (int)threadIdx.x % ROPE_LANES;
  const int h0 = (int)blockIdx.y * ROPE_BLOCK_HEADS + sub;
  const int rows = p.q_heads + 2 * p.kv_heads;
  const int n_rot = p.rot_dim / 16;     // threads of a head that rotate
  const bool half = p.layout == ATTN_F16_ROPE_HALF;
  // This thread's two 16-byte vectors of 8 numbers, whether they turn, and where
  // the four pairs whose angles each needs first stand in `cs`: there, pairs that
  // the threads of a head need at the same time are neighbours.
  int va, vb, ca, cb, step;
  bool turn_a, turn_b;
  if (half) {
    turn_a = turn_b = i < n_rot;
    va = turn_a ? i : n_rot + i;                 // the rest begins at vector 2 n_rot
    vb = turn_a ? i + n_rot : 16 + i;
    ca = i;                                      // pair 8i + k at 16k + i
    cb = i + 64;
    step = 16;
  } else {
    va = i;
    vb = i + 16;
    turn_a = va < 2 * n_rot;
    turn_b = vb < 2 * n_rot;
    ca = va;                                     // pair 4v + k at 32k + v
    cb = vb;
    step = 32;
  }
  int64_t slot = -1, page = 0, row = 0;
  if (p.kv_heads > 0) {
    slot = p.slots[t];
    if (slot >= p.num_slots || slot < -1) {
      if (threadIdx.x == 0) report(p.status, GEMM_F16_ERR_BAD_INDEX);
      slot = -1;
    }
    page = slot / p.page_size;
    row = slot - page * p.page_size;
  }
  uint4 xa[ROPE_EACH], xb[ROPE_EACH];
#pragma unroll
  for (int e = 0; e < ROPE_EACH; ++e) {
    const int r = h0 + e * ROPE_HEADS;
    if (r < rows && (r < p.q_heads || slot >= 0)) {
      const __half* src;
      if (r < p.q_heads)
        src = p.Q + t * p.q_st[0] + (int64_t)r * p.q_st[1];
      else if (r < p.q_heads + p.kv_heads)
        src = p.K + t * p.k_st[0] + (int64_t)(r - p.q_heads) * p.k_st[1];
      else
        src = p.V + t * p.v_st[0] + (int64_t)(r - p.q_heads - p.kv_heads) * p.v_st[1];
      xa[e] = *reinterpret_cast<const uint4*>(src + va * 8);
      xb[e] = *reinterpret_cast<const uint4*>(src + vb * 8);
    }
  }
  if ((int)threadIdx.x < p.rot_dim / 2) {
    const uint64_t angle = p.turns[threadIdx.x] * (uint64_t)(int64_t)p.positions[t];
    const int32_t top = (int32_t)(uint32_t)(angle >> 32);   // 2^-32 turns, in [-1/2, 1/2)
    float s, c;
    sincospif((float)top * 0x1p-31f, &s, &c);
    const int pair = (int)threadIdx.x;
    cs[half ? (pair & 7) * 16 + (pair >> 3) : (pair & 3) * 32 + (pair >> 2)] =
        make_float2(c * p.factor, (p.inverse ? -s : s) * p.factor);
  }
  __syncthreads();
  float2 w[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (turn_a) w[k] = cs[ca + k * step];
    if (turn_b) w[4 + k] = cs[cb + k * step];
  }
#pragma unroll
  for (int e = 0; e < ROPE_EACH; ++e) {
    const int r = h0 + e * ROPE_HEADS;
    if (r < rows && (r < p.q_heads || slot >= 0)) {
      uint4 a = xa[e], b = xb[e];
      if (r < p.q_heads + p.kv_heads) {
        if (half) {
          if (turn_a) {
            a.x = rotate_pair(a.x, b.x, w[0], w[1], &b.x);
            a.y = rotate_pair(a.y, b.y, w[2], w[3], &b.y);
            a.z = rotate_pair(a.z, b.z, w[4], w[5], &b.z);
            a.w = rotate_pair(a.w, b.w, w[6], w[7], &b.w);
          }
        } else {
          if (turn_a)
            a = make_uint4(rotate_neighbours(a.x, w[0]), rotate_neighbours(a.y, w[1]),
                           rotate_neighbours(a.z, w[2]), rotate_neighbours(a.w, w[3]));
          if (turn_b)
            b = make_uint4(rotate_neighbours(b.x, w[4]), rotate_neighbours(b.y, w[5]),
                           rotate_neighbours(b.z, w[6]), rotate_neighbours(b.w, w[7]));
        }
      }
      __half* dst;
      if (r < p.q_heads)
        dst = p.Qo + t * p.qo_st[0] + (int64_t)r * p.qo_st[1];
      else if (r < p.q_heads + p.kv_heads)
        dst = p.Kc + page * p.kc_st[0] + row * p.kc_st[1] + (int64_t)(r - p.q_heads) * p.kc_st[2];
      else
        dst = p.Vc + page * p.vc_st[0] + row * p.vc_st[1] +
              (int64_t)(r - p.q_heads - p.kv_heads) * p.vc_st[2];
      *reinterpret_cast<uint4*>(dst + va * 8) = a;
      *reinterpret_cast<uint4*>(dst + vb * 8) = b;
    }
  }
}

bool off(const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) != 0; }

// The 32-bit integers of a buffer that a call reads or writes.
struct Ints {
  const int32_t* at;
  int64_t n;
};
bool meet(const Ints& a, const Ints& b) {
  return a.n > 0 && b.n > 0 && a.at < b.at + b.n && b.at < a.at + a.n;
}
// Whether it meets one of a table's rows (`wide` entries, `stride` apart).
bool meets_rows(const Ints& a, const int32_t* table, int rows, int64_t stride, int wide) {
  if (a.n <= 0) return false;
  const int64_t o = a.at - table;
  if (o < 0) return o + a.n > 0;
  const int64_t r = o / stride, in = o - r * stride;
  return r < rows && (in < wide || (r + 1 < rows && a.n > stride - in));
}

// Strides of [a][b][256] or [a][b][c][256] storage: positive and at least a
// head's length where the dimension's extent is above 1.
int check_strides(const int64_t* st, const int* extent, int n) {
  if (!st) return GEMM_F16_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && (st[i] < HEAD_DIM || st[i] >= ((int64_t)1 << 38)))
      return GEMM_F16_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && (st[i] & 7)) return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

template <typename Params>
cudaError_t launch(void (*kernel)(Params), dim3 grid, int threads, gemm_f16_stream_t stream,
                   const Params& prm) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, prm);
}

}  // namespace

extern "C" {

int attn_f16_paged_maps_validate(int batch, const int32_t* cached, const int32_t* added,
                                 const int32_t* block_table, int64_t table_stride, int max_pages,
                                 const int32_t* free_pages, int num_free,
                                 const int32_t* free_head, int page_size, int max_tokens,
                                 const int32_t* starts, const int32_t* kv_lens,
                                 const int32_t* positions, const int32_t* slots,
                                 const int32_t* free_head_out) {
  if (batch < 1 || batch > 65535 || max_pages < 1 || max_pages > (1 << 24) || page_size < 1 ||
      page_size > (1 << 20) || num_free < 0 || max_tokens < 0 || table_stride < max_pages)
    return GEMM_F16_ERR_INVALID_ARG;
  if (!cached || !added || !block_table || !free_head || !starts || !kv_lens || !free_head_out ||
      (num_free > 0 && !free_pages) || (max_tokens > 0 && (!positions || !slots)) ||
      free_head == free_head_out)
    return GEMM_F16_ERR_INVALID_ARG;
  const void* ptrs[] = {cached, added, block_table, free_pages, free_head,
                        starts, kv_lens, positions, slots, free_head_out};
  for (const void* ptr : ptrs)
    if (off(ptr, 3)) return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

int attn_f16_paged_maps_overlap(int batch, const int32_t* cached, const int32_t* added,
                                const int32_t* block_table, int64_t table_stride, int max_pages,
                                const int32_t* free_pages, int num_free, const int32_t* free_head,
                                int max_tokens, const int32_t* starts, const int32_t* kv_lens,
                                const int32_t* positions, const int32_t* slots,
                                const int32_t* free_head_out) {
  const Ints written[] = {{starts, (int64_t)batch + 1}, {kv_lens, batch}, {positions, max_tokens},
                          {slots, max_tokens}, {free_head_out, 1}};
  const Ints read[] = {{cached, batch}, {added, batch}, {free_pages, num_free}, {free_head, 1}};
  const int n = sizeof(written) / sizeof(written[0]);
  for (int i = 0; i < n; ++i) {
    for (int j = i + 1; j < n; ++j)
      if (meet(written[i], written[j])) return GEMM_F16_ERR_INVALID_ARG;
    for (const Ints& r : read)
      if (meet(written[i], r)) return GEMM_F16_ERR_INVALID_ARG;
    if (meets_rows(written[i], block_table, batch, table_stride, max_pages))
      return GEMM_F16_ERR_INVALID_ARG;
  }
  for (const Ints& r : read)
    if (meets_rows(r, block_table, batch, table_stride, max_pages)) return GEMM_F16_ERR_INVALID_ARG;
  return GEMM_F16_OK;
}

int attn_f16_paged_maps(gemm_f16_plan_t p, int batch, const int32_t* cached, const int32_t* added,
                        int32_t* block_table, int64_t table_stride, int max_pages,
                        const int32_t* free_pages, int num_free, const int32_t* free_head,
                        int page_size, int max_tokens, int32_t* starts, int32_t* kv_lens,
                        int32_t* positions, int32_t* slots, int32_t* free_head_out,
                        gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  int rc = attn_f16_paged_maps_validate(batch, cached, added, block_table, table_stride, max_pages,
                                        free_pages, num_free, free_head, page_size, max_tokens,
                                        starts, kv_lens, positions, slots, free_head_out);
  if (rc) return rc;
  // Each block reads all lengths while others write: no buffer may serve twice.
  rc = attn_f16_paged_maps_overlap(batch, cached, added, block_table, table_stride, max_pages,
                                   free_pages, num_free, free_head, max_tokens, starts, kv_lens,
                                   positions, slots, free_head_out);
  if (rc) return rc;
  DeviceGuard g(p->device);
  MapsParams prm;
  prm.batch = batch;
  prm.cached = cached;
  prm.added = added;
  prm.table = block_table;
  prm.table_stride = table_stride;
  prm.rows = (int64_t)max_pages * page_size;
  prm.free_pages = free_pages;
  prm.num_free = num_free;
  prm.free_head = free_head;
  prm.page_size = page_size;
  prm.max_tokens = max_tokens;
  prm.starts = starts;
  prm.kv_lens = kv_lens;
  prm.positions = positions;
  prm.slots = slots;
  prm.free_head_out = free_head_out;
  prm.status = p->status_dev;
  const unsigned grid = (unsigned)std::max<int64_t>(1, ceil_div(max_tokens, MAP_CHUNK));
  GF16_CUDA(launch(paged_maps_kernel, dim3(grid, 1, 1), MAP_THREADS, stream, prm),
            "launch paged_maps_kernel");
  return GEMM_F16_OK;
}

int attn_f16_rope_turns(const double* radians, int n, uint64_t* turns) {
  if (!radians || !turns || n < 0) return GEMM_F16_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586;
  for (int i = 0; i < n; ++i)
    if (!(radians[i] >= 0.0 && radians[i] < two_pi)) return GEMM_F16_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) turns[i] = (uint64_t)std::ldexp(radians[i] / two_pi, 64);
  return GEMM_F16_OK;
}

int attn_f16_rope_validate(int tokens, int q_heads, int kv_heads, int head_dim, int rot_dim,
                           int layout, float factor, const uint64_t* turns,
                           const int32_t* positions, const void* Q, const int64_t q_strides[2],
                           const void* Qo, const int64_t qo_strides[2], const void* K,
                           const int64_t k_strides[2], const void* V, const int64_t v_strides[2],
                           const int32_t* slots, const void* Kc, const int64_t kc_strides[3],
                           const void* Vc, const int64_t vc_strides[3], int num_pages,
                           int page_size) {
  if (tokens < 0 || q_heads < 0 || kv_heads < 0 || q_heads > 65535 || kv_heads > 65535 ||
      q_heads + kv_heads < 1 || head_dim != HEAD_DIM)
    return GEMM_F16_ERR_INVALID_ARG;
  if (rot_dim < 16 || rot_dim > HEAD_DIM || rot_dim % 16) return GEMM_F16_ERR_INVALID_ARG;
  if (layout != ATTN_F16_ROPE_HALF && layout != ATTN_F16_ROPE_INTERLEAVED)
    return GEMM_F16_ERR_INVALID_ARG;
  if (!(std::fabs(factor) <= 3.0e38f)) return GEMM_F16_ERR_INVALID_ARG;
  const bool any = tokens > 0;
  if (!turns || (any && !positions)) return GEMM_F16_ERR_INVALID_ARG;
  if (q_heads > 0 && any && (!Q || !Qo)) return GEMM_F16_ERR_INVALID_ARG;
  if (kv_heads > 0 && (num_pages < 1 || page_size < 1 || !Kc || !Vc))
    return GEMM_F16_ERR_INVALID_ARG;
  if (kv_heads > 0 && any && (!K || !V || !slots)) return GEMM_F16_ERR_INVALID_ARG;
  if (off(turns, 7) || off(positions, 3)) return GEMM_F16_ERR_MISALIGNED;
  int rc;
  if (q_heads > 0) {
    const int e[2] = {tokens, q_heads};
    if ((rc = check_strides(q_strides, e, 2)) || (rc = check_strides(qo_strides, e, 2))) return rc;
    if (off(Q, 15) || off(Qo, 15)) return GEMM_F16_ERR_MISALIGNED;
    if (Q == Qo && any &&
        ((tokens > 1 && q_strides[0] != qo_strides[0]) ||
         (q_heads > 1 && q_strides[1] != qo_strides[1])))
      return GEMM_F16_ERR_INVALID_ARG;
  }
  if (kv_heads > 0) {
    const int e[2] = {tokens, kv_heads}, ce[3] = {num_pages, page_size, kv_heads};
    if ((rc = check_strides(k_strides, e, 2)) || (rc = check_strides(v_strides, e, 2)) ||
        (rc = check_strides(kc_strides, ce, 3)) || (rc = check_strides(vc_strides, ce, 3)))
      return rc;
    if (off(K, 15) || off(V, 15) || off(Kc, 15) || off(Vc, 15) || off(slots, 3))
      return GEMM_F16_ERR_MISALIGNED;
  }
  return GEMM_F16_OK;
}

int attn_f16_rope(gemm_f16_plan_t p, int tokens, int q_heads, int kv_heads, int head_dim,
                  int rot_dim, int layout, int inverse, float factor, const uint64_t* turns,
                  const int32_t* positions, const void* Q, const int64_t q_strides[2], void* Qo,
                  const int64_t qo_strides[2], const void* K, const int64_t k_strides[2],
                  const void* V, const int64_t v_strides[2], const int32_t* slots, void* Kc,
                  const int64_t kc_strides[3], void* Vc, const int64_t vc_strides[3],
                  int num_pages, int page_size, gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  const int rc = attn_f16_rope_validate(tokens, q_heads, kv_heads, head_dim, rot_dim, layout,
                                        factor, turns, positions, Q, q_strides, Qo, qo_strides, K,
                                        k_strides, V, v_strides, slots, Kc, kc_strides, Vc,
                                        vc_strides, num_pages, page_size);
  if (rc) return rc;
  if (tokens == 0) return GEMM_F16_OK;
  DeviceGuard g(p->device);
  RopeParams prm = {};
  prm.q_heads = q_heads;
  prm.kv_heads = kv_heads;
  prm.rot_dim = rot_dim;
  prm.layout = layout;
  prm.inverse = inverse != 0;
  prm.factor = factor;
  prm.turns = turns;
  prm.positions = positions;
  prm.slots = slots;
  prm.Q = static_cast<const __half*>(Q);
  prm.K = static_cast<const __half*>(K);
  prm.V = static_cast<const __half*>(V);
  prm.Qo = static_cast<__half*>(Qo);
  prm.Kc = static_cast<__half*>(Kc);
  prm.Vc = static_cast<__half*>(Vc);
  for (int i = 0; i < 2; ++i) {
    if (q_heads > 0) {
      prm.q_st[i] = q_strides[i];
      prm.qo_st[i] = qo_strides[i];
    }
    if (kv_heads > 0) {
      prm.k_st[i] = k_strides[i];
      prm.v_st[i] = v_strides[i];
    }
  }
  for (int i = 0; i < 3 && kv_heads > 0; ++i) {
    prm.kc_st[i] = kc_strides[i];
    prm.vc_st[i] = vc_strides[i];
  }
  prm.page_size = kv_heads > 0 ? page_size : 1;
  prm.num_slots = kv_heads > 0 ? (int64_t)num_pages * page_size : 0;
  prm.status = p->status_dev;
  const dim3 grid((unsigned)tokens, (unsigned)ceil_div(q_heads + 2 * kv_heads, ROPE_BLOCK_HEADS), 1);
  GF16_CUDA(launch(rope_kernel, grid, ROPE_THREADS, stream, prm),
            "launch rope_kernel");
  return GEMM_F16_OK;
}

}  // extern "C"
