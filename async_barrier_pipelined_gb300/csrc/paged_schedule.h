// How the attention over a paged cache (paged_attn.cu) reads a step's
// lengths, which key blocks a tile of queries needs, where the copies of a
// block start and which keys a query sees.  Plain integer arithmetic, no CUDA
// types: the kernels and the host-side tests share it.
#pragma once

#include <stdint.h>

#include "schedule.h"

namespace gf16 {
namespace paged {

constexpr int BLOCK_KEYS = 128;  // keys per block

GF16_HD int imin(int a, int b) { return a < b ? a : b; }
GF16_HD int imax(int a, int b) { return a > b ? a : b; }
GF16_HD int64_t lmin(int64_t a, int64_t b) { return a < b ? a : b; }
GF16_HD int64_t lmax(int64_t a, int64_t b) { return a > b ? a : b; }

// One request of the step, with everything out of range cut off (`bad` then):
// 0 <= start, start + n <= total_q, 0 <= n <= max_q, 0 <= len <= rows.
struct Request {
  int start, n, len;
  bool bad;
};
GF16_HD Request read_request(int s0, int s1, int len, int total_q, int max_q, int64_t rows) {
  Request r;
  const int64_t room = lmin(rows, 2147483647 - 1024);  // positions and block ends stay in 32 bits
  r.bad = s0 < 0 || s1 < s0 || s1 > total_q || (int64_t)s1 - s0 > max_q || len < 0 || len > room;
  r.start = imin(imax(s0, 0), total_q);
  r.n = imin(imin(imax(s1, r.start), total_q) - r.start, max_q);
  r.len = (int)lmin(lmax(len, 0), room);
  return r;
}

// What the kernels need to know of a call's masks and pages.
struct Masks {
  int window, sinks;
};

// Key blocks that a tile of a request's new tokens i0 .. i1 (inclusive) looks
// at: the blocks of the first `sinks` keys that lie before the window, then
// fb, fb + 1, ...; nb in all, at least one (of a tile that sees no key, too,
// so that its rows are written).  `first` is the first key of the window of
// token i0, `end` one past the last key of token i1.
struct Span {
  int sblk, fb, nb;
  int first, end;
};
GF16_HD Span tile_span(const Request& r, int i0, int i1, const Masks& m) {
  Span s;
  const int p0 = r.len - r.n + i0, p1 = r.len - r.n + i1;  // positions, p1 < len
  s.end = imax(p1 + 1, 0);
  s.first = m.window > 0 ? (int)lmax(0, (int64_t)p0 - m.window + 1) : 0;
  s.first = imin(s.first, s.end);
  if (s.end == 0) {
    s.sblk = s.fb = 0;
    s.nb = 1;
    return s;
  }
  const int last = (s.end - 1) / BLOCK_KEYS;
  s.fb = imin(s.first / BLOCK_KEYS, last);
  s.sblk = 0;
  if (m.window > 0 && m.sinks > 0) s.sblk = imin((m.sinks - 1) / BLOCK_KEYS + 1, s.fb);
  s.nb = s.sblk + last - s.fb + 1;
  return s;
}
GF16_HD int span_block(const Span& s, int j) { return j < s.sblk ? j : s.fb + (j - s.sblk); }

// A block is copied in groups of `rows` keys (the largest power of two that
// divides the page size, at most a block): key group k0 .. k0 + rows - 1 of a
// tile with span s.  `need`: some query may see a key of it; groups that are
// not needed read as zeros.  The last needed group may hold keys past the end
// whose memory may hold anything: its copy starts `shift` rows early (before
// the page's first row it reads as zeros), so that key k0 + i sits in row
// i + shift of the group, its last row is the tile's last key, and no row
// past it is ever read.
struct Group {
  bool need;
  int shift;
};
GF16_HD Group key_group(const Span& s, int k0, int rows, const Masks& m) {
  Group g;
  const int left = s.end - k0;
  g.need = left > 0 && (m.window == 0 || k0 + rows > s.first || k0 < m.sinks);
  g.shift = left > 0 && left < rows ? rows - left : 0;
  return g;
}

// The key that row `r` of block `blk` holds, or -1 for a row of zeros (or of
// an earlier key a second time) in front of a shifted group.
GF16_HD int row_key(const Span& s, int blk, int r, int rows) {
  const int k0 = blk * BLOCK_KEYS + (r & ~(rows - 1));
  const int left = s.end - k0;
  const int shift = left > 0 && left < rows ? rows - left : 0;
  const int i = (r & (rows - 1)) - shift;
  return i < 0 || left <= 0 ? -1 : k0 + i;
}

// Whether the query at position p sees key k >= 0.
GF16_HD bool sees(int p, int k, const Masks& m) {
  return k <= p && (m.window == 0 || (int64_t)k > (int64_t)p - m.window || k < m.sinks);
}

// The tile rows (row n: new token n / group of the tile, whose first token
// stands at pos0) that see the key in row `r` of block `blk`: lo <= n < hi.
GF16_HD void rows_that_see(const Span& s, int blk, int r, int rows, int pos0, int group,
                           const Masks& m, int tile_rows, int* lo, int* hi) {
  const int k = row_key(s, blk, r, rows);
  *lo = 0;
  *hi = 0;
  if (k < 0) return;
  *lo = (int)lmin(lmax((int64_t)k - pos0, 0) * group, tile_rows);
  *hi = tile_rows;
  if (m.window > 0 && k >= m.sinks)
    *hi = (int)lmin(lmax((int64_t)k - pos0 + m.window, 0) * group, tile_rows);
}

// Bits a .. b - 1 of a word, a and b cut to 0 .. 32.
GF16_HD uint32_t bits(int a, int b) {
  const int lo = imin(imax(a, 0), 32), hi = imin(imax(b, 0), 32);
  const uint32_t below_hi = (uint32_t)(((uint64_t)1 << hi) - 1);
  const uint32_t below_lo = (uint32_t)(((uint64_t)1 << lo) - 1);
  return below_hi & ~below_lo;
}

// Which rows of block `blk` hold keys that the query at position p (of the
// tile of span s) sees, as 128 bits (right for groups of up to 128 rows).
GF16_HD void seen_words(const Span& s, int blk, int rows, int p, const Masks& m,
                        uint32_t (&see)[4]) {
  // Keys of the query's window and its sinks as rows lo .. hi - 1 and 0 .. sk - 1
  // of a block without a shifted group, cut to the block.
  const int k0 = blk * BLOCK_KEYS;
  const int hi = imin(imax(p - k0 + 1, 0), BLOCK_KEYS);
  int lo = 0, sk = 0;
  if (m.window > 0) {
    lo = (int)lmin(lmax((int64_t)p - k0 + 1 - m.window, 0), BLOCK_KEYS);
    sk = imin(imax(m.sinks - k0, 0), hi);
  }
#pragma unroll
  for (int w = 0; w < 4; ++w)
    see[w] = bits(lo - 32 * w, hi - 32 * w) | bits(-32 * w, sk - 32 * w);
  const int left = s.end - k0;
  if (left >= BLOCK_KEYS) return;
  if (left <= 0) {   // a tile that sees no key
#pragma unroll
    for (int w = 0; w < 4; ++w) see[w] = 0;
    return;
  }
  const int over = left & (rows - 1);
  const int gs = left - over;   // rows from here on: the last needed group, `shift` rows late
  if (over == 0) return;        // (hi ends the block's keys)
  const int shift = rows - over;
  uint64_t late0 = ((uint64_t)(see[1] & bits(gs - 32, BLOCK_KEYS)) << 32) | (see[0] & bits(gs, BLOCK_KEYS));
  uint64_t late1 = ((uint64_t)(see[3] & bits(gs - 96, BLOCK_KEYS)) << 32) | (see[2] & bits(gs - 64, BLOCK_KEYS));
  if (shift >= 64) {            // only with rows of 128: the chunk kernel's are at most 64
    late1 = late0 << (shift - 64);
    late0 = 0;
  } else {                      // shift >= 1
    late1 = (late1 << shift) | (late0 >> (64 - shift));
    late0 <<= shift;
  }
  see[0] = (see[0] & bits(0, gs)) | (uint32_t)late0;
  see[1] = (see[1] & bits(0, gs - 32)) | (uint32_t)(late0 >> 32);
  see[2] = (see[2] & bits(0, gs - 64)) | (uint32_t)late1;
  see[3] = (see[3] & bits(0, gs - 96)) | (uint32_t)(late1 >> 32);
}

// Whether every query of the tile (positions p0 .. p1) sees every key of the
// block, which then needs no mask.
GF16_HD bool block_is_full(int p0, int p1, int blk, const Masks& m) {
  const int k0 = blk * BLOCK_KEYS, k1 = k0 + BLOCK_KEYS - 1;
  return k1 <= p0 && (m.window == 0 || (int64_t)k0 > (int64_t)p1 - m.window || k1 < m.sinks);
}

// Work is a line of key blocks: of every request in order, its key/value
// heads, their tiles of tokens, and the tiles' blocks.  Worker w of `workers`
// takes blocks w * per .. (w + 1) * per - 1, so all have the same to do
// whatever the lengths are; a tile that is cut is merged from partial sums.
GF16_HD int64_t per_worker(int64_t blocks, int workers) {
  return lmax(1, (blocks + workers - 1) / workers);
}

// Where the large kernel deals out whole tiles first, as many of its `tiles` as
// make full rounds of the workers but one, so that the rest (one to two rounds)
// holds a tile for each of them; none with fewer than two rounds, or with more
// tiles than its prologue should add up.
constexpr int MOST_TILES = 16384;
GF16_HD int whole_tiles(int tiles, int workers) {
  return tiles > MOST_TILES || tiles < 2 * workers ? 0 : (tiles / workers - 1) * workers;
}

// The blocks of the rest bring every worker, `load` blocks of whole tiles before
// it, to a common level, and are one at least for each.  Shares at the level
// deal_level_enough are enough for the rest; where they are more than it, the
// last workers give the difference up: worker c's share begins `before` blocks
// (the shares of those before it) into the rest, or as far as leaves a block to
// each worker from it on.
GF16_HD int deal_share(int level, int load) { return imax(1, level - load); }
GF16_HD int deal_level_enough(int most_load, int rest, int workers) {
  return most_load + (rest + workers - 1) / workers;
}
// The lowest level above the `least` load at which the shares of all workers,
// shares(level), are enough for the rest.
#ifdef __CUDACC__
#pragma nv_exec_check_disable
#endif
template <typename Shares>
GF16_HD int deal_level(int least, int most, int rest, int workers, const Shares& shares) {
  int lo = least, hi = deal_level_enough(most, rest, workers);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (shares(mid) < rest) lo = mid; else hi = mid;
  }
  return hi;
}
GF16_HD int deal_start(int before, int rest, int workers, int c) {
  return imin(before, rest - (workers - c));
}

// Partial sums: at most two per worker, of the tile that its range begins in
// (slot 2w) and of the one that it ends in (slot 2w + 1) if that is another.
// The parts of a tile whose blocks are L .. L + nb - 1 belong to the workers
// L / per .. (L + nb - 1) / per.
GF16_HD int part_slot(int64_t L, int64_t per, int w) {
  return 2 * w + ((int64_t)w * per < L ? 1 : 0);
}

}  // namespace paged
}  // namespace gf16
