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

// Bits a .. b - 1 (cut to 0 .. 31) of a word.
GF16_HD uint32_t bits(int64_t a, int64_t b) {
  const int lo = (int)lmin(lmax(a, 0), 32), hi = (int)lmin(lmax(b, 0), 32);
  if (lo >= hi) return 0;
  return (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
}

// The rows 32 * word .. + 31 of block `blk` whose keys the query at position
// p (of the tile of span s) sees, as bits.
GF16_HD uint32_t seen_word(const Span& s, int blk, int word, int rows, int p, const Masks& m) {
  // Keys of the query's window and its sinks, as row numbers of an unshifted block.
  const int64_t k0 = (int64_t)blk * BLOCK_KEYS;
  const int64_t lo = m.window > 0 ? (int64_t)p - m.window + 1 - k0 : 0, hi = (int64_t)p + 1 - k0;
  const int64_t sk = m.window > 0 ? lmin(m.sinks, (int64_t)p + 1) - k0 : 0;
  // Rows before the last needed group are unshifted; that group (its first
  // row gs) has its keys `shift` rows later.
  const int64_t left = s.end - k0;
  int64_t gs = BLOCK_KEYS, shift = 0;
  if (left > 0 && left < BLOCK_KEYS && left % rows) {
    gs = left - left % rows;
    shift = rows - left % rows;
  } else if (left <= 0) {
    gs = 0;
    shift = BLOCK_KEYS;
  }
  const int64_t w0 = 32 * word;
  const uint32_t plain =
      (bits(lo - w0, hi - w0) | bits(-w0, sk - w0)) & bits(-w0, gs - w0);
  const uint32_t late = (bits(lmax(lo, gs) + shift - w0, hi + shift - w0) |
                         bits(gs + shift - w0, sk + shift - w0)) &
                        bits(gs + shift - w0, gs + rows - w0);
  return plain | (gs < BLOCK_KEYS ? late : 0u);
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

// Partial sums: at most two per worker, of the tile that its range begins in
// (slot 2w) and of the one that it ends in (slot 2w + 1) if that is another.
// The parts of a tile whose blocks are L .. L + nb - 1 belong to the workers
// L / per .. (L + nb - 1) / per.
GF16_HD int part_slot(int64_t L, int64_t per, int w) {
  return 2 * w + ((int64_t)w * per < L ? 1 : 0);
}

}  // namespace paged
}  // namespace gf16
