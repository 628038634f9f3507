// Host-side checks of paged_schedule.h: what the kernels read of a step's
// lengths, which blocks, pages and rows their copies touch, and which keys
// their masks let through, against plain loops over every key.
// Prints "ok <cases>" or the first thing that is wrong.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "paged_schedule.h"

using namespace gf16::paged;

#define CHECK(c)                                                                        \
  do {                                                                                  \
    if (!(c)) {                                                                         \
      std::printf("line %d: %s\n", __LINE__, #c);                                       \
      std::exit(1);                                                                     \
    }                                                                                   \
  } while (0)

static void check_tile(const Request& r, int i0, int i1, const Masks& m, int page_size, int group) {
  const int rows = std::min(page_size & -page_size, BLOCK_KEYS);
  const Span s = tile_span(r, i0, i1, m);
  const int p0 = r.len - r.n + i0, p1 = r.len - r.n + i1;
  CHECK(s.nb >= 1 && s.sblk >= 0 && s.sblk <= s.nb && s.end >= 0 && s.end <= r.len);
  std::map<int, std::pair<int, int>> where;
  std::set<int> blocks;
  for (int j = 0; j < s.nb; ++j) {
    const int blk = span_block(s, j);
    CHECK(blk >= 0 && blocks.insert(blk).second);
    bool all = true;
    for (int g = 0; g < BLOCK_KEYS / rows; ++g) {
      const int k0 = blk * BLOCK_KEYS + g * rows;
      const Group grp = key_group(s, k0, rows, m);
      CHECK(grp.shift >= 0 && grp.shift < rows);
      if (grp.need) {
        // the copied rows lie in the page and before the tile's end
        const int row = k0 % page_size - grp.shift;
        CHECK(k0 % page_size + rows <= page_size && row + rows <= page_size && row > -rows);
        CHECK(k0 - grp.shift + rows <= s.end && k0 < r.len);
      }
      bool any = false;
      for (int i = 0; i < rows; ++i) {
        const int br = g * rows + i, k = row_key(s, blk, br, rows);
        if (k < 0) {
          all = false;
        } else {
          CHECK(k < s.end && k >= k0 && k < k0 + rows);
          CHECK(i - grp.shift == k - k0);
          for (int t = i0; t <= i1; ++t) {
            const bool v = sees(r.len - r.n + t, k, m);
            any |= v;
            all &= v;
          }
          CHECK(where.emplace(k, std::make_pair(blk, br)).second);
        }
        int lo, hi;
        const int tile_rows = (i1 - i0 + 1) * group;
        rows_that_see(s, blk, br, rows, p0, group, m, tile_rows, &lo, &hi);
        for (int n = 0; n < tile_rows; ++n)
          CHECK((n >= lo && n < hi) == (k >= 0 && sees(p0 + n / group, k, m)));
      }
      CHECK(!any || grp.need);
    }
    CHECK(!block_is_full(p0, p1, blk, m) || all);
    for (int t = i0; t <= i1; ++t) {
      const int p = r.len - r.n + t;
      uint32_t see[4];
      seen_words(s, blk, rows, p, m, see);
      for (int w = 0; w < 4; ++w) {
        const uint32_t word = see[w];
        for (int i = 0; i < 32; ++i) {
          const int k = row_key(s, blk, 32 * w + i, rows);
          CHECK(((word >> i) & 1u) == (k >= 0 && sees(p, k, m) ? 1u : 0u));
        }
      }
    }
  }
  for (int k = 0; k < r.len; ++k) {
    bool any = false;
    for (int t = i0; t <= i1; ++t) any |= sees(r.len - r.n + t, k, m);
    CHECK(!any || where.count(k));
  }
}

// The line dealt out to workers: every block once, parts where they are said to be.
static void check_line(const std::vector<int>& tiles, int workers) {
  int64_t total = 0;
  for (int nb : tiles) total += nb;
  const int64_t per = per_worker(total, workers);
  CHECK(per * workers >= total);
  std::map<int, int> slot_users;
  int64_t L = 0;
  for (int nb : tiles) {
    const int c0 = (int)(L / per), c1 = (int)((L + nb - 1) / per);
    CHECK(c1 < workers);
    int64_t done = 0;
    for (int c = c0; c <= c1; ++c) {
      const int64_t a = std::max<int64_t>(L, c * per), b = std::min<int64_t>(L + nb, (c + 1) * per);
      CHECK(b > a);
      done += b - a;
      if (b - a < nb) {
        const int slot = part_slot(L, per, c);
        CHECK(slot == (c == c0 ? part_slot(L, per, c0) : 2 * c));
        CHECK(slot < 2 * workers && ++slot_users[slot] == 1);
      }
    }
    CHECK(done == nb);
    L += nb;
  }
}

// Whole tiles in turn, the rest by blocks to a common level.
static void check_deal(const std::vector<int>& tiles, int workers) {
  const int n = (int)tiles.size(), whole = whole_tiles(n, workers);
  CHECK(whole % workers == 0 && (whole == 0) == (n < 2 * workers || n > MOST_TILES));
  if (whole == 0) return;
  CHECK(n - whole >= workers && n - whole < 2 * workers);
  std::vector<int> load(workers, 0), start(workers + 1);
  int dealt = 0, rest = 0, biggest = 0;
  for (int i = 0; i < n; ++i) {
    biggest = std::max(biggest, tiles[i]);
    if (i < whole) {
      load[i % workers] += tiles[i];
      dealt += tiles[i];
    } else {
      rest += tiles[i];
    }
  }
  const int least = *std::min_element(load.begin(), load.end());
  const int most = *std::max_element(load.begin(), load.end());
  auto shares = [&](int level) {
    int64_t sum = 0;
    for (int l : load) sum += deal_share(level, l);
    return sum;
  };
  int lo = least, hi = deal_level_enough(most, rest, workers);
  CHECK(shares(hi) >= rest);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (shares(mid) < rest) lo = mid; else hi = mid;
  }
  CHECK(shares(hi) >= rest);
  int before = 0;
  for (int c = 0; c < workers; ++c) {
    start[c] = dealt + deal_start(before, rest, workers, c);
    before += deal_share(hi, load[c]);
  }
  start[workers] = dealt + rest;
  CHECK(start[0] == dealt);
  for (int c = 0; c < workers; ++c) {
    const int share = start[c + 1] - start[c];
    CHECK(share >= 1);
    CHECK(load[c] + share <= std::max(hi, most + 1));   // nobody is over the level
  }
  // Parts: slot 2c + 1 of the tile that worker c begins, 2c of one begun before.
  std::map<int, int> slot_users;
  int L = dealt;
  for (int i = whole; i < n; L += tiles[i], ++i) {
    int c0 = 0, done = 0;
    while (start[c0 + 1] <= L) ++c0;
    int last = c0;
    while (start[last + 1] < L + tiles[i]) ++last;
    CHECK(last < workers);
    for (int c = c0; c <= last; ++c) {
      const int a = std::max(L, start[c]), b = std::min(L + tiles[i], start[c + 1]);
      CHECK(b > a);
      done += b - a;
      if (b - a < tiles[i]) CHECK(++slot_users[2 * c + (a == L ? 1 : 0)] == 1);
      CHECK((a == L) == (c == c0));
    }
    CHECK(done == tiles[i]);
  }
}

int main() {
  std::mt19937 rng(1);
  auto pick = [&](int a, int b) { return (int)(a + rng() % (unsigned)(b - a + 1)); };
  int cases = 0;
  const int pages[] = {8, 16, 24, 32, 40, 48, 64, 96, 128, 136, 256, 1000};
  for (int i = 0; i < 3000; ++i, ++cases) {
    Request r{0, pick(1, 40), 0, false};
    r.len = pick(0, 4) == 0 ? pick(0, r.n) : r.n + pick(0, 700);
    const int i0 = pick(0, r.n - 1), i1 = pick(i0, r.n - 1);
    const Masks masks[] = {{0, 0}, {0, 7}, {pick(1, 300), 0}, {pick(1, 300), pick(1, 300)},
                           {1, 1}, {2147483647, 2147483647}, {pick(100, 2000), 4}};
    check_tile(r, i0, i1, masks[pick(0, 6)], pages[pick(0, 11)], pick(1, 9));
  }
  for (int i = 0; i < 2000; ++i, ++cases) {
    std::vector<int> tiles(pick(1, 60));
    for (int& t : tiles) t = pick(1, pick(1, 3) == 1 ? 200 : 4);
    check_line(tiles, pick(1, 160));
  }
  for (int i = 0; i < 2000; ++i, ++cases) {
    const int workers = pick(1, 128);
    std::vector<int> tiles(pick(0, 5) == 0 ? pick(1, 300) : workers * pick(2, 9) + pick(-1, workers));
    const int mode = pick(0, 3);
    for (size_t t = 0; t < tiles.size(); ++t)
      tiles[t] = mode == 0 ? 1 : mode == 1 ? pick(1, 300) : mode == 2 ? 1 + (int)t % 40
                                                               : (t + 1 == tiles.size() ? 100000 : 1);
    check_deal(tiles, workers);
  }
  const int edge[] = {-2147483647 - 1, -5, -1, 0, 1, 7, 100, 2147483000, 2147483647};
  for (int s0 : edge)
    for (int s1 : edge)
      for (int len : edge)
        for (int total : {0, 1, 100, 2147483647})
          for (int most : {0, 1, 50, 2147483647})
            for (int64_t rows : {(int64_t)8, (int64_t)4096, (int64_t)1 << 39}) {
              const Request r = read_request(s0, s1, len, total, most, rows);
              CHECK(r.start >= 0 && r.n >= 0 && r.n <= most && (int64_t)r.start + r.n <= total);
              CHECK(r.len >= 0 && r.len <= rows);
              const bool good = s0 >= 0 && s1 >= s0 && s1 <= total && (int64_t)s1 - s0 <= most &&
                                len >= 0 && len <= rows && len <= 2147483647 - 1024;
              CHECK(r.bad == !good);
              if (good) CHECK(r.start == s0 && r.n == s1 - s0 && r.len == len);
              for (const Masks& m : {Masks{0, 0}, Masks{5, 2}, Masks{2147483647, 2147483647}})
                if (r.n > 0) {
                  const Span s = tile_span(r, 0, r.n - 1, m);
                  CHECK(s.nb >= 1 && s.end <= r.len && s.first >= 0);
                  const int blk = span_block(s, s.nb - 1);
                  CHECK(blk >= 0 && (s.end == 0 || blk * (int64_t)BLOCK_KEYS < s.end));
                }
              ++cases;
            }
  std::printf("ok %d\n", cases);
  return 0;
}
