// Host-side check of deal_level (paged_schedule.h): the lowest level above the
// least load at which the workers' shares are enough for the rest, against a
// plain walk over the levels.  Prints "ok <cases>" or the first thing wrong.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "paged_schedule.h"

using namespace gf16::paged;

int main() {
  std::mt19937 rng(2);
  auto pick = [&](int a, int b) { return (int)(a + rng() % (unsigned)(b - a + 1)); };
  int cases = 0;
  for (; cases < 20000; ++cases) {
    const int workers = pick(1, 128), spread = pick(0, 2) == 0 ? 0 : pick(0, 60);
    std::vector<int> load(workers);
    for (int& l : load) l = 12 + pick(0, spread);
    const int rest = workers + pick(0, pick(0, 1) ? 40 * workers : 3);
    auto shares = [&](int level) {
      int sum = 0;
      for (int l : load) sum += deal_share(level, l);
      return sum;
    };
    const int least = *std::min_element(load.begin(), load.end());
    const int most = *std::max_element(load.begin(), load.end());
    int want = least + 1;
    while (shares(want) < rest) ++want;
    const int got = deal_level(least, most, rest, workers, shares);
    if (got != want) {
      std::printf("case %d: level %d, not %d\n", cases, got, want);
      return 1;
    }
  }
  std::printf("ok %d\n", cases);
  return 0;
}
