// The planner's arithmetic where KV tiles come from spans of each query (any number of them a query tile): prints one line for
// each drawn call whose items or partial rows do not fit their room.  Arguments: seed, number of calls.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "extend_plan.h"

using namespace pkv::plan;

int main(int argc, char** argv) {
  (void)argc;
  std::mt19937_64 rng(atoi(argv[1]));
  auto upto = [&](int64_t n) { return (int64_t)(rng() % (uint64_t)n) + 1; };
  auto log_upto = [&](int64_t n) { return upto(std::max<int64_t>(1, n >> (rng() % 18))); };
  int failures = 0;
  for (int call = 0; call < atoi(argv[2]); ++call) {
    const int group = (int)upto(16), pair = pair_positions(group), hkv = (int)log_upto(64), sms = (int)(rng() % 2 ? 152 : upto(200));
    const int n = (int)log_upto(60);
    int64_t num_tokens = 0, tiles = 0, work = 0;
    int max_q = 0;
    struct T {
      int n, npos;
      int64_t seq_rows;
    };
    std::vector<T> list;
    for (int s = 0; s < n; ++s) {
      const int q = (int)log_upto(40000 / n + 1), nt = tiles_of(q, pair);
      num_tokens += q;
      max_q = std::max(max_q, q);
      tiles += nt;
      const int most = (int)log_upto(2000);
      for (int i = 0; i < nt; ++i) {
        const int kv = rng() % 4 ? (int)upto(most) : 0;              // (0: no query of the tile attends anything)
        list.push_back({kv, std::min(pair, q - i * pair), (int64_t)nt * std::min(pair, q) * group * hkv});
        work += kv;
      }
    }
    const int64_t longest = longest_part(work, tiles, hkv, sms), row_room = max_rows(std::min(max_q, pair) * group, sms);
    int64_t items = 0, rows = 0;
    bool covered = true;
    for (const T& t : list) {
      const int parts = parts_of(t.n, t.n, t.seq_rows, longest, row_room);
      items += parts;
      if (parts > 1) rows += (int64_t)parts * t.npos * group * hkv;
      int at = 0;
      for (int k = 0; k < parts; ++k) {
        int from;
        const int len = part_range(t.n, parts, k, from);
        if ((len > 0 && from != at) || (len == 0 && parts > 1)) covered = false;
        at += len;
      }
      if (at != t.n) covered = false;
    }
    if (items > max_items(max_tiles((int)num_tokens, n, pair), sms) || rows > row_room || !covered) {
      ++failures;
      printf("call %d: group %d, %d kv heads, %d SMs: %lld items, %lld rows (room %lld)%s\n", call, group, hkv, sms, (long long)items,
             (long long)rows, (long long)row_room, covered ? "" : ", not covered");
    }
  }
  return failures != 0;
}
