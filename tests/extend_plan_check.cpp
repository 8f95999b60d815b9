// The planner's arithmetic over drawn calls: prints one line for each call whose
// items or partial rows do not fit their room, or whose parts do not cover a query
// tile's KV tiles exactly once.  Arguments: seed, number of calls, kv heads (0: drawn).
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "extend_plan.h"

using namespace pkv::plan;

struct Sequence {
  int q_len, ctx;
};

static int failures = 0;
static int64_t most_items = 0, most_rows = 0;    // per mille of the room beside one item a tile / of the rows

static void check(const std::vector<Sequence>& seqs, int group, int hkv, int sms, int window, int ring, int bs) {
  const int pair = pair_positions(group);
  int64_t num_tokens = 0, tiles = 0, work = 0;
  int max_q = 0;
  struct T {
    int tile0, n, npos, first, last, n_last;
    int64_t seq_rows;
  };
  std::vector<T> list;
  for (const Sequence& s : seqs) {
    num_tokens += s.q_len;
    max_q = std::max(max_q, s.q_len);
    const int64_t h = ring ? ((int64_t)((s.ctx - 1) / bs) - ring + 1) * bs : 0;
    const int held = h > 0 ? (int)h : 0, nt = tiles_of(s.q_len, pair);
    for (int i = 0; i < nt; ++i) {
      T t;
      t.npos = std::min(pair, s.q_len - i * pair);
      const int pos0 = s.ctx - s.q_len + i * pair;
      t.n = tile_range(pos0, t.npos, window, held, t.tile0);
      int unused;
      t.n_last = tile_range(s.ctx - s.q_len + (nt - 1) * pair, s.q_len - (nt - 1) * pair, window, held, unused);
      t.seq_rows = (int64_t)nt * std::min(pair, s.q_len) * group * hkv;
      // the same from the definition: positions attended by any query of the tile
      t.first = INT32_MAX;
      t.last = -1;
      for (int p = pos0; p < pos0 + t.npos; ++p) {
        const int from = std::max(held, window ? std::max(0, p - window + 1) : 0);
        if (from > p) continue;
        t.first = std::min(t.first, from);
        t.last = std::max(t.last, p);
      }
      list.push_back(t);
      work += t.n;
    }
    tiles += nt;
  }
  const int64_t longest = longest_part(work, tiles, hkv, sms);
  const int tile_rows = std::min(max_q, pair) * group;
  const int64_t room = max_items(max_tiles((int)num_tokens, (int)seqs.size(), pair), sms), row_room = max_rows(tile_rows, sms);
  int64_t items = 0, rows = 0;
  bool covered = tiles <= max_tiles((int)num_tokens, (int)seqs.size(), pair);
  for (const T& t : list) {
    const int parts = parts_of(t.n, t.n_last, t.seq_rows, longest, (int64_t)1 << 60), chosen = parts_of(t.n, t.n_last, t.seq_rows, longest, row_room);
    if (chosen != parts && chosen != 1) covered = false;     // cut as its length asks, or whole
    items += parts;
    if (parts > 1) rows += (int64_t)parts * t.npos * group * hkv;
    int at = 0;
    for (int k = 0; k < parts; ++k) {
      int from;
      const int n = part_range(t.n, parts, k, from);
      if (n > 0 && from != at) covered = false;
      if (n == 0 && parts > 1) covered = false;              // an empty part
      if (n > longest) covered = false;
      at += n;
    }
    if (at != t.n) covered = false;
    if (t.last >= 0 && (t.first / kKv < t.tile0 || t.last / kKv != t.tile0 + t.n - 1)) covered = false;
  }
  most_items = std::max(most_items, 1000 * (items - tiles) / (max_items(0, sms)));
  most_rows = std::max(most_rows, 1000 * rows / row_room);
  if (items > room || rows > row_room || !covered) {
    ++failures;
    printf("group %d, %d kv heads, %d SMs, window %d, ring %d, %zu sequences (first %d of %d): %lld items (room %lld), %lld rows (room %lld)%s\n",
           group, hkv, sms, window, ring, seqs.size(), seqs[0].q_len, seqs[0].ctx, (long long)items, (long long)room, (long long)rows,
           (long long)row_room, covered ? "" : ", not covered");
  }
}

int main(int argc, char** argv) {
  std::mt19937_64 rng(atoi(argv[1]));
  const int calls = atoi(argv[2]), heads = atoi(argv[3]);
  auto upto = [&](int64_t n) { return (int)(rng() % (uint64_t)n) + 1; };
  auto log_upto = [&](int64_t n) { return std::min<int64_t>(n, upto(std::max<int64_t>(1, n >> (rng() % 18)))); };
  const int hs[] = {1, 1, 1, 2, 3, 4, 8, 32}, sms_of[] = {152, 152, 152, 148, 132, 20, 1};
  for (int g : {4, 8, 8, 16, 1}) {                                  // long prompts and chunks of one kv head
    check({{8192, 8192}}, g, 1, 152, 0, 0, 16);
    check({{1483, 1483 + 22277}}, g, 1, 152, 0, 0, 16);
    check({{4880, 4880}}, g, 1, 152, 0, 0, 16);
    check({{7057, 7057}}, g, 1, 152, 0, 0, 16);
    check({{21000, 21000}}, g, 1, 152, 0, 0, 16);
    check({{32768, 131072}}, g, 1, 152, 0, 0, 16);
  }
  for (int i = 0; i < calls; ++i) {
    const int group = upto(16), hkv = heads ? heads : hs[rng() % 8], sms = sms_of[rng() % 7];
    const int window = rng() % 3 ? 0 : (int)log_upto(20000), bs = 1 << (rng() % 6);
    const int n = (int)log_upto(60), longest = (int)log_upto(40000 / n + 1);
    std::vector<Sequence> seqs;
    for (int s = 0; s < n; ++s) {
      const int q = (int)log_upto(longest);
      seqs.push_back({q, q + (rng() % 3 ? (int)log_upto(130000) : 0)});
    }
    const int ring = window && rng() % 2 ? upto((window + longest) / bs + 2) : 0;
    check(seqs, group, hkv, sms, window, ring, bs);
  }
  printf("%d failures; beyond one item a tile %lld/1000 of the room, rows %lld/1000\n", failures, (long long)most_items, (long long)most_rows);
  return failures != 0;
}
