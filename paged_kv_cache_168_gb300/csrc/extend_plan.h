// extend_plan.h -- how pa_extend's work is cut into items: plain arithmetic, the
// same for the planner kernel, the layout of its workspace and a host program.
//
// A sequence's new tokens are query tiles of `pair` positions (two tiles of 128
// rows, row = position * group + head); tile i attends n_i KV tiles of 128 tokens
// and is cut into ceil(n_i / longest) parts.  With W = sum of n_i over the call's
// query tiles, longest is at least W * hkv / want for some want <= kPartsPerSm *
// sms.  So
//   parts beyond the first of their tile: sum (ceil(n_i / longest) - 1) <= W /
//     longest <= want / hkv, which is what the item list has room for beside one
//     item a tile;
//   parts of cut tiles (n_i > longest): ceil(n_i / longest) < 2 n_i / longest, in
//     all at most 2 want / hkv; with hkv heads of at most tile_rows rows each, the
//     partial results are at most 2 want tile_rows rows.
// Both hold for any lengths, so no item is ever without room.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PKV_PLAN __host__ __device__ __forceinline__
#else
#define PKV_PLAN inline
#endif

namespace pkv {
namespace plan {

constexpr int kRows = 128;                 // MMA M: rows of one query tile
constexpr int kKv = 128;                   // tokens of a KV tile
constexpr int kMinPartTiles = 2;           // shortest part of a split context (1, 2 or 4: the same within 2%)
constexpr int kPartsPerSm = 4;             // most parts wanted per SM where contexts are split

// Positions of an item: two query tiles.
PKV_PLAN int pair_positions(int group) { return 2 * (kRows / group); }

// Query tiles of q_len tokens.
PKV_PLAN int tiles_of(int q_len, int pair) { return (q_len + pair - 1) / pair; }

// First position that the query at position pos attends.
PKV_PLAN int attend_from(int pos, int window, int held) {
  const int w = window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0;
  return w > held ? w : held;
}

// KV tiles [tile0, tile0 + n) that the queries at pos0 .. pos0 + npos - 1 attend.
PKV_PLAN int tile_range(int pos0, int npos, int window, int held, int& tile0) {
  const int first = attend_from(pos0, window, held), last = pos0 + npos - 1;
  tile0 = first / kKv;
  return first > last ? 0 : last / kKv - tile0 + 1;
}

// Most query tiles of num_seqs sequences of num_tokens tokens together (each
// sequence's last one may be shorter), items, and rows of partial results.
PKV_PLAN int64_t max_tiles(int num_tokens, int num_seqs, int pair) { return (int64_t)num_tokens / pair + num_seqs; }
PKV_PLAN int64_t max_items(int64_t tiles, int sms) { return tiles + (int64_t)kPartsPerSm * sms; }
PKV_PLAN int64_t max_rows(int tile_rows, int sms) { return 2 * (int64_t)kPartsPerSm * sms * tile_rows; }

// The part length in KV tiles, from the `work` (KV tiles) of all `tiles` query
// tiles together.  With K parts a SM the call takes about (work / sms) (1 + 1 / K)
// -- the last round is half empty -- and K times an item's own cost, about 3 KV
// tiles: least at K = sqrt(work / sms / 3).  32 + 8 heads, us, this rule / K = 1 /
// K = 4: 4 tokens over 30000: 56 / 48 / 75; 4 x 4 over 8000: 51 / 59 / 61; 2 x 512
// over 8000, 8 + 1 heads: 84 / 83 / 104; 8 x 4 over 32K to 128K, 64 + 8 heads: 543 /
// 736 / 543.
PKV_PLAN int64_t longest_part(int64_t work, int64_t tiles, int hkv, int sms) {
  const int64_t per_sm = work * hkv / sms;
  const int64_t want = (int64_t)(per_sm >= 48 ? kPartsPerSm : per_sm >= 27 ? 3 : per_sm >= 12 ? 2 : 1) * sms;
  int64_t longest = (work * hkv + want - 1) / want;
  if (longest < kMinPartTiles) longest = kMinPartTiles;
  // Query tiles that cover half of the SMs are not cut for less than a dozen KV tiles (13
  // chunks over windows of 1000 tokens: 43 us, cut 81).
  if (tiles * hkv * 2 >= sms && longest < 12) longest = 12;
  return longest;
}

// Parts of a query tile that attends n KV tiles, of a sequence whose last query
// tile attends n_last and whose tiles have seq_rows rows together (all heads).  A
// sequence stays whole if its tiles, were all cut like the last, would leave more
// partial rows than there is room for: it has tiles enough to keep the SMs busy, and
// merging costs more than it gives (prompts, us, whole / cut: 4096 tokens of 32 + 8
// heads 160 / 252, 8192 of 8 + 2 196 / 222; but 1483 tokens over 22277, 8 + 1 heads,
// which are below the limit: 303 / 182).
PKV_PLAN int parts_of(int n, int n_last, int64_t seq_rows, int64_t longest, int64_t row_room) {
  if (n <= longest || (n_last + longest - 1) / longest * seq_rows > row_room) return 1;
  return (int)((n + longest - 1) / longest);
}

// Part `part` of n KV tiles in `parts` parts: `from` on, that many (equal but for
// the last; none is empty when n > 0).
PKV_PLAN int part_range(int n, int parts, int part, int& from) {
  const int len = (n + parts - 1) / parts;
  from = part * len;
  const int left = n - from;
  return left < 0 ? 0 : left < len ? left : len;
}

}  // namespace plan
}  // namespace pkv
