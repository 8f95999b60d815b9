// extend_tc.cuh -- attention of a chunk of new tokens per sequence over any paged
// cache, on the tensor cores (tcgen05 + TMEM); instantiated by extend_tc.cu (plain
// scores), extend_spans.cu, extend_cap.cu, extend_slopes.cu and extend_scored.cu
// (shaped scores, below).
//
// Sequence s owns the packed query tokens query_start_loc[s] .. [s + 1]; query j
// of its q_len sits at position ctx - q_len + j and attends the positions from
// its window's (or ring's) start up to its own.  Three launches:
//
//   plan_kernel    one CTA: from the lengths, the list of work items in the
//                  workspace.  An item is up to two query tiles of 128 rows (row
//                  = position * group + head) of one sequence, over its context
//                  or a part of it; contexts are cut only where the whole call
//                  has too few items for the SMs (extend_plan.h).
//   extend_kernel  one persistent CTA per SM draws (item, kv head) pairs from a
//                  counter, a sequence's heads and tiles next to each other so
//                  that its K and V are read from L2 while they are hot.
//   finish_kernel  merges parts by log-sum-exp, zeroes the rows of items with a
//                  bad block id, and recomputes on CUDA cores the items whose
//                  results are not finite: an infinite or NaN V reaches rows that
//                  do not attend it through the second product (0 * NaN = NaN).
//
// extend_kernel, per 128-token KV tile c and query tile t (0 or 1):
//     S_t  = Q_t K_c^T     (M = 128 rows, N = 128 tokens, K = D)  -> TMEM (fp32)
//     O_t += P_t V_c       (M = 128 rows, N = D, K = 128 tokens)  -> TMEM (fp32)
// P_t is written by the softmax threads over the S_t columns they have read and
// is the A operand straight from TMEM.  The two query tiles share every K and V
// tile and take turns: while one's softmax runs, the other's products do.  An
// item with at most 128 rows lets both share its one query tile instead: tile t
// takes every other KV tile, and the two results are merged in the epilogue.
// Roles (one warp each but for the softmax), numbered as they are but where two
// threads share a row (Cfg::kHalves): there the softmax has warps 0-15, 0-7 for query
// tile 0, four for each half of the columns, and the others follow as 16-19.
//   warps 0-3, 4-7  softmax of query tile 0 and 1: thread = TMEM lane = row.
//                   Base-2 online softmax; the running maximum is raised only
//                   when a tile's exceeds it by more than 8 (a factor 256), and
//                   only then is O rescaled in TMEM.  Statistics are fp32;
//                   weights are rounded to the cache's 16-bit type (fp16 for an
//                   8-bit cache), the sum takes them unrounded.  (One 16-bit word a
//                   weight: a second one would double the second product.  Errors
//                   against 64 bits are up to 1.4 times those of 32-bit arithmetic.)
//   warp 8          issues the products, in a fixed order that alternates between
//                   the query tiles.
//   warp 9          draws items, publishes them in a ring, and copies K tiles (a
//                   lane a block, one tensor copy each) into the ring of K and V.
//   warp 10         copies V tiles.
//   warp 11         copies Q rows (positions x heads of the kv head) into the
//                   swizzled K-major operand.
//   warps 12-15     (caches whose chunks are not operands: 8-bit codes, blocks
//                   of fewer than 8 tokens) fill the K and V stages in place of
//                   the copies: codes become exact 16-bit integers, and the
//                   scales are applied in the softmax: K's to the scores, V's to
//                   the weights, whose maximum is taken with the tile's largest V
//                   scale, so that they stay at most 2^15 whatever the scales are.
// Every wait is bounded; a timeout sets PA_DEVERR_TIMEOUT, the call's results are
// then not to be used, and the CTA drains its own copies and products before
// releasing TMEM.
//
// What bounds it.  A pair of query tiles and one KV tile are four batches of eight
// products, 2048 clocks at the tensor cores' rate.  Measured: 16 prompts of 2048
// tokens, 32 + 8 heads of 128 in bf16: 570 us, 0.96 PFLOP/s; 32 chunks of 512 over 512
// to 3584: 546 us, 1.18 PFLOP/s (heads of 64, half of the products against the same
// softmax a tile: 552 and 503 us); 3200 clocks a pair and KV tile, and 5000 to 9000
// around the end of an item: the chain scores - softmax - second product of a query
// tile (TMEM has room for two), whose every hand-over costs some 300 clocks, because
// shared memory answers slowly while products read their operands from it.  8 x 4
// tokens over 32K to 128K: 545 us, 6.1 TB/s, bound by HBM.  8-bit caches: 32 chunks of
// up to 700 tokens 750 us, 0.55 PFLOP/s, 6000 clocks a pair and KV tile, 3500 of them
// softmax (two scales a score; the converters next to it slow both down; with eight
// converter warps, whose registers come from the softmax, 884 us).  A warpgroup of its
// own for the results took 637 us instead of 593 on the prompts; two issuing warps,
// one a query tile, each in its own order, 628 instead of 588 (and the chunks 634
// instead of 549: both softmaxes run at once and the tensor cores idle).
//
// Shaped scores.  A score s = scale q.k becomes c tanh(s / c) (a cap c), then less
// slope_h |distance|, and a query attends the positions of its own span [first, last]
// instead of all up to its own.  The softmax threads shape the scores that they have read:
//   cap       c tanh(y) = y P(y^2) c for y = s / c of at most 3/4 (P: 5 terms, relative error
//             6e-7, the division folded into them): seven packed fp32 operations for two
//             scores, in the loop that takes the powers.  2^x and 1 / x instead would triple
//             the load of the special-function units.  A warp that meets a larger |y| in a
//             tile takes the exact form for that tile.
//   distance  slope (t - p) is linear in the column up to the query's own position: a packed
//             FMA, split into 16 columns' part and their first one's.  KV tiles are taken from
//             the last one backwards: from left to right the maximum, and with it a rescaling
//             of the results, would move with every tile (16 prompts of 2048 tokens: 876 us
//             instead of 705; now 676).  Behind a query (prefixes) the warp takes the exact form.
//   spans     the planner finds each query tile's first and last position, and which
//             positions all of its queries attend; only KV tiles outside of those are masked.
// What bounds it: beside what bounds the plain scores, instructions.  A softmax warp has its
// quarter of the SM nearly to itself, and straight code beyond about 160 instructions costs it
// 2.6 clocks an instruction, beyond about 700 in all roles 5 (measured with rows of independent
// FMAs); packed FMAs take 2.3 clocks.  So a tile's code is what counts: each shape has kernels
// of its own, without conditions, and rare forms stand behind what is common.  Measured (us, bf16
// but for the slopes, the rate counts the attended pairs): 32 capped chunks of 512 over 512 to
// 3584, 32 + 8 heads, 645 (1.0 PFLOP/s; plain scores 540; in fp16, with a maximum, 1034; what takes
// kAny: cap 56 in bf16 1166, cap and slopes 1088; blocks of 4 tokens 1016, heads of 64 612); 16
// prompts of 2048 with slopes, 32 + 32 heads in fp16, 676 (0.81; plain 592); 2 rows of 8192 tokens of
// packed documents with prefixes 312 (0.57; most KV tiles are masked somewhere; capped as well 362,
// with slopes 488); capped chunks over an 8-bit cache in a window of 1500 691 (0.37; plain 526); 8 x
// 4 tokens over 32K to 128K, capped, 566 (5.9 TB/s).  The planner's pass over spans is one CTA's: 18
// us of these documents' (7 without spans), 114 of 2150 for 128K tokens of them.
#pragma once

#include <cuda.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "extend_plan.h"
#include "kernels.h"
#include "scores.cuh"
#include "tc_common.cuh"

namespace pkv {
namespace {

using plan::attend_from;
using plan::kKv;
using plan::kRows;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kRescaleThreshold = 8.f;   // base-2 units
// 8-bit caches: weights (with V's scales) and their sums are 2^kLift times as large.
// Stored in fp16 they reach 2^15 at most, and a token that holds nearly all of a
// row's weight keeps 11 bits of it down to a V scale 2^-21 times its tile's largest
// one (unlifted: 2^-14, and at 2^-21 its row was off by 6%).
constexpr float kLift = 7.f;

// Flags of a query tile and kv head.
constexpr uint32_t kBadBlock = 1, kRedo = 2;

// ------------------------------------------------------------------ workspace
struct Header {
  int32_t next;                            // (item, head) pairs handed out
  int32_t total;                           // items * kv heads
  int32_t num_split;                       // query tiles whose contexts are split
  int32_t any_flag;
};

// One work item, for every kv head.
struct __align__(16) Item {
  int32_t seq, base, count;                // its sequence, the sequence's first item and number of items
  int32_t row0, pos0, npos;                // first token row, position and number of positions
  int32_t tile0, ntiles;                   // KV tiles [tile0, tile0 + ntiles) of this part
  int32_t first;                           // first position any of its queries attends
  int32_t held;                            // first position a ring still holds
  int32_t part_row;                        // first row of its partial results for kv head 0, or -1
  int32_t head_rows;                       // partial rows between kv heads
  int32_t flag;                            // the item whose flags it raises: its query tile's first
  int32_t parts;                           // of its query tile's context
  int32_t rows;                            // partial rows of one part
  int32_t tile;                            // its query tile
};

struct Space {
  Header* head;
  int32_t* seq_tile;                       // [num_seqs + 1] number of a sequence's first query tile
  int2* tiles;                             // [max_tiles] a query tile's first item and first partial row
  int4* spans;                             // [max_tiles] with spans: where a query tile's first span begins and its last
                                           // one does, where the first one ends and the last one does
  Item* items;                             // [max_items]
  int32_t* splits;                         // [max_items] first items of the split query tiles
  uint32_t* flags;                         // [max_items * kv heads]
  float* o;                                // [max_rows][D]
  float* ml;                               // [max_rows][2]
  int32_t max_tiles;
  int32_t max_items;
  int32_t tile_rows;                       // most rows an item can have
  int64_t max_rows;
};

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// The workspace of these shapes, laid out from `base`; its size in *bytes.
Space lay_out(uint8_t* base, int num_seqs, int num_tokens, int num_kv_heads, int group, int max_query_len,
              int head_size, int sms, bool scored, size_t* bytes) {
  const int pair = plan::pair_positions(group);
  Space w{};
  w.tile_rows = (max_query_len < pair ? max_query_len : pair) * group;
  w.max_tiles = (int32_t)plan::max_tiles(num_tokens, num_seqs, pair);
  w.max_items = (int32_t)plan::max_items(w.max_tiles, sms);
  w.max_rows = plan::max_rows(w.tile_rows, sms);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at = align_up(at + n);
    return base + here;
  };
  w.head = reinterpret_cast<Header*>(take(sizeof(Header)));
  w.seq_tile = reinterpret_cast<int32_t*>(take(((size_t)num_seqs + 1) * 4));
  w.tiles = reinterpret_cast<int2*>(take((size_t)w.max_tiles * sizeof(int2)));
  w.spans = reinterpret_cast<int4*>(take(scored ? (size_t)w.max_tiles * sizeof(int4) : 0));
  w.items = reinterpret_cast<Item*>(take((size_t)w.max_items * sizeof(Item)));
  w.splits = reinterpret_cast<int32_t*>(take((size_t)w.max_items * 4));
  w.flags = reinterpret_cast<uint32_t*>(take((size_t)w.max_items * num_kv_heads * 4));
  w.o = reinterpret_cast<float*>(take((size_t)w.max_rows * head_size * 4));
  w.ml = reinterpret_cast<float*>(take((size_t)w.max_rows * 8));
  *bytes = at;
  return w;
}

// Programmatic launches: let the next kernel on the stream begin / wait for the one before to be done.
__device__ __forceinline__ void launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void launch_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------------ planner
constexpr int kPlanThreads = 1024;
constexpr int kPlanCache = 4096;           // sequences and query tiles whose numbers are searched in shared memory

struct Seq {
  int start, q_len, ctx, held;
  bool listed, zero;                       // has items; only zero rows
};

template <bool kScored>
__device__ __forceinline__ Seq read_seq(const ExtendParams& p, int s, uint32_t& err) {
  Seq q;
  const bool single = kScored && !p.query_start_loc;          // one token a sequence
  q.start = single ? s : p.query_start_loc[s];
  const int64_t end = single ? s + 1 : p.query_start_loc[s + 1];
  q.ctx = p.context_lens[s];
  q.held = 0;
  q.zero = false;
  q.listed = q.start >= 0 && end > q.start && end <= p.num_tokens;
  q.q_len = q.listed ? (int)(end - q.start) : 0;
  if (!q.listed) {
    if (end != q.start || q.start < 0 || end > p.num_tokens) err |= PA_DEVERR_CONTEXT;
    return q;
  }
  if (single && q.ctx <= 0) {                                 // a padded sequence
    q.zero = true;
    return q;
  }
  if (q.q_len > p.max_query_len || (kScored && q.ctx > p.max_context) || q.q_len > q.ctx || q.ctx > INT32_MAX - kKv ||      // (tile ends stay in int32)
      (p.ring_blocks == 0 && (int64_t)q.ctx > (int64_t)p.bt_width * p.block_size)) {
    q.zero = true;
    err |= PA_DEVERR_CONTEXT;
    return q;
  }
  if (p.ring_blocks > 0) {
    const int64_t h = ((int64_t)((q.ctx - 1) / p.block_size) - p.ring_blocks + 1) * p.block_size;
    q.held = h > 0 ? (int)h : 0;
  }
  return q;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive prefix of v over the CTA, and the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* tmp, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t in = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) tmp[warp] = in;
  __syncthreads();
  const int64_t w = warp_scan(tmp[lane], lane);
  total = __shfl_sync(kFull, w, 31);
  const int64_t before = __shfl_sync(kFull, w, (warp + 31) & 31);
  return in - v + (warp ? before : 0);
}

// First and last position that the query at position pos, token row `row`, attends; ctx: the end of the positions that
// any query of its tile attends, or of its sequence's.
template <bool kScored>
__device__ __forceinline__ int span_from(const ExtendParams& p, int pos, int held, int row) {
  const int a = attend_from(pos, p.window, held);
  return kScored && p.first_pos ? max(a, p.first_pos[row]) : a;
}
template <bool kScored>
__device__ __forceinline__ int span_to(const ExtendParams& p, int pos, int ctx, int row) {
  return kScored && p.last_pos ? max(min(p.last_pos[row], ctx - 1), -1) : pos;
}

// Distances of a row count from a position of its own, which the softmax does not see: its nearest attended one, `near`,
// or with a slope below 0 its farthest one (`far_from` further).  The largest bias is 0 then: beside one of 2^30, scores and
// the maximum would be rounded by more than a power of two can hold.
__device__ __forceinline__ int far_from(const ExtendParams& p, int near, int pos, int held, int ctx, int row) {
  return max(near - span_from<true>(p, pos, held, row), span_to<true>(p, pos, ctx, row) - near);
}

// A query tile: positions pos0 .. pos0 + npos - 1 of a sequence, from token row row0 on.
struct Tile {
  int seq, row0, pos0, npos, held;
  int first;                               // first position any of its queries attends
  int tile0, n;                            // the KV tiles that it attends
  int n_last;                              // those of the sequence's last query tile
  int64_t seq_rows;                        // rows of the sequence's query tiles, all heads
};

// One CTA.  Three passes with a scan each: over sequences (thread t owns [t * per,
// (t + 1) * per)), which numbers their query tiles; over query tiles, whose KV
// tiles give the call's work and with it the part length, and whose parts give the
// items' and the partial rows' numbers; over items.  What has to be looked up
// backwards -- a tile's sequence, an item's tile -- is searched in shared memory.
template <bool kScored>
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const __grid_constant__ ExtendParams p,
                                                              const __grid_constant__ Space ws, int sms) {
  __shared__ int64_t tmp[32];
  __shared__ int32_t seq_tile[kPlanCache], tile_item[kPlanCache];
  __shared__ uint32_t errs;
  __shared__ int nsplit;
  const int S = p.num_seqs, G = p.group, pair = plan::pair_positions(G), tid = threadIdx.x, hkv = p.num_kv_heads;
  const bool spans = kScored && (p.first_pos || p.last_pos);
  if (tid == 0) errs = nsplit = 0;
  launch_next();

  // ---- sequences
  const int per = (S + kPlanThreads - 1) / kPlanThreads;
  const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
  uint32_t err = 0, none = 0;
  int64_t count = 0, all;
  for (int s = s0; s < s1; ++s) {
    const Seq q = read_seq<kScored>(p, s, err);
    if (q.listed) count += plan::tiles_of(q.q_len, pair);
  }
  int64_t at = block_scan(count, tmp, all);
  if (all > ws.max_tiles) err |= PA_DEVERR_CONTEXT;           // sequences overlap: the last ones are left out
  const int tiles = (int)min(all, (int64_t)ws.max_tiles);
  for (int s = s0; s < s1; ++s) {
    const int base = (int)min(at, (int64_t)tiles);
    ws.seq_tile[s] = base;
    if (s < kPlanCache) seq_tile[s] = base;
    if (per > 1) {
      const Seq q = read_seq<kScored>(p, s, none);
      if (q.listed) at += plan::tiles_of(q.q_len, pair);
    }
  }
  if (tid == 0) ws.seq_tile[S] = tiles;
  if (err) atomicOr(&errs, err);
  __syncthreads();

  // ---- query tiles
  auto place = [&](int i, Tile& t) {
    int lo = 0, hi = S;                                       // the last sequence whose first tile is <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((mid < kPlanCache ? seq_tile[mid] : ws.seq_tile[mid]) <= i) lo = mid; else hi = mid;
    }
    const Seq q = read_seq<kScored>(p, lo, none);
    // the longest contexts first
    const int q0 = (plan::tiles_of(q.q_len, pair) - 1 - (i - (lo < kPlanCache ? seq_tile[lo] : ws.seq_tile[lo]))) * pair;
    t.seq = lo;
    t.row0 = q.start + q0;
    t.pos0 = q.ctx - q.q_len + q0;
    t.npos = min(pair, q.q_len - q0);
    t.held = q.held;
    return q;
  };
  auto tile = [&](int i) {
    Tile t;
    const Seq q = place(i, t);
    t.first = attend_from(t.pos0, p.window, q.held);
    t.n = plan::tile_range(t.pos0, t.npos, p.window, q.held, t.tile0);
    if (kScored && spans) {
      const int4 v = ws.spans[i];
      t.first = v.x;
      t.tile0 = v.x / kKv;
      t.n = v.w < v.x ? 0 : v.w / kKv - t.tile0 + 1;          // (no query of the tile attends anything: v.w is -1)
    }
    if (q.zero) t.n = 0;
    const int nt = plan::tiles_of(q.q_len, pair), l0 = (nt - 1) * pair;
    int unused;
    t.n_last = plan::tile_range(q.ctx - q.q_len + l0, q.q_len - l0, p.window, q.held, unused);
    if (kScored && spans) t.n_last = t.n;
    t.seq_rows = (int64_t)nt * min(pair, q.q_len) * G * hkv;
    return t;
  };
  auto parts_of = [&](const Tile& t, int64_t longest) {
    return plan::parts_of(t.n, t.n_last, t.seq_rows, longest, ws.max_rows);
  };
  if (kScored && spans) {                                     // a warp a query tile
    for (int i = tid >> 5; i < tiles; i += kPlanThreads / 32) {
      Tile t;
      const Seq q = place(i, t);
      int first = INT32_MAX, first_max = 0, last_min = INT32_MAX - 1, last = -1;
      for (int j = tid & 31; j < t.npos && !q.zero; j += 32) {
        const int a = span_from<kScored>(p, t.pos0 + j, t.held, t.row0 + j);
        const int b = span_to<kScored>(p, t.pos0 + j, q.ctx, t.row0 + j);
        if (a > b) continue;                                  // it attends nothing; its row is zeroed in the end
        first = min(first, a);
        first_max = max(first_max, a);
        last_min = min(last_min, b);
        last = max(last, b);
      }
      first = __reduce_min_sync(kFull, first);
      first_max = __reduce_max_sync(kFull, first_max);
      last_min = __reduce_min_sync(kFull, last_min);
      last = __reduce_max_sync(kFull, last);
      if ((tid & 31) == 0) ws.spans[i] = make_int4(first, first_max, last_min, last);
    }
    __syncthreads();
  }
  Tile mine{};                                                // tile tid: most calls have no more
  int64_t work = 0, total;
  for (int i = tid; i < tiles; i += kPlanThreads) {
    const Tile t = tile(i);
    if (i == tid) mine = t;
    work += t.n;
  }
  block_scan(work, tmp, total);
  const int64_t longest = plan::longest_part(total, tiles, hkv, sms);
  int64_t done = 0;                                           // items << 32 | partial rows of the tiles before
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int64_t add = 0, sum;
    if (i < tiles) {
      const Tile t = i0 == 0 ? mine : tile(i);
      const int parts = parts_of(t, longest);
      add = (int64_t)parts << 32 | (uint32_t)(parts > 1 ? parts * t.npos * G * hkv : 0);
    }
    const int64_t before = done + block_scan(add, tmp, sum);
    if (i < tiles) {
      ws.tiles[i] = make_int2((int)(before >> 32), (int)(uint32_t)before);
      if (i < kPlanCache) tile_item[i] = (int)(before >> 32);
    }
    done += sum;
  }
  const int items = (int)(done >> 32);
  __syncthreads();

  // ---- items
  auto first_item = [&](int t) { return t == tiles ? items : t < kPlanCache ? tile_item[t] : ws.tiles[t].x; };
  for (int i = tid; i < items; i += kPlanThreads) {
    int k = i;                                                // its query tile, where none is cut
    if (items > tiles) {
      k = 0;
      int hi = tiles;
      while (hi - k > 1) {
        const int mid = (k + hi) >> 1;
        if (first_item(mid) <= i) k = mid; else hi = mid;
      }
    }
    const Tile t = k == tid ? mine : tile(k);
    const int first = first_item(k), part = i - first;
    Item it;
    it.seq = t.seq;
    it.base = first_item(t.seq < kPlanCache ? seq_tile[t.seq] : ws.seq_tile[t.seq]);
    it.count = first_item(t.seq + 1 < min(S, kPlanCache) ? seq_tile[t.seq + 1] : ws.seq_tile[t.seq + 1]) - it.base;
    it.row0 = t.row0;
    it.pos0 = t.pos0;
    it.npos = t.npos;
    it.parts = parts_of(t, longest);
    int from;
    it.ntiles = plan::part_range(t.n, it.parts, part, from);
    it.tile0 = t.tile0 + from;
    it.first = t.first;
    it.held = t.held;
    it.rows = t.npos * G;
    it.part_row = it.parts > 1 ? ws.tiles[k].y + part * it.rows : -1;
    it.head_rows = it.parts * it.rows;
    it.flag = first;
    it.tile = k;
    ws.items[i] = it;
    if (it.parts > 1 && part == 0) ws.splits[atomicAdd(&nsplit, 1)] = i;
  }
  for (int64_t i = tid; i < (int64_t)items * hkv; i += kPlanThreads) ws.flags[i] = 0;
  __syncthreads();
  if (tid == 0) {
    ws.head->next = 0;
    ws.head->total = items * hkv;
    ws.head->num_split = nsplit;
    ws.head->any_flag = 0;
    if (errs) report(p.dev_err, errs);
  }
}

// ------------------------------------------------------------------ the attention kernel
// What scores become, in kernels of their own: with conditions inside, a tile's code outgrows the instruction cache,
// and a warp alone with it waits 2 to 5 clocks for each instruction.
enum Shape {
  kNone,                                   // pa_extend
  kSpans,                                  // spans of each query alone
  kCap,                                    // a cap that folds (scores.cuh), in bf16 one of at most 80 in base 2
  kSlope,                                  // slopes alone, no position behind the query's own
  kAny                                     // both, slopes with such positions, or a cap that does not fold
};

// How the K and V stages are filled.
enum Fill { kBulk, kGather, kCodes };

constexpr int kRing = 4;                   // items between the drawing warp and the others
// Tiles' scales (8-bit caches).  They have no barriers of their own.  They are
// written before their tile's K, and so before its scores.  When tile c's are
// written, tiles up to c - 2 have gone through their first product, and a softmax
// warpgroup can then be at most six tiles behind (items of one tile each, all for
// query tile 0: their epilogues meet).
constexpr int kScaleRing = 8;
constexpr int kScalePitch = 36;

// An item as the roles see it.
struct Work {
  int kvh;                                 // -1: no more
  int seq, row0, pos0, npos;
  int tile0, n[2];                         // first KV tile; KV tiles of query tile t (alt: its every other one)
  int alt;                                 // both take query tile 0's rows
  int first, held, kv_end;                 // attended positions lie in [first, kv_end)
  int edge_lo, edge_hi;                    // KV tiles (counted from tile0) below / from which on some pair is masked
  int c0;                                  // ring number of the first KV tile
  int qload[2];                            // load number of Q tile t, if it has one
  int part_row, flag;
};

template <typename T, int D, Fill F, int kShape>
struct Cfg {
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int kTileBytes = kKv * D * 2;              // K (or V) of one KV tile
  static constexpr int kGroupBytes = 8 * D * 2;               // 8 tokens of it
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr bool kConvert = F != kBulk;
  // Where no maximum is needed (kFixed below) and registers allow, two threads share a row, 64 columns each: a softmax
  // warp is otherwise alone with its tile on its quarter of the SM, and waits for every result and every instruction by
  // itself.  (Capped chunks 835 -> 742 us.  With a maximum the halves have to meet in every tile: slopes 876 -> 987,
  // plain scores 552 -> 632.)
  static constexpr int kHalves = kShape == kCap && kBf16 && !kConvert ? 2 : 1;
  static constexpr int kSoft = 8 * kHalves;                   // softmax warps; the other roles' follow
  static constexpr int kThreads = 32 * (kSoft + 4 + (kConvert ? 4 : 0));
  // registers a thread, whose sum over the warpgroups is the launch's: the softmax
  // warpgroups hold a row's 128 scores (8-bit caches: 64), the converters of 8-bit
  // caches half of a tile's codes (8 registers more or fewer for the softmax: within 2%)
  static constexpr int kRegsSoftmax = kHalves == 2 ? 96 : F == kBulk ? 200 : F == kGather ? 176 : 160;
  static constexpr int kRegsRest = kHalves == 2 ? 96 : F == kBulk ? 104 : F == kGather ? 88 : 96;
  static constexpr int kRegsConvert = F == kGather ? 72 : 96;
  static_assert((kThreads == 640 ? 96 * 5 : kThreads == 512 ? 128 * 4 : 168 * 3) ==
                2 * kHalves * kRegsSoftmax + kRegsRest + (kConvert ? kRegsConvert : 0), "register split");
  // K and V tiles take turns in one ring: K of tile c is fill 2c, V fill 2c + 1, fill
  // n sits in buffer n % kBufs.  Five buffers of 32 KiB beside the query tiles are
  // all that fits (K and V in rings of two each: 1200 more clocks a tile, waiting for
  // copies); the converting variants need the rest for scales and staged codes.
  static constexpr int kBufs = kConvert ? 4 : 5;
  static constexpr size_t kRingBytes = (size_t)kBufs * kTileBytes;
};

struct __align__(16) Shared {
  uint64_t full[5], empty[5];              // the buffers of K and V tiles
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2];
  // PV of tile number n of query tile t completes pv_done[t][n & 1]: a waiter is never two phases behind
  uint64_t pv_done[2][2];
  uint64_t item_full[kRing], item_empty[kRing];
  uint64_t xbar;                           // all softmax warps (items that share a query tile)
  uint64_t rows[2][4];                     // the two warps of a query tile's 32 rows (64 columns each)
  uint64_t mma_drain;
  Work work[kRing];
  volatile int bad[kRing];                 // a block id out of range was met
  volatile int odd[kRing];                 // (8-bit caches) a V scale that is not finite was met
  float red[2][kRows][2];                  // of each query tile: (maximum, sum), or its halves' sums
  uint32_t tmem_base;
  volatile int abort_flag;
  int last_fill[5], last_q[2];             // the last copies into each buffer, -1: none
  int pad[3];
};
struct __align__(16) Scales {
  // column 8 n + 2 q + b at q * kScalePitch + 2 n + b: what a softmax thread reads is
  // contiguous, and the four of a row read different banks
  float k[kScaleRing][4 * kScalePitch], v[kScaleRing][4 * kScalePitch];    // (K's times the softmax scale, base 2)
  float top[kScaleRing][4], low[kScaleRing][4];    // largest and smallest (but 0) V scale of each 32 tokens
};

// Bound of every wait: about a second, far above any wait of a healthy call.
constexpr uint32_t kPolls = 1u << 20;
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kPolls; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pack2f(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2f(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2f(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2f(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2f(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// tanh(y) / y times c for two y: |y| <= 3/4 (kTerms 5) or <= 1 (kTerms 6).
template <int kTerms>
__device__ __forceinline__ uint64_t cap_quotient2(const ScoreShape& w, uint64_t y) {
  const float* c = kTerms == 5 ? w.three_quarters : w.poly;
  const uint64_t s = mul2f(y, y);
  uint64_t v = pack2f(c[kTerms - 1], c[kTerms - 1]);
#pragma unroll
  for (int k = kTerms - 2; k >= 0; --k) v = fma2f(v, s, pack2f(c[k], c[k]));
  return v;
}
// The base-2 score of any y (s / c where scores are capped, else s log2(e)), dist positions from the row's nearest one;
// shift: far_from, or 0.
__device__ __forceinline__ float shaped_score(const ScoreShape& w, float y, float slope2, int dist, int shift) {
  const float v = w.capped ? score::any_cap(w, y) : y;
  return w.slopes ? v - slope2 * (float)(abs(dist) - shift) : v;
}

// 32 TMEM lanes x 64 columns; the wait is part of the statement.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
        "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
        "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 TMEM lanes x 128 columns (16 x 256 bits, 16 times): lane l of the warp gets columns 8 n + 2 (l % 4) + {0, 1} of
// rows l / 4 (v[4 n], v[4 n + 1]) and l / 4 + 8 (v[4 n + 2], v[4 n + 3]).
__device__ __forceinline__ void tmem_ld16x256(uint32_t taddr, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, "
      "%51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]),
        "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]),
        "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]),
        "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]),
        "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
// The same of 32 columns, both ways.
__device__ __forceinline__ void tmem_ld16x256_32(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16x256_32(uint32_t taddr, const float* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
               "%13, %14, %15, %16};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
               "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
// 16 lanes x 64 columns (16 x 128 bits, 16 times): column 4 n + l % 4 of rows l / 4 (r[2 n]) and l / 4 + 8
// (r[2 n + 1]).
__device__ __forceinline__ void tmem_st16x128(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
               "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, "
               "%31, %32};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
               "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
               "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
               "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}

// 32 TMEM lanes x 32 columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <int N>
__device__ __forceinline__ void set_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 bytes; `wide`: they are 32-byte aligned (else 16).
__device__ __forceinline__ void store32(void* at, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(at)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(at)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  const int n = take ? 16 : 0;             // 0: the destination is zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Tensor copies global -> shared, completing their bytes on `bar`.
__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load4(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// Offset of the 16-byte piece (8 dims) of token r in a K or V stage (8-token groups, a group's 64-dim atoms together).
template <int D>
__device__ __forceinline__ uint32_t kv_offset(int r, int piece) {
  return (uint32_t)((r >> 3) * (8 * D * 2) + (piece >> 3) * 1024 + (r & 7) * 128 + (((piece & 7) ^ (r & 7)) << 4));
}

// Whether KV tile jt of the item holds places without a token of the context.
__device__ __forceinline__ bool ragged(const Work& w, int jt) {
  const int t0 = (w.tile0 + jt) * kKv;
  return t0 < w.first || t0 + kKv > w.kv_end;
}

// Table entry and validity of the block that holds position pos.
__device__ __forceinline__ int block_of(const ExtendParams& p, const int32_t* row, int blk) {
  return row[p.ring_blocks > 0 ? blk % p.ring_blocks : blk];
}

template <typename T, int D, Fill F, int kShape>
__global__ void __launch_bounds__(Cfg<T, D, F, kShape>::kThreads, 1) extend_kernel(const __grid_constant__ ExtendParams p,
                                                                       const __grid_constant__ Space ws,
                                                                       const __grid_constant__ CUtensorMap q_map,
                                                                       const __grid_constant__ CUtensorMap kv_map) {
  using C = Cfg<T, D, F, kShape>;
  constexpr bool kI8 = F == kCodes, kScored = kShape != kNone;
  constexpr bool kBF16 = std::is_same<T, __nv_bfloat16>::value;
  using PT = typename std::conditional<kI8, __half, T>::type;      // type of the weights and of V's operand
  // (no static shared memory: the operands start 1024-byte aligned without padding)
  extern __shared__ __align__(1024) uint8_t qbuf[];
  uint8_t* ring = qbuf + 2 * C::kQBytes;
  Shared& sh = *reinterpret_cast<Shared*>(ring + C::kRingBytes);
  Scales& scales = *reinterpret_cast<Scales*>(&sh + 1);            // 8-bit caches alone
  // Capped scores lie in [-c, c]: with bf16 weights, whose range is fp32's, and c up to 80 in base 2 they are taken
  // against 0, without a maximum.  Sums of 2^80 over 2^31 tokens stay finite beside values up to 2^16; larger results are
  // seen as infinities, and those of rows near -c whose products leave fp32 at its lower end by their size: such items are
  // redone on CUDA cores against a maximum.  What is not seen is below 2^-126 a token beside weights of 2^-40 or more.
  constexpr bool kFixed = kShape == kCap && kBF16 && !kI8;
  // Scores that fall with distance are largest where the queries are: with the last KV tile first the running maximum is
  // found at once, from left to right it would rise, and the results be rescaled, with every tile.
  constexpr bool kBackwards = kShape == kSlope || kShape == kAny;
  constexpr int NB = C::kBufs, kH = C::kHalves, kSoft = C::kSoft, kCols = kKv / kH;
  if (smem_u32(qbuf) & 1023u) {                                    // never, as laid out
    if (threadIdx.x == 0) report(p.dev_err, PA_DEVERR_TIMEOUT);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group, ptile = kRows / G;                        // positions of one query tile
  const int bs = p.block_size;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4 * kH);
      mbar_init(&sh.pv_done[i][0], 1);
      mbar_init(&sh.pv_done[i][1], 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&sh.full[i], C::kConvert ? 4 : 1);
      mbar_init(&sh.empty[i], 1);
      sh.last_fill[i] = -1;
    }
    sh.last_q[0] = sh.last_q[1] = -1;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.item_full[i], 1);
      // the softmax warps, the issuing warp, the Q warp, and the V warp or 4 converter warps
      mbar_init(&sh.item_empty[i], kSoft + (C::kConvert ? 6 : 3));
    }
    mbar_init(&sh.xbar, kSoft);
    for (int i = 0; i < 8; ++i) mbar_init(&sh.rows[i >> 2][i & 3], 2);
    mbar_init(&sh.mma_drain, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kSoft) {
    tc::tmem_alloc(&sh.tmem_base, 512);
    tc::tmem_relinquish();
  }
  launch_next();
  launch_wait();                                                   // the planner's items
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;                              // S_t at 128 t, O_t at 256 + 128 t

  // a role gave up: tell the others
  auto give_up = [&]() {
    report(p.dev_err, PA_DEVERR_TIMEOUT);
    sh.abort_flag = 1;
  };
  // waits of whole warps; false (in every lane): it ran out, or another role gave up
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(kFull, bar_wait(bar, parity) && !sh.abort_flag);
  };
  // the next item of the ring
  auto next_item = [&](int i, Work& w) -> bool {
    if (!wait(&sh.item_full[i % kRing], (i / kRing) & 1)) return false;
    w = sh.work[i % kRing];
    return true;
  };
  auto done_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.item_empty[i % kRing]);
  };
  // fill n's buffer: free to be filled / filled
  auto wait_empty = [&](int n) -> bool { return n < NB || wait(&sh.empty[n % NB], (n / NB - 1) & 1); };
  auto buffer = [&](int n) { return ring + (n % NB) * C::kTileBytes; };
  // fill n: the K (part 0) or V (part 1) vectors of the blocks `id` of the lanes that take one, one copy a block
  auto copy_blocks = [&](int n, int part, int id, int kvh, bool take) {
    const uint32_t bytes = bs / 8 * C::kGroupBytes;
    const unsigned m = __ballot_sync(kFull, take);
    uint64_t* bar = &sh.full[n % NB];
    if (lane == 0) {
      sh.last_fill[n % NB] = n;
      mbar_arrive_expect_tx(bar, (uint32_t)__popc(m) * bytes);
    }
    __syncwarp();
    if (take)
      tma_load4(buffer(n) + lane * bytes, &kv_map, 0, 0, part, (id * p.num_kv_heads + kvh) * (bs / 8), bar);
    __syncwarp();
  };
  // KV tiles of an item
  auto tiles_of = [](const Work& w) { return w.alt ? w.n[0] + w.n[1] : max(w.n[0], w.n[1]); };
  // the number in its item of the j-th KV tile of n that is worked on
  auto nth = [](int j, int n) { return kBackwards ? n - 1 - j : j; };

  if (warp >= kSoft && warp < kSoft + 4) {
    set_regs_dec<C::kRegsRest>();
    if (warp == kSoft + 1) {
      // ================================================================= items, and K copies
      int32_t w_next = 0;
      int total = ws.head->total;
      if (lane == 0) w_next = atomicAdd(&ws.head->next, 1);
      w_next = __shfl_sync(kFull, w_next, 0);
      int c = 0, q0 = 0, q1 = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        Work w;
        w.kvh = -1;
        if (w_next < total) {
          // heads outside, items inside: a sequence's (head, tile) pairs are numbered head by head
          const Item a = ws.items[w_next / p.num_kv_heads];
          const int local = w_next - a.base * p.num_kv_heads;
          const int h = local / a.count, k = a.base + local % a.count;
          const Item it = ws.items[k];
          w.kvh = h;
          w.seq = it.seq;
          w.row0 = it.row0;
          w.pos0 = it.pos0;
          w.npos = it.npos;
          w.tile0 = it.tile0;
          w.alt = it.npos <= ptile;
          w.first = it.first;
          w.held = it.held;
          w.kv_end = it.pos0 + it.npos;
          if (w.alt) {
            w.n[0] = (it.ntiles + 1) / 2;
            w.n[1] = it.ntiles / 2;
          } else {
            // tile 0's last position may need one KV tile less
            w.n[0] = kBackwards ? it.ntiles : max(0, min(it.ntiles, (it.pos0 + ptile - 1) / kKv + 1 - it.tile0));
            w.n[1] = it.ntiles;
          }
          int last_first = attend_from(w.kv_end - 1, p.window, it.held), first_last = it.pos0;
          if (kScored && (p.first_pos || p.last_pos)) {
            const int4 v = ws.spans[it.tile];
            w.kv_end = v.w + 1;
            last_first = v.y;
            first_last = v.z;
            if (!w.alt) w.n[0] = it.ntiles;
          }
          w.edge_lo = (last_first + kKv - 1) / kKv - it.tile0;
          w.edge_hi = (first_last + 1) / kKv - it.tile0;
          w.c0 = c;
          w.qload[0] = q0;
          w.qload[1] = q1;
          if (w.n[0] > 0) ++q0;
          if (!w.alt && w.n[1] > 0) ++q1;
          w.part_row = it.part_row < 0 ? -1 : it.part_row + h * it.head_rows;
          w.flag = it.flag * p.num_kv_heads + h;
        }
        const int slot = i % kRing;
        if (i >= kRing && !wait(&sh.item_empty[slot], ((i / kRing) - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          sh.work[slot] = w;
          sh.bad[slot] = 0;
          sh.odd[slot] = 0;
          mbar_arrive(&sh.item_full[slot]);
        }
        __syncwarp();
        if (w.kvh < 0) break;
        if (lane == 0) w_next = atomicAdd(&ws.head->next, 1);
        const int n = tiles_of(w);
        if constexpr (!C::kConvert) {
          const int32_t* row = p.block_tables + w.seq * p.bt_stride;
          const int fb = w.first / bs, nblk = (w.kv_end + bs - 1) / bs;   // blocks [fb, nblk) are read
          for (int j = 0; j < n; ++j, ++c) {
            // lane l copies the tile's block l
            const int blk = (w.tile0 + nth(j, n)) * (kKv / bs) + lane;
            const bool take = lane < kKv / bs && blk >= fb && blk < nblk;
            int id = take ? block_of(p, row, blk) : 0;
            if (take && (unsigned)id >= (unsigned)p.num_blocks) {
              id = 0;
              sh.bad[slot] = 1;
            }
            if (!wait_empty(2 * c)) {
              ok = false;
              break;
            }
            copy_blocks(2 * c, 0, id, w.kvh, take);
          }
        } else {
          c += n;
        }
        w_next = __shfl_sync(kFull, w_next, 0);
      }
      if (!ok && lane == 0) give_up();
      __syncwarp();
    } else if (warp == kSoft + 2) {
      // ================================================================= V copies
      if constexpr (!C::kConvert) {
        int c = 0;
        bool ok = true;
        for (int i = 0; ok; ++i) {
          Work w;
          if (!next_item(i, w)) {
            ok = false;
            break;
          }
          if (w.kvh < 0) break;
          const int n = tiles_of(w);
          const int32_t* row = p.block_tables + w.seq * p.bt_stride;
          const int fb = w.first / bs, nblk = (w.kv_end + bs - 1) / bs;
          for (int j = 0; j < n; ++j, ++c) {
            const int blk = (w.tile0 + nth(j, n)) * (kKv / bs) + lane;
            const bool take = lane < kKv / bs && blk >= fb && blk < nblk;
            int id = take ? block_of(p, row, blk) : 0;
            if ((unsigned)id >= (unsigned)p.num_blocks) id = 0;      // reported by the K copies
            if (!wait_empty(2 * c + 1)) {
              ok = false;
              break;
            }
            copy_blocks(2 * c + 1, 1, id, w.kvh, take);
          }
          if (ok) done_item(i);
        }
        if (!ok && lane == 0) give_up();
        __syncwarp();
      }
    } else if (warp == kSoft + 3) {
      // ================================================================= Q rows
      bool ok = true;
      for (int i = 0; ok; ++i) {
        Work w;
        if (!next_item(i, w)) {
          ok = false;
          break;
        }
        if (w.kvh < 0) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || w.n[t] == 0 || (w.alt && t == 1)) continue;
          const int load = w.qload[t];
          if (load > 0 && !wait(&sh.q_empty[t], (load - 1) & 1)) {
            ok = false;
            continue;
          }
          // ptile positions x group heads, 64 dims a copy; rows past the sequence's are
          // the next sequence's (or zero behind the last token), and are not used
          if (lane == 0) {
            sh.last_q[t] = load;
            mbar_arrive_expect_tx(&sh.q_full[t], (uint32_t)((kScored ? min(ptile, p.max_query_len) : ptile) * G * D * 2));
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
              tma_load3(qbuf + t * C::kQBytes + a * (kRows * 128), &q_map, a * 64, w.kvh * G, w.row0 + t * ptile,
                        &sh.q_full[t]);
          }
          __syncwarp();
        }
        if (ok) done_item(i);
      }
      if (!ok && lane == 0) give_up();
      __syncwarp();
    } else {
      // ================================================================= products
      // The whole warp runs the schedule, so that operands stay in uniform registers;
      // one elected lane issues.  Order: items in turn, and per item, KV tile by KV
      // tile, for query tile t = 0, 1: PV_t of its tile before, then QK_t of this one.
      // While one query tile's weights are being made, the other's products run.
      const uint32_t id_qk = tc::idesc_f16(kRows, kKv, kBF16, false, false);
      const uint32_t id_pv = tc::idesc_f16(kRows, D, kBF16 && !kI8, false, true);
      const uint64_t qd0 = tc::smem_desc(smem_u32(qbuf), 16, 1024, tc::kSwizzle128B);
      const uint64_t kd0 = tc::smem_desc(smem_u32(ring), 16, C::kGroupBytes, tc::kSwizzle128B);
      const uint64_t vd0 = tc::smem_desc(smem_u32(ring), 1024, C::kGroupBytes, tc::kSwizzle128B);
      bool ok = true;
      // Every instruction between two batches of products is felt: the tensor cores
      // queue only about four of them ahead (256 clocks).
      auto spin = [&](uint64_t* bar, uint32_t parity, bool there) {
        if (!__all_sync(kFull, there)) {
          for (uint32_t i = 0; ok && !__all_sync(kFull, mbar_test_wait(bar, parity)); ++i)
            if ((i & 255) == 255 && (i > 8 * kPolls || __any_sync(kFull, sh.abort_flag))) ok = false;
        }
        tc::fence_after_sync();
      };
      // The ring's buffer and phase of the next K fill; its V fill is the one after.
      // Fills are used, and so waited for, in order, each at least once: no phase of a
      // barrier is skipped, so its parity never stands for one two phases back.
      struct Fills {
        int kb = 0;
        uint32_t kp = 0;
        __device__ int vb() const { return kb == NB - 1 ? 0 : kb + 1; }
        __device__ uint32_t vp() const { return kb == NB - 1 ? kp ^ 1u : kp; }
        __device__ void next() {
          kb += 2;
          if (kb >= NB) {
            kb -= NB;
            kp ^= 1u;
          }
        }
      };
      // the product that each query tile still owes
      struct Owed {
        int buf = -1, steps = 0;           // V's buffer; steps of 16 tokens
        uint32_t phase = 0, num = 0;       // V's phase; KV tiles of this query tile so far
        bool first = false, wait_v = false, last_user = false;
      };
      Owed owed0, owed1;
      Fills fill;
      bool k_there = false;
      // where the weights of 16 tokens are: each half of the columns has its own over the scores it has read
      auto p_column = [](int k) { return kH == 2 ? (k >> 2) * 64 + (k & 3) * 8 : k * 8; };
      auto pv = [&](auto which, Owed& x) {
        constexpr int t = decltype(which)::value;
        if (x.buf < 0) return;
        const bool p_there = mbar_test_wait(&sh.p_full[t], x.num & 1);
        if (x.wait_v) spin(&sh.full[x.buf], x.phase, mbar_test_wait(&sh.full[x.buf], x.phase));
        spin(&sh.p_full[t], x.num & 1, p_there);
        // the next K is looked at now: shared memory is slow to answer while products read it
        k_there = mbar_test_wait(&sh.full[fill.kb], fill.kp);
        const uint64_t vd = vd0 + (uint64_t)((x.buf * C::kTileBytes) >> 4);
        if (ok && tc::elect()) {
          tc::mma_f16_ta(tmem + 256 + t * 128, tmem + t * kKv, vd, id_pv, (uint32_t)!x.first);
          if (x.steps == kKv / 16) {
#pragma unroll
            for (int k = 1; k < kKv / 16; ++k)
              tc::mma_f16_ta(tmem + 256 + t * 128, tmem + t * kKv + p_column(k), vd + (uint64_t)((k * 2 * C::kGroupBytes) >> 4),
                             id_pv, 1u);
          } else {
            for (int k = 1; k < x.steps; ++k)
              tc::mma_f16_ta(tmem + 256 + t * 128, tmem + t * kKv + p_column(k), vd + (uint64_t)((k * 2 * C::kGroupBytes) >> 4),
                             id_pv, 1u);
          }
          tc::commit(&sh.pv_done[t][x.num & 1]);
          if (x.last_user) tc::commit(&sh.empty[x.buf]);
        }
        __syncwarp();
        ++x.num;
        x.buf = -1;
      };
      auto flush = [&]() {
        pv(std::integral_constant<int, 0>{}, owed0);
        pv(std::integral_constant<int, 1>{}, owed1);
      };
      uint32_t q_num0 = 0, q_num1 = 0;                               // loads of each query tile so far
      auto uni = [&](int v) { return __shfl_sync(kFull, v, 0); };
      for (int i = 0; ok; ++i) {
        const int slot = i % kRing;
        uint64_t* bar = &sh.item_full[slot];
        const uint32_t par = (i / kRing) & 1;
        if (!__all_sync(kFull, mbar_test_wait(bar, par))) flush();   // nothing to go on with: what is owed first
        spin(bar, par, false);
        if (!ok) break;
        const Work& w = sh.work[slot];
        if (uni(w.kvh) < 0) break;
        const int n0 = uni(w.n[0]), n1 = uni(w.n[1]);
        const bool alt = uni(w.alt) != 0;
        const int tok = uni(w.kv_end) - uni(w.tile0) * kKv;          // tokens from the first KV tile on
        const int skip = uni(w.first) - uni(w.tile0) * kKv;          // of them, before the first attended one
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[slot]);
        const int rounds = max(n0, n1);
        if (rounds == 0) continue;
        // its rows may still be on their way: then what is owed goes first
        const bool load0 = n0 > 0, load1 = !alt && n1 > 0;
        pv(std::integral_constant<int, 0>{}, owed0);
        if (load0) {
          const bool there = mbar_test_wait(&sh.q_full[0], q_num0 & 1);
          if (!__all_sync(kFull, there)) pv(std::integral_constant<int, 1>{}, owed1);
          spin(&sh.q_full[0], q_num0 & 1, there);
          ++q_num0;
        }
        auto turn = [&](auto which, Owed& x, int j, int n, int other) {
          constexpr int t = decltype(which)::value;
          pv(which, x);
          if (j >= n) return;
          const int jt = nth(alt ? 2 * j + t : j, alt ? n0 + n1 : rounds);   // KV tile of the item
          // the last of the (one or two) query tiles that use this K and V
          const bool both = !alt && j < other, last_k = !both || t == 1;
          const int kb = fill.kb, vb = fill.vb();
          const uint32_t vp = fill.vp();
          if (!both || t == 0) spin(&sh.full[kb], fill.kp, k_there);
          k_there = false;
          if (t == 1 && load1 && j == 0) {
            spin(&sh.q_full[1], q_num1 & 1, false);
            ++q_num1;
          }
          const int after = tok - jt * kKv;                          // tokens from this KV tile on
          if (F == kBulk && (jt * kKv < skip || after < kKv)) spin(&sh.full[vb], vp, false);   // its softmax writes V
          const uint64_t qd = qd0 + (uint64_t)((t == 0 || alt ? 0 : C::kQBytes) >> 4);
          const uint64_t kd = kd0 + (uint64_t)((kb * C::kTileBytes) >> 4);
          const bool last_q = j == n - 1 && (!alt || (t == 0 ? other < n : other <= n));
          if (ok && tc::elect()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_f16(tmem + t * kKv, qd + (uint64_t)(((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4),
                          kd + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_qk, kk > 0);
            tc::commit(&sh.s_full[t]);
            if (last_k) tc::commit(&sh.empty[kb]);
            if (last_q) tc::commit(&sh.q_empty[alt ? 0 : t]);
          }
          __syncwarp();
          x.buf = vb;
          x.phase = vp;
          x.steps = after >= kKv ? kKv / 16 : (after + 15) >> 4;
          x.first = j == 0;
          x.wait_v = !both || t == 0;
          x.last_user = last_k;
          if (last_k) fill.next();
        };
        for (int j = 0; j < rounds && ok; ++j) {
          turn(std::integral_constant<int, 0>{}, owed0, j, n0, n1);
          turn(std::integral_constant<int, 1>{}, owed1, j, n1, n0);
        }
      }
      flush();
      if (!ok && lane == 0) give_up();
      // every product issued completes before TMEM can be freed
      if (tc::elect()) {
        tc::commit(&sh.mma_drain);
      }
      __syncwarp();
      if (!__all_sync(kFull, bar_wait(&sh.mma_drain, 0)) && lane == 0) report(p.dev_err, PA_DEVERR_TIMEOUT);
    }
    __syncwarp();
  } else if (warp >= kSoft + 4) {
    // =================================================================== converters
    if constexpr (C::kConvert) {
      set_regs_dec<C::kRegsConvert>();
      const int ct = threadIdx.x - 32 * (kSoft + 4);                              // 0 .. 127
      const int shift = __ffs(bs) - 1;
      constexpr int kPer = kI8 ? 8 : D / 8;                          // 16-byte source pieces of one vector
      constexpr int kLoads = kKv * kPer / 128;                       // of one thread, K or V
      const int u0 = ct / kPer, piece = ct % kPer;                   // load e: piece `piece` of token u0 + e * 128 / kPer
      const I8Layout L8{bs, p.num_kv_heads};
      int c = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        Work w;
        if (!next_item(i, w)) {
          ok = false;
          break;
        }
        if (w.kvh < 0) break;
        const int n = tiles_of(w);
        const int32_t* row = p.block_tables + w.seq * p.bt_stride;
        // the block of token u of KV tile j, or -1: no query attends it, or its id is bad
        auto find = [&](int j, int u) -> int {
          const int pos = (w.tile0 + nth(j, n)) * kKv + u;
          if (pos < w.first || pos >= w.kv_end) return -1;
          const int id = block_of(p, row, pos >> shift);
          if ((unsigned)id < (unsigned)p.num_blocks) return id;
          sh.bad[i % kRing] = 1;
          return -1;
        };
        // a warp's loads touch 32 tokens: lane 32 / kPer * e + r keeps the block of the r-th of load e
        constexpr int kTok = 32 / kPer;
        static_assert(kTok * kLoads == 32, "one token a lane");
        int mine = -1;
        auto look_up = [&](int j) { return find(j, (ct >> 5) * kTok + lane % kTok + lane / kTok * (128 / kPer)); };
        auto block = [&](int e) { return __shfl_sync(kFull, mine, e * kTok + lane / kPer); };
        auto place = [&](int j, int e) { return ((w.tile0 + nth(j, n)) * kKv + u0 + e * (128 / kPer)) & (bs - 1); };
        if constexpr (!kI8) {
          // 16-byte pieces by asynchronous copies, absent tokens as zeros; a token's K and V
          // together (their addresses differ by a constant).  A tile is completed after
          // the next one has been issued.
          auto issue = [&](int j) {
            const uint32_t k_dst = smem_u32(buffer(2 * c)), v_dst = smem_u32(buffer(2 * c + 1));
#pragma unroll
            for (int e = 0; e < kLoads; ++e) {
              const int id = block(e), s = place(j, e);
              // a block of fewer than 8 tokens is one group: K atoms, then V atoms, of bs rows each
              const int in_block = ((piece >> 3) * bs + s) * 64 + (((piece & 7) ^ s) << 3);
              const uint8_t* src = p.cache;
              if (id >= 0) src += 2 * (((int64_t)id * p.num_kv_heads + w.kvh) * (2 * D * bs) + in_block);
              const uint32_t at = kv_offset<D>(u0 + e * (128 / kPer), piece);
              cp_async16(k_dst + at, src, id >= 0);
              cp_async16(v_dst + at, id >= 0 ? src + 2 * D * bs : src, id >= 0);
            }
            cp_async_commit();
          };
          auto complete = [&](int tile) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&sh.full[2 * tile % NB]);
              mbar_arrive(&sh.full[(2 * tile + 1) % NB]);
            }
          };
          int next = n > 0 ? look_up(0) : -1;
          for (int j = 0; j < n; ++j, ++c) {
            mine = next;
            if (j + 1 < n) next = look_up(j + 1);
            // the tile before this one is completed now if this one's buffers are not free yet
            bool pending = j > 0;
            if (pending && c >= 2 && !__all_sync(kFull, mbar_test_wait(&sh.empty[(2 * c + 1) % NB], ((2 * c + 1) / NB - 1) & 1))) {
              cp_async_wait<0>();
              complete(c - 1);
              pending = false;
            }
            if (!wait_empty(2 * c) || !wait_empty(2 * c + 1)) {
              ok = false;
              break;
            }
            issue(j);
            if (pending) {
              cp_async_wait<1>();
              complete(c - 1);
            }
          }
          cp_async_wait<0>();
          if (ok && n > 0) complete(c - 1);
        } else {
          // A thread converts the 16-byte pieces that it has loaded itself: K's are staged
          // in shared memory by asynchronous copies, V's in registers (there is no room
          // for both in either), each asked for as soon as the tile before is converted.
          const uint32_t stage = smem_u32(&scales + 1) + ct * 16;
          uint4 v[kLoads];
          auto load = [&](int j, auto which) {
            constexpr int part = decltype(which)::value;
#pragma unroll
            for (int e = 0; e < kLoads; ++e) {
              const int id = block(e);
              const uint8_t* src = id < 0 ? p.cache : p.cache + L8.code(id, w.kvh, part, place(j, e), piece * 16);
              if (part == 0) {
                cp_async16(stage + e * 2048, src, id >= 0);
              } else {
                v[e] = id < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(src);
              }
            }
            if (part == 0) cp_async_commit();
          };
          constexpr std::integral_constant<int, 0> kK{};
          constexpr std::integral_constant<int, 1> kV{};
          float sk = 0.f, sv = 0.f;
          auto load_scales = [&](int j) {
            const int id = find(j, ct), t = ((w.tile0 + nth(j, n)) * kKv + ct) & (bs - 1);
            sk = id < 0 ? 0.f : *reinterpret_cast<const float*>(p.cache + L8.scale(id, w.kvh, 0, t));
            sv = id < 0 ? 0.f : *reinterpret_cast<const float*>(p.cache + L8.scale(id, w.kvh, 1, t));
            // (0 * inf would reach rows that do not attend the token)
            if (!(fabsf(sv) < INFINITY)) {
              sv = 0.f;
              sh.odd[i % kRing] = 1;
            }
          };
          auto write = [&](auto which) {
            constexpr int part = decltype(which)::value;
            uint8_t* dst = buffer(2 * c + part);
            auto convert = [&](const uint32_t (&in)[4], int e) {
              uint32_t y[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (part == 1 || !kBF16) {
                  // fp16 1024 + (code + 128), less 1152: exact
                  const uint32_t b = in[k] ^ 0x80808080u;
                  const __half2 off = __half2half2(__ushort_as_half((unsigned short)0x6480));
                  const uint32_t a0 = __byte_perm(b, 0x64646464u, 0x4140), a1 = __byte_perm(b, 0x64646464u, 0x4342);
                  const __half2 h0 = __hsub2(*reinterpret_cast<const __half2*>(&a0), off);
                  const __half2 h1 = __hsub2(*reinterpret_cast<const __half2*>(&a1), off);
                  y[2 * k] = *reinterpret_cast<const uint32_t*>(&h0);
                  y[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                } else {
                  // bf16 128 + (low 7 bits), less 128 (code >= 0) or 256: exact
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t b = __byte_perm(in[k], 0, hf ? 0x4342 : 0x4140);
                    const uint32_t a = 0x43004300u | (b & 0x007f007fu), s = 0x43004300u | (b & 0x00800080u);
                    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                                     *reinterpret_cast<const __nv_bfloat162*>(&s));
                    y[2 * k + hf] = *reinterpret_cast<const uint32_t*>(&r);
                  }
                }
              }
              const int u = u0 + e * (128 / kPer);
              *reinterpret_cast<uint4*>(dst + kv_offset<D>(u, 2 * piece)) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(dst + kv_offset<D>(u, 2 * piece + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
            };
            if (part == 0) {
              cp_async_wait<0>();
#pragma unroll 2
              for (int e = 0; e < kLoads; ++e) {
                uint32_t in[4];
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(in[0]), "=r"(in[1]), "=r"(in[2]), "=r"(in[3])
                             : "r"(stage + e * 2048)
                             : "memory");
                convert(in, e);
              }
            } else {
#pragma unroll
              for (int e = 0; e < kLoads; ++e) {
                const uint32_t in[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
                convert(in, e);
              }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full[(2 * c + part) % NB]);
          };
          int next = -1;
          if (n > 0) {
            mine = look_up(0);
            load(0, kK);
            load(0, kV);
            load_scales(0);
          }
          for (int j = 0; j < n; ++j, ++c) {
            if (j + 1 < n) next = look_up(j + 1);
            if (!wait_empty(2 * c)) {
              ok = false;
              break;
            }
            {
              const int r = c % kScaleRing;
              // the tile's largest V scale bounds its weights (floats above 0 order like integers)
              const unsigned top = __reduce_max_sync(kFull, __float_as_uint(fmaxf(sv, 0.f)));
              const unsigned low = __reduce_min_sync(kFull, __float_as_uint(sv > 0.f ? sv : INFINITY));
              const int at = (ct % 8 / 2) * kScalePitch + ct / 8 * 2 + ct % 2;
              scales.k[r][at] = sk * (kScored && p.shape.capped ? p.shape.cap_in : p.scale_log2);
              scales.v[r][at] = sv;
              if (lane == 0) {
                scales.top[r][ct >> 5] = __uint_as_float(top);
                scales.low[r][ct >> 5] = __uint_as_float(low);
              }
            }
            write(kK);
            mine = next;
            if (j + 1 < n) {
              load(j + 1, kK);
              load_scales(j + 1);
            }
            if (!wait_empty(2 * c + 1)) {
              ok = false;
              break;
            }
            write(kV);
            if (j + 1 < n) load(j + 1, kV);
          }
        }
        if (ok) done_item(i);
      }
      if (!ok && lane == 0) give_up();
      __syncwarp();
    }
  } else {
    // =================================================================== softmax warpgroups
    set_regs_inc<C::kRegsSoftmax>();
    const int t = warp / (4 * kH);                                   // query tile
    const int half = kH == 2 ? (warp >> 2) & 1 : 0;                  // of its columns
    const int row = threadIdx.x & 127;                               // TMEM lane
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + quarter + t * kKv + half * kCols, o_addr = tmem + quarter + 256 + t * 128;
    const int ipos = row / G, head = row - ipos * G;
    int num = 0, nx = 0, nr = 0;                                     // KV tiles, exchanges so far
    bool ok = true;
    // an exchange of the two warpgroups: everything before it is seen after it
    auto meet = [&]() {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.xbar);
      if (!wait(&sh.xbar, nx & 1)) ok = false;
      ++nx;
      tc::fence_after_sync();
    };
    // an exchange of the two warps that share their rows
    auto meet_rows = [&]() {
      tc::fence_before_sync();
      __syncwarp();
      uint64_t* bar = &sh.rows[t][warp & 3];
      if (lane == 0) mbar_arrive(bar);
      if (!wait(bar, nr & 1)) ok = false;
      ++nr;
      tc::fence_after_sync();
    };
    // thread = token here: V rows of fill 2 c + 1 that hold no token of the context become zero (V has landed: the issuer
    // waited for it); true: the wait ran out
    auto zero_rows = [&](const Work& w, int jt, int c) -> bool {
      if constexpr (F == kBulk) {
        if (ragged(w, jt)) {
          if (!wait(&sh.full[(2 * c + 1) % NB], ((2 * c + 1) / NB) & 1)) {
            ok = false;
            return true;
          }
          const int at = (w.tile0 + jt) * kKv + row;
          if (half == 0 && (at >= w.kv_end || at < w.first)) {
            uint8_t* v = buffer(2 * c + 1);
#pragma unroll 2
            for (int e = 0; e < D / 8; ++e) *reinterpret_cast<uint4*>(v + kv_offset<D>(row, e)) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
        }
      }
      return false;
    };
    for (int i = 0; ok; ++i) {
      if (!wait(&sh.item_full[i % kRing], (i / kRing) & 1)) {
        ok = false;
        break;
      }
      const Work& w = sh.work[i % kRing];                            // (read where needed: registers are scarce here)
      if (w.kvh < 0) break;
      const bool alt = w.alt != 0;
      const int my0 = alt ? 0 : t * ptile;                           // my tile's first position in the item
      const bool row_ok = ipos < (alt ? w.npos : min(ptile, w.npos - my0));
      const int pos = w.pos0 + my0 + ipos;
      auto token = [&]() { return w.row0 + (row_ok ? pos - w.pos0 : 0); };
      const int from = kScored ? 0 : attend_from(pos, p.window, w.held);
      const float slope2 = kScored && p.shape.slopes ? p.shape.slopes[w.kvh * G + head] * score::kLog2e : 0.f;
      const int n = t == 0 ? w.n[0] : w.n[1];
      // (with two threads a row there are registers for little else: read where needed)
      using Held = typename std::conditional<kH == 2, const int&, const int>::type;
      Held tile0 = w.tile0, c0 = w.c0, edge_lo = w.edge_lo, edge_hi = w.edge_hi;
      float m = kFixed ? 0.f : -INFINITY, l = 0.f;
      // 8-bit caches: a thread has rows gr + 8 i of its warp's 32 (and a quarter of their columns)
      float m4[4], l4[4];
      int pos4[4];
      uint32_t ok4 = 0;
      if constexpr (kI8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = (warp & 3) * 32 + (lane >> 2) + 8 * k, ip = r / G;
          pos4[k] = w.pos0 + my0 + ip;
          if (ip < (alt ? w.npos : min(ptile, w.npos - my0))) ok4 |= 1u << k;
          m4[k] = -INFINITY;
          l4[k] = 0.f;
        }
      }
      for (int j = 0; j < n; ++j, ++num) {
        const int turn = alt ? 2 * j + t : j, c = c0 + turn;
        const int jt = kBackwards ? tiles_of(w) - 1 - turn : turn;
        const int t0 = (tile0 + jt) * kKv + half * kCols;              // my first column's token
        if (!wait(&sh.s_full[t], num & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const bool edge = jt < edge_lo || jt >= edge_hi;
        if constexpr (kI8) {
          // Scales are per token, that is per column: a thread that held a whole row
          // would read all 128 of K's and of V's, and those reads alone would keep the
          // SM's shared memory busy for 2000 clocks a tile.  Read as 16 x 256 bits, a
          // thread holds 32 columns (8 n + 2 q, + 1) of four rows (gr + 8 i) instead.
          // (They were written before this tile's K was, which the scores have waited for.)
          const int slot = c % kScaleRing;
          const float4 tops = *reinterpret_cast<const float4*>(scales.top[slot]);
          const float4* ks = reinterpret_cast<const float4*>(&scales.k[slot][(lane & 3) * kScalePitch]);
          const float4* vs = reinterpret_cast<const float4*>(&scales.v[slot][(lane & 3) * kScalePitch]);
          // 16 rows each; one copy of the code (it has to stay in the instruction cache),
          // so the rows' state changes places after each
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const uint32_t half = (uint32_t)(16 * h) << 16;
            float x[64];                                             // [n][row 2 h, 2 h + 1][2]
            tmem_ld16x256(s_addr + half, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 k = ks[e];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                unpack2f(mul2f(pack2f(x[8 * e + 2 * r], x[8 * e + 2 * r + 1]), pack2f(k.x, k.y)), x[8 * e + 2 * r],
                         x[8 * e + 2 * r + 1]);
                unpack2f(mul2f(pack2f(x[8 * e + 4 + 2 * r], x[8 * e + 5 + 2 * r]), pack2f(k.z, k.w)), x[8 * e + 4 + 2 * r],
                         x[8 * e + 5 + 2 * r]);
              }
            }
            if constexpr (kShape != kNone && kShape != kSpans) {
              // (K's scales made x base-2 scores, or quotients by the cap)
              bool exact = false;
              float sl[2] = {0.f, 0.f};
              int at[2] = {0, 0}, shift[2] = {0, 0};                 // my first column less the row's nearest position
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const bool is_row = ok4 >> r & 1;
                if constexpr (kShape != kCap) {
                  const int rr = (warp & 3) * 32 + (lane >> 2) + 8 * (2 * h + r);
                  int nearest = pos4[r];
                  const int tok = w.row0 + (is_row ? pos4[r] - w.pos0 : 0);
                  if (kShape == kAny && p.last_pos) {
                    nearest = min(nearest, span_to<true>(p, pos4[r], w.kv_end, tok));
                    exact |= is_row && t0 + kKv - 1 > nearest;
                  }
                  if (p.shape.slopes) sl[r] = p.shape.slopes[w.kvh * G + rr % G] * score::kLog2e;
                  at[r] = t0 + 2 * (lane & 3) - nearest;
                  if (sl[r] < 0.f) shift[r] = far_from(p, nearest, pos4[r], w.held, w.kv_end, tok);
                }
                if constexpr (kShape != kSlope) {
                  float big[2] = {0.f, 0.f};
#pragma unroll
                  for (int n = 0; n < 16; ++n) big[n & 1] = fmaxf(fmaxf(big[n & 1], fabsf(x[4 * n + 2 * r])), fabsf(x[4 * n + 2 * r + 1]));
                  exact |= is_row && p.shape.capped && fmaxf(big[0], big[1]) > (kShape == kCap ? 0.75f : 1.f);
                }
              }
              if (kShape != kSlope && __builtin_expect(__any_sync(kFull, exact), 0)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) tmem_st16x256_32(s_addr + half + 32 * e, x + 16 * e);
                tc::tmem_wait_st();
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                  float v[16];
                  tmem_ld16x256_32(s_addr + half + 32 * e, v);
#pragma unroll
                  for (int k = 0; k < 16; ++k)
                    v[k] = kShape == kCap ? score::any_cap(p.shape, v[k])
                                          : shaped_score(p.shape, v[k], sl[k >> 1 & 1],
                                                         at[k >> 1 & 1] + 32 * e + 8 * (k >> 2) + (k & 1), shift[k >> 1 & 1]);
                  tmem_st16x256_32(s_addr + half + 32 * e, v);
                }
                tc::tmem_wait_st();
                tmem_ld16x256(s_addr + half, x);
              } else {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  // a slope's part: that of 32 columns' first one, and that within those (no sum of many steps)
                  uint64_t in[4], off[4];
                  if constexpr (kShape != kCap) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                      const float v = sl[r] * (float)(at[r] + shift[r] + 32 * k);
                      in[k] = pack2f(sl[r] * (8.f * k), sl[r] * (8.f * k + 1.f));
                      off[k] = pack2f(v, v);
                    }
                  }
#pragma unroll
                  for (int n = 0; n < 16; ++n) {
                    const int e = 4 * n + 2 * r;
                    const uint64_t y = pack2f(x[e], x[e + 1]);
                    if constexpr (kShape == kCap)
                      unpack2f(mul2f(y, cap_quotient2<5>(p.shape, y)), x[e], x[e + 1]);
                    else if (kShape == kSlope || !p.shape.capped)
                      unpack2f(add2f(add2f(y, in[n & 3]), off[n >> 2]), x[e], x[e + 1]);
                    else
                      unpack2f(add2f(fma2f(y, cap_quotient2<6>(p.shape, y), in[n & 3]), off[n >> 2]), x[e], x[e + 1]);
                  }
                }
              }
            }
            // weights carry V's scales: what is kept at most 2^8 is 2^(x - m) times the
            // tile's largest one (bounded below: sums stay finite), and 2^kLift times that
            // is stored
            float bias[2];
            bias[0] = bias[1] = log2f(fmaxf(fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w)), 0x1p-93f));
            if (__builtin_expect(edge, 0)) {
              uint32_t on[2];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int tok = w.row0 + (ok4 >> r & 1 ? pos4[r] - w.pos0 : 0);
                const int lo = span_from<kScored>(p, pos4[r], w.held, tok) - t0;
                const int hi = ok4 >> r & 1 ? span_to<kScored>(p, pos4[r], w.kv_end, tok) + 1 - t0 : 0;
                // how many of this thread's columns lie below a limit
                auto below = [&](int v) {
                  const int u = min(max(v, 0), kKv);
                  return 2 * (u >> 3) + min(max((u & 7) - 2 * (lane & 3), 0), 2);
                };
                on[r] = (uint32_t)((1ull << below(hi)) - 1) & ~(uint32_t)((1ull << below(lo)) - 1);
              }
              if (__any_sync(kFull, (on[0] & on[1]) != kFull)) {
#pragma unroll
                for (int n = 0; n < 16; ++n)
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    x[4 * n + k] = (on[k >> 1] >> (2 * n + (k & 1))) & 1 ? x[4 * n + k] : -INFINITY;
                // Where scales differ by more than 2^4, of the tokens that the row attends:
                // beside a masked token's large scale the others' weights would leave
                // fp16's range.
                const float4 lows = *reinterpret_cast<const float4*>(scales.low[slot]);
                const float low = fminf(fminf(lows.x, lows.y), fminf(lows.z, lows.w));
                if (fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w)) > 16.f * low) {
                  float big[2] = {0.f, 0.f};
#pragma unroll 1
                  for (int e = 0; e < 8; ++e) {
                    const float4 v = vs[e];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                      const uint32_t o = on[r] >> (4 * e);
                      big[r] = fmaxf(fmaxf(big[r], o & 1 ? v.x : 0.f), o & 2 ? v.y : 0.f);
                      big[r] = fmaxf(fmaxf(big[r], o & 4 ? v.z : 0.f), o & 8 ? v.w : 0.f);
                    }
                  }
#pragma unroll
                  for (int r = 0; r < 2; ++r) {
                    big[r] = fmaxf(big[r], __shfl_xor_sync(kFull, big[r], 1));
                    big[r] = fmaxf(big[r], __shfl_xor_sync(kFull, big[r], 2));
                    bias[r] = log2f(fmaxf(big[r], 0x1p-93f));
                  }
                }
              }
            }
            float mt[2];
            bool more = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int n = 0; n < 16; ++n) top[n & 1] = fmaxf(fmaxf(top[n & 1], x[4 * n + 2 * r]), x[4 * n + 2 * r + 1]);
              mt[r] = fmaxf(top[0], top[1]) + bias[r];
              more |= m4[r] == -INFINITY || mt[r] > m4[r] + kRescaleThreshold;
            }
            // Shuffles are slow here (they queue with the converters' shared-memory
            // accesses): a row's maximum is put together only where some maximum may change.
            if (__builtin_expect(__any_sync(kFull, more), 0)) {
              float alpha[2];
              bool any = false;
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                mt[r] = fmaxf(mt[r], __shfl_xor_sync(kFull, mt[r], 1));
                mt[r] = fmaxf(mt[r], __shfl_xor_sync(kFull, mt[r], 2));
                const float m_new = fmaxf(m4[r], mt[r]);
                const bool need = (ok4 >> r & 1) && m4[r] != -INFINITY && m_new > m4[r] + kRescaleThreshold;
                alpha[r] = need ? exp2f(m4[r] - m_new) : 1.f;
                if (need || m4[r] == -INFINITY) m4[r] = m_new;
                l4[r] *= alpha[r];
                any |= need;
              }
              if (__any_sync(kFull, any)) {
                if (!wait(&sh.pv_done[t][(num - 1) & 1], ((num - 1) >> 1) & 1)) ok = false;
                tc::fence_after_sync();
                for (int e = 0; ok && e < D / 32; ++e) {
                  float o[16];
                  tmem_ld16x256_32(o_addr + half + e * 32, o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] *= alpha[(k >> 1) & 1];
                  tmem_st16x256_32(o_addr + half + e * 32, o);
                }
              }
            }
            uint32_t y[32];
            uint64_t sum[2] = {0, 0};
            uint64_t nm[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float v = m4[r] == -INFINITY ? 0.f : kLift - m4[r];
              nm[r] = pack2f(v, v);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = vs[e];
#pragma unroll
              for (int k = 0; k < 4; ++k) {                          // (n = 2 e + k / 2, row k & 1)
                float a, b;
                unpack2f(add2f(pack2f(x[8 * e + 2 * k], x[8 * e + 2 * k + 1]), nm[k & 1]), a, b);
                const uint64_t ab = pack2f(ex2_approx(a), ex2_approx(b));
                sum[k & 1] = add2f(ab, sum[k & 1]);
                unpack2f(mul2f(ab, k < 2 ? pack2f(v.x, v.y) : pack2f(v.z, v.w)), a, b);
                y[4 * e + k] = Elem<PT>::pack2(a, b);
              }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float a, b;
              unpack2f(sum[r], a, b);
              l4[r] += a + b;
            }
            tmem_st16x128(s_addr + half, y);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float mm = m4[r], ll = l4[r];
              const int pp = pos4[r];
              m4[r] = m4[r + 2];
              l4[r] = l4[r + 2];
              pos4[r] = pos4[r + 2];
              m4[r + 2] = mm;
              l4[r + 2] = ll;
              pos4[r + 2] = pp;
            }
            ok4 = (ok4 >> 2 | ok4 << 2) & 15u;
          }
          if (!ok) break;
        } else if constexpr (kFixed) {
          // 32 columns at a time, weights against 0.  The weights wait in registers until it is known that every score was
          // near enough for the polynomial: one vote a tile, and its other form out of the way (votes in every part, with
          // that form between them: 742 us instead of 642).
          const int lo = edge ? span_from<true>(p, pos, w.held, token()) - t0 : 0;       // attended columns [lo, hi)
          const int hi = edge ? (row_ok ? span_to<true>(p, pos, w.kv_end, token()) + 1 - t0 : 0) : kCols;
          if (edge && zero_rows(w, jt, c)) break;
          auto mask = [&](float (&x)[32], int e) {
            const int a = min(max(lo - e * 32, 0), 32), b = min(max(hi - e * 32, 0), 32);
            const uint32_t on = (uint32_t)((1ull << b) - 1) & ~(uint32_t)((1ull << a) - 1);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = (on >> k) & 1 ? x[k] : -INFINITY;
          };
          uint64_t sum[2] = {0, 0};
          auto powers = [&](const float (&x)[32], uint32_t* y) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float a = ex2_approx(x[2 * k]), b = ex2_approx(x[2 * k + 1]);
              sum[k & 1] = add2f(pack2f(a, b), sum[k & 1]);
              y[k] = Elem<PT>::pack2(a, b);
            }
          };
          uint32_t y[kCols / 2];
          float big[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < kCols / 32; ++e) {
            float x[32];
            tmem_ld32(s_addr + e * 32, x);
#pragma unroll
            for (int k = 0; k < 32; k += 4)
#pragma unroll
              for (int i = 0; i < 2; ++i) big[i] = fmaxf(fmaxf(big[i], fabsf(x[k + i])), fabsf(x[k + 2 + i]));
            const float* f = p.shape.folded;
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const uint64_t xx = pack2f(x[k], x[k + 1]), z = mul2f(xx, xx);
              uint64_t v = pack2f(f[4], f[4]);
#pragma unroll
              for (int i = 3; i >= 0; --i) v = fma2f(v, z, pack2f(f[i], f[i]));
              unpack2f(mul2f(xx, v), x[k], x[k + 1]);
            }
            if (__builtin_expect(edge, 0)) mask(x, e);
            powers(x, y + e * 16);
          }
          if (__builtin_expect(__any_sync(kFull, row_ok && fmaxf(big[0], big[1]) * p.shape.cap_in > 0.75f), 0)) {
            sum[0] = sum[1] = 0;
#pragma unroll 1
            for (int e = 0; e < kCols / 32; ++e) {
              float x[32];
              tmem_ld32(s_addr + e * 32, x);
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = score::any_cap(p.shape, x[k] * p.shape.cap_in);
              mask(x, e);
              powers(x, y);
              tc::tmem_st16u(s_addr + e * 16, y);
            }
          } else {
#pragma unroll
            for (int e = 0; e < kCols / 32; ++e) tc::tmem_st16u(s_addr + e * 16, y + e * 16);
          }
          float a, b;
          unpack2f(add2f(sum[0], sum[1]), a, b);
          l += a + b;
        } else {
          float x[kCols];
          tmem_ld64(s_addr, x);
          if constexpr (kH == 1) tmem_ld64(s_addr + 64, x + 64);
          // Shaped scores: x unit + ahead(column / 16) is the base-2 score; under a cap x stays q.k (fly) and is capped in
          // the loop that takes the powers.
          float unit = p.scale_log2, so = 0.f, base = 0.f;
          bool fly = kShape == kCap;
          if constexpr (kShape != kNone && kShape != kSpans) {
            int ref = pos, shift = 0;                                // the nearest attended position
            bool exact = false;
            if (kShape == kAny && p.last_pos) {
              ref = min(pos, span_to<true>(p, pos, w.kv_end, token()));
              exact = row_ok && t0 + kCols - 1 > ref;
            }
            if (kShape != kCap && slope2 < 0.f) shift = far_from(p, ref, pos, w.held, w.kv_end, token());
            if constexpr (kShape != kSlope) {
              float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int e = 0; e < kCols; e += 8)
#pragma unroll
                for (int k = 0; k < 4; ++k) big[k] = fmaxf(fmaxf(big[k], fabsf(x[e + k])), fabsf(x[e + 4 + k]));
              exact |= row_ok && fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3])) * p.shape.cap_in > (kShape == kCap ? 0.75f : 1.f);
              // (uncapped: cap_in is 0)
            }
            if (kShape != kSlope && __builtin_expect(__any_sync(kFull, exact), 0)) {
              // any form, 16 columns at a time through TMEM
#pragma unroll 1
              for (int e = 0; e < kCols; e += 16) {
                float v[16];
                tc::tmem_ld16(s_addr + e, v);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  v[k] = kShape == kCap ? score::any_cap(p.shape, v[k] * p.shape.cap_in)
                                        : shaped_score(p.shape, v[k] * (p.shape.capped ? p.shape.cap_in : p.scale_log2), slope2,
                                                       t0 + e + k - ref, shift);
                tc::tmem_st16(s_addr + e, v);
              }
              tc::tmem_wait_st();
              tmem_ld64(s_addr, x);
              if constexpr (kH == 1) tmem_ld64(s_addr + 64, x + 64);
              unit = 1.f;
              fly = false;
            } else if constexpr (kShape != kCap) {
              if (p.shape.slopes) {
                so = slope2;
                base = slope2 * (float)(t0 - ref + shift);
              }
              uint64_t in[8];                                        // the slope's part within 16 columns
#pragma unroll
              for (int k = 0; k < 8; ++k) in[k] = pack2f(so * (2.f * k), so * (2.f * k + 1.f));
              const bool straight = kShape == kSlope || !p.shape.capped;
              const float u = straight ? p.scale_log2 : p.shape.cap_in;
              const uint64_t u2 = pack2f(u, u);
#pragma unroll
              for (int e = 0; e < kCols; e += 2) {
                if (straight) {
                  unpack2f(fma2f(pack2f(x[e], x[e + 1]), u2, in[e / 2 % 8]), x[e], x[e + 1]);
                } else {
                  const uint64_t y = mul2f(pack2f(x[e], x[e + 1]), u2);
                  unpack2f(fma2f(y, cap_quotient2<6>(p.shape, y), in[e / 2 % 8]), x[e], x[e + 1]);
                }
              }
              unit = 1.f;
            }
          }
          auto ahead = [&](int k) { return kShape == kSlope || kShape == kAny ? fmaf(so, 16.f * k, base) : 0.f; };
          if (edge) {
            // attended columns [lo, hi)
            const int lo = (kScored ? span_from<kScored>(p, pos, w.held, token()) : from) - t0;
            const int hi = row_ok ? span_to<kScored>(p, pos, w.kv_end, token()) + 1 - t0 : 0;
#pragma unroll
            for (int e = 0; e < kCols / 32; ++e) {
              const int a = min(max(lo - e * 32, 0), 32), b = min(max(hi - e * 32, 0), 32);
              const uint32_t on = (uint32_t)((1ull << b) - 1) & ~(uint32_t)((1ull << a) - 1);
              if (__any_sync(kFull, on != kFull)) {
#pragma unroll
                for (int k = 0; k < 32; ++k) x[e * 32 + k] = (on >> k) & 1 ? x[e * 32 + k] : -INFINITY;
              }
            }
            if (zero_rows(w, jt, c)) break;
          }
          float mt;
          if constexpr (kShape == kSlope || kShape == kAny) {
            float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < kCols / 16; ++k) {
              float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int e = 0; e < 16; e += 4)
#pragma unroll
                for (int i = 0; i < 2; ++i) top[i] = fmaxf(fmaxf(top[i], x[16 * k + e + i]), x[16 * k + e + 2 + i]);
              best[k & 1] = fmaxf(best[k & 1], fmaxf(top[0], top[1]) + ahead(k));
            }
            mt = fmaxf(best[0], best[1]);
          } else {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // four chains: latency
#pragma unroll
            for (int e = 0; e < kCols; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], x[e + k]), x[e + 4 + k]);
            mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            if (kShape == kCap && fly)
              mt = mt == -INFINITY ? mt : score::any_cap(p.shape, mt * p.shape.cap_in);      // (the cap keeps the order)
            else
              mt *= unit;
          }
          const float m_new = fmaxf(m, mt);
          const bool need = row_ok && m != -INFINITY && m_new > m + kRescaleThreshold;
          if (m == -INFINITY) m = m_new;
          if (__any_sync(kFull, need)) {
            // O holds exactly the tiles before this one once the last PV has completed
            if (!wait(&sh.pv_done[t][(num - 1) & 1], ((num - 1) >> 1) & 1)) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const float alpha = need ? exp2f(m - m_new) : 1.f;
            if (need) {
              l *= alpha;
              m = m_new;
            }
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
              float o[16];
              tc::tmem_ld16(o_addr + e * 16, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= alpha;
              tc::tmem_st16(o_addr + e * 16, o);
            }
          }
          // a masked place holds what the polynomial takes to far below 0
          if (kShape == kCap && fly && edge) {
#pragma unroll
            for (int e = 0; e < kCols; ++e) x[e] = x[e] == -INFINITY ? -64.f * p.shape.cap_out : x[e];
          }
          // weights 2^(x - m), the sum of the unrounded ones in fp32
          const float nm = m == -INFINITY ? 0.f : -m;
          uint64_t sum[2] = {0, 0};
          // to_power(pair, column): what two powers are of
          auto weigh = [&](auto to_power) {
#pragma unroll
            for (int e = 0; e < kCols / 32; ++e) {
              uint32_t y[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const int col = e * 32 + 2 * k;
                float a, b;
                unpack2f(to_power(pack2f(x[col], x[col + 1]), col), a, b);
                a = ex2_approx(a);
                b = ex2_approx(b);
                sum[k & 1] = add2f(pack2f(a, b), sum[k & 1]);
                y[k] = Elem<PT>::pack2(a, b);
              }
              tc::tmem_st16u(s_addr + e * 16, y);
            }
          };
          const uint64_t unit2 = pack2f(unit, unit), nm2 = pack2f(nm, nm);
          if (kShape == kCap && fly) {
            weigh([&](uint64_t xx, int) {
              const float* f = p.shape.folded;
              const uint64_t z = mul2f(xx, xx);
              uint64_t v = pack2f(f[4], f[4]);
#pragma unroll
              for (int k = 3; k >= 0; --k) v = fma2f(v, z, pack2f(f[k], f[k]));
              return fma2f(xx, v, nm2);
            });
          } else if (kShape == kSlope || kShape == kAny) {
            weigh([&](uint64_t xx, int col) {
              const float v = nm + ahead(col / 16);
              return add2f(xx, pack2f(v, v));
            });
          } else {
            weigh([&](uint64_t xx, int) { return fma2f(xx, unit2, nm2); });
          }
          {
            float a, b;
            unpack2f(add2f(sum[0], sum[1]), a, b);
            l += a + b;
          }
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t]);
      }
      if constexpr (kI8) {
        // to one row a lane: row lane is number lane / 8 of the lanes 4 (lane % 8) ..
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          l4[k] += __shfl_xor_sync(kFull, l4[k], 1);
          l4[k] += __shfl_xor_sync(kFull, l4[k], 2);
          const float mk = __shfl_sync(kFull, m4[k], (lane & 7) * 4), lk = __shfl_sync(kFull, l4[k], (lane & 7) * 4);
          if (lane >> 3 == k) {
            m = mk;
            l = lk;
          }
        }
      }
      // a row that attends nothing has not made its tiles masked ones: it was worked out like the others, and is left out
      if (kScored && (p.first_pos || p.last_pos) &&
          span_from<kScored>(p, pos, w.held, token()) > span_to<kScored>(p, pos, w.kv_end, token())) {
        m = -INFINITY;
        l = 0.f;
      }
      if (ok && n > 0 && !wait(&sh.pv_done[t][(num - 1) & 1], ((num - 1) >> 1) & 1)) ok = false;
      if (!ok) break;
      tc::fence_after_sync();
      if (lane == 0 && sh.bad[i % kRing]) {
        atomicOr(&ws.flags[w.flag], kBadBlock);
        atomicOr(reinterpret_cast<uint32_t*>(&ws.head->any_flag), 1u);
        report(p.dev_err, PA_DEVERR_BLOCK_ID);
      }
      if (kI8 && lane == 0 && sh.odd[i % kRing]) {
        atomicOr(&ws.flags[w.flag], kRedo);
        atomicOr(reinterpret_cast<uint32_t*>(&ws.head->any_flag), 1u);
      }
      // ---- results: columns [c0, c0 + nc) of my row
      float f[2] = {1.f, 1.f};
      int col0 = half * (D / kH), ncol = D / kH;
      bool have0 = n > 0, have1 = false;
      float lo = 0.f;                                                // alt: the other tile's sum
      if constexpr (kH == 2) {
        // the halves' sums; whoever writes here next waits until they have been read
        auto both = [&]() { if (alt) meet(); else meet_rows(); };
        sh.red[t][row][half] = l;
        both();
        if (!ok) break;
        l = sh.red[t][row][0] + sh.red[t][row][1];
        if (alt) lo = sh.red[t ^ 1][row][0] + sh.red[t ^ 1][row][1];
        both();
        if (!ok) break;
      }
      uint32_t o0 = o_addr, o1 = o_addr;
      if (alt) {
        sh.red[t][row][0] = m;                                       // (the same in both halves)
        if (kH == 1) sh.red[t][row][1] = l;
        meet();
        if (!ok) break;
        const float mo = sh.red[t ^ 1][row][0];
        if (kH == 1) lo = sh.red[t ^ 1][row][1];
        const float mm = fmaxf(m, mo);
        const float fm = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - mm);
        const float fo = mo == -INFINITY ? (lo == 0.f ? 0.f : 1.f) : exp2f(mo - mm);
        // in the order of the tiles, whichever half this is
        l = t == 0 ? l * fm + lo * fo : lo * fo + l * fm;
        m = mm;
        f[0] = t == 0 ? fm : fo;
        f[1] = t == 0 ? fo : fm;
        have0 = w.n[0] > 0;
        have1 = w.n[1] > 0;
        o0 = tmem + quarter + 256;
        o1 = o0 + 128;
        if (D / 2 / kH >= 32) {                                      // (32 columns at a time)
          ncol = D / 2 / kH;
          col0 = (t * kH + half) * ncol;
        } else {
          ncol = half == 0 ? D / 2 : 0;
          col0 = t * (D / 2) + half;
        }
      }
      const bool part = w.part_row >= 0;
      const float scale = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
      // Weights against 0 (kFixed) whose sum is below 2^-40: products with small values may have left fp32.
      const bool faint = kFixed && row_ok && l > 0.f && l < 0x1p-40f;
      float least = INFINITY;                                        // of such a row's |o|
      const int rr = (my0 + ipos) * G + head;                        // row within the item
      const int part_row = w.part_row;
      float* prow = ws.o + (int64_t)(part_row + rr) * D;
      T* tile = static_cast<T*>(p.out) + ((int64_t)(w.row0 + my0) * p.num_q_heads + w.kvh * G) * D;
      // Rows leave 64 bytes at a time, a pair of lanes a row: a store of 16 bytes a row
      // and lane asks for 32 lines, and the stores alone took 6000 clocks an item.  The
      // lanes of a pair exchange halves, then both store of one row, then of the other
      // (16 prompts of 2048 tokens: 570 us; rows of four lanes 578; 32 bytes a row and
      // lane, no exchange, 581).
      const int mine = row_ok ? (ipos * p.num_q_heads + head) * D : -1;   // my row in the tile's output
      const int other = __shfl_xor_sync(kFull, mine, 1);
      const bool upper = lane & 1, wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
      const int row_a = upper ? other : mine, row_b = upper ? mine : other;
      uint64_t odd[2] = {0, 0};                                      // NaN once any value is not finite
      const uint64_t scale2 = pack2f(scale, scale);
      // A row that attends nothing is zero, whatever the tiles that it was worked out with made of it: a K scale that is
      // not finite, which all other rows attend, and 0 * NaN is NaN.  (Over a 16-bit cache such values are seen below,
      // and parts are left out by their sum of 0.)
      const bool blank = kI8 && kScored && row_ok && l == 0.f;
      const bool blanks = kI8 && kScored && __any_sync(kFull, blank);
      for (int e = col0; e < col0 + ncol; e += 32) {
        float o[32];
        if (have0) {
          tmem_ld32(o0 + e, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (alt) {
          float b[32];
          if (have1) {
            tmem_ld32(o1 + e, b);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) b[k] = 0.f;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = o[k] * f[0] + b[k] * f[1];
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) odd[k & 1] = fma2f(pack2f(o[2 * k], o[2 * k + 1]), 0, odd[k & 1]);
        if (kFixed && faint) {
#pragma unroll
          for (int k = 0; k < 32; ++k) least = fminf(least, fabsf(o[k]));
        }
        if (blanks) {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = blank ? 0.f : o[k];
        }
        if (!part) {
          uint32_t y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float a, b;
            unpack2f(mul2f(pack2f(o[2 * k], o[2 * k + 1]), scale2), a, b);
            y[k] = Elem<T>::pack2(a, b);
          }
          uint32_t ya[8], yb[8];                                     // of the even lane's row, of the odd lane's
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t got = __shfl_xor_sync(kFull, upper ? y[k] : y[k + 8], 1);
            ya[k] = upper ? got : y[k];
            yb[k] = upper ? y[k + 8] : got;
          }
          T* at = tile + e + (upper ? 16 : 0);
          if (row_a >= 0) store32(at + row_a, ya, wide);
          if (row_b >= 0) store32(at + row_b, yb, wide);
        } else if (row_ok) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4*>(prow + e + 4 * k) = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (row_ok && part && col0 == 0)
        *reinterpret_cast<float2*>(ws.ml + 2 * (int64_t)(part_row + rr)) = make_float2(m, l);
      // A V that is not finite reaches rows that do not attend it (0 * NaN = NaN):
      // finish_kernel redoes the item.  (8-bit codes are finite; scales that are not
      // have been seen above.)  The same where a faint row has results so small that
      // products of 2^-126 and less, or the lack of them, may matter.
      float odd_a, odd_b;
      unpack2f(add2f(odd[0], odd[1]), odd_a, odd_b);
      const bool lost = faint && least < 0x1p-96f;
      if (!kI8 && __any_sync(kFull, (row_ok && !(odd_a + odd_b == 0.f)) || lost) && lane == 0) {
        atomicOr(&ws.flags[w.flag], kRedo);
        atomicOr(reinterpret_cast<uint32_t*>(&ws.head->any_flag), 1u);
      }
      // both halves have read both accumulators before either is overwritten
      if (alt) meet(); else tc::fence_before_sync();
      if (!ok) break;
      done_item(i);
    }
    if (!ok && lane == 0) give_up();
    __syncwarp();
  }

  tc::fence_before_sync();
  __syncthreads();
  // Never leave copies in flight: all have been waited for by the products, unless a role gave up.
  if (threadIdx.x == 0 && sh.abort_flag) {
    for (int i = 0; i < NB; ++i) {
      const int n = sh.last_fill[i];
      if (n >= 0 && !bar_wait(&sh.full[i], (n / NB) & 1)) report(p.dev_err, PA_DEVERR_TIMEOUT);
    }
    for (int i = 0; i < 2; ++i)
      if (sh.last_q[i] >= 0 && !bar_wait(&sh.q_full[i], sh.last_q[i] & 1)) report(p.dev_err, PA_DEVERR_TIMEOUT);
  }
  if (warp == kSoft) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ finish
// Attention of one row on CUDA cores by one warp, for tiles that the tensor
// cores cannot take: positions [from, pos], fp32 online softmax.
template <typename T, int D, bool kI8, bool kScored>
__device__ void row_on_cuda_cores(const ExtendParams& p, const Item& it, int kvh, int r, int lane) {
  constexpr int kDims = D / 32;
  const int bs = p.block_size, j = r / p.group, h = kvh * p.group + r % p.group;
  const int pos = it.pos0 + j, from = span_from<kScored>(p, pos, it.held, it.row0 + j);
  const int to = span_to<kScored>(p, pos, p.context_lens[it.seq], it.row0 + j), ref = min(pos, to);
  const float unit = kScored && p.shape.capped ? p.shape.cap_in : p.scale_log2;
  const float slope2 = kScored && p.shape.slopes ? p.shape.slopes[h] * score::kLog2e : 0.f;
  const int shift = kScored && slope2 < 0.f ? far_from(p, ref, pos, it.held, p.context_lens[it.seq], it.row0 + j) : 0;
  const T* q = static_cast<const T*>(p.q) + (int64_t)(it.row0 + j) * p.q_token_stride + (int64_t)h * D + lane * kDims;
  float x[kDims], o[kDims], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int d = 0; d < kDims; ++d) {
    x[d] = (float)q[d] * unit;
    o[d] = 0.f;
  }
  const Layout L{bs, D, p.num_kv_heads};
  const I8Layout L8{bs, p.num_kv_heads};
  const int32_t* row = p.block_tables + it.seq * p.bt_stride;
  for (int t = from; t <= to; ++t) {
    const int b = block_of(p, row, t / bs), at = t & (bs - 1);
    if ((unsigned)b >= (unsigned)p.num_blocks) continue;             // its tile is flagged as bad
    // element lane * kDims + d of the token's K (part 0) or V
    auto element = [&](int part, int d) -> float {
      if constexpr (kI8)
        return (float)(int8_t)p.cache[L8.code(b, kvh, part, at, lane * kDims + d)] *
               *reinterpret_cast<const float*>(p.cache + L8.scale(b, kvh, part, at));
      else
        return (float)reinterpret_cast<const T*>(p.cache)[L.offset(b, kvh, part, at, lane * kDims + d)];
    };
    float z = 0.f;
#pragma unroll
    for (int d = 0; d < kDims; ++d) z = fmaf(x[d], element(0, d), z);
#pragma unroll
    for (int i = 16; i; i >>= 1) z += __shfl_xor_sync(kFull, z, i);
    if constexpr (kScored) z = shaped_score(p.shape, z, slope2, t - ref, shift);
    // (a score of -inf has weight 0, before any finite one too: there mn is -inf as well)
    const float mn = fmaxf(m, z), a = m == -INFINITY ? 0.f : exp2f(m - mn), e = z == -INFINITY ? 0.f : exp2f(z - mn);
    l = l * a + e;
#pragma unroll
    for (int d = 0; d < kDims; ++d) o[d] = o[d] * a + e * element(1, d);
    m = mn;
  }
  T* out = static_cast<T*>(p.out) + ((int64_t)(it.row0 + j) * p.num_q_heads + h) * D + lane * kDims;
#pragma unroll
  for (int d = 0; d < kDims; ++d) out[d] = Elem<T>::from_float(l == 0.f ? 0.f : o[d] / l);
}

// Warps take rows of split query tiles: out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p, in the order of the
// parts; then, where any flag was raised, the rows of flagged items.
template <typename T, int D, bool kI8, bool kScored>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ ExtendParams p,
                                                     const __grid_constant__ Space ws) {
  constexpr int kDims = D / 32;
  const int lane = threadIdx.x & 31, hkv = p.num_kv_heads, G = p.group;
  launch_wait();
  const int64_t w0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5, nw = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const Header hd = *ws.head;
  for (int64_t u = w0; u < (int64_t)hd.num_split * hkv * ws.tile_rows; u += nw) {
    const int r = (int)(u % ws.tile_rows), h = (int)(u / ws.tile_rows % hkv);
    const int item = ws.splits[u / ws.tile_rows / hkv];
    const Item& it = ws.items[item];
    if (r >= it.npos * G || (hd.any_flag && ws.flags[item * hkv + h])) continue;
    const int64_t first = it.part_row + (int64_t)h * it.head_rows + r;
    const int rows = it.rows, parts = it.parts;
    float M = -INFINITY;
    for (int k = lane; k < parts; k += 32) M = fmaxf(M, ws.ml[2 * (first + (int64_t)k * rows)]);
#pragma unroll
    for (int i = 16; i; i >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, i));
    float l = 0.f, o[kDims] = {};
    // (no branch: a part's loads need not wait for those of the part before)
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const int64_t at = first + (int64_t)k * rows;
      const float2 ml = *reinterpret_cast<const float2*>(ws.ml + 2 * at);
      // nothing attended in this part: its o is finite and counts nothing; -inf with a sum: NaN scores
      const float f = ml.y == 0.f ? 0.f : ml.x == -INFINITY ? 1.f : exp2f(ml.x - M);
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] = fmaf(ws.o[at * D + lane * kDims + d], f, o[d]);
    }
    T* out = static_cast<T*>(p.out) +
             ((int64_t)(it.row0 + r / G) * p.num_q_heads + h * G + r % G) * D + lane * kDims;
#pragma unroll
    for (int d = 0; d < kDims; ++d) out[d] = Elem<T>::from_float(l == 0.f ? 0.f : o[d] / l);
  }
  if (!hd.any_flag) return;
  for (int u = 0; u < hd.total; ++u) {
    const int item = u / hkv, h = u % hkv;
    const uint32_t f = ws.flags[u];
    if (!f) continue;
    const Item& it = ws.items[item];
    for (int64_t r = w0; r < it.npos * G; r += nw) {
      if (f & kBadBlock) {
        T* out = static_cast<T*>(p.out) +
                 ((int64_t)(it.row0 + r / G) * p.num_q_heads + h * G + r % G) * D + lane * kDims;
#pragma unroll
        for (int d = 0; d < kDims; ++d) out[d] = Elem<T>::from_float(0.f);
      } else {
        row_on_cuda_cores<T, D, kI8, kScored>(p, it, h, (int)r, lane);
      }
    }
  }
}

// ------------------------------------------------------------------ launch
// A launch that may begin while the kernel before it on the stream runs; it waits
// (launch_wait) before it touches that kernel's results.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The driver's encoder of tensor maps (looked up once).
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
cudaError_t encoder(EncodeTiled* f) {
  static std::atomic<EncodeTiled> known{nullptr};
  *f = known.load(std::memory_order_acquire);
  if (*f) return cudaSuccess;
  void* at = nullptr;
  cudaDriverEntryPointQueryResult found;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess || !at) return cudaErrorSymbolNotFound;
  *f = reinterpret_cast<EncodeTiled>(at);
  known.store(*f, std::memory_order_release);
  return cudaSuccess;
}

// q as [token][head][dim], copied as ptile tokens x group heads x 64 dims into 128B-swizzled rows; the pool as
// [8-token group][K, V][D * 8 elements in rows of 256], copied as a block's groups of one part.
template <int D, Fill F, bool kScored>
cudaError_t encode_maps(const ExtendParams& p, int act_dtype, CUtensorMap* q_map, CUtensorMap* kv_map) {
  EncodeTiled f;
  const cudaError_t e = encoder(&f);
  if (e != cudaSuccess) return e;
  const CUtensorMapDataType type = act_dtype == PA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.num_q_heads, (cuuint64_t)p.num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)p.q_token_stride * 2};
    // (where no sequence has as many queries as a tile, no more than there can be)
    const int ptile = kRows / p.group, positions = kScored && p.max_query_len < ptile ? p.max_query_len : ptile;
    const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)positions};
    if (f(q_map, type, 3, const_cast<void*>(p.q), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (F == kBulk) {
    const cuuint64_t groups = (cuuint64_t)p.num_blocks * p.num_kv_heads * (p.block_size / 8);
    const cuuint64_t dims[4] = {256, D / 32, 2, groups};
    const cuuint64_t strides[3] = {512, (cuuint64_t)D * 16, (cuuint64_t)D * 32};
    const cuuint32_t box[4] = {256, D / 32, 1, (cuuint32_t)(p.block_size / 8)};
    if (f(kv_map, type, 4, const_cast<uint8_t*>(p.cache), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

template <typename T, int D, Fill F, int kShape>
cudaError_t launch_fill(const ExtendParams& p, const Space& ws, int sms, cudaStream_t stream) {
  using C = Cfg<T, D, F, kShape>;
  constexpr bool kScored = kShape != kNone;
  constexpr size_t smem = 2 * C::kQBytes + C::kRingBytes + sizeof(Shared) + (F == kCodes ? sizeof(Scales) + kKv * D : 0);
  static_assert(smem <= 227 * 1024 && sizeof(Shared) % 16 == 0, "shared memory");
  cudaError_t e = set_smem_attribute_once<extend_kernel<T, D, F, kShape>>(smem);
  if (e != cudaSuccess) return e;
  CUtensorMap q_map{}, kv_map{};
  e = encode_maps<D, F, kScored>(p, std::is_same<T, __half>::value ? PA_F16 : PA_BF16, &q_map, &kv_map);
  if (e != cudaSuccess) return e;
  plan_kernel<kScored><<<1, kPlanThreads, 0, stream>>>(p, ws, sms);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_early(extend_kernel<T, D, F, kShape>, sms, C::kThreads, smem, stream, p, ws, q_map, kv_map);
  if (e != cudaSuccess) return e;
  return launch_early(finish_kernel<T, D, F == kCodes, kScored>, 2 * sms, 256, 0, stream, p, ws);
}

template <int kShape, typename T>
cudaError_t launch_typed(const ExtendParams& p, const Space& ws, int sms, int head_size, bool i8, cudaStream_t stream) {
  if (i8) return launch_fill<T, 128, kCodes, kShape>(p, ws, sms, stream);
  const bool bulk = p.block_size >= 8;                               // whole 8-token groups
  if (head_size == 128)
    return bulk ? launch_fill<T, 128, kBulk, kShape>(p, ws, sms, stream)
                : launch_fill<T, 128, kGather, kShape>(p, ws, sms, stream);
  return bulk ? launch_fill<T, 64, kBulk, kShape>(p, ws, sms, stream)
              : launch_fill<T, 64, kGather, kShape>(p, ws, sms, stream);
}

template <int kShape>
cudaError_t launch(const ExtendParams& p, void* workspace, int sms, int act_dtype, int head_size, bool i8,
                   cudaStream_t stream) {
  size_t bytes;
  const Space ws = lay_out(static_cast<uint8_t*>(workspace), p.num_seqs, p.num_tokens, p.num_kv_heads, p.group,
                           p.max_query_len, head_size, sms, kShape != kNone, &bytes);
  return act_dtype == PA_F16 ? launch_typed<kShape, __half>(p, ws, sms, head_size, i8, stream)
                             : launch_typed<kShape, __nv_bfloat16>(p, ws, sms, head_size, i8, stream);
}

}  // namespace
}  // namespace pkv
