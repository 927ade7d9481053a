// Index arithmetic of the attention of packed rows, plain C++ for host and device (internal; not part
// of the C ABI): how the rows of a request form tiles, which key tiles a block of them sees, and the
// line that all key tiles of a call form.
//
// A request of c rows over a group of rep query heads: a tile has 128 rows of one head or, where the
// request has 64 rows or fewer, all its rows of several heads.  A block is what a pair of tiles covers:
// the same rows of two tiles' heads, or two tiles' rows of one head where the group's tiles are odd.
#pragma once

#include "window_index.h"

namespace mikv {

struct RowTiles {
  int32_t tb, hb;       // rows of a tile, and heads
  int32_t groups;       // tiles side by side in a group of query heads
  int32_t blocks, per;  // blocks of rows, and pairs of tiles of one block and key head
  bool pair_heads;
};
MIKV_HD RowTiles row_tiles_of(int32_t rows, int32_t rep) {
  RowTiles t;
  t.hb = rows <= kKeyRows / 2 ? min_of(rep, kKeyRows / max_of(rows, 1)) : 1;
  t.tb = t.hb > 1 ? max_of(rows, 1) : kKeyRows;
  t.groups = (rep + t.hb - 1) / t.hb;
  const int32_t tiles = (rows + t.tb - 1) / t.tb;
  t.pair_heads = t.groups % 2 == 0 || tiles <= 1;
  t.blocks = t.pair_heads ? tiles : (tiles + 1) / 2;
  t.per = t.pair_heads ? (t.groups + 1) / 2 : t.groups;
  return t;
}
MIKV_HD int32_t block_row(const RowTiles& t, int32_t blk) { return (t.pair_heads ? blk : 2 * blk) * t.tb; }

// A request's rows: `rows` of them, the first at position `off` (below 0: it sees nothing), over `keys` keys.
struct Rows {
  int32_t rows, off, keys;
};
constexpr int32_t kMaxPos = 1 << 30;   // positions of a request's first row are held here, and slots lie below
// `held`: slots of its sequence.  A request that is refused has no keys: a start below 0, or without starts
// more rows than slots, as in the row maps.
MIKV_HD Rows rows_of(int32_t rows, int32_t held, bool from_start, int32_t start) {
  Rows r;
  r.rows = rows;
  r.off = from_start ? min_of(max_of(start, -1), kMaxPos) : held - rows;
  // keys that its last row sees: below 2^30 + 2^20
  r.keys = (from_start ? start < 0 : rows > held) || held <= 0 ? 0 : max_of(0, min_of(held, r.off + rows));
  return r;
}

// The key tiles of KT keys that the rows of a block see, as KeyTiles says.
template <int KT>
MIKV_HD KeyTiles chunk_tiles(const RowTiles& t, const Rows& r, int32_t window, int32_t sinks, int32_t blk) {
  const int32_t q0 = block_row(t, blk);
  const int32_t p1 = r.off + min_of(q0 + (t.pair_heads ? t.tb : 2 * t.tb), r.rows) - 1;   // the largest position
  const int32_t last = min_of(p1, r.keys - 1);
  const int32_t lo = window > 0 ? max_of(r.off + q0 - window + 1, 0) : 0;
  const int32_t end = last < 0 ? 0 : last / KT + 1;
  const int32_t st = window > 0 && sinks > 0 ? (min_of(sinks, max_of(r.keys, 1)) - 1) / KT + 1 : 0;
  KeyTiles k;
  k.tw0 = min_of(lo / KT, end);
  k.ts = min_of(st, k.tw0);
  k.tiles = k.ts + end - k.tw0;
  k.ns = max_of(k.ts, min_of(st, st > k.tw0 ? k.tiles : k.ts));
  return k;
}
// The line: every item takes kChunkPlaces places for what it costs beside its key tiles, and `weight` a tile: eight
// where two tiles of rows meet it, five where one does.  (Four chunks beside sixty single tokens, 304 us with equal
// weights: 276 with 3 to 4, 258 with 5 to 8, 272 with 1 to 2; 8192 causal rows of 32 heads, 424 us with two tiles'
// places an item, 377 with three, 370 with four, 374 with five.)  INT8 tiles cost the same, whatever the rows: their
// codes' conversion.
constexpr int kChunkPlaces = 32;
template <int KT>
MIKV_HD int32_t tile_weight(const RowTiles& t) {
  return KT == kKeyRows && t.groups == 1 && t.blocks <= 1 ? 5 : 8;
}
// Places of each item of a block; the tile that a boundary `at` places behind an item's begin names (0: its begin).
template <int KT>
MIKV_HD int32_t chunk_places(const RowTiles& t, const Rows& r, int32_t window, int32_t sinks, int32_t blk) {
  return kChunkPlaces + tile_weight<KT>(t) * max_of(1, chunk_tiles<KT>(t, r, window, sinks, blk).tiles);
}
MIKV_HD int32_t chunk_tile(int32_t at, int32_t weight) { return max_of(0, at - kChunkPlaces) / weight; }
// CTAs that get a part: not fewer than two tiles each, as far as there are any.
MIKV_HD int32_t chunk_workers(int64_t total, int32_t ctas) {
  return total / 16 >= ctas ? ctas : max_of(1, static_cast<int32_t>(total / 16));
}

}  // namespace mikv
