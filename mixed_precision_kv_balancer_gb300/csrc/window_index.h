// Index arithmetic of windowed attention, plain C++ for host and device (internal; not part of
// the C ABI): which key tiles the query rows of an item see, and the line that all key tiles of a
// call form where they are shared out over the CTAs in equal parts.
#pragma once

#include "page_index.h"

namespace mikv {

constexpr int kKeyRows = 128;   // rows of a key tile

// The row blocks of a call: tb rows (a pair of heads' tiles) or 2 tb (two tiles of one head) each.
struct QueryBlocks {
  int32_t window, sinks, blocks, tb;
  bool pair_heads;
};
MIKV_HD int32_t min_of(int32_t x, int32_t y) { return x < y ? x : y; }
MIKV_HD int32_t max_of(int32_t x, int32_t y) { return x > y ? x : y; }
MIKV_HD int32_t first_row(const QueryBlocks& q, int32_t blk) { return (q.pair_heads ? blk : 2 * blk) * q.tb; }

// The key tiles that the rows of a block see: ts of the sinks, then tw0, tw0 + 1, ...; `tiles` of
// them, the first `ns` with sinks.
struct KeyTiles {
  int32_t ts, tw0, tiles, ns;
};
MIKV_HD KeyTiles key_tiles(const QueryBlocks& q, int32_t ql, int32_t kl, int32_t blk) {
  const int32_t q0 = first_row(q, blk), off = kl - ql;
  const int32_t p1 = off + min_of(q0 + (q.pair_heads ? q.tb : 2 * q.tb), ql) - 1;   // the largest position
  const int32_t lo = q.window > 0 ? max_of(off + q0 - q.window + 1, 0) : 0;
  const int32_t end = p1 < 0 ? 0 : p1 / kKeyRows + 1;
  const int32_t sinks = q.window > 0 ? (min_of(q.sinks, kl) + kKeyRows - 1) / kKeyRows : 0;
  KeyTiles k;
  k.tw0 = min_of(lo / kKeyRows, end);
  k.ts = min_of(sinks, k.tw0);
  k.tiles = k.ts + end - k.tw0;
  // where the window begins among the sinks the list is 0, 1, 2, ... and its first `sinks` hold
  // sinks, which a later query tile sees though its own window begins behind them
  k.ns = max_of(k.ts, min_of(sinks, sinks > k.tw0 ? k.tiles : k.ts));
  return k;
}

// The line: entry e is row block blocks - 1 - e % blocks of batch row e / blocks.  Each of its items, one
// after the other, takes kItemPlaces places for what it costs beside its tiles and one place a tile;
// rows that count take a tile's place even where they see nothing: an answer is due.  CTA c of
// `workers` takes places [line_begin(total, workers, c), line_begin(total, workers, c + 1)), where a boundary among an item's first kItemPlaces places, or on its first tile, is the item's begin.
constexpr int kItemPlaces = 3;
MIKV_HD int32_t entry_places(const QueryBlocks& q, int32_t ql, int32_t kl, int32_t blk) {
  return first_row(q, blk) >= ql ? 0 : kItemPlaces + max_of(1, key_tiles(q, ql, kl, blk).tiles);
}
// The tile of an item of `places` that a boundary `at` places behind its begin names.
MIKV_HD int32_t line_tile(int32_t at) { return max_of(0, at - kItemPlaces); }
// CTAs that get a part: not fewer than two places each, as far as there are any.
MIKV_HD int32_t line_workers(int32_t total, int32_t ctas) { return max_of(1, min_of(ctas, total / 2)); }

// split_begin in 32 bits: total c / workers for c <= workers < 2^15.
MIKV_HD int32_t line_begin(int32_t total, int32_t workers, int32_t c) {
  const int32_t each = total / workers, rest = total - each * workers;
  return each * c + rest * c / workers;
}

}  // namespace mikv
