"""Index arithmetic of the attention of packed rows, compiled for the host: how rows form tiles, the key tiles of a
block of them, and the parts of the line of all key tiles."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "chunk_index.h"
using namespace mikv;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
static unsigned seed = 1;
static int pick(int lo, int hi) { seed = seed * 1664525u + 1013904223u; return lo + (int)((seed >> 8) % (unsigned)(hi - lo + 1)); }

// every (row, query head) of a request is in one tile, and no tile has more than 128 rows
static int check_rows(int rows, int rep) {
  const RowTiles t = row_tiles_of(rows, rep);
  CHECK(t.blocks <= rows / kKeyRows + 1 && (rows > 0) == (t.blocks > 0));
  CHECK(t.tb >= 1 && t.hb >= 1 && t.tb * t.hb <= kKeyRows && min_of(t.tb, rows) * t.hb <= rows * rep);
  std::vector<int> seen(rows * rep, 0);
  for (int blk = 0; blk < t.blocks; ++blk)
    for (int u = 0; u < t.per; ++u)
      for (int i = 0; i < 2; ++i) {
        const int group = t.pair_heads ? 2 * u + i : u, heads = min_of(t.hb, rep - group * t.hb);
        const int q0 = block_row(t, blk) + (t.pair_heads ? 0 : i * t.tb);
        if (i == 0) CHECK(heads > 0 && q0 < rows);
        if (q0 >= rows || heads <= 0) continue;
        for (int r = 0; r < kKeyRows; ++r) {
          const int sub = r / t.tb, q = q0 + r - sub * t.tb;
          if (sub < heads && q < rows) ++seen[q * rep + group * t.hb + sub];
        }
      }
  for (int x : seen) CHECK(x == 1);
  return 0;
}

// the tiles of a block's list are those that one of its rows sees, each once, sinks first
template <int KT>
static int check_tiles(const RowTiles& t, const Rows& r, int window, int sinks) {
  for (int blk = 0; blk < t.blocks; ++blk) {
    const int q0 = block_row(t, blk), q1 = min_of(q0 + (t.pair_heads ? t.tb : 2 * t.tb), r.rows);
    const KeyTiles k = chunk_tiles<KT>(t, r, window, sinks, blk);
    std::vector<int> sees(r.keys / KT + 1, 0), sink(sees.size(), 0), listed(sees.size(), 0);
    for (int i = q0; i < q1; ++i) {
      const int p = r.off + i;
      for (int j = 0; j <= p && j < r.keys; ++j)
        if (window == 0 || j > p - window || j < sinks) sees[j / KT] = 1;
    }
    for (int j = 0; j < min_of(sinks, r.keys); ++j) sink[j / KT] = window > 0;
    for (int i = 0; i < k.tiles; ++i) {
      const int tile = i < k.ts ? i : k.tw0 + i - k.ts;
      CHECK(tile >= 0 && tile < (int)sees.size() && !listed[tile]);
      listed[tile] = 1;
      if (sink[tile]) CHECK(i < k.ns);
    }
    for (size_t x = 0; x < sees.size(); ++x) CHECK(!sees[x] || listed[x]);
    int seen = 0;
    for (int x : sees) seen += x;
    CHECK(k.tiles <= seen + 1);
    CHECK(chunk_places<KT>(t, r, window, sinks, blk) == kChunkPlaces + tile_weight<KT>(t) * max_of(1, k.tiles));
  }
  return 0;
}

// CTAs walk their parts as the kernel does: every item's tiles are taken once and in order; an item that is cut has
// its parts in slots of their own, which the CTA that begins it can tell
template <int KT>
static int check_line(const std::vector<Rows>& reqs, int rep, int heads, int window, int sinks, int ctas) {
  struct Entry { int req, blk, places, items, weight; long long base; };
  std::vector<Entry> line;
  long long total = 0;
  for (size_t i = 0; i < reqs.size(); ++i) {
    const RowTiles t = row_tiles_of(reqs[i].rows, rep);
    for (int b = 0; b < t.blocks; ++b) {
      const int p = chunk_places<KT>(t, reqs[i], window, sinks, b);
      line.push_back({(int)i, b, p, heads * t.per, tile_weight<KT>(t), total});
      total += (long long)p * heads * t.per;
    }
  }
  if (total == 0) return 0;
  const int workers = chunk_workers(total, ctas);
  struct Seg { int t0, t1, slot; };
  struct Cut { long long begin; int last, before; };
  std::vector<std::vector<Seg>> parts(total);
  std::vector<Cut> cuts;
  const auto find = [&](long long x) { int e = 0; while (e + 1 < (int)line.size() && line[e + 1].base <= x) ++e; return e; };
  for (int c = 0; c < workers; ++c) {
    long long x = split_begin(total, workers, c), y = split_begin(total, workers, c + 1);
    CHECK(x < y);
    int e = find(x), in = (int)((x - line[e].base) % line[e].places), item = (int)((x - line[e].base) / line[e].places);
    int left = line[e].items - 1 - item, t0 = chunk_tile(in, line[e].weight);
    if (t0 == 0) x -= in;
    const long long begin = x - (t0 == 0 ? 0 : in);
    Cut cut = {0, -1, 0};
    if (y < total) {
      const int f = find(y);
      const long long b = line[f].base + (y - line[f].base) / line[f].places * line[f].places;
      if (chunk_tile((int)(y - b), line[f].weight) == 0) y = b;
      else if (b >= x) cut = {b, split_owner(total, workers, b + line[f].places - 1), b > x};
    }
    cuts.push_back(cut);
    if (x >= y) continue;
    long long to_go = y - begin, at = begin;
    int places = line[e].places;
    const auto end = [&] { return chunk_tile((int)(to_go < places ? to_go : places), line[e].weight); };
    int t1 = end();
    for (int n = 0;; ++n) {
      const int tiles = (places - kChunkPlaces) / line[e].weight;
      const bool whole = t0 == 0 && t1 == tiles;
      CHECK(t1 > t0 && t1 <= tiles);
      parts[at].push_back({t0, t1, whole ? -1 : 2 * c + (n > 0)});
      CHECK(whole || n == 0 || to_go <= places);   // cut items: a CTA's first and last
      to_go -= places;
      at += places;
      if (to_go <= 0) break;
      if (--left < 0) {
        ++e;
        left = line[e].items - 1;
        places = line[e].places;
      }
      t0 = 0;
      t1 = end();
    }
  }
  std::vector<char> used(2 * ctas, 0), joined(total, 0);
  for (int c0 = 0; c0 < (int)cuts.size(); ++c0) {
    if (cuts[c0].last < 0) continue;
    const auto& segs = parts[cuts[c0].begin];
    CHECK(cuts[c0].last > c0 && cuts[c0].last < workers && (int)segs.size() == cuts[c0].last - c0 + 1);
    for (size_t i = 0; i < segs.size(); ++i) {
      const int slot = 2 * (c0 + (int)i) + (i == 0 ? cuts[c0].before : 0);
      CHECK(segs[i].slot == slot && !used[slot]);
      used[slot] = 1;
    }
    joined[cuts[c0].begin] = 1;
  }
  for (const Entry& e : line)
    for (int i = 0; i < e.items; ++i) {
      const auto& segs = parts[e.base + (long long)i * e.places];
      int next = 0;
      for (const Seg& s : segs) { CHECK(s.t0 == next); next = s.t1; }
      CHECK(next == (e.places - kChunkPlaces) / e.weight);
      CHECK((segs.size() > 1) == (joined[e.base + (long long)i * e.places] != 0) && (segs.size() == 1) == (segs[0].slot < 0));
    }
  return 0;
}

static Rows request() {
  const int rows = pick(0, 2) ? pick(0, 9) : pick(0, 700), held = pick(0, 4) ? pick(0, 900) : 0;
  return rows_of(rows, held, pick(0, 2) == 0, pick(-1, 800));
}

int main() {
  for (int rows = 0; rows < 700; ++rows)
    for (int rep : {1, 2, 3, 4, 5, 7, 8, 16, 17, 40, 130}) if (check_rows(rows, rep)) return 1;
  for (int n = 0; n < 4000; ++n) {
    const Rows r = request();
    CHECK(r.keys >= 0 && r.keys <= 900);
    const int window = pick(0, 3) ? pick(1, 700) : 0, sinks = pick(0, 2) ? pick(0, 300) : 0;
    const RowTiles t = row_tiles_of(r.rows, pick(1, 17));
    if (check_tiles<128>(t, r, window, sinks) || check_tiles<64>(t, r, window, sinks)) return 1;
  }
  for (int n = 0; n < 4000; ++n) {
    std::vector<Rows> reqs(pick(1, 30));
    for (Rows& r : reqs) r = request();
    const int rep = pick(1, 17), heads = pick(1, 4), window = pick(0, 1) * pick(1, 500), sinks = pick(0, 200), ctas = pick(0, 3) ? 152 : pick(1, 152);
    if (check_line<128>(reqs, rep, heads, window, sinks, ctas) || check_line<64>(reqs, rep, heads, window, sinks, ctas)) return 1;
  }
  // positions at their limits stay inside 32 bits
  for (int rows : {1, 64, 65, 1 << 20})
    for (int held : {0, 1, 1 << 30})
      for (int start : {-1, 0, 1 << 30, 0x7fffffff})
        for (int window : {0, 1, 1 << 30})
          for (int sinks : {0, 1, 1 << 30}) {
            const Rows r = rows_of(rows, held, true, start);
            const RowTiles t = row_tiles_of(rows, 3);
            CHECK(r.off <= kMaxPos && r.keys <= held);
            for (int blk : {0, t.blocks - 1}) CHECK(chunk_tiles<64>(t, r, window, sinks, blk).tiles >= 0);
          }
  CHECK(rows_of(1 << 20, 5, false, 0).off == 5 - (1 << 20));
  return 0;
}
"""


def test_index_arithmetic_of_packed_rows(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "chunk_index.cpp"
    src.write_text(HARNESS)
    inc = os.path.join(ROOT, "mixed_precision_kv_balancer_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover", "-I", inc, str(src),
                    "-o", str(tmp_path / "chunk_index")], check=True)
    res = subprocess.run([str(tmp_path / "chunk_index")], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr


BELOW = r"""
#include <initializer_list>
#include "chunk_index.h"
using namespace mikv;
int main() {   // requests that are refused, however far below 0: they see nothing, and no sum leaves 32 bits
  for (int start : {-1, -2, -(1 << 30), -0x7fffffff - 1})
    for (int window : {0, 1, 1 << 30})
      for (int rows : {1, 65, 1 << 20}) {
        const Rows r = rows_of(rows, 100, true, start);
        const RowTiles t = row_tiles_of(rows, 3);
        if (r.keys != 0 || chunk_tiles<128>(t, r, window, 4, 0).tiles != 0 || r.off >= 0) return 1;
      }
  return 0;
}
"""


def test_positions_far_below_zero(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "below.cpp"
    src.write_text(BELOW)
    inc = os.path.join(ROOT, "mixed_precision_kv_balancer_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover", "-I", inc, str(src),
                    "-o", str(tmp_path / "below")], check=True)
    res = subprocess.run([str(tmp_path / "below")], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr


MORE = r"""
#include <cstdio>
#include <initializer_list>
#include "chunk_index.h"
using namespace mikv;
int main() {   // without a start, a request with more rows than its sequence has slots is refused: none of its rows sees a key
  for (int held : {0, 1, 8, 300})
    for (int rows : {1, 2, 8, 10, 64, 65, 301, 1 << 20})
      for (int window : {0, 1, 100, 1 << 30})
        for (int sinks : {0, 4}) {
          const Rows r = rows_of(rows, held, false, 0);
          const RowTiles t = row_tiles_of(rows, 3);
          if (r.keys != (rows > held ? 0 : held)) return std::printf("%d rows, %d slots: %d keys\n", rows, held, r.keys), 1;
          for (int blk = 0; rows > held && blk < t.blocks; ++blk)
            if (chunk_tiles<128>(t, r, window, sinks, blk).tiles || chunk_tiles<64>(t, r, window, sinks, blk).tiles) return 1;
        }
  return 0;
}
"""


def test_more_rows_than_slots_see_nothing(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "more.cpp"
    src.write_text(MORE)
    inc = os.path.join(ROOT, "mixed_precision_kv_balancer_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover", "-I", inc, str(src),
                    "-o", str(tmp_path / "more")], check=True)
    res = subprocess.run([str(tmp_path / "more")], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
