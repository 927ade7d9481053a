"""Index arithmetic of windowed attention, compiled for the host: the key tiles of a row block, and
the line of all key tiles that is shared out in equal parts."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "window_index.h"
using namespace mikv;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
static unsigned seed = 1;
static int pick(int lo, int hi) { seed = seed * 1664525u + 1013904223u; return lo + (int)((seed >> 8) % (unsigned)(hi - lo + 1)); }

// the tiles of a block's list are those that one of its rows sees, each once, sinks first
static int check_tiles(const QueryBlocks& q, int ql, int kl) {
  for (int blk = 0; blk < q.blocks; ++blk) {
    const int q0 = first_row(q, blk), q1 = min_of(q0 + (q.pair_heads ? q.tb : 2 * q.tb), ql);
    if (q0 >= ql) { CHECK(entry_places(q, ql, kl, blk) == 0); continue; }
    const KeyTiles k = key_tiles(q, ql, kl, blk);
    std::vector<int> sees((kl + kKeyRows - 1) / kKeyRows, 0), sink(sees.size(), 0), listed(sees.size(), 0);
    for (int i = q0; i < q1; ++i) {
      const int p = kl - ql + i;
      for (int j = 0; j <= p && j < kl; ++j)
        if (q.window == 0 || j > p - q.window || j < q.sinks) sees[j / kKeyRows] = 1;
    }
    for (int j = 0; j < min_of(q.sinks, kl); ++j) sink[j / kKeyRows] = q.window > 0;
    for (int i = 0; i < k.tiles; ++i) {
      const int tile = i < k.ts ? i : k.tw0 + i - k.ts;
      CHECK(tile >= 0 && tile < (int)sees.size() && !listed[tile]);
      listed[tile] = 1;
      if (sink[tile]) CHECK(i < k.ns);
    }
    for (size_t t = 0; t < sees.size(); ++t) CHECK(!sees[t] || listed[t]);
    int seen = 0;
    for (int x : sees) seen += x;
    CHECK(k.tiles <= seen + 1);   // two blocks' windows may leave one tile between them that neither sees
    CHECK(entry_places(q, ql, kl, blk) == kItemPlaces + max_of(1, k.tiles));
  }
  return 0;
}

// every item's tiles are taken once and in order; an item that is cut has its parts in slots of their own, and
// one boundary, the first inside of it, finds all of them
static int check_line(const std::vector<int>& places, int items, int ctas) {
  int total = 0;
  for (int t : places) total += t * items;
  const int workers = line_workers(total, ctas);
  CHECK(workers >= 1 && workers <= ctas);
  if (total == 0) return 0;
  struct Seg { int t0, t1, slot; };
  struct Cut { int begin, last, second; };   // of a CTA: the item that begins in it and goes on in later ones
  std::vector<Cut> cuts;
  std::vector<std::vector<Seg>> per_item(total);
  for (int c = 0; c < workers; ++c) {
    int x = line_begin(total, workers, c), y = line_begin(total, workers, c + 1);
    CHECK(x == split_begin(total, workers, c) && y == split_begin(total, workers, c + 1));
    CHECK(x < y);
    int e = 0, base = 0;
    while (base + places[e] * items <= x) base += places[e++] * items;
    const int first = (x - base) % places[e];
    if (line_tile(first) == 0) x -= first;
    cuts.push_back({0, -1, 0});
    if (y < total) {
      int f = 0, fbase = 0;
      while (fbase + places[f] * items <= y) fbase += places[f++] * items;
      const int in = (y - fbase) % places[f];
      if (line_tile(in) == 0) y -= in;
      else if (y - in >= x) cuts.back() = {y - in, split_owner(total, workers, y - in + places[f] - 1), y - in > x};
    }
    for (int n = 0; x < y; ++n) {
      const int in = (x - base) % places[e], tiles = places[e] - kItemPlaces;
      const int t0 = line_tile(in), t1 = min_of(tiles, line_tile(in + y - x));
      CHECK(t1 > t0);
      const bool whole = t1 - t0 == tiles;
      const int next = x + places[e] - in;
      CHECK(whole || n == 0 || next >= y);   // cut items: a CTA's first and last
      per_item[x - in].push_back({t0, t1, whole ? -1 : 2 * c + (n > 0)});
      x = next;
      if (x < y && x == base + places[e] * items) {
        base = x;
        do ++e; while (places[e] == 0);
      }
    }
  }
  std::vector<int> used(2 * ctas, 0), joined(total, 0);
  for (int c0 = 0; c0 < (int)cuts.size(); ++c0) {
    const Cut& cut = cuts[c0];
    if (cut.last < 0) continue;
    const auto& segs = per_item[cut.begin];
    CHECK(cut.last > c0 && cut.last < workers && (int)segs.size() == cut.last - c0 + 1);
    for (size_t i = 0; i < segs.size(); ++i) {
      const int slot = 2 * (c0 + (int)i) + (i == 0 ? cut.second : 0);
      CHECK(segs[i].slot == slot && !used[slot]);
      used[slot] = 1;
    }
    CHECK(!joined[cut.begin]);
    joined[cut.begin] = 1;
  }
  int at = 0;
  for (int t : places)
    for (int i = 0; i < (t ? items : 0); ++i, at += t) {
      const auto& segs = per_item[at];
      int next = 0;
      for (const Seg& s : segs) { CHECK(s.t0 == next); next = s.t1; }
      CHECK(next == t - kItemPlaces);
      CHECK((segs.size() > 1) == (joined[at] != 0) && (segs.size() == 1) == (segs[0].slot < 0));
    }
  CHECK(at == total);
  return 0;
}

int main() {
  for (int n = 0; n < 3000; ++n) {
    QueryBlocks q;
    q.window = pick(0, 3) ? pick(1, 700) : 0;
    q.sinks = pick(0, 2) ? pick(0, 300) : 0;
    q.pair_heads = pick(0, 1);
    q.tb = pick(0, 2) ? kKeyRows : pick(1, 64);
    const int Tq = q.tb < kKeyRows ? q.tb : pick(1, 600), per = q.pair_heads ? q.tb : 2 * q.tb;
    q.blocks = (Tq + per - 1) / per;
    if (check_tiles(q, pick(0, Tq), pick(0, 900))) return 1;
  }
  for (int n = 0; n < 20000; ++n) {
    std::vector<int> places(pick(1, 40));
    for (int& t : places) t = pick(0, 3) ? kItemPlaces + pick(1, 1 << pick(0, 7)) : 0;
    if (check_line(places, pick(1, 12), pick(0, 3) ? 152 : pick(1, 152))) return 1;
  }
  // the largest line: no sum passes 32 bits
  const int total = 0x7fffffff, workers = line_workers(total, 152);
  CHECK(workers == 152);
  for (int c = 0; c <= workers; ++c) CHECK(line_begin(total, workers, c) == split_begin(total, workers, c));
  CHECK(split_owner(total, workers, total - 1) == 151);
  return 0;
}
"""


def test_index_arithmetic_of_windowed_attention(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "window_index.cpp"
    src.write_text(HARNESS)
    inc = os.path.join(ROOT, "mixed_precision_kv_balancer_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover", "-I", inc, str(src),
                    "-o", str(tmp_path / "window_index")], check=True)
    res = subprocess.run([str(tmp_path / "window_index")], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
