"""Paged cache and windowed attention without a GPU: the calls' refusals, the index arithmetic
of the kernels (compiled for the host), and hand-checked scenarios of the oracle."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle.paged as op
from conftest import ROOT

EINVAL, ESHAPE, EALIGN, EUNSUP = -1, -2, -3, -4
FAKE = 4096      # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def lib():
    from mixed_precision_kv_balancer_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build_library()
    return _lib.load()


def _pages(**kw):
    from mixed_precision_kv_balancer_gb300 import _lib
    p = _lib.mikv_pages()
    p.layers, p.n_pages, p.page_size, p.Hkv, p.D, p.type, p.max_seqs, p.max_pages = 2, 8, 16, 2, 128, 0, 4, 4
    p.k = p.v = p.table = p.lens = p.refs = FAKE
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


def _rows(data=FAKE, sb=1024, sh=512, st=128):
    from mixed_precision_kv_balancer_gb300 import _lib
    return ctypes.byref(_lib.mikv_rows(data, sb, sh, st))


BAD_PAGES = [(None, EINVAL), (dict(type=3), EINVAL), (dict(D=64), EUNSUP), (dict(page_size=0), ESHAPE),
             (dict(page_size=4097), ESHAPE), (dict(layers=0), ESHAPE), (dict(n_pages=0), ESHAPE),
             (dict(Hkv=0), ESHAPE), (dict(Hkv=1025), ESHAPE), (dict(max_seqs=0), ESHAPE),
             (dict(max_pages=0), ESHAPE), (dict(max_pages=1 << 27), ESHAPE),
             (dict(n_pages=1 << 27, page_size=16), ESHAPE), (dict(k=None), EINVAL), (dict(table=None), EINVAL),
             (dict(refs=None), EINVAL), (dict(type=2), EINVAL), (dict(v=FAKE + 8), EALIGN),
             (dict(type=2, k_meta=FAKE, v_meta=FAKE + 4), EALIGN)]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_every_paged_call_checks_the_cache(lib, kw, code):
    p = None if kw is None else _pages(**kw)
    big = 1 << 34
    assert lib.mikv_page_reserve(p, None, FAKE, 1, FAKE, FAKE, big, None) == code
    assert lib.mikv_page_fork(p, FAKE, FAKE, 1, FAKE, FAKE, big, None) == code
    assert lib.mikv_page_free(p, None, 1, FAKE, None) == code
    assert lib.mikv_page_copy(p, FAKE, FAKE, 1, FAKE, None) == code
    assert lib.mikv_page_compact(p, None, FAKE, FAKE, 1, 1, FAKE, FAKE, big, None) == code
    assert lib.mikv_paged_append(p, 0, _rows(), _rows(), 1, 1, None, None, None, None) == code
    assert lib.mikv_paged_gather(p, 0, None, 1, 1, _rows(), _rows(), None) == code
    assert lib.mikv_paged_attention(FAKE, p, 0, None, 1, 4, 0, 0, FAKE, None, FAKE, big, None) == code
    assert lib.mikv_paged_attention_workspace_bytes(p, 1, 4, 0, 0) == 0


def test_page_calls_refuse(lib):
    p, big = _pages(), 1 << 30
    ws = lib.mikv_page_workspace_bytes(p, 3)
    assert ws >= 8 * 4 + 3 * 4 and lib.mikv_page_workspace_bytes(p, 0) == 0 and lib.mikv_page_workspace_bytes(p, 4097) == 0
    for call in (lambda n, a, o, w, nb: lib.mikv_page_reserve(p, FAKE, a, n, o, w, nb, None),
                 lambda n, a, o, w, nb: lib.mikv_page_fork(p, FAKE, a, n, o, w, nb, None),
                 lambda n, a, o, w, nb: lib.mikv_page_compact(p, FAKE, FAKE, a, n, 1, o, w, nb, None)):
        assert call(0, None, None, None, 0) == 0                  # nothing to do
        assert call(-1, FAKE, FAKE, FAKE, big) == ESHAPE
        assert call(4097, FAKE, FAKE, FAKE, big) == ESHAPE
        assert call(1, None, FAKE, FAKE, big) == EINVAL
        assert call(1, FAKE, None, FAKE, big) == EINVAL
        assert call(1, FAKE, FAKE, None, big) == EINVAL
        assert call(1, FAKE, FAKE, FAKE + 4, big) == EALIGN
        assert call(3, FAKE, FAKE, FAKE, ws - 1) == ESHAPE
        assert b"workspace" in lib.mikv_last_error()
    assert lib.mikv_page_reserve(p, None, FAKE, 5, FAKE, FAKE, big, None) == ESHAPE      # 4 sequences
    assert lib.mikv_page_free(p, None, 5, FAKE, None) == ESHAPE
    assert lib.mikv_page_free(p, FAKE, 65536, FAKE, None) == ESHAPE
    assert lib.mikv_page_free(p, FAKE, 1, None, None) == EINVAL
    assert lib.mikv_page_free(p, None, 0, None, None) == 0
    assert lib.mikv_page_copy(p, None, FAKE, 1, FAKE, None) == EINVAL
    assert lib.mikv_page_copy(p, FAKE, FAKE, -1, FAKE, None) == ESHAPE
    assert lib.mikv_page_copy(p, None, None, 0, None, None) == 0
    assert lib.mikv_page_compact(p, None, FAKE, FAKE, 1, -1, FAKE, FAKE, big, None) == ESHAPE
    assert lib.mikv_page_compact(p, None, FAKE, FAKE, 1, 65, FAKE, FAKE, big, None) == ESHAPE   # 64 slots a sequence
    assert lib.mikv_page_compact(p, None, None, FAKE, 1, 1, FAKE, FAKE, big, None) == EINVAL


def test_row_calls_refuse(lib):
    p = _pages()
    for call in (lambda layer, k, n, T: lib.mikv_paged_append(p, layer, k, _rows(), n, T, None, None, None, None),
                 lambda layer, k, n, T: lib.mikv_paged_gather(p, layer, None, n, T, k, _rows(), None)):
        assert call(2, _rows(), 1, 1) == ESHAPE
        assert call(-1, _rows(), 1, 1) == ESHAPE
        assert call(0, _rows(), 5, 1) == ESHAPE
        assert call(0, _rows(), 1, -1) == ESHAPE
        assert call(0, _rows(), 0, 1) == 0
        assert call(0, _rows(), 1, 0) == 0
        assert call(0, None, 1, 1) == EINVAL
        assert call(0, _rows(data=None), 1, 1) == EINVAL
        assert call(0, _rows(data=FAKE + 2), 1, 1) == EALIGN
        assert call(0, _rows(st=129), 1, 1) == EALIGN
        assert call(0, _rows(sh=-128), 1, 1) == EINVAL


def test_attention_calls_refuse(lib):
    p, big = _pages(), 1 << 30
    pa = lambda q=FAKE, layer=0, n=1, Hq=4, window=0, sinks=0, out=FAKE, ws=FAKE, nb=big: lib.mikv_paged_attention(
        q, p, layer, None, n, Hq, window, sinks, out, None, ws, nb, None)
    assert pa(n=0, q=None, ws=None) == 0
    for kw in (dict(layer=2), dict(n=-1), dict(n=5), dict(Hq=3), dict(Hq=0), dict(nb=64)):
        assert pa(**kw) == ESHAPE, kw
    for kw in (dict(window=-1), dict(sinks=-1), dict(q=None), dict(out=None), dict(ws=None)):
        assert pa(**kw) == EINVAL, kw
    for kw in (dict(q=FAKE + 2), dict(out=FAKE + 8), dict(ws=FAKE + 4)):
        assert pa(**kw) == EALIGN, kw
    assert lib.mikv_paged_attention_workspace_bytes(p, 1, 3, 0, 0) == 0
    assert lib.mikv_paged_attention_workspace_bytes(p, 1, 4, 0, 0) > 0
    # a workspace for no window serves every window
    assert lib.mikv_paged_attention_workspace_bytes(p, 2, 4, 0, 0) >= lib.mikv_paged_attention_workspace_bytes(p, 2, 4, 17, 3)

    def wa(q=_rows(), k=_rows(), v=_rows(), out=_rows(), B=1, Hq=4, Hkv=2, Tq=8, Tk=8, D=128, type=0, window=0, sinks=0, ws=None, nb=0):
        return lib.mikv_window_attention(q, k, v, B, Hq, Hkv, Tq, Tk, D, type, None, None, window, sinks, out, None, ws, nb, None)
    assert wa(B=0) == 0
    for kw in (dict(B=-1), dict(B=65536), dict(Hq=5), dict(Hkv=0), dict(Tq=0), dict(Tk=0)):
        assert wa(**kw) == ESHAPE, kw
    for kw in (dict(type=2), dict(window=-1), dict(sinks=-1), dict(q=None), dict(out=None), dict(v=_rows(sb=-8))):
        assert wa(**kw) == EINVAL, kw
    assert wa(D=64) == EUNSUP
    # a chunk of few rows behind many keys is split, and needs a workspace
    many = dict(Tk=8192, Tq=16, k=_rows(sb=1 << 21, sh=1 << 20), v=_rows(sb=1 << 21, sh=1 << 20))
    need = lib.mikv_window_attention_workspace_bytes(1, 4, 2, 16, 8192, 0, 0)
    assert need >= 2 * 4 * 16 * 130 * 4
    assert wa(**many) == EINVAL and wa(ws=FAKE, nb=need - 1, **many) == ESHAPE and wa(ws=FAKE + 16, nb=need, **many) == EALIGN
    assert lib.mikv_window_attention_workspace_bytes(8, 64, 8, 4096, 4096, 0, 0) == 0
    assert lib.mikv_window_attention_workspace_bytes(1, 5, 2, 16, 8192, 0, 0) == 0
    assert wa(q=_rows(st=64)) == EINVAL and wa(out=_rows(sh=0)) == EINVAL and wa(k=_rows(st=0)) == EINVAL   # rows overlap
    for kw in (dict(q=_rows(st=132)), dict(k=_rows(data=FAKE + 4)), dict(v=_rows(sh=4)), dict(out=_rows(sb=2))):
        assert wa(**kw) == EALIGN, kw


HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "page_index.h"
using namespace mikv;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  const uint32_t top = 0x7fffffffu;
  for (uint32_t d = 1; d <= 4096; ++d) {
    const FastDiv f = make_fast_div(d);
    for (uint32_t q = 0; q < 200; ++q)
      for (int e = -1; e <= 1; ++e) {
        const uint32_t x = q * d + e;
        if (x <= top) CHECK(div_of(x, f) == x / d);
        const uint32_t y = (top / d - q) * d + e;
        if (y <= top) CHECK(div_of(y, f) == y / d);
      }
    for (int32_t len : {0, 1, (int)d - 1, (int)d, (int)d + 1, 0x7fffffff - 4096})
      CHECK(pages_of(len, f) == (int32_t)(((int64_t)len + d - 1) / d));
  }
  for (int len = 0; len < 40; ++len)
    for (int window = 0; window < 45; ++window)
      for (int sinks = 0; sinks < 45; ++sinks) {
        const Visible v = visible_slots(len, window, sinks);
        int i = 0;
        for (int j = 0; j < len; ++j)
          if (window == 0 || j > len - 1 - window || j < sinks) {
            CHECK(i < v.count && visible_slot(v, i) == j);
            ++i;
          }
        CHECK(i == v.count);
      }
  // pages outside the pool have no row, pages inside it a row below n_pages * heads * ps
  const int32_t n = 7, heads = 3;
  const uint32_t ps = 5;
  for (int32_t page : {-1, -2147483647 - 1, 7, 8, 2147483647})
    CHECK(pool_row(page, n, heads, 2, ps, 4) == kNoRow);
  for (int32_t page = 0; page < n; ++page)
    for (int h = 0; h < heads; ++h)
      for (uint32_t r = 0; r < ps; ++r) CHECK(pool_row(page, n, heads, h, ps, r) == (uint32_t)((page * heads + h) * ps + r));
  CHECK(pool_row(16777214, 16777215, 16, 15, 16, 15) == 4294967039u);   // the largest pools: 32 bits hold every row
  // the split: parts are in order, cover every tile once, and differ by at most one tile
  for (int64_t total : {1LL, 2LL, 7LL, 303LL, 304LL, 305LL, 32768LL, 70368744177663LL})
    for (int workers : {1, 2, 5, 304}) {
      CHECK(split_begin(total, workers, 0) == 0 && split_begin(total, workers, workers) == total);
      for (int c = 0; c < workers; ++c) {
        const int64_t b = split_begin(total, workers, c), e = split_begin(total, workers, c + 1);
        CHECK(b <= e && e - b <= total / workers + 1);
        if (total >= workers) CHECK(b < e);   // with no more workers than tiles no part is empty
        if (b < e) CHECK(split_owner(total, workers, b) == c && split_owner(total, workers, e - 1) == c);
      }
    }
  return 0;
}
"""


def test_index_arithmetic_of_the_kernels(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "index.cpp"
    src.write_text(HARNESS)
    inc = os.path.join(ROOT, "mixed_precision_kv_balancer_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", inc, str(src),
                    "-o", str(tmp_path / "index")], check=True)
    res = subprocess.run([str(tmp_path / "index")], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr


# --- the oracle, by hand ----------------------------------------------------------------

def _oracle(n_pages=6, ps=4, seqs=4, width=4):
    k = np.arange(n_pages * ps, dtype=np.float64).reshape(1, n_pages, 1, ps, 1)
    return op.Pages(k, -k, np.full((seqs, width), -1, np.int32), np.zeros(seqs, np.int32), np.zeros(n_pages, np.int32))


def test_oracle_pages_by_hand():
    o = _oracle()
    assert o.reserve([0, 1, 0], [6, 1, 1]).tolist() == [0, 0, -1]        # the repeated request is refused
    assert o.table[:2].tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]] and o.refs.tolist() == [1, 1, 1, 0, 0, 0]
    assert o.fork([0, 0, 1], [2, 1, 3]).tolist() == [1, 0, 1]            # 1 is not empty (and a parent)
    assert o.table[2].tolist() == [0, 3, -1, -1] and o.table[3].tolist() == [4, -1, -1, -1]
    assert o.refs.tolist() == [2, 1, 1, 1, 1, 0]
    assert o.k[0, 3, 0, :, 0].tolist() == [4, 5, 14, 15]                 # two filled rows copied
    assert o.reserve([0, 1, 2], [3, 9, 3]).tolist() == [6, -1, -1]       # one free page: 1 and all after it wait
    assert o.reserve([2], [2]).tolist() == [6]                           # no page needed
    assert o.compact([2], np.array([[[[7, 0, 4]]]]), [3]).tolist() == [0]  # no free page for the new ones
    assert o.free([1, 1, 9]).tolist() == [1, 0, 0]
    assert o.compact([2], np.array([[[[7, 0, 4]]]]), [3]).tolist() == [1]
    assert o.k[0, 2, 0, :3, 0].tolist() == [15, 0, 4] and o.table[2].tolist() == [2, -1, -1, -1]
    assert o.refs.tolist() == [1, 1, 1, 0, 1, 1] and o.lens.tolist() == [9, 0, 3, 1]
    assert o.copy([0, 0, 1, 9], [3, 3, 0, 1]).tolist() == [1, 0, 0, 0]   # 0 is read by a pair: not written


def test_oracle_visibility_by_hand():
    assert np.flatnonzero(op.visible(9, 12, 3, 2)).tolist() == [0, 1, 7, 8, 9]
    assert np.flatnonzero(op.visible(2, 12, 3, 2)).tolist() == [0, 1, 2]
    assert np.flatnonzero(op.visible(-1, 12, 3, 2)).tolist() == []
    q, k, v = np.ones((1, 1, 2, 4)), np.zeros((1, 1, 3, 4)), np.arange(12.0).reshape(1, 1, 3, 4)
    out, lse, _ = op.window_attention(q, k, v, 2, 0)
    np.testing.assert_allclose(out[0, 0], [(v[0, 0, 0] + v[0, 0, 1]) / 2, (v[0, 0, 1] + v[0, 0, 2]) / 2])
    np.testing.assert_allclose(lse[0, 0], np.log([2.0, 2.0]))
    out, lse, _ = op.window_attention(q, k, v, 0, 0, q_lens=[2], k_lens=[1])
    assert out[0, 0, 0].tolist() == [0] * 4 and lse[0, 0, 0] == -np.inf  # one key, two queries: the first sees none
