"""Packed batches without a GPU: the calls' refusals, and the oracle by hand."""
import os

import numpy as np
import pytest

import oracle.batch as ob
from test_paged_host import BAD_PAGES, EALIGN, EINVAL, ESHAPE, FAKE, _pages, _rows


@pytest.fixture(scope="module")
def lib():
    from mixed_precision_kv_balancer_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build_library()
    return _lib.load()


BIG = 1 << 34


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_every_call_checks_the_cache(lib, kw, code):
    p = None if kw is None else _pages(**kw)
    assert lib.mikv_batch_rows(p, None, None, FAKE, 1, 1, FAKE, FAKE, FAKE, FAKE, None) == code
    assert lib.mikv_slot_append(p, 0, _rows(), _rows(), 1, FAKE, None) == code
    assert lib.mikv_page_bounds(p, 0, FAKE, FAKE, 1, FAKE, FAKE, None) == code
    assert lib.mikv_block_select(FAKE, p, 0, FAKE, FAKE, None, None, 1, 4, 2, 0, 1, FAKE, FAKE, FAKE, BIG, None) == code
    assert lib.mikv_block_attention(FAKE, p, 0, None, None, FAKE, FAKE, 1, 4, 2, FAKE, None, FAKE, BIG, None) == code
    assert lib.mikv_chunk_attention(_rows(), p, 0, None, None, FAKE, 1, 1, 4, 0, 0, _rows(), None, FAKE, BIG, None) == code
    assert lib.mikv_block_select_workspace_bytes(p, 1, 4) == 0
    assert lib.mikv_block_attention_workspace_bytes(p, 1, 4, 2) == 0
    assert lib.mikv_chunk_attention_workspace_bytes(p, 1, 1, 4) == 0


def test_batch_rows_refuses(lib):
    call = lambda p=_pages(), counts=FAKE, n=2, rows=5, a=FAKE, b=FAKE: lib.mikv_batch_rows(
        p, None, None, counts, n, rows, a, b, FAKE, FAKE, None)
    assert call(n=0, rows=0, counts=None, a=None, b=None) == 0
    for kw in (dict(n=-1), dict(n=5), dict(n=4097), dict(rows=-1), dict(p=_pages(n_pages=1 << 28, Hkv=1))):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(counts=None), dict(a=None), dict(b=None)):
        assert call(**kw) == EINVAL, kw
    assert lib.mikv_batch_rows(_pages(), FAKE, None, FAKE, 4097, 5, FAKE, FAKE, FAKE, FAKE, None) == ESHAPE


def test_slot_append_and_bounds_refuse(lib):
    p = _pages()
    call = lambda layer=0, k=_rows(), v=_rows(), rows=3, slots=FAKE: lib.mikv_slot_append(p, layer, k, v, rows, slots, None)
    assert call(rows=0, slots=None, k=None) == 0
    assert call(layer=2) == ESHAPE and call(layer=-1) == ESHAPE and call(rows=-1) == ESHAPE
    assert call(slots=None) == EINVAL and call(k=None) == EINVAL and call(v=_rows(data=None)) == EINVAL
    assert call(k=_rows(sh=-128)) == EINVAL and call(k=_rows(data=FAKE + 2)) == EALIGN and call(v=_rows(st=129)) == EALIGN
    call = lambda layer=0, a=FAKE, b=FAKE, rows=3, c=FAKE, d=FAKE: lib.mikv_page_bounds(p, layer, a, b, rows, c, d, None)
    assert call(rows=0, a=None) == 0
    assert call(layer=2) == ESHAPE and call(rows=-1) == ESHAPE
    for kw in (dict(a=None), dict(b=None), dict(c=None), dict(d=None)):
        assert call(**kw) == EINVAL, kw
    assert call(c=FAKE + 8) == EALIGN


def test_block_calls_refuse(lib):
    p = _pages()
    need = lib.mikv_block_select_workspace_bytes(p, 3, 4)
    assert need >= 3 * 2 * 4 * 4 and lib.mikv_block_select_workspace_bytes(p, 0, 4) == 0
    assert lib.mikv_block_select_workspace_bytes(p, 32768, 4) == 0                   # 2 key heads: 65536 units
    call = lambda q=FAKE, layer=0, b=FAKE, s=FAKE, seq=None, rows=3, Hq=4, keep=3, first=1, recent=1, sel=FAKE, n_sel=FAKE, ws=FAKE, nb=BIG: \
        lib.mikv_block_select(q, p, layer, b, s, seq, None, rows, Hq, keep, first, recent, sel, n_sel, ws, nb, None)
    assert call(rows=0, q=None, ws=None) == 0
    for kw in (dict(layer=2), dict(rows=-1), dict(rows=5), dict(rows=32768, seq=FAKE), dict(Hq=3), dict(Hq=0), dict(nb=need - 1)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(keep=0), dict(first=-1), dict(recent=0), dict(first=3), dict(recent=3), dict(recent=2 ** 31 - 1), dict(q=None),
               dict(b=None), dict(s=None), dict(sel=None), dict(n_sel=None), dict(ws=None)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(q=FAKE + 2), dict(b=FAKE + 4), dict(ws=FAKE + 8)):
        assert call(**kw) == EALIGN, kw
    need = lib.mikv_block_attention_workspace_bytes(p, 3, 4, 3)
    assert need > 0 and lib.mikv_block_attention_workspace_bytes(p, 3, 5, 3) == 0 and lib.mikv_block_attention_workspace_bytes(p, 3, 4, 0) == 0
    call = lambda q=FAKE, layer=0, seq=None, sel=FAKE, n_sel=FAKE, rows=3, Hq=4, keep=3, out=FAKE, ws=FAKE, nb=BIG: \
        lib.mikv_block_attention(q, p, layer, seq, None, sel, n_sel, rows, Hq, keep, out, None, ws, nb, None)
    assert call(rows=0, q=None, ws=None) == 0
    for kw in (dict(layer=-1), dict(rows=-1), dict(rows=5), dict(rows=32768, seq=FAKE), dict(Hq=5), dict(keep=0), dict(keep=1 << 27),
               dict(nb=need - 1)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(q=None), dict(sel=None), dict(n_sel=None), dict(out=None), dict(ws=None)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(q=FAKE + 2), dict(out=FAKE + 8), dict(ws=FAKE + 4)):
        assert call(**kw) == EALIGN, kw


def test_chunk_attention_refuses(lib):
    p = _pages()
    need = lib.mikv_chunk_attention_workspace_bytes(p, 2, 7, 4)
    assert need > 0
    assert lib.mikv_chunk_attention_workspace_bytes(p, 4097, 7, 4) == 0 and lib.mikv_chunk_attention_workspace_bytes(p, 2, 0, 4) == 0
    rows = lambda data=FAKE, sh=128, st=512: _rows(data=data, sb=0, sh=sh, st=st)
    call = lambda q=rows(), layer=0, rs=FAKE, n=2, r=7, Hq=4, window=0, sinks=0, out=rows(), ws=FAKE, nb=BIG: lib.mikv_chunk_attention(
        q, p, layer, None, None, rs, n, r, Hq, window, sinks, out, None, ws, nb, None)
    assert call(n=0, q=None, ws=None) == 0 and call(r=0, q=None, ws=None) == 0
    for kw in (dict(layer=2), dict(n=-1), dict(n=5), dict(n=4097), dict(r=-1), dict(Hq=3), dict(Hq=0), dict(nb=need - 1)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(window=-1), dict(sinks=-1), dict(q=None), dict(out=None), dict(rs=None), dict(ws=None), dict(q=rows(data=None)),
               dict(out=rows(sh=0)), dict(out=rows(st=64)), dict(q=rows(sh=-128))):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(q=rows(data=FAKE + 2)), dict(out=rows(st=516)), dict(ws=FAKE + 8)):
        assert call(**kw) == EALIGN, kw


def test_rows_by_hand():
    table = np.array([[5, 2, -1], [7, -1, -1], [0, 1, 3]], np.int32)
    lens = np.array([6, 3, 12], np.int32)
    start, seq, pos, slot = ob.batch_rows(table, lens, 4, 8, [2, 0, 2, 9, 1], [7, -1, 0, 0, 2], [2, 1, 1, 1, 3], 10)
    assert start.tolist() == [0, 2, 3, 4, 5, 8]
    assert seq.tolist() == [2, 2, -1, -1, -1, 1, 1, 1, -1, -1]       # refused, named twice, no such sequence, past the end
    assert pos.tolist() == [7, 8, -1, -1, -1, 2, 3, 4, -1, -1]
    assert slot.tolist() == [7, 12, -1, -1, -1, 30, -1, -1, -1, -1]  # positions 3 and 4 of three
    start, seq, pos, slot = ob.batch_rows(table, lens, 4, 8, None, None, [7, 1], 8)
    assert seq.tolist() == [-1] * 7 + [1] and slot.tolist() == [-1] * 7 + [30]   # more rows than slots


def test_bounds_and_choice_by_hand():
    codes, s = ob.bounds(np.array([[127.0, -50.5, 0.0], [10.25, 25.0, 0.0]], np.float32))
    assert s == 1 and codes.tolist() == [[10, -51, 0], [127, 25, 0]]
    assert ob.bounds(np.array([[np.nan, 1.0]]))[1] == np.inf and ob.bounds(np.zeros((2, 3)))[1] == 0
    b = np.array([[[-1, 2], [3, 5]], [[-4, -4], [0, 0]]], np.int8)
    got = ob.scores(np.array([[127.0, -127.0]]), b, np.array([1.0, 2.0], np.float32))
    assert got.tolist() == [127 * 3 - 127 * 2, 2 * 127 * 4]
    assert ob.pick([1.0, 5.0, 5.0, 0.0, 5.0, 2.0], 4, 1, 1) == [0, 1, 2, 5]
    assert ob.pick([1.0, 5.0], 4, 1, 1) == [0, 1]


def test_a_score_bounds_every_logit():
    """Up to the rounding of the query's codes: half a step of s_q a channel, times the key's size."""
    rng = np.random.RandomState(0)
    for _ in range(20):
        k, q = rng.randn(16, 128).astype(np.float32), rng.randn(1, 128).astype(np.float32)
        codes, s = ob.bounds(k)
        top = ob.scores(q, codes[None], np.array([s]))[0]
        slack = 0.5 * np.abs(q).max() / 127 * (np.abs(k).sum(1).max() + 128 * s) + 1e-3
        assert top >= (k @ q[0]).max() - slack


def test_rows_beyond_what_a_call_numbers_are_refused(lib):
    most = (1 << 30) + 1
    assert lib.mikv_batch_rows(_pages(), None, None, FAKE, 2, most, FAKE, FAKE, FAKE, FAKE, None) == ESHAPE
    assert lib.mikv_slot_append(_pages(), 0, _rows(), _rows(st=0), most, FAKE, None) == ESHAPE


def test_rows_over_picked_blocks_go_in_parts():
    """Each part is one that a call takes, and they are the rows in order."""
    import types

    import torch
    from mixed_precision_kv_balancer_gb300.paged import PagedCache
    for Hkv in (1, 2, 8, 32, 40000, 70000):
        cache = types.SimpleNamespace(k=torch.empty(1, 1, Hkv, 1, 0), device="cpu")
        cache._row_parts = lambda n, c=cache: PagedCache._row_parts(c, n)
        for rows in (0, 1, 2, 100, 8191, 8192, 65535, 65536, 200001):
            if Hkv >= 40000 and rows > 100:
                continue
            parts = cache._row_parts(rows)
            assert all((b - a) * Hkv <= 65535 or b - a == 1 for a, b in parts) and max([b - a for a, b in parts], default=0) <= -(-rows // max(1, len(parts)))
            assert [a for a, _ in parts] + [rows] * bool(parts) == [0] * bool(parts) + [b for _, b in parts]
            assert (len(parts) <= 1) == (rows * Hkv <= 65535 or rows <= 1 or rows <= 65535 // Hkv)
            if rows > 30000:                         # (longer tensors start threads)
                continue
            q, sel = torch.arange(rows), torch.arange(rows) + 7
            got = PagedCache._in_parts(cache, None, q, sel)
            if len(parts) > 1:
                assert torch.equal(torch.cat([g[0] for g in got]), q.int()) and all(g[1] is None for g in got)
                assert torch.equal(torch.cat([g[3] for g in got]), sel)
                with pytest.raises(ValueError, match="rows"):
                    PagedCache._in_parts(cache, None, q, sel[1:])
            else:
                assert len(got) == 1 and got[0][0] is None and got[0][2] is q and got[0][3] is sel
