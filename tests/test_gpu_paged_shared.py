"""Appends into pages that several sequences own: they are left as they are, and reported."""
import numpy as np
import pytest
import torch

import paged_helpers as ph
from mixed_precision_kv_balancer_gb300 import _lib

pytestmark = pytest.mark.gpu
ints = ph.ints
SHARED = 128


def _rows(type, n, T, seed=3):
    return ph.normal((n, 2, T, 128), seed, ph.DTYPE[type]).to(ph.DEV)


def _stored(cache, s):
    """Everything the cache holds of sequence s, slot by slot."""
    L, ps = int(cache.lens[s]), cache.k.shape[3]
    j = torch.arange(L, device=ph.DEV)
    page = cache.table[s].long()[j // ps]
    return [ph.raw(x[:, page, :, j % ps]) for x in (cache.k, cache.v, cache.k_meta, cache.v_meta) if x is not None]


def _same(a, b, slots=slice(None)):
    return all(np.array_equal(x[slots], y[slots]) for x, y in zip(a, b))


@pytest.fixture(autouse=True)
def _clear():
    _lib.mikv_wait_status()


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("by_start", [True, False])
def test_a_shared_prefix_is_not_written(type, by_start):
    """40 slots: two full pages that parent and child share, and 8 slots of a page that each owns."""
    cache = ph.make([40, 0], 16, 2, type, spare=6, poison=False, layers=2)
    assert cache.fork(ints([0]), ints([1])).tolist() == [1]
    before, mine = _stored(cache, 1), _stored(cache, 0)
    x = _rows(type, 1, 15)
    cache.append(1, x, x, seqs=ints([0]), start=ints([25]) if by_start else None)        # slots 25 .. 39
    assert _lib.mikv_wait_status() == SHARED and _lib.mikv_wait_status() == 0
    assert _same(_stored(cache, 1), before)
    after = _stored(cache, 0)
    assert _same(after, mine, slice(0, 32)) and not _same(after, mine, slice(32, 40))
    # once the child has gone the pages are the parent's alone
    cache.free(ints([1]))
    cache.append(1, x, x, seqs=ints([0]), start=ints([25]))
    assert _lib.mikv_wait_status() == 0
    now = _stored(cache, 0)
    assert _same(now, mine, slice(0, 25)) and not _same(now, mine, slice(25, 32)) and _same(now, after, slice(32, 40))


@pytest.mark.parametrize("type", ["fp16", "int8"])
def test_slots_reserved_before_a_fork(type):
    """They are shared as far as their pages are full: an append behind the fork reaches only the parent's own."""
    cache = ph.make([8, 0], 16, 2, type, spare=8, max_pages=4, poison=False)
    start = cache.reserve(ints([32]), seqs=ints([0]))                # slots 8 .. 39
    assert start.tolist() == [8]
    assert cache.fork(ints([0]), ints([1])).tolist() == [1]
    child, parent = _stored(cache, 1), _stored(cache, 0)
    x = _rows(type, 1, 32)
    cache.append(0, x, x, seqs=ints([0]), start=start)
    assert _lib.mikv_wait_status() == SHARED
    assert _same(_stored(cache, 1), child)
    assert _same(_stored(cache, 0), parent, slice(0, 32)) and not _same(_stored(cache, 0), parent, slice(32, 40))


def test_appends_of_slots_reserved_behind_a_fork():
    """Parent, children and a sequence of whole pages grow; nothing is reported and every token arrives."""
    cache = ph.make([40, 64, 0, 0, 0], 16, 2, "fp16", spare=20, max_pages=8, poison=False)
    assert cache.fork(ints([0, 0, 1]), ints([2, 3, 4])).tolist() == [1, 1, 1]
    before = [_stored(cache, s) for s in range(5)]
    x = _rows("fp16", 5, 20)
    start = cache.reserve(ints([20] * 5))
    cache.append(0, x, x, start=start)
    assert _lib.mikv_wait_status() == 0
    for s in range(5):
        L = 64 if s in (1, 4) else 40
        got = _stored(cache, s)
        assert _same(got, before[s], slice(0, L))
        np.testing.assert_array_equal(got[0][L:], ph.raw(x[s].transpose(0, 1)[:, None]))


def test_a_page_that_the_caller_holds_too():
    """Its count is above one: what it holds stays."""
    cache = ph.make([30], 16, 2, "fp16", poison=False)
    cache.refs[int(cache.table[0, 0])] += 1
    before = _stored(cache, 0)
    x = _rows("fp16", 1, 30)
    cache.append(0, x, x)
    assert _lib.mikv_wait_status() == SHARED
    assert _same(_stored(cache, 0), before, slice(0, 16)) and not _same(_stored(cache, 0), before, slice(16, 30))
