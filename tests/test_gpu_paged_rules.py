"""Which requests of one call are served when free pages run out, by hand."""
import numpy as np
import pytest
import torch

import paged_helpers as ph
import test_paged_rules as rules
from mixed_precision_kv_balancer_gb300.paged import PagedCache

pytestmark = pytest.mark.gpu
ints = ph.ints


def _cache(lens, n_pages):
    cache = PagedCache(1, n_pages, 4, 1, 128, len(lens), 4)
    table, refs = rules.table_of(lens, n_pages)
    for x, y in ((cache.table, table), (cache.refs, refs), (cache.lens, np.array(lens, np.int32))):
        x.copy_(torch.from_numpy(y))
    return cache


def test_requests_behind_a_shortage():
    lens, n_pages, add, start, after = rules.shortage()
    cache = _cache(lens, n_pages)
    assert cache.reserve(ints(add)).tolist() == start and cache.lens.tolist() == after
    assert cache.refs.tolist() == [1, 1, 1, 1, 1, 0]
    assert cache.reserve(ints([1]), seqs=ints([2])).tolist() == [4]


def test_requests_behind_a_bad_position():
    lens, n_pages, pos, keep, ok = rules.bad_position()
    cache = _cache(lens, n_pages)
    assert cache.compact(ints(pos.tolist()), ints(keep)).tolist() == ok
    assert cache.lens.tolist() == [8, 8, 0] and cache.refs.tolist() == [1, 1, 1, 1, 0, 0, 0, 0]
    assert cache.compact(ints(pos[:, 1:2].tolist()), ints(keep[1:2]), seqs=ints([1])).tolist() == [1]
