"""Calls of several threads at once, each on a stream of its own: what one asks of a kernel does not fail another's launch."""
import ctypes
import threading

import pytest
import torch

from mixed_precision_kv_balancer_gb300 import _lib
from mixed_precision_kv_balancer_gb300.cache import MikvCache

pytestmark = pytest.mark.gpu


def _together(calls, times):
    """Each of the calls `times` times in a thread of its own; the threads begin together."""
    failed, begin = [], threading.Barrier(len(calls))

    def run(call):
        torch.cuda.set_device(0)
        stream = torch.cuda.Stream()
        fn, args = call
        begin.wait()
        codes = {fn(*args, stream.cuda_stream) for _ in range(times)}
        stream.synchronize()
        if codes != {0}:
            failed.append((fn.__name__, codes))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("lengths", [(500, 3000, 8000, 1200), (9000, 20000, 40000, 12000), (41000, 100000, 131072, 65000)])
def test_selections_of_different_lengths(lengths):
    g = torch.Generator(device="cuda").manual_seed(1)
    cache, work = MikvCache(1, 2, 2, 128, 16, 2, 1, 1, torch.device("cuda:0")), []
    for L in lengths:
        scores = torch.rand(1, 2, L, generator=g, device="cuda")
        keep = torch.empty(1, 2, L // 5, dtype=torch.int32, device="cuda")
        evict = torch.empty(1, 2, L - L // 5, dtype=torch.int32, device="cuda")
        _lib.mikv_select(_lib.MIKV_H2O, cache, L, 20, 0, 0.5, scores=scores, keep_pos=keep, evict_pos=evict)
        work.append((L, scores, keep, evict, keep.clone()))

    def call(L, scores, keep, evict, _):
        return _lib.load().mikv_select, (_lib.MIKV_H2O, ctypes.byref(cache.struct), L, 20, 0, 0.5, scores.data_ptr(), None, None, None, 0, None,
                                         keep.data_ptr(), evict.data_ptr(), None, None, 0)

    _together([call(*w) for w in work], 3000)
    assert all(torch.equal(w[2], w[4]) for w in work)


def test_perturbations_of_different_head_counts():
    g = torch.Generator(device="cuda").manual_seed(2)
    hidden, work = 16384, []          # a CTA a column block: its heads are all of them
    for Hq in (1, 8, 24, 40):
        o = torch.randn(1, Hq, 128, generator=g, device="cuda")
        w = torch.randn(hidden, Hq * 128, generator=g, device="cuda").half()
        y = torch.empty(1, hidden, device="cuda")
        ws = torch.empty(_lib.load().mikv_output_perturbation_workspace_bytes(1, Hq, hidden), dtype=torch.uint8, device="cuda")
        _lib.mikv_output_perturbation(o, None, w, y=y, ws=ws)
        work.append((o, w, y, ws, y.clone()))

    def call(o, w, y, ws, _):
        return _lib.load().mikv_output_perturbation, (o.data_ptr(), None, w.data_ptr(), 1, o.shape[1], 128, hidden, y.data_ptr(), None,
                                                      ws.data_ptr(), ws.numel())

    _together([call(*w) for w in work], 1500)
    assert all(torch.equal(w[2], w[4]) for w in work)
