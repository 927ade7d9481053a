"""A compaction of a paged cache to the positions that a selection writes."""
import pytest
import torch

import paged_helpers as ph
from mixed_precision_kv_balancer_gb300 import _lib
from mixed_precision_kv_balancer_gb300.cache import MikvCache, n_keep

pytestmark = pytest.mark.gpu
ints = ph.ints


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
def test_compaction_to_the_positions_of_a_selection(type):
    """keep_pos [layers][n][Hkv][max_keep]: each layer's part is what mikv_select writes for a batch of the
    n sequences."""
    layers, n, Hkv, L, pct, window = 3, 2, 2, 150, 20, 8
    cache = ph.make([L, L, 33], 16, Hkv, type, layers=layers, spare=8, poison=False)
    read = lambda l, T: cache.gather(l, *(torch.zeros(n, Hkv, T, 128, dtype=ph.DTYPE[type], device=ph.DEV) for _ in range(2)))
    rows = [read(l, L) for l in range(layers)]
    sel = MikvCache(n, 2 * Hkv, Hkv, 128, 16, 2, L, L, torch.device(ph.DEV))
    keep = n_keep(L, pct, window)
    keep_pos = torch.full((layers, n, Hkv, keep), -7, dtype=torch.int32, device=ph.DEV)
    scores = torch.rand(layers, n, Hkv, L, generator=torch.Generator().manual_seed(4)).to(ph.DEV)
    for l in range(layers):
        evict = torch.empty(n, Hkv, L - keep, dtype=torch.int32, device=ph.DEV)
        _lib.mikv_select(_lib.MIKV_H2O, sel, L, pct, window, scores=scores[l], keep_pos=keep_pos[l], evict_pos=evict)
    assert cache.compact(keep_pos, ints([keep, keep])).tolist() == [1, 1]
    assert cache.lens.tolist() == [keep, keep, 33]
    for l in range(layers):
        # the window, and of the older positions those of the highest scores
        top = scores[l, :, :, :L - window].topk(keep - window, -1).indices
        want = torch.cat([top, torch.arange(L - window, L, device=ph.DEV).expand(n, Hkv, window)], -1).sort(-1).values
        assert torch.equal(keep_pos[l].long(), want)
        for a, b in zip(read(l, keep), rows[l]):
            assert torch.equal(a, b.gather(2, want.unsqueeze(-1).expand(n, Hkv, keep, 128)))
    assert _lib.mikv_wait_status() == 0
