"""INT8 codes of rows that hold values which are no numbers, against the definition."""
import numpy as np
import pytest
import torch

import paged_helpers as ph
from mixed_precision_kv_balancer_gb300 import _lib
from mixed_precision_kv_balancer_gb300.cache import MikvCache

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _definition(x):
    """Codes and (scale, zero) of fp16 rows [T][128]: NaN does not count for a group's extremes, and a
    quotient that is no number gives code 0."""
    x = x.astype(np.float32).reshape(len(x), 2, 64)
    with np.errstate(all="ignore"):
        lo, hi = np.fmin.reduce(x, axis=-1), np.fmax.reduce(x, axis=-1)
        s, z = ((hi - lo) / np.float32(255)).astype(np.float16), lo.astype(np.float16)
        sf, zf = s.astype(np.float32)[..., None], z.astype(np.float32)[..., None]
        c = np.clip(np.rint((x - zf) / sf), 0, 255)
    c = np.where((sf == 0) | np.isnan(c), 0, c).astype(np.uint8)
    return c.reshape(len(x), 128), np.stack([s, z], -1)


def _rows():
    """Rows of 128 normal values; each pattern spoils some channels of one group or of both."""
    spoil = [{}, {3: NAN}, {3: INF}, {3: -INF}, {3: INF, 9: -INF}, {3: NAN, 9: INF}, {3: NAN, 9: -INF}, {0: NAN, 63: NAN},
             {64: INF, 127: NAN}, {i: NAN for i in range(64)}, {i: INF for i in range(64)}, {i: -INF for i in range(64, 128)},
             {i: (INF, -INF, NAN)[i % 3] for i in range(128)}, {i: NAN for i in range(1, 64)}, {i: (1.5 if i % 2 else NAN) for i in range(64)},
             {2: 65504.0, 5: -65504.0, 7: NAN}]
    x = ph.normal((len(spoil), 128), 8, torch.float16)
    for t, at in enumerate(spoil):
        for c, y in at.items():
            x[t, c] = y
    return x


def test_codes_of_values_that_are_no_numbers():
    x = _rows()
    T = len(x)
    cache = ph.make([T], 4, 1, "int8", poison=False)
    v = x.flip(0)
    cache.append(0, x[None, None].to(ph.DEV), v[None, None].to(ph.DEV))
    at = torch.arange(T)
    page = cache.table[0].cpu().long()[at // 4]
    for rows, stored, meta in ((x, cache.k, cache.k_meta), (v, cache.v, cache.v_meta)):
        codes, m = _definition(rows.numpy())
        np.testing.assert_array_equal(stored[0].cpu()[page, 0, at % 4].numpy(), codes)
        np.testing.assert_array_equal(meta[0].cpu()[page, 0, at % 4].numpy(), m)   # NaN equals NaN


def test_infinities_as_in_the_contiguous_cache():
    x = _rows()
    x = x[~torch.isnan(x).any(-1)]
    T = len(x)
    paged = ph.make([T], 4, 1, "int8", poison=False)
    paged.append(0, x[None, None].to(ph.DEV), x[None, None].to(ph.DEV))
    flat = MikvCache(1, 1, 1, 128, 8, 2, T, 1, torch.device(ph.DEV), use_balancer=False)
    pos = torch.arange(T, dtype=torch.int32, device=ph.DEV).view(1, 1, T)
    _lib.mikv_quantize_append(_lib.MIKV_TIER_HI, flat, x[None, None].to(ph.DEV), x[None, None].to(ph.DEV), pos, T)
    at = torch.arange(T, device=ph.DEV)
    page = paged.table[0].long()[at // 4]
    for name in ("k", "v"):
        assert torch.equal(getattr(paged, name)[0, page, 0, at % 4], getattr(flat, name + "_hi")[0, 0, :T])
        np.testing.assert_array_equal(getattr(paged, name + "_meta")[0, page, 0, at % 4].cpu().numpy(),
                                      getattr(flat, name + "_hi_meta")[0, 0, :T].cpu().numpy())
