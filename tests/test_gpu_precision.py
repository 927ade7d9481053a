"""How exact the softmax weights and sums of the attention over pages and of windowed attention are, on
inputs whose outputs do not hide it, against 64 bits."""
import numpy as np
import pytest
import torch

import paged_helpers as ph
import precision_cases as pc
from mixed_precision_kv_balancer_gb300 import _lib

pytestmark = pytest.mark.gpu


def _cache(k, v, type, ps=16):
    """One sequence a batch row: k, v [n][Hkv][N][128] in pages of `ps`."""
    n, Hkv, N, _ = k.shape
    cache = ph.make([N] * n, ps, Hkv, type, poison=False)
    j = torch.arange(N)
    for name, x in (("k", k), ("v", v)):
        x = torch.from_numpy(x).to(ph.DTYPE[type])
        stored, meta = ph.quantize(x) if type == "int8" else (x, None)
        for i in range(n):
            page = cache.table[i].cpu().long()[j // ps]
            getattr(cache, name)[0, page, :, j % ps] = stored[i].transpose(0, 1).to(ph.DEV)
            if meta is not None:
                getattr(cache, name + "_meta")[0, page, :, j % ps] = meta[i].transpose(0, 1).to(ph.DEV)
    return cache


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("rep", [4, 16])
@pytest.mark.parametrize("n_keys", [2, 4, 16, 18, 40, 64, 200])
def test_weights_of_two_parts_and_fp32_sums_over_pages(type, rep, n_keys):
    """2^-11 or 2^-8 of a part squared: what two 16-bit parts leave of a weight."""
    n, Hkv = 3, 2
    q, k, v = (np.stack(x) for x in zip(*(pc.rows(n_keys, Hkv * rep, Hkv, 100 * i + n_keys) for i in range(n))))
    cache = _cache(k, v, type)
    out, lse = cache.attend(0, torch.from_numpy(q).to(ph.DTYPE[type]).to(ph.DEV))
    two = pc.HALF_STEP[type] ** 2
    for i in range(n):
        want, wl = pc.softmax64(q[i], *ph.sequence(cache, 0, i))
        assert pc.out_error(ph.f64(out[i]), want, pc.HALF_STEP[type], two, n_keys) < 1
        assert pc.lse_error(ph.f64(lse[i]), wl, n_keys) < 1


@pytest.mark.parametrize("type", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,rep", [(1, 4), (1, 16), (7, 5), (64, 2), (200, 3)])
@pytest.mark.parametrize("n_keys", [2, 18, 64, 200])
def test_weights_rounded_once_and_fp32_sums_of_chunks(type, rows, rep, n_keys):
    """All rows ask with one query, so the last one of each head sees all keys and an earlier one those up
    to its position; the sums are taken before the weights are rounded."""
    Hkv = 2
    q, k, v = pc.rows(n_keys, Hkv * rep, Hkv, rows + n_keys)
    dt = ph.DTYPE[type]
    dev = lambda x: torch.from_numpy(x).to(dt).to(ph.DEV)
    out = torch.empty(1, Hkv * rep, rows, 128, dtype=dt, device=ph.DEV)
    lse = torch.empty(1, Hkv * rep, rows, device=ph.DEV)
    _lib.mikv_window_attention(dev(q)[None, :, None].repeat(1, 1, rows, 1), dev(k)[None], dev(v)[None], 0, 0, out, lse)
    for i in range(rows):
        seen = n_keys - rows + i + 1
        if seen < 1:
            continue
        want, wl = pc.softmax64(q, k[:, :seen], v[:, :seen])
        assert pc.out_error(ph.f64(out[0, :, i]), want, pc.HALF_STEP[type], pc.HALF_STEP[type], n_keys) < 1
        assert pc.lse_error(ph.f64(lse[0, :, i]), wl, n_keys) < 1


def test_split_keys_keep_fp32_sums():
    """Keys that several CTAs hold and a second kernel joins: n copies of a few keys add log n to the lse."""
    q, k, v = pc.rows(64, 8, 2, 3)
    times = 128
    dev = lambda x: torch.from_numpy(x).half().to(ph.DEV)
    qd, kd, vd = dev(q)[None, :, None], dev(np.tile(k, (1, times, 1)))[None], dev(np.tile(v, (1, times, 1)))[None]
    assert _lib.load().mikv_window_attention_workspace_bytes(1, 8, 2, 1, 64 * times, 0, 0) > 0
    out, lse = torch.empty_like(qd), torch.empty(1, 8, 1, device=ph.DEV)
    _lib.mikv_window_attention(qd, kd, vd, 0, 0, out, lse)
    want, wl = pc.softmax64(q, k, v)
    assert pc.out_error(ph.f64(out[0, :, 0]), want, 2.0 ** -11, 2.0 ** -11, 64 * times) < 1
    # a thread's serial sum of at most 128 weights a tile and 64 tiles, each addition 2^-24 of it
    assert np.abs(ph.f64(lse[0, :, 0]) - wl - np.log(times)).max() < 2.0 ** -18 + 2.0 ** -20 + 192 * 2.0 ** -24
