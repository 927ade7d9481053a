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


# INT8 keys enter the products of packed rows as two fp16 numbers, 22 bits: a score, whose sum |q k| is at most 4 here, is off
# by 4 * 2^-22 for that and by 4 * 2^-23 for each of 17 additions that may cut what they add; times 1 / sqrt(128) below 2^-20 of
# a logit, so that a weight is off by that share and a normalised one by twice it.  The values' two numbers leave 2^-22 of them.
def _codes_share(type):
    return (2.0 ** -19 + 2.0 ** -22, 2.0 ** -20) if type == "int8" else (0.0, 0.0)


def _close(out, lse, want, wl, type, weights, n_keys):
    of_out, of_lse = _codes_share(type)
    assert pc.out_error(ph.f64(out), want, pc.HALF_STEP[type], weights + of_out, n_keys) < 1
    err = np.abs(ph.f64(lse) - wl) - of_lse
    assert pc.lse_error(wl + err, wl, n_keys) < 1


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("rows,rep", [(1, 4), (1, 16), (2, 16), (7, 5)])
@pytest.mark.parametrize("n_keys", [2, 4, 16, 18, 40, 64, 200])
def test_fp32_sums_of_few_packed_rows(type, rows, rep, n_keys):
    """Single tokens and drafts by both calls that take them: packed rows round a weight once, picked blocks keep two parts of
    it.  All rows ask with one query."""
    n, Hkv = 3, 2
    rows = min(rows, n_keys)
    q, k, v = (np.stack(x) for x in zip(*(pc.rows(n_keys, Hkv * rep, Hkv, 100 * i + n_keys) for i in range(n))))
    cache = _cache(k, v, type)
    batch = cache.rows(ph.ints([rows] * n), n * rows)
    qd = torch.from_numpy(q).to(ph.DTYPE[type]).to(ph.DEV).repeat_interleave(rows, 0)
    buf = cache.bounds_buffers()
    cache.renew(0, cache.rows(ph.ints([n_keys] * n), n * n_keys), buf)
    half = pc.HALF_STEP[type]
    calls = ((*cache.attend_rows(0, qd, batch), half),
             (*cache.attend_blocks(0, qd, *cache.pick(0, qd, buf, -(-n_keys // 16), batch=batch), batch), half ** 2))
    for i in range(n):
        ki, vi = ph.sequence(cache, 0, i)
        for t in range(rows):
            seen = n_keys - rows + t + 1
            want, wl = pc.softmax64(q[i], ki[:, :seen], vi[:, :seen])
            for out, lse, weights in calls:
                _close(out[i * rows + t], lse[i * rows + t], want, wl, type, weights, n_keys)


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("rows,rep", [(65, 3), (64, 4), (200, 1), (33, 4)])
@pytest.mark.parametrize("n_keys", [18, 64, 200])
def test_weights_rounded_once_and_fp32_sums_of_packed_chunks(type, rows, rep, n_keys):
    """Requests of two tiles or more; sums are taken before the weights are rounded."""
    Hkv = 2
    q, k, v = pc.rows(n_keys, Hkv * rep, Hkv, rows + n_keys)
    cache = _cache(k[None], v[None], type)
    qd = torch.from_numpy(q).to(ph.DTYPE[type]).to(ph.DEV)[None].repeat(rows, 1, 1)
    first = max(n_keys - rows, 0)                    # rows past the last slot see all of them
    out, lse = cache.attend_rows(0, qd, cache.rows(ph.ints([rows]), rows, start=ph.ints([first])))
    ki, vi = ph.sequence(cache, 0, 0)
    for t in range(rows):
        seen = min(first + t + 1, n_keys)
        want, wl = pc.softmax64(q, ki[:, :seen], vi[:, :seen])
        _close(out[t], lse[t], want, wl, type, pc.HALF_STEP[type], n_keys)


@pytest.mark.parametrize("rows,rep", [(1, 4), (7, 5), (64, 4), (200, 1)])
@pytest.mark.parametrize("n_keys", [2, 18, 64, 200])
def test_codes_that_no_16_bit_number_holds(rows, rep, n_keys):
    """8-bit keys show in the lse, 8-bit values in outputs whose weights are all alike, and so not rounded."""
    Hkv = 2
    q, k, v = pc.codes_beyond_16_bits(n_keys, Hkv * rep, Hkv, n_keys)
    cache = ph.make([n_keys], 16, Hkv, "int8", poison=False)
    j = torch.arange(n_keys)
    page = cache.table[0].cpu().long()[j // 16]
    for name, (codes, meta) in (("k", k), ("v", v)):
        getattr(cache, name)[0, page, :, j % 16] = torch.from_numpy(codes).transpose(0, 1).to(ph.DEV)
        getattr(cache, name + "_meta")[0, page, :, j % 16] = torch.from_numpy(meta).transpose(0, 1).to(ph.DEV)
    ki, vi = pc.code_values(*k), pc.code_values(*v)
    first = max(n_keys - rows, 0)
    batch = cache.rows(ph.ints([rows]), rows, start=ph.ints([first]))
    for x, weights in ((q, 2.0 ** -11), (0 * q, 0.0)):
        qd = torch.from_numpy(x).half().to(ph.DEV)[None].repeat(rows, 1, 1)
        out, lse = cache.attend_rows(0, qd, batch)
        for t in range(rows):
            seen = min(first + t + 1, n_keys)
            want, wl = pc.softmax64(x, ki[:, :seen], vi[:, :seen])
            if weights:
                _close(out[t], lse[t], want, wl, "int8", weights, n_keys)
            else:
                assert pc.out_error(ph.f64(out[t]), want, 2.0 ** -11, 2.0 ** -22, n_keys) < 1
