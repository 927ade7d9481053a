"""Paged cache on the GPU: attention of one token, rows in and out, page operators, and a whole
serving sequence, against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import paged_helpers as ph
from mixed_precision_kv_balancer_gb300 import _lib
from mixed_precision_kv_balancer_gb300.paged import PagedCache

pytestmark = pytest.mark.gpu
ints = ph.ints


def _query(n, Hq, type, seed=5, scale=1.0):
    return ph.normal((n, Hq, 128), seed, ph.DTYPE[type], scale).to(ph.DEV)


def _check(cache, q, window=0, sinks=0, seqs=None, layer=0):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=ph.DEV)
    _lib.mikv_paged_attention(q, cache, layer, window, sinks, out, lse, seqs=None if seqs is None else ints(seqs))
    want, wlse, mag = ph.expect(cache, q, layer, window, sinks, seqs)
    ph.close(out, want, mag, ph.HALF_STEP[cache.type], weights=2.0 ** -16)   # two 16-bit parts: bf16 2^-8 * 2^-8
    ph.close_lse(lse, wlse)
    return out, lse


# --- attention of one token -------------------------------------------------------------

@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("lens,ps,Hkv,rep", [
    ([1], 16, 1, 1), ([0, 1, 2, 15, 16, 17], 16, 2, 4), ([63, 64, 65, 127, 128, 129, 300], 7, 1, 8),
    ([1000, 3, 0, 517], 1, 2, 5), ([257, 31], 128, 3, 9), ([333], 20, 1, 16), ([100, 200], 64, 2, 17),
    ([90, 0], 16, 1, 40), ([2500], 4096, 2, 2)])
def test_attention(type, lens, ps, Hkv, rep):
    cache = ph.make(lens, ps, Hkv, type)
    _check(cache, _query(len(lens), Hkv * rep, type))
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 4), (100, 130), (1000, 1), (4096, 4), (0, 9)])
def test_window_and_sinks(type, window, sinks):
    cache = ph.make([0, 1, 5, 6, 64, 131, 700], 16, 2, type)
    _check(cache, _query(7, 6, type), window, sinks)


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
def test_long_and_ragged_batches_split_over_the_sms(type):
    cache = ph.make([9001, 1, 0, 4500, 70, 0, 333, 128], 32, 4, type, layers=2)
    out, lse = _check(cache, _query(8, 16, type), layer=1)
    for _ in range(3):     # the joins' order is fixed: the same bits every time
        o2, l2 = cache.attend(1, _query(8, 16, type))
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    _check(cache, _query(8, 16, type), 2000, 5, layer=1)


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
def test_sequences_in_any_order_repeated_and_out_of_range(type):
    cache = ph.make([40, 0, 77, 130], 16, 2, type)
    seqs = [3, 2, 3, -1, 0, 4, 1, 2147483647]
    out, lse = _check(cache, _query(8, 4, type), seqs=seqs)
    for i in (3, 5, 6, 7):
        assert (out[i] == 0).all() and torch.isneginf(lse[i]).all()


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("drop", [9.0, 10.5, 14.0])
def test_many_small_weights_beside_a_large_one(type, drop):
    """One key `drop` above 4000 others that share most of the mass: their weights lie below
    fp16's smallest normal number."""
    cache = ph.make([4001], 32, 1, type, poison=False)
    q = torch.ones(1, 1, 128, dtype=ph.DTYPE[type], device=ph.DEV) * 0.25
    k = torch.zeros_like(cache.k if cache.k_meta is None else cache.k.half())
    page, r = int(cache.table[0, 17]), 5
    k[0, page, 0, r] = drop / (0.25 * 128 ** 0.5)
    if type == "int8":
        codes, meta = ph.quantize(k.cpu())
        cache.k.copy_(codes)
        cache.k_meta.copy_(meta)
    else:
        cache.k.copy_(k)
    _check(cache, q)


def test_bad_table_entries_are_not_seen():
    _lib.mikv_wait_status()
    cache = ph.make([200, 64, 30], 16, 2, "fp16")
    q = _query(3, 4, "fp16")
    cache.table[0, 3] = -1
    cache.table[0, 5] = cache.refs.numel()
    cache.table[1, :4] = 2 ** 31 - 1
    out, lse = cache.attend(0, q)
    assert _lib.mikv_wait_status() == 64 and _lib.mikv_wait_status() == 0
    k, v = (np.nan_to_num(x) for x in ph.sequence(_patched(cache), 0, 0))
    seen = np.ones(200, bool)
    seen[48:64] = seen[80:96] = False
    for h in range(4):
        want, wl, mag = op.attend_row(ph.f64(q)[0, h], k[h // 2], v[h // 2], seen)
        ph.close(out[0, h], want, mag, 2.0 ** -11, 2.0 ** -16)
        assert abs(float(lse[0, h]) - wl) < 1e-3
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert torch.isfinite(out[2]).all()


def _patched(cache):
    """The cache with its bad entries pointing at page 0 (their slots are masked by the caller)."""
    n = cache.refs.numel()
    t = torch.where((cache.table < 0) | (cache.table >= n), 0, cache.table)
    return PagedCache.over(k=cache.k, v=cache.v, k_meta=cache.k_meta, v_meta=cache.v_meta, table=t, lens=cache.lens,
                           refs=cache.refs, type=cache.type)


def test_lengths_are_held_inside_the_table():
    cache = ph.make([64, 64], 16, 1, "bf16")
    want, wl = cache.attend(0, _query(2, 1, "bf16"))
    cache.lens[0] = 1000
    cache.lens[1] = -5
    out, lse = cache.attend(0, _query(2, 1, "bf16"))
    assert torch.equal(out[0], want[0]) and torch.equal(lse[0], wl[0])
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("type", ["fp16", "int8"])
def test_pools_past_32_bit_offsets(type):
    """The sequence's pages are the last ones of a pool of 2^25 rows a tensor and more."""
    Hkv, ps = 8, 64
    n_pages = (1 << 25) // (Hkv * ps) + 40
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    small = ph.make([700, 90], ps, Hkv, type, poison=False)
    big = PagedCache(1, n_pages, ps, Hkv, 128, 2, small.table.shape[1], type)
    m = small.refs.numel()
    for x, y in ((big.k, small.k), (big.v, small.v), (big.k_meta, small.k_meta), (big.v_meta, small.v_meta)):
        if x is not None:
            x[:, -m:] = y
    big.table.copy_(torch.where(small.table >= 0, small.table + (n_pages - m), -1))
    big.lens.copy_(small.lens)
    q = _query(2, 16, type)
    for a, b in zip(big.attend(0, q), small.attend(0, q)):
        assert torch.equal(a, b)
    shape = (2, Hkv, 700, 128)
    a, b = (c.gather(0, torch.zeros(shape, dtype=torch.float16, device=ph.DEV),
                     torch.zeros(shape, dtype=torch.float16, device=ph.DEV)) for c in (big, small))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert big.copy(ints([n_pages - m]), ints([n_pages // 2])).tolist() == [1]
    assert torch.equal(big.k[0, n_pages // 2], small.k[0, 0])


def test_other_streams_and_two_calls_at_once():
    caches = [ph.make([900, 20, 333], 16, 2, "fp16", seed=s) for s in (0, 50)]
    qs = [_query(3, 8, "fp16", seed=s) for s in (1, 2)]
    want = [c.attend(0, q) for c, q in zip(caches, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(caches[i].attend(0, qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_a_stream_given_by_name_owns_its_workspace():
    """Calls on a stream that is not the current one, whose workspaces the binding makes itself."""
    cache = ph.make([4000, 700], 16, 2, "fp16")
    q = _query(2, 8, "fp16")
    k, v = (ph.normal((1, 1, 5000, 128), s, torch.float16).to(ph.DEV) for s in (1, 2))
    x = ph.normal((1, 2, 9, 128), 3, torch.float16).to(ph.DEV)
    want = cache.attend(0, q)
    ww = torch.empty_like(x)
    _lib.mikv_window_attention(x, k, v, 0, 0, ww)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        out, lse, wo = torch.empty_like(q), torch.empty(2, 8, device=ph.DEV), torch.empty_like(x)
        side.wait_stream(torch.cuda.current_stream())
        _lib.mikv_paged_attention(q, cache, 0, 0, 0, out, lse, stream=side)
        _lib.mikv_window_attention(x, k, v, 0, 0, wo, stream=side)
        torch.full((1 << 22,), float("nan"), device=ph.DEV)          # memory of the current stream, written at once
        got.append((out, lse, wo))
    torch.cuda.synchronize()
    for out, lse, wo in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(wo, ww)


# --- rows in and out --------------------------------------------------------------------

def _strided(shape, dtype, seed, layout):
    """A [n][H][T][D] tensor whose memory is laid out otherwise."""
    n, H, T, D = shape
    if layout == "bthd":
        return ph.normal((n, T, H, D), seed, dtype).to(ph.DEV).transpose(1, 2)
    if layout == "padded":
        return ph.normal((n, H, T + 3, D + 8), seed, dtype).to(ph.DEV)[:, :, 1:T + 1, :D]
    return ph.normal(shape, seed, dtype).to(ph.DEV)


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("ps,T,layout", [(1, 5, "bhtd"), (16, 1, "bthd"), (7, 130, "padded"), (64, 64, "bthd"), (128, 65, "bhtd")])
def test_append_and_gather(type, ps, T, layout):
    lens = [T, T + 9, 3 * T + 2, 200]
    cache = ph.make(lens, ps, 3, type, layers=2, poison=False)
    counts, start = [T, max(T - 1, 0), T, 0], [0, 4, 2 * T + 2, 5]
    k, v = _strided((4, 3, T, 128), ph.DTYPE[type], 11, layout), _strided((4, 3, T, 128), ph.DTYPE[type], 12, layout)
    before = [ph.raw(x) for x in (cache.k, cache.v)]
    o = op.Pages(*before, ph.raw(cache.table), ph.raw(cache.lens), ph.raw(cache.refs))
    metas = None
    if type == "int8":
        metas = op.Pages(ph.raw(cache.k_meta), ph.raw(cache.v_meta), o.table, o.lens, o.refs)
    for name, x in (("k", k), ("v", v)):
        x = x.cpu()
        stored, meta = ph.quantize(x) if type == "int8" else (x, None)
        for i in range(4):
            for t in range(counts[i]):
                slot = start[i] + t
                page = o.table[i, slot // ps]
                getattr(o, name)[1, page, :, slot % ps] = ph.raw(stored[i, :, t])
                if metas is not None:
                    getattr(metas, name)[1, page, :, slot % ps] = ph.raw(meta[i, :, t])
    cache.append(1, k, v, start=ints(start), counts=ints(counts))
    np.testing.assert_array_equal(ph.raw(cache.k), o.k)
    np.testing.assert_array_equal(ph.raw(cache.v), o.v)
    if metas is not None:
        np.testing.assert_array_equal(ph.raw(cache.k_meta), metas.k)
        np.testing.assert_array_equal(ph.raw(cache.v_meta), metas.v)
    # back: every layer, a length below and above the sequences'
    for layer in (0, 1):
        for top in (T, max(lens) + 3):
            ko = _strided((4, 3, top, 128), ph.DTYPE[type], 21, layout)
            vo = _strided((4, 3, top, 128), ph.DTYPE[type], 22, layout)
            k0, v0 = ko.clone(), vo.clone()
            cache.gather(layer, ko, vo)
            for s in range(4):
                n = min(top, lens[s])
                want = [torch.from_numpy(x).to(ph.DTYPE[type]) for x in ph.sequence(cache, layer, s)]
                assert torch.equal(ko[s, :, :n].cpu(), want[0][:, :n]) and torch.equal(vo[s, :, :n].cpu(), want[1][:, :n])
                assert torch.equal(ko[s, :, n:], k0[s, :, n:]) and torch.equal(vo[s, :, n:], v0[s, :, n:])


def test_codes_at_halves_and_extremes():
    """Groups whose quotients lie on halves, tiny and huge ranges, equal values: the codes are the
    definition's, which divides in fp32."""
    T = 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 1, T, 128, generator=g)
    for t in range(40):                        # scale 2^e / 8: quotients k / 2 of many codes are exact halves
        step = 2.0 ** (t % 10 - 5)
        x[0, 0, t] = torch.randint(0, 511, (128,), generator=g) * (step / 2)
        x[0, 0, t, ::64], x[0, 0, t, 1::64] = 0.0, 255 * step
    x[0, 0, 40:44] *= 1e-6                     # scales among fp16's subnormal numbers, and below them
    x[0, 0, 44:46] *= 6e-8
    x[0, 0, 46:50] = torch.randn(4, 128, generator=g) * 2e4
    x[0, 0, 50, 3], x[0, 0, 50, 70] = 65504.0, -65504.0
    x[0, 0, 51] = 1.25
    x[0, 0, 52] = 65504.0
    x[0, 0, 52, ::2] = -65504.0
    x = x.half()
    cache = ph.make([T], 16, 1, "int8", poison=False)
    cache.append(0, x.to(ph.DEV), x.to(ph.DEV))
    codes, meta = ph.quantize(x)
    at = torch.arange(T)
    page = cache.table[0].cpu().long()[at // 16]
    for stored, sm in ((cache.k, cache.k_meta), (cache.v, cache.v_meta)):
        assert torch.equal(stored[0].cpu()[page, 0, at % 16], codes[0, 0])
        assert torch.equal(sm[0].cpu()[page, 0, at % 16], meta[0, 0])


def test_append_skips_what_it_may_not_write():
    cache = ph.make([40, 40, 40], 16, 2, "fp16", poison=False)
    x = ph.normal((4, 2, 10, 128), 3, torch.float16).to(ph.DEV)
    before = ph.raw(cache.k)
    # refused reservations, starts at or past the end, sequences out of range, negative counts
    cache.append(0, x, x, seqs=ints([0, 1, 3, -1]), start=ints([-1, 40, 0, 0]))
    cache.append(0, x, x, seqs=ints([0, 1, 2, 0]), start=ints([0, 0, 2147483647, 0]), counts=ints([0, -3, 10, 0]))
    np.testing.assert_array_equal(ph.raw(cache.k), before)
    # a repeated sequence: the first row counts; a row that runs past the end is cut; counts above T are T
    cache.append(0, x, x, seqs=ints([2, 0, 2, 1]), start=ints([35, 0, 0, 20]), counts=ints([10, 99, 10, 1]))
    at = lambda s, j: cache.k[0, int(cache.table[s, j // 16]), :, j % 16]
    assert torch.equal(at(2, 35), x[0, :, 0]) and torch.equal(at(2, 39), x[0, :, 4])
    assert torch.equal(at(0, 9), x[1, :, 9]) and torch.equal(at(1, 20), x[3, :, 0])
    changed = (ph.raw(cache.k) != before).any(axis=(0, 2, 4)).sum()
    assert changed == 5 + 10 + 1
    # no start: the sequence's last slots; more tokens than slots: nothing
    before = ph.raw(cache.k)
    cache.append(0, x[:2], x[:2], counts=ints([3, 10]))
    assert torch.equal(at(0, 37), x[0, :, 0]) and torch.equal(at(1, 30), x[1, :, 0]) and torch.equal(at(1, 39), x[1, :, 9])
    cache.lens[2] = 5
    before = ph.raw(cache.k)
    cache.append(0, x[:1], x[:1], seqs=ints([2]))
    np.testing.assert_array_equal(ph.raw(cache.k), before)


def test_rows_of_bad_pages():
    _lib.mikv_wait_status()
    cache = ph.make([40], 16, 2, "bf16", poison=False)
    cache.table[0, 1] = 10 ** 6
    x = ph.normal((1, 2, 40, 128), 3, torch.bfloat16).to(ph.DEV)
    before = ph.raw(cache.k)
    cache.append(0, x, x)
    assert _lib.mikv_wait_status() == 64
    changed = (ph.raw(cache.k) != before).any(axis=(0, 2, 4)).sum()
    assert changed == 24
    ko, vo = torch.ones_like(x), torch.ones_like(x)
    cache.gather(0, ko, vo)
    assert _lib.mikv_wait_status() == 64
    assert (ko[:, :, 16:32] == 0).all() and torch.equal(ko[:, :, :16], x[:, :, :16]) and torch.equal(vo[:, :, 32:], x[:, :, 32:])


# --- page operators ---------------------------------------------------------------------

def _same(cache, o, om=None):
    np.testing.assert_array_equal(ph.raw(cache.lens), o.lens)
    np.testing.assert_array_equal(ph.raw(cache.table), o.table)
    np.testing.assert_array_equal(ph.raw(cache.refs), o.refs)
    np.testing.assert_array_equal(ph.raw(cache.k), o.k)
    np.testing.assert_array_equal(ph.raw(cache.v), o.v)
    if om is not None:
        np.testing.assert_array_equal(ph.raw(cache.k_meta), om.k)
        np.testing.assert_array_equal(ph.raw(cache.v_meta), om.v)


def _oracles(cache):
    rest = [ph.raw(x) for x in (cache.table, cache.lens, cache.refs)]
    o = op.Pages(ph.raw(cache.k), ph.raw(cache.v), *rest)
    om = None if cache.k_meta is None else op.Pages(ph.raw(cache.k_meta), ph.raw(cache.v_meta), *rest)
    return o, om


def _random_call(rng, cache, oracles):
    """One random call, valid requests and broken ones mixed, on the cache and its oracles."""
    S, n_pages = cache.lens.numel(), cache.refs.numel()
    n = int(rng.randint(1, 6))
    some = lambda: rng.randint(-1, S + 1, size=n) if rng.rand() < 0.3 else rng.choice(S, size=min(n, S), replace=False)
    kind = rng.choice(["reserve", "fork", "free", "copy", "compact"], p=[0.35, 0.25, 0.15, 0.1, 0.15])
    seqs = some()
    n = len(seqs)
    if kind == "reserve":
        add = rng.randint(-1, 30, size=n)
        got = cache.reserve(ints(add.tolist()), seqs=ints(seqs.tolist()))
        want = [o.reserve(seqs.tolist(), add.tolist()) for o in oracles]
    elif kind == "fork":
        child = rng.randint(-1, S + 1, size=n)
        got = cache.fork(ints(seqs.tolist()), ints(child.tolist()))
        want = [o.fork(seqs.tolist(), child.tolist()) for o in oracles]
    elif kind == "free":
        got = cache.free(ints(seqs.tolist()))
        want = [o.free(seqs.tolist()) for o in oracles]
    elif kind == "copy":
        src, dst = rng.randint(-1, n_pages + 1, size=n), rng.randint(-1, n_pages + 1, size=n)
        got = cache.copy(ints(src.tolist()), ints(dst.tolist()))
        want = [o.copy(src.tolist(), dst.tolist()) for o in oracles]
    else:
        most = int(rng.randint(1, 25))
        lens = oracles[0].lens
        top = np.array([lens[s] if 0 <= s < S else 1 for s in seqs])
        pos = (rng.rand(cache.k.shape[0], n, cache.k.shape[2], most) * np.maximum(top, 1)[None, :, None, None]).astype(np.int32)
        if rng.rand() < 0.3:
            pos[rng.randint(pos.shape[0]), rng.randint(n), 0, 0] = rng.choice([-1, 10 ** 6])
        keep = rng.randint(-1, most + 2, size=n)
        got = cache.compact(ints(pos.tolist()), ints(keep.tolist()), seqs=ints(seqs.tolist()))
        want = [o.compact(seqs.tolist(), pos, keep.tolist()) for o in oracles]
    for w in want:
        np.testing.assert_array_equal(ph.raw(got), w, err_msg=kind)
    return int(np.sum(want[0] >= (0 if kind == "reserve" else 1)))


@pytest.mark.parametrize("type,ps,seed", [("fp16", 4, 0), ("bf16", 7, 1), ("int8", 4, 2), ("int8", 1, 3), ("fp16", 16, 4)])
def test_random_page_calls(type, ps, seed):
    rng = np.random.RandomState(seed)
    cache = ph.make([0, 9, 0, 5, 0, 20, 1, 0], ps, 2, type, seed=seed, layers=2, spare=int(12 + 60 / ps), max_pages=-(-64 // ps))
    o, om = _oracles(cache)
    served = 0
    for step in range(120):
        served += _random_call(rng, cache, [x for x in (o, om) if x is not None])
        _same(cache, o, om)
        owned = np.zeros_like(o.refs)                 # every reference is a table's
        for s, L in enumerate(o.lens):
            np.add.at(owned, o.table[s, :o.pages_of(L)], 1)
        np.testing.assert_array_equal(owned, o.refs)
    assert served > 60


@pytest.mark.parametrize("n_pages", [1, 15, 16, 16383, 16384, 16385, 70001])
def test_free_pages_are_found_anywhere(n_pages):
    """The last free pages of pools around the search's pass of 16384 references."""
    cache = PagedCache(1, n_pages, 1, 1, 128, 3, max(4, min(n_pages, 4)))
    cache.refs.fill_(1)
    free = sorted({0, n_pages // 2, n_pages - 1})
    cache.refs[torch.tensor(free, device=ph.DEV)] = 0
    start = cache.reserve(ints([1, len(free) - 1, 1]))
    assert start.tolist() == [0, 0, -1]
    got = cache.table[0, :1].tolist() + cache.table[1, :len(free) - 1].tolist()
    assert got == free and int(cache.refs.min()) == 1 and cache.lens.tolist() == [1, len(free) - 1, 0]


def test_requests_whose_sum_passes_32_bits():
    """4096 requests of 600000 pages each: only those that fit, in order, are served, and those that
    need no page; the sum of all is 2.4e9."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of device memory")
    S, width = 4096, 600000
    cache = PagedCache(1, 700000, 1, 1, 128, S, width)
    add = torch.full((S,), width, dtype=torch.int32, device=ph.DEV)
    add[5] = add[S - 1] = 0
    add[0] = 100000
    start = cache.reserve(add)
    want = torch.full((S,), -1, dtype=torch.int32, device=ph.DEV)
    want[0] = want[1] = want[5] = want[S - 1] = 0
    assert torch.equal(start, want)
    assert int(cache.refs.sum()) == 700000 and cache.lens[:3].tolist() == [100000, 600000, 0] and int(cache.lens[2:].sum()) == 0
    assert torch.equal(cache.table[1], torch.arange(100000, 700000, dtype=torch.int32, device=ph.DEV))
    assert (cache.table[2:] == -1).all()


def test_many_requests_of_one_call():
    S = 4096
    cache = PagedCache(1, 3 * S, 2, 1, 128, S, 4)
    add = torch.arange(S, device=ph.DEV, dtype=torch.int32) % 4
    o, _ = _oracles(cache)
    ws = cache.page_workspace(S)
    assert torch.equal(cache.reserve(add, ws=ws), torch.zeros(S, dtype=torch.int32, device=ph.DEV))
    o.reserve(list(range(S)), add.tolist())
    _same(cache, o)
    half = S // 2
    cache.free(torch.arange(half, S, device=ph.DEV, dtype=torch.int32))
    o.free(list(range(half, S)))
    parent = torch.arange(half, device=ph.DEV, dtype=torch.int32)
    ok = cache.fork(parent, parent + half, ws=ws)
    np.testing.assert_array_equal(ph.raw(ok), o.fork(list(range(half)), list(range(half, S))))
    _same(cache, o)


def test_unaligned_references():
    """The reference counts of a cache may begin at any int32."""
    hold = torch.zeros(101, dtype=torch.int32, device=ph.DEV)
    cache = PagedCache(1, 100, 4, 1, 128, 2, 25)
    cache = PagedCache.over(k=cache.k, v=cache.v, table=cache.table, lens=cache.lens, refs=hold[1:])
    hold[1:3] = 7
    assert cache.reserve(ints([9, 80])).tolist() == [0, 0]
    assert cache.table[0, :3].tolist() == [2, 3, 4] and int(hold[0]) == 0


# --- run together -----------------------------------------------------------------------

@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
def test_a_serving_sequence(type):
    """Prompts in chunks, a fork, decode steps with a window, an eviction, a finished sequence:
    what each step answers is the oracle's attention over the rows that were appended."""
    layers, Hkv, rep, ps, dt = 2, 2, 3, 16, ph.DTYPE[type]
    Hq, window, sinks = Hkv * rep, 50, 3
    cache = PagedCache(layers, 40, ps, Hkv, 128, 4, 12, type)
    ws, wa = cache.page_workspace(4), cache.attention_workspace(4, Hq)
    rng = iter(range(1000, 9999))
    rows = [[[], []] for _ in range(4)]       # per sequence: [layer] -> list of (k, v) [Hkv][D]
    stored = lambda x: ph.values(*ph.quantize(x)) if type == "int8" else x.double()

    def put(seqs, counts):
        start = cache.reserve(ints(counts), seqs=ints(seqs), ws=ws)
        assert (start >= 0).all()
        T = max(counts)
        for layer in range(layers):
            k, v = (ph.normal((len(seqs), Hkv, T, 128), next(rng), dt) for _ in range(2))
            cache.append(layer, k.to(ph.DEV), v.to(ph.DEV), seqs=ints(seqs), start=start, counts=ints(counts))
            for i, s in enumerate(seqs):
                for t in range(counts[i]):
                    rows[s][layer].append((stored(k[i, :, t]).numpy(), stored(v[i, :, t]).numpy()))

    def chunk(seqs, counts):
        """Prompt attention of the tokens just put, over the rows read back."""
        Tq, Tk = max(counts), max(len(rows[s][0]) for s in seqs)
        for layer in range(layers):
            kc, vc = (torch.full((len(seqs), Hkv, Tk, 128), float("nan"), dtype=dt, device=ph.DEV) for _ in range(2))
            cache.gather(layer, kc, vc, seqs=ints(seqs))
            q = ph.normal((len(seqs), Hq, Tq, 128), next(rng), dt).to(ph.DEV)
            out = torch.empty_like(q)
            lse = torch.empty(q.shape[:3], device=ph.DEV)
            kl = [len(rows[s][0]) for s in seqs]
            _lib.mikv_window_attention(q, kc, vc, window, sinks, out, lse, q_lens=ints(counts), k_lens=ints(kl))
            kn, vn = (np.zeros((len(seqs), Hkv, Tk, 128)) for _ in range(2))
            for i, s in enumerate(seqs):
                for j, (a, b) in enumerate(rows[s][layer]):
                    # the rows read back are rounded to 16 bits once
                    kn[i, :, j], vn[i, :, j] = (torch.from_numpy(x).float().to(dt).double().numpy() for x in (a, b))
            want, wl, mag = op.window_attention(ph.f64(q), kn, vn, window, sinks, counts, kl)
            ph.close(out, want, mag, ph.HALF_STEP[type], weights=ph.HALF_STEP[type])
            ph.close_lse(lse, wl)

    def attend(seqs):
        for layer in range(layers):
            q = _query(len(seqs), Hq, type, seed=next(rng))
            out, lse = cache.attend(layer, q, window, sinks, seqs=ints(seqs), ws=wa)
            for i, s in enumerate(seqs):
                k = np.stack([r[0] for r in rows[s][layer]], 1)
                v = np.stack([r[1] for r in rows[s][layer]], 1)
                seen = op.visible(k.shape[1] - 1, k.shape[1], window, sinks)
                for h in range(Hq):
                    want, wl, mag = op.attend_row(ph.f64(q)[i, h], k[h // rep], v[h // rep], seen)
                    ph.close(out[i, h], want, mag, ph.HALF_STEP[type], weights=2.0 ** -16)
                    assert abs(float(lse[i, h]) - wl) <= 2 * ph.FP32 + 2.0 ** -22 * abs(wl)

    put([0, 2], [70, 33])
    chunk([0, 2], [70, 33])
    put([0, 2], [21, 40])
    chunk([0, 2], [21, 40])
    assert cache.fork(ints([0, 0]), ints([1, 3]), ws=ws).tolist() == [1, 1]
    rows[1], rows[3] = ([list(x) for x in rows[0]] for _ in range(2))
    for _ in range(7):
        put([0, 1, 2, 3], [1, 1, 1, 1])
        attend([0, 1, 2, 3])
    keep = np.sort(np.stack([np.stack([np.stack([np.random.RandomState(l * 9 + h).permutation(98)[:30]
                                                 for h in range(Hkv)])] * 1) for l in range(layers)]), -1)   # [layers][1][Hkv][30]
    assert cache.compact(ints(keep.tolist()), ints([30]), seqs=ints([1]), ws=ws).tolist() == [1]
    rows[1] = [[(np.stack([rows[1][l][keep[l, 0, h, j]][0][h] for h in range(Hkv)]),
                 np.stack([rows[1][l][keep[l, 0, h, j]][1][h] for h in range(Hkv)])) for j in range(30)] for l in range(layers)]
    attend([1, 0])
    put([1, 0], [2, 1])
    attend([0, 1, 2, 3])
    assert cache.free(ints([0, 2])).tolist() == [1, 1]
    attend([3, 1])
    assert cache.free(ints([1, 3])).tolist() == [1, 1] and int(cache.refs.abs().max()) == 0


def test_a_decode_step_in_a_graph():
    """Captured once and replayed, a step reserves, appends and attends over caches that grow."""
    def step(cache, q, k, v, bufs):
        cache.reserve(bufs["one"], start=bufs["start"], ws=bufs["ws"])
        cache.append(0, k, v, start=bufs["start"])
        cache.attend(0, q, 40, 2, out=bufs["out"], lse=bufs["lse"], ws=bufs["wa"])

    caches = [ph.make([5, 62, 0], 16, 2, "fp16", spare=40, max_pages=16, poison=False) for _ in range(2)]
    q, k = torch.empty(3, 4, 128, dtype=torch.float16, device=ph.DEV), torch.empty(3, 2, 1, 128, dtype=torch.float16, device=ph.DEV)
    v = torch.empty_like(k)
    bufs = [{"one": ints([1, 1, 1]), "start": ints([0, 0, 0]), "ws": c.page_workspace(3), "wa": c.attention_workspace(3, 4),
             "out": torch.empty_like(q), "lse": torch.empty(3, 4, device=ph.DEV)} for c in caches]
    state = [x.clone() for x in (caches[0].table, caches[0].lens, caches[0].refs, caches[0].k, caches[0].v)]
    for x in (q, k, v):
        x.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[0], q, k, v, bufs[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], q, k, v, bufs[0])
    for x, y in zip((caches[0].table, caches[0].lens, caches[0].refs, caches[0].k, caches[0].v), state):
        x.copy_(y)
    for i in range(60):
        for x in (q, k, v):
            x.normal_()
        graph.replay()
        step(caches[1], q, k, v, bufs[1])
        for name in ("start", "out", "lse"):
            assert torch.equal(bufs[0][name], bufs[1][name]), (i, name)
    for x in ("table", "lens", "refs", "k", "v"):
        assert torch.equal(getattr(caches[0], x), getattr(caches[1], x))
    assert caches[0].lens.tolist() == [65, 122, 60]


def test_page_calls_in_a_graph():
    """Release, fork, compact, reserve and copy, captured once and replayed as sequences grow."""
    def calls(c, b):
        c.free(b["child"], ok=b["ok"][0])
        c.fork(b["parent"], b["child"], ok=b["ok"][1], ws=b["ws"])
        c.compact(b["keep"], b["kn"], seqs=b["child"], ok=b["ok"][2], ws=b["ws"])
        c.reserve(b["add"], seqs=b["both"], start=b["start"], ws=b["ws"])
        c.copy(b["src"], b["dst"], ok=b["ok"][3])

    caches = [ph.make([37, 64, 0, 0], 16, 2, "int8", layers=2, spare=60, max_pages=30, poison=False) for _ in range(2)]
    g = torch.Generator().manual_seed(9)
    keep = torch.stack([torch.randperm(30, generator=g)[:20].sort().values for _ in range(8)]).view(2, 2, 2, 20).int().to(ph.DEV)
    bufs = [{"child": ints([2, 3]), "parent": ints([0, 1]), "ok": torch.zeros(4, 2, dtype=torch.int32, device=ph.DEV), "keep": keep,
             "kn": ints([20, 7]), "add": ints([3, 5]), "both": ints([0, 1]), "start": ints([0, 0]), "src": ints([1, 2]),
             "dst": ints([5, 6]), "ws": c.page_workspace(2)} for c in caches]
    names = ("table", "lens", "refs", "k", "v", "k_meta", "v_meta")
    state = [getattr(caches[0], x).clone() for x in names]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(caches[0], bufs[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(caches[0], bufs[0])
    for x, y in zip(names, state):
        getattr(caches[0], x).copy_(y)
    for _ in range(40):
        graph.replay()
        calls(caches[1], bufs[1])
        assert torch.equal(bufs[0]["ok"], bufs[1]["ok"]) and torch.equal(bufs[0]["start"], bufs[1]["start"])
        for x in names:
            assert torch.equal(getattr(caches[0], x), getattr(caches[1], x)), x
    assert caches[0].lens.tolist() == [157, 264, 20, 7]


@pytest.mark.parametrize("type", ["fp16", "bf16", "int8"])
@pytest.mark.parametrize("n", [129, 256, 257, 700])
def test_batches_past_one_pass_of_the_search(type, n):
    """More rows than the threads that look for a warp's first one; long, short and empty sequences."""
    lens = np.random.RandomState(n).choice([0, 0, 1, 17, 60, 333], size=n)
    cache = ph.make(lens, 16, 2, type)
    _check(cache, _query(n, 4, type))
    _check(cache, _query(n, 4, type), 40, 3)


@pytest.mark.parametrize("type", ["fp16", "int8"])
def test_the_largest_batch(type):
    """65535 sequences of one to three slots: one of length 1 answers with its own value row."""
    n = 65535
    lens = 1 + np.arange(n) % 3
    cache = ph.make(lens, 2, 1, type, poison=False)
    q = _query(n, 2, type)
    out, lse = cache.attend(0, q)
    for i in (0, 3, 6, 32766, 65532):
        assert lens[i] == 1
        _, v = ph.sequence(cache, 0, i)
        want = torch.from_numpy(v[0, 0]).to(ph.DTYPE[type]).to(ph.DEV)
        assert torch.equal(out[i, 0], want) and torch.equal(out[i, 1], want)
    pick = [1, 2, 40000, 65534]
    want, wl, mag = ph.expect(cache, q[pick], 0, 0, 0, pick)
    ph.close(out[pick], want, mag, ph.HALF_STEP[type], 2.0 ** -16)
    ph.close_lse(lse[pick], wl)


def test_the_binding_refuses():
    cache = ph.make([20, 20], 16, 2, "bf16")
    q = _query(2, 4, "bf16")
    with pytest.raises(ValueError, match="q:"):
        cache.attend(0, q.half())
    with pytest.raises(ValueError, match="q:"):
        cache.attend(0, q.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="seqs"):
        cache.attend(0, q, seqs=torch.zeros(2, dtype=torch.int64, device=ph.DEV))
    with pytest.raises(ValueError, match="seqs"):
        cache.attend(0, q, seqs=ints([0]))
    with pytest.raises(ValueError, match="seqs"):
        cache.attend(0, q, seqs=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(_lib.MikvError) as e:
        cache.attend(3, q)
    assert e.value.code == -2
    with pytest.raises(_lib.MikvError):
        cache.attend(0, q, ws=torch.empty(16, dtype=torch.uint8, device=ph.DEV))
    x = ph.normal((2, 2, 4, 128), 1, torch.bfloat16).to(ph.DEV)
    with pytest.raises(ValueError, match="v:"):
        cache.append(0, x, x[:, :1])
    with pytest.raises(ValueError, match="k:"):
        cache.append(0, x.half(), x)
    with pytest.raises(ValueError, match="contiguous last"):
        cache.append(0, x.transpose(2, 3).contiguous().transpose(2, 3), x)
    with pytest.raises(ValueError, match="keep_pos"):
        cache.compact(torch.zeros(1, 2, 3, 1, dtype=torch.int32, device=ph.DEV), ints([1, 1]))
    with pytest.raises(ValueError, match="CUDA"):
        PagedCache(1, 1, 1, 1, 128, 1, 1, device="cpu")
    with pytest.raises(ValueError, match="v:"):
        PagedCache.over(k=cache.k, v=cache.v[:, :1], table=cache.table, lens=cache.lens, refs=cache.refs, type="bf16")
