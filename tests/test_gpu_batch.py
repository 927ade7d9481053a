"""Packed batches on the GPU: row maps, rows into slots, bounds of pages' keys, and the choice of blocks, against
the oracle to the bit; attention over picked blocks and a whole serving step against it in 64 bits."""
import threading

import numpy as np
import pytest
import torch

import oracle.batch as ob
import paged_helpers as ph
from mixed_precision_kv_balancer_gb300 import _lib
from mixed_precision_kv_balancer_gb300.paged import PagedCache

pytestmark = pytest.mark.gpu
ints = ph.ints
TYPES = ["fp16", "bf16", "int8"]


def _query(rows, Hq, type, seed=5):
    q = ph.normal((rows, Hq, 128), seed, ph.DTYPE[type])
    q[..., 3::29] *= 2
    return q.to(ph.DEV)


def keys32(cache, layer, s):
    """Sequence s's stored keys in slot order, [len][Hkv][D] fp32 (INT8: one rounding)."""
    return ph.sequence(cache, layer, s)[0].transpose(1, 0, 2).astype(np.float32)


# --- row maps ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,ps,counts,seqs,start,rows", [
    ([5], 4, [1], None, None, 1), ([9, 0, 30, 4], 4, [2, 0, 7, 4], None, None, 13), ([9, 3, 30, 4], 7, [3, 4, 9, 1], None, None, 40),
    ([9, 3, 30, 4], 1, [3, 5, 40, -2], [2, 0, 1, 3], [25, -1, 0, 2], 50), ([50, 60], 16, [8, 8, 8, 8, 8], [1, 1, -1, 2, 0], [52, 0, 0, 0, 44], 44),
    ([300] * 70, 16, [1 + i % 5 for i in range(70)], None, None, 150), ([8], 4, [0], None, None, 3),
    ([8, 8], 4, [2 ** 31 - 1, 2], None, [0, 6], 9), ([8, 8], 4, [3, 2], None, [2 ** 31 - 2, 6], 9)])
def test_row_maps(lens, ps, counts, seqs, start, rows):
    cache = ph.make(lens, ps, 1, "fp16")
    b = cache.rows(ints(counts), rows, seqs=None if seqs is None else ints(seqs), start=None if start is None else ints(start))
    short = [min(c, rows + 1) for c in counts]
    want = ob.batch_rows(cache.table.cpu().numpy(), lens, ps, cache.refs.numel(), seqs, start, short, rows)
    if counts[0] > rows and start is not None:
        want = [np.minimum(w.astype(np.int64), 2 ** 31 - 1) for w in want]
    for got, w in zip(b[:4], want):
        np.testing.assert_array_equal(got.cpu().numpy(), w if not (start and max(start) > 2 ** 30) else
                                      np.where(w < -1, 2 ** 31 - 1, w))
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("n", [257, 1500, 4096])
def test_row_maps_of_many_requests(n):
    rng = np.random.RandomState(n)
    lens = rng.randint(0, 40, n)
    cache = ph.make(lens, 8, 1, "fp16")
    seqs = rng.randint(-1, n + 1, n)
    counts = rng.randint(0, 6, n)
    rows = int(counts.sum()) + 17
    b = cache.rows(ints(counts), rows, seqs=ints(seqs))
    table, seen = cache.table.cpu().numpy(), set()
    row_start, want, at = [0], np.full((3, rows), -1, np.int64), 0
    for s, c in zip(seqs.tolist(), counts.tolist()):
        if 0 <= s < n and s not in seen and lens[s] >= c:
            p = lens[s] - c + np.arange(c)
            want[:, at:at + c] = np.full(c, s), p, table[s, p // 8] * 8 + p % 8
        seen.add(s)
        at += c
        row_start.append(at)
    for got, w in zip(b[:4], (row_start, *want)):
        np.testing.assert_array_equal(got.cpu().numpy(), w)


def test_row_maps_meet_bad_pages():
    _lib.mikv_wait_status()
    cache = ph.make([40, 20], 8, 1, "fp16")
    cache.table[0, 4] = cache.refs.numel()
    b = cache.rows(ints([10, 2]), 12)
    assert (b.slot[2:10] == -1).all() and (b.slot[:2] >= 0).all() and (b.slot[10:] >= 0).all() and (b.seq[:10] == 0).all()
    assert _lib.mikv_wait_status() == 64


# --- rows into slots --------------------------------------------------------------------

def _strided(shape, type, seed, layout):
    rows, H, D = shape
    if layout == "heads":                # [H][rows][D]
        return ph.normal((H, rows, D), seed, ph.DTYPE[type]).to(ph.DEV).transpose(0, 1)
    if layout == "packed":               # as one projection writes queries, keys and values
        return ph.normal((rows, 3, H, D), seed, ph.DTYPE[type]).to(ph.DEV)[:, 1]
    if layout == "padded":
        return ph.normal((rows + 1, H, D + 8), seed, ph.DTYPE[type]).to(ph.DEV)[1:, :, :D]
    return ph.normal(shape, seed, ph.DTYPE[type]).to(ph.DEV)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("layout", ["rows", "heads", "packed", "padded"])
@pytest.mark.parametrize("lens,ps,Hkv,counts", [([1], 16, 1, [1]), ([40, 0, 33, 70], 16, 2, [40, 0, 1, 65]), ([100, 37], 7, 3, [90, 2]), ([9], 1, 2, [9])])
def test_rows_into_slots(type, layout, lens, ps, Hkv, counts):
    a, b = (ph.make(lens, ps, Hkv, type, layers=2) for _ in range(2))
    rows = sum(counts) + 3
    k, v = (_strided((rows, Hkv, 128), type, seed, layout) for seed in (3, 4))
    batch = a.rows(ints(counts), rows)
    a.put(1, k, v, batch)
    # the same rows, padded, through the call that takes sequences
    T = max(counts)
    at, kp, vp = 0, *(torch.zeros(len(lens), Hkv, T, 128, dtype=k.dtype, device=ph.DEV) for _ in range(2))
    for i, c in enumerate(counts):
        kp[i, :, :c], vp[i, :, :c] = k[at:at + c].transpose(0, 1), v[at:at + c].transpose(0, 1)
        at += c
    b.append(1, kp, vp, counts=ints(counts))
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_meta, b.k_meta), (a.v_meta, b.v_meta)):
        if x is not None:
            np.testing.assert_array_equal(ph.raw(x), ph.raw(y))
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", TYPES)
def test_slots_that_are_skipped(type):
    _lib.mikv_wait_status()
    cache = ph.make([40, 20], 8, 2, type, poison=False)
    before = cache.k.clone()
    k = ph.normal((4, 2, 128), 1, ph.DTYPE[type]).to(ph.DEV)
    n = cache.refs.numel() * 8
    shared = int(cache.table[1, 0])
    cache.refs[shared] = 2
    _lib.mikv_slot_append(cache, 0, k, k, ints([-1, -2 ** 31, n, 2 ** 31 - 1]))
    assert _lib.mikv_wait_status() == 64 and torch.equal(cache.k, before)
    _lib.mikv_slot_append(cache, 0, k, k, ints([shared * 8 + 3, -1, -7, -1]))
    assert _lib.mikv_wait_status() == 128 and torch.equal(cache.k, before)
    _lib.mikv_slot_append(cache, 0, k, k, ints([-1, n - 1, 0, -1]))
    changed = (cache.k != before).any(-1).nonzero()[:, 1:]
    assert {(int(p), int(r)) for p, _, r in changed} <= {(cache.refs.numel() - 1, 7), (0, 0)} and len(changed)


# --- bounds of pages --------------------------------------------------------------------

def _bounds_of_all(cache, layer=0):
    buf = cache.bounds_buffers()
    lens = cache.lens.clone()
    cache.renew(layer, cache.rows(lens, int(lens.sum())), buf)
    return buf


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("lens,ps,Hkv", [([1], 16, 1), ([40, 0, 33, 70], 16, 2), ([100, 37], 7, 3), ([9], 1, 2), ([300, 5], 100, 1), ([700], 512, 2)])
def test_bounds(type, lens, ps, Hkv):
    cache = ph.make(lens, ps, Hkv, type, layers=2)
    bounds, scales = _bounds_of_all(cache, 1)
    assert (bounds[0] == 0).all() and (scales[0] == 0).all()
    touched = set()
    for s, L in enumerate(lens):
        k = keys32(cache, 1, s)
        for b in range(-(-L // ps)):
            page = int(cache.table[s, b])
            touched.add(page)
            for h in range(Hkv):
                codes, scale = ob.bounds(k[b * ps:(b + 1) * ps, h])
                assert float(scales[1, page, h]) == scale
                np.testing.assert_array_equal(bounds[1, page, h].cpu().numpy(), codes)
    rest = [p for p in range(cache.refs.numel()) if p not in touched]
    assert (bounds[1, rest] == 0).all() and (scales[1, rest] == 0).all()
    assert _lib.mikv_wait_status() == 0


def test_bounds_of_what_is_no_number_and_of_zeros():
    cache = ph.make([64], 8, 1, "bf16", poison=False)
    page = cache.table[0].long()
    cache.k[0, page[0], 0, 3, 5] = float("nan")
    cache.k[0, page[1], 0, 7, 127] = float("-inf")
    cache.k[0, page[2]] = 0
    cache.k[0, page[3]] = 1e-40                      # the scale is 0, or below what is normal
    bounds, scales = _bounds_of_all(cache)
    assert torch.isinf(scales[0, page[:2], 0]).all() and (bounds[0, page[:2]] == 0).all()
    assert scales[0, page[2], 0] == 0 and (bounds[0, page[2]] == 0).all()
    codes, scale = ob.bounds(keys32(cache, 0, 0)[24:32, 0])
    assert float(scales[0, page[3], 0]) == scale and (bounds[0, page[3], 0].cpu().numpy() == codes).all()


def test_bounds_of_rows_without_a_place():
    _lib.mikv_wait_status()
    cache = ph.make([20, 8], 8, 1, "fp16")
    buf = cache.bounds_buffers()
    _lib.mikv_page_bounds(cache, 0, ints([-1, 2, 0, 0, 1, 1]), ints([0, 0, -1, 20, 8, 2 ** 31 - 1]), *buf)
    assert (buf[0] == 0).all() and _lib.mikv_wait_status() == 0
    cache.table[0, 1] = -1
    _lib.mikv_page_bounds(cache, 0, ints([0, 0, 1]), ints([9, 17, 3]), *buf)
    assert _lib.mikv_wait_status() == 64
    assert set(buf[1][0, :, 0].nonzero()[:, 0].tolist()) == {int(cache.table[0, 2]), int(cache.table[1, 0])}


# --- the choice of blocks ---------------------------------------------------------------

def _choice(cache, q, buf, row_seq, row_pos, keep, first, recent, layer=0):
    """Expected (sel, n_sel) and, per row and head, the blocks."""
    rows, Hq, _ = q.shape
    Hkv, ps = cache.k.shape[2], cache.k.shape[3]
    rep = Hq // Hkv
    sel, n_sel = np.full((rows, Hkv, keep), -1, np.int32), np.zeros((rows, Hkv), np.int32)
    bounds, scales, table = buf[0].cpu().numpy(), buf[1].cpu().numpy(), cache.table.cpu().numpy()
    qn = q.float().cpu().numpy()
    for r in range(rows):
        s = row_seq[r]
        if not 0 <= s < cache.lens.numel():
            continue
        p = min(row_pos[r], int(cache.lens[s]) - 1)
        nb = p // ps + 1
        page = table[s, :max(nb, 0)]
        for h in range(Hkv):
            got = ob.pick(ob.scores(qn[r, h * rep:(h + 1) * rep], bounds[layer, page, h], scales[layer, page, h]), keep, first, recent)
            sel[r, h, :len(got)] = got
            n_sel[r, h] = len(got)
    return sel, n_sel


def _check_choice(cache, q, keep, first=0, recent=1, row_seq=None, row_pos=None, buf=None, layer=0):
    buf = _bounds_of_all(cache, layer) if buf is None else buf
    rows = q.shape[0]
    seq = list(range(rows)) if row_seq is None else row_seq
    pos = [int(cache.lens[s]) - 1 if 0 <= s < cache.lens.numel() else 0 for s in seq] if row_pos is None else row_pos
    want, wn = _choice(cache, q, buf, seq, pos, keep, first, recent, layer)
    sel = torch.full(want.shape, 77, dtype=torch.int32, device=ph.DEV)
    n_sel = torch.full(wn.shape, 77, dtype=torch.int32, device=ph.DEV)
    _lib.mikv_block_select(q, cache, layer, *buf, first, recent, sel, n_sel, row_seq=None if row_seq is None else ints(row_seq),
                           row_pos=None if row_pos is None else ints(row_pos))
    np.testing.assert_array_equal(n_sel.cpu().numpy(), wn)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)
    return sel, n_sel


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("lens,ps,Hkv,rep,keep,first,recent", [
    ([1], 16, 1, 1, 1, 0, 1), ([0, 1, 15, 16, 17, 200], 16, 2, 4, 3, 1, 1), ([333, 500], 7, 1, 8, 10, 2, 3), ([600], 1, 2, 5, 64, 0, 1),
    ([1000, 40], 20, 3, 9, 5, 0, 2), ([900], 16, 1, 16, 57, 1, 4), ([900], 16, 1, 17, 56, 1, 4), ([5000, 0], 8, 1, 2, 300, 1, 2),
    ([2500], 1, 1, 1, 1, 0, 1), ([300, 300], 64, 2, 40, 2, 1, 1)])
def test_choice(type, lens, ps, Hkv, rep, keep, first, recent):
    cache = ph.make(lens, ps, Hkv, type, layers=2)
    _check_choice(cache, _query(len(lens), Hkv * rep, type), keep, first, recent, layer=1)
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", ["fp16", "int8"])
def test_choice_among_very_many_blocks(type):
    cache = ph.make([20000, 9000], 1, 1, type)
    for keep in (1, 255, 4000):
        _check_choice(cache, _query(2, 3, type), keep, 1 if keep > 1 else 0, 1)


def test_choice_of_rows_in_any_order():
    cache = ph.make([90, 0, 400, 33], 16, 2, "bf16")
    seq, pos = [2, 2, 2, 0, -1, 4, 1, 3, 3, 2], [399, 0, 250, 80, 5, 5, 0, 1000, -1, 2 ** 31 - 1]
    _check_choice(cache, _query(10, 8, "bf16"), 4, 1, 2, seq, pos)


def test_equal_scores_go_to_the_lower_block():
    cache = ph.make([640], 16, 1, "fp16", poison=False)
    cache.k[:] = 1.0
    buf = _bounds_of_all(cache)
    q = torch.ones(1, 2, 128, dtype=torch.float16, device=ph.DEV)
    sel, _ = _check_choice(cache, q, 7, 1, 2, buf=buf)
    assert sel[0, 0].tolist() == [0, 1, 2, 3, 4, 38, 39]
    # zero queries, zero keys, queries and bounds that are no numbers
    for x in (0.0, float("nan"), float("inf"), -float("inf")):
        q[0, 1, 9] = x
        _check_choice(cache, q, 7, 1, 2, buf=buf)
    q = torch.zeros_like(q)
    _check_choice(cache, q, 7, 1, 2, buf=buf)
    buf[1][0, cache.table[0, 20].long()] = float("inf")
    buf[0][0, cache.table[0, 20].long()] = 0
    assert 20 in _check_choice(cache, q, 4, 0, 1, buf=buf)[0].tolist()[0][0]


# --- attention over picked blocks -------------------------------------------------------

def _check_blocks(cache, q, sel, n_sel, row_seq, row_pos, layer=0):
    rows, Hq, D = q.shape
    Hkv, ps = cache.k.shape[2], cache.k.shape[3]
    out = torch.full_like(q, float("nan"))
    lse = torch.full((rows, Hq), float("nan"), device=ph.DEV)
    _lib.mikv_block_attention(q, cache, layer, sel, n_sel, out, lse, row_seq=ints(row_seq), row_pos=ints(row_pos))
    want, wl, mag = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf), np.zeros((rows, Hq, D))
    qn, sn, nn = ph.f64(q), sel.cpu().numpy(), n_sel.cpu().numpy()
    kept = {s: ph.sequence(cache, layer, s) for s in set(row_seq) if 0 <= s < cache.lens.numel() and int(cache.lens[s]) > 0}
    for r, (s, p) in enumerate(zip(row_seq, row_pos)):
        if s not in kept:
            continue
        k, v = kept[s]
        p = min(p, k.shape[1] - 1)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            j = [b * ps + i for b in sn[r, hk, :max(0, min(nn[r, hk], sel.shape[2]))] if 0 <= b <= p // ps for i in range(ps)]
            j = np.array([x for x in j if x <= p], int)
            want[r, h], wl[r, h], mag[r, h] = ob_attend(qn[r, h], k[hk][j], v[hk][j])
    ph.close(out, want, mag, ph.HALF_STEP[cache.type], weights=2.0 ** -16)
    ph.close_lse(lse, wl)
    return out, lse


def ob_attend(q, k, v):
    import oracle.paged as op
    return op.attend_row(q, k, v, np.ones(len(k), bool))


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("lens,ps,Hkv,rep,keep", [([1], 16, 1, 1, 1), ([0, 1, 15, 16, 17, 200], 16, 2, 4, 3), ([333, 500], 7, 1, 8, 10),
                                                  ([600], 1, 2, 5, 64), ([1000, 40], 20, 3, 9, 5), ([900], 16, 1, 17, 40),
                                                  ([300, 300], 128, 2, 16, 2), ([3000, 2000, 100], 32, 4, 3, 60)])
def test_block_attention(type, lens, ps, Hkv, rep, keep):
    cache = ph.make(lens, ps, Hkv, type, layers=2)
    q = _query(len(lens), Hkv * rep, type)
    sel, n_sel = cache.pick(1, q, _bounds_of_all(cache, 1), keep)
    seq, pos = list(range(len(lens))), [max(L - 1, -1) for L in lens]
    out, lse = _check_blocks(cache, q, sel, n_sel, seq, pos, layer=1)
    again = cache.attend_blocks(1, q, sel, n_sel)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", TYPES)
def test_blocks_in_any_order_repeated_and_out_of_range(type):
    _lib.mikv_wait_status()
    cache = ph.make([90, 0, 400, 33], 16, 2, type)
    seq, pos = [2, 2, 2, 0, -1, 4, 1, 3, 3, 2], [399, 0, 250, 80, 5, 5, 0, 1000, -1, 2 ** 31 - 1]
    rng = np.random.RandomState(1)
    sel = torch.from_numpy(rng.randint(0, 25, (10, 2, 6)).astype(np.int32)).to(ph.DEV)
    sel[2, 0] = 3                                    # six times the same block
    sel[0, 1, 2:4] = torch.tensor([-1, 2 ** 31 - 1])
    n_sel = torch.from_numpy(rng.randint(0, 7, (10, 2)).astype(np.int32)).to(ph.DEV)
    n_sel[0, 1], n_sel[1, 0], n_sel[2, 1], n_sel[9, 0] = 6, 0, 2 ** 31 - 1, -5
    _check_blocks(cache, _query(10, 8, type), sel, n_sel, seq, pos)
    assert _lib.mikv_wait_status() == 64             # blocks that are none of their row's
    cache.table[2, 3] = -1                           # a block without a page is not seen
    n_sel.fill_(1)
    sel[:3] = torch.tensor([[3] * 6, [0] * 6])
    out, lse = cache.attend_blocks(0, _query(3, 8, type), sel[:3], n_sel[:3],
                                   cache.rows(ints([3]), 3, seqs=ints([2])))
    assert (out[:, :4] == 0).all() and torch.isneginf(lse[:, :4]).all() and torch.isfinite(lse[:, 4:]).all()
    assert _lib.mikv_wait_status() == 64


@pytest.mark.parametrize("type", TYPES)
def test_all_blocks_are_dense_attention(type):
    cache = ph.make([700, 33, 0, 260], 16, 2, type)
    q = _query(4, 8, type)
    sel, n_sel = cache.pick(0, q, _bounds_of_all(cache), 44)
    out, lse = cache.attend_blocks(0, q, sel, n_sel)
    want, wl, mag = ph.expect(cache, q, 0, 0, 0)
    ph.close(out, want, mag, ph.HALF_STEP[type], weights=2.0 ** -16)
    ph.close_lse(lse, wl)


def test_bounds_behind_a_row_past_the_length():
    """A row past its sequence's length does nothing, so that the next one on its page does the page."""
    cache = ph.make([13], 8, 1, "fp16")
    buf, want = cache.bounds_buffers(), _bounds_of_all(cache)
    _lib.mikv_page_bounds(cache, 0, ints([0, 0, 0]), ints([15, 14, 9]), *buf)
    page = int(cache.table[0, 1])
    assert torch.equal(buf[0][0, page], want[0][0, page]) and torch.equal(buf[1][0, page], want[1][0, page]) and buf[1][0, page, 0] > 0


def test_row_maps_of_several_threads():
    """Calls of different sizes whose tables of sequences need more shared memory than a kernel has unasked, each thread's
    on a stream of its own: none fails for what another asks."""
    lib, failed, done = _lib.load(), [], []
    sizes = [2049, 2600, 3300, 4096]
    cache = ph.make([3] * 4096, 8, 1, "fp16")
    work = []
    for n in sizes:
        seqs, counts = torch.randperm(4096, device=ph.DEV)[:n].int(), torch.ones(n, dtype=torch.int32, device=ph.DEV)
        work.append((n, seqs, counts, torch.empty(n + 1, dtype=torch.int32, device=ph.DEV),
                     torch.empty(3, n, dtype=torch.int32, device=ph.DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    begin = threading.Barrier(len(work))

    def run(n, seqs, counts, row_start, maps, stream):
        torch.cuda.set_device(0)
        args = (cache.ref, seqs.data_ptr(), None, counts.data_ptr(), n, n, row_start.data_ptr(), *(m.data_ptr() for m in maps),
                stream.cuda_stream)
        begin.wait()
        codes = {lib.mikv_batch_rows(*args) for _ in range(3000)}
        stream.synchronize()
        (done if codes == {0} else failed).append((n, codes))

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(done) == len(work), failed
    for n, seqs, _, row_start, maps, _ in work:
        assert torch.equal(row_start, torch.arange(n + 1, dtype=torch.int32, device=ph.DEV)) and torch.equal(maps[0], seqs)
        assert (maps[1] == 2).all() and torch.equal(maps[2], cache.table[seqs.long(), 0] * 8 + 2)


def _alike(a, la, b, lb, half_step, weights):
    """Two answers of which each is off by half a step of itself, and its weights' and fp32's share of values below 8."""
    a, b, slack = a.double(), b.double(), 8 * (weights + ph.FP32)
    assert ((a - b).abs() <= 2 * half_step * (torch.maximum(a.abs(), b.abs()) + slack) + 2 * slack).all()
    assert ((la - lb).abs() <= 4 * ph.FP32 + 2.0 ** -21 * lb.abs()).all()


@pytest.mark.parametrize("type", TYPES)
def test_more_rows_than_a_call_over_picked_blocks_takes(type):
    """A batch of 2100 rows and 32 key heads, 67200 pairs: the same as its halves, and attention of packed rows over all blocks."""
    H, n = 32, 2100
    cache = ph.make([n - 300, 300], 64, H, type)
    q = _query(n, H, type)
    batch = cache.rows(ints([n - 300, 300]), n)
    buf = cache.bounds_buffers()
    cache.renew(0, batch, buf)
    ws = cache.block_workspace(n, H, 3)
    sel, n_sel = cache.pick(0, q, buf, 3, 1, 1, batch=batch, ws=ws)
    out, lse = cache.attend_blocks(0, q, sel, n_sel, batch, ws=ws)
    for at in (slice(0, 1000), slice(1000, n)):
        half = batch._replace(seq=batch.seq[at].contiguous(), pos=batch.pos[at].contiguous())
        s, c = cache.pick(0, q[at], buf, 3, 1, 1, batch=half)
        assert torch.equal(s, sel[at]) and torch.equal(c, n_sel[at])
    rows = [0, 1, 1049, 1050, 1051, 1799, 1800, 2098, 2099]
    some = batch._replace(seq=batch.seq[rows].contiguous(), pos=batch.pos[rows].contiguous())
    got = _check_blocks(cache, q[rows], sel[rows], n_sel[rows], some.seq.tolist(), some.pos.tolist())
    _alike(out[rows], lse[rows], *got, ph.HALF_STEP[type], 2.0 ** -16)
    all_blocks = -(-n // 64)
    out, lse = cache.attend_blocks(0, q, *cache.pick(0, q, buf, all_blocks, batch=batch), batch)
    dense, dense_lse = cache.attend_rows(0, q, batch)
    _alike(out, lse, dense, dense_lse, ph.HALF_STEP[type], ph.HALF_STEP[type])


def test_more_sequences_than_a_call_over_picked_blocks_takes():
    """Without a batch, row r is sequence r in every part."""
    H, n = 32, 2060
    cache = ph.make([1 + i % 5 for i in range(n)], 2, H, "fp16")
    q = _query(n, H, "fp16")
    buf = _bounds_of_all(cache)
    sel, n_sel = cache.pick(0, q, buf, 3)
    assert torch.equal(n_sel, ((cache.lens + 1) // 2)[:, None].expand(-1, H))
    out, lse = cache.attend_blocks(0, q, sel, n_sel)
    want, wl = cache.attend(0, q)
    _alike(out, lse, want, wl, 2.0 ** -11, 2.0 ** -16)


@pytest.mark.parametrize("type", TYPES)
def test_batches_without_rows_do_nothing(type):
    cache = ph.make([40, 0], 16, 2, type)
    buf, dt = cache.bounds_buffers(), ph.DTYPE[type]
    before = [ph.raw(t) for t in (cache.k, cache.v, *buf)]
    for counts in ([], [0], [0, -3]):
        batch = cache.rows(ints(counts), 0)
        if counts:
            assert batch.row_start.tolist() == [0] * (len(counts) + 1)
        q, k = torch.empty(0, 8, 128, dtype=dt, device=ph.DEV), torch.empty(0, 2, 128, dtype=dt, device=ph.DEV)
        cache.put(0, k, k, batch)
        cache.renew(0, batch, buf)
        out, lse = cache.attend_rows(0, q, batch)
        sel, n_sel = cache.pick(0, q, buf, 3, batch=batch)
        picked = cache.attend_blocks(0, q, sel, n_sel, batch)
        assert [t.shape[0] for t in (out, lse, sel, n_sel, *picked)] == [0] * 6
    batch = cache.rows(ints([]), 5)                  # rows of no request
    assert batch.row_start.tolist() == [0] and all((t == -1).all() for t in batch[1:4])
    q = _query(5, 8, type)
    out, lse = cache.attend_rows(0, q, batch)
    sel, n_sel = cache.pick(0, q, buf, 3, batch=batch)
    picked = cache.attend_blocks(0, q, sel, n_sel, batch)
    assert (out == 0).all() and (lse == 0).all() and (n_sel == 0).all() and (sel == -1).all()
    assert (picked[0] == 0).all() and torch.isneginf(picked[1]).all()
    cache.renew(0, batch, buf)
    assert all((a == ph.raw(b)).all() for a, b in zip(before, (cache.k, cache.v, *buf))) and _lib.mikv_wait_status() == 0
