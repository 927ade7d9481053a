"""Attention of packed rows over pages against the oracle in 64 bits, and whole serving steps of packed batches."""
import subprocess
import sys

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


def _rows(rows, Hq, type, layout="rows", seed=5):
    if layout == "heads":
        return ph.normal((Hq, rows, 128), seed, ph.DTYPE[type]).to(ph.DEV).transpose(0, 1)
    if layout == "padded":
        return ph.normal((rows + 2, Hq + 1, 136), seed, ph.DTYPE[type]).to(ph.DEV)[1:rows + 1, 1:, :128]
    return ph.normal((rows, Hq, 128), seed, ph.DTYPE[type]).to(ph.DEV)


held = ph.sequence      # a sequence's keys and values, as stored


def expect(cache, q, row_start, window, sinks, seqs=None, start=None, layer=0):
    """(out, lse, mag); NaN for rows of no request."""
    rows, Hq, D = q.shape
    out, mag, lse = np.full((rows, Hq, D), np.nan), np.full((rows, Hq, D), np.nan), np.full((rows, Hq), np.nan)
    qn = ph.f64(q)
    for i in range(len(row_start) - 1):
        r0, r1 = min(max(row_start[i], 0), rows), min(max(row_start[i + 1], 0), rows)
        if r1 <= r0:
            continue
        s = i if seqs is None else seqs[i]
        out[r0:r1], mag[r0:r1], lse[r0:r1] = 0, 0, -np.inf
        if not 0 <= s < cache.lens.numel() or int(cache.lens[s]) <= 0 or (start is not None and start[i] < 0):
            continue
        k, v = held(cache, layer, s)
        first = k.shape[1] - (r1 - r0) if start is None else start[i]
        out[r0:r1], lse[r0:r1], mag[r0:r1] = ob.attend(qn[r0:r1], k, v, first + np.arange(r1 - r0), window, sinks)
    return out, lse, mag


def check(cache, q, row_start, window=0, sinks=0, seqs=None, start=None, layer=0, status=0):
    rows, Hq, _ = q.shape
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=ph.DEV)
    lse = torch.full((rows, Hq), 7.0, device=ph.DEV)
    _lib.mikv_chunk_attention(q, cache, layer, ints(row_start), window, sinks, out, lse, seqs=None if seqs is None else ints(seqs),
                              start=None if start is None else ints(start))
    want, wl, mag = expect(cache, q, row_start, window, sinks, seqs, start, layer)
    ph.close(out, want, mag, ph.HALF_STEP[cache.type], weights=ph.HALF_STEP[cache.type])   # weights rounded once
    ph.close_lse(lse, wl)
    left = np.isnan(wl)
    assert (ph.f64(out)[left] == 7).all() and (ph.f64(lse)[left] == 7).all()
    assert _lib.mikv_wait_status() == status
    return out, lse


def starts(counts):
    return [0] + np.cumsum(counts).tolist()


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("lens,ps,Hkv,rep,counts", [
    ([1], 16, 1, 1, [1]), ([9], 4, 1, 2, [9]), ([0, 1, 15, 16, 17, 200], 16, 2, 4, [0, 1, 3, 16, 5, 1]), ([333, 500], 7, 1, 8, [130, 40]),
    ([600, 30], 1, 2, 5, [64, 30]), ([1000, 40], 20, 3, 9, [257, 1]), ([900], 16, 1, 17, [128]), ([300, 300], 128, 2, 16, [300, 7]),
    ([1500, 2000, 100], 32, 2, 3, [700, 1, 100]), ([130], 64, 1, 1, [129]), ([700], 100, 1, 3, [385]), ([258, 257, 256], 16, 1, 1, [258, 257, 256])])
def test_chunks(type, lens, ps, Hkv, rep, counts):
    cache = ph.make(lens, ps, Hkv, type, layers=2)
    check(cache, _rows(sum(counts), Hkv * rep, type), starts(counts), layer=1)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 0), (64, 4), (128, 130), (200, 1), (513, 300), (5000, 9), (0, 5)])
def test_window_and_sinks(type, window, sinks):
    cache = ph.make([0, 1, 5, 700, 64, 900], 16, 2, type)
    counts = [0, 1, 2, 300, 64, 1]
    check(cache, _rows(sum(counts), 6, type), starts(counts), window, sinks)


@pytest.mark.parametrize("type", ["fp16", "int8"])
@pytest.mark.parametrize("layout", ["heads", "padded"])
def test_strided_rows(type, layout):
    cache = ph.make([300, 77], 16, 2, type)
    q = _rows(150, 8, type, layout)
    out, lse = check(cache, q, [0, 140, 150])
    into = _rows(150, 8, type, layout, seed=9)
    cache.attend_rows(0, q, cache.rows(ints([140, 10]), 150), out=into)
    assert torch.equal(into, out)


@pytest.mark.parametrize("type", TYPES)
def test_many_single_tokens_beside_chunks(type):
    rng = np.random.RandomState(3)
    lens = rng.randint(1, 900, 90).tolist()
    counts = [1] * 90
    counts[3], counts[40], lens[3], lens[40] = 200, 33, 700, 33
    cache = ph.make(lens, 16, 2, type)
    q = _rows(sum(counts), 8, type)
    out, lse = check(cache, q, starts(counts))
    again = cache.attend_rows(0, q, cache.rows(ints(counts), sum(counts)))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("type", TYPES)
def test_long_sequences_are_shared_out(type):
    cache = ph.make([20000, 6000, 3, 0, 9000], 64, 1, type)
    counts = [3, 150, 3, 0, 1]
    q = _rows(sum(counts), 4, type)
    out, lse = check(cache, q, starts(counts))
    for _ in range(3):
        again = cache.attend_rows(0, q, cache.rows(ints(counts), sum(counts)))
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    check(cache, q, starts(counts), 5000, 130)


@pytest.mark.parametrize("type", TYPES)
def test_requests_of_every_kind(type):
    """Refused, out of range, empty, named twice, behind the length, not the last rows; rows of no request."""
    cache = ph.make([90, 0, 400, 33], 16, 2, type)
    seqs = [2, 0, -1, 4, 1, 3, 2, 3, 0]
    start = [250, -1, 0, 0, 0, 30, 399, 2 ** 31 - 3, 0]
    counts = [40, 5, 3, 3, 4, 8, 1, 5, 0]
    rows = sum(counts) + 9
    check(cache, _rows(rows, 8, type), starts(counts), seqs=seqs, start=start)
    check(cache, _rows(rows, 8, type), starts(counts), 50, 3, seqs=seqs, start=start)
    check(cache, _rows(rows, 8, type), starts(counts), seqs=seqs)                # more rows than slots: some see nothing
    at = starts(counts)
    at[1], at[-1] = 38, rows + 100                                               # rows between requests, past the end
    check(cache, _rows(rows, 8, type), [min(x, rows) if i else -3 for i, x in enumerate(at)], seqs=seqs, start=start)


def test_pages_outside_the_pool_read_as_zeros():
    _lib.mikv_wait_status()
    cache = ph.make([200, 64], 16, 2, "fp16", poison=False)
    q = _rows(41, 4, "fp16")
    cache.table[0, 3] = -1
    cache.table[1, :4] = 2 ** 31 - 1
    out, lse = cache.attend_rows(0, q, cache.rows(ints([40, 1]), 41))
    assert _lib.mikv_wait_status() == 64
    cache.table[0, 3] = 0
    k, v = held(cache, 0, 0)
    k[:, 48:64], v[:, 48:64] = 0, 0
    seen = np.arange(200)[None] <= 160 + np.arange(40)[:, None]
    for h in range(4):
        l = np.where(seen, ph.f64(q)[:40, h] @ k[h // 2].T / 128 ** 0.5, -np.inf)
        w = np.exp(l - l.max(1, keepdims=True))
        want = (w @ v[h // 2]) / w.sum(1, keepdims=True)
        mag = (w @ np.abs(v[h // 2])) / w.sum(1, keepdims=True)
        ph.close(out[:40, h], want, mag, 2.0 ** -11, 2.0 ** -11)
    assert (out[40] == 0).all() and (lse[40] - np.log(64)).abs().max() < 1e-6


@pytest.mark.parametrize("type", TYPES)
def test_slots_that_no_row_sees_hold_anything(type):
    cache = ph.make([500], 16, 1, type, poison=False)
    q = _rows(3, 2, type)
    want = check(cache, q, [0, 3], 100, 5)
    page = cache.table[0].long()
    bad = cache.k if cache.k_meta is None else cache.k_meta
    badv = cache.v if cache.v_meta is None else cache.v_meta
    for t in (bad, badv):
        t[0, page[1:24]] = float("nan")              # slots 16 .. 383: the first row sees 0 .. 4 and 398 ..
        t[0, page[0], :, 5:] = float("inf")
        t[0, page[31], :, 4:] = float("nan")         # behind the last slot
    got = cache.attend_rows(0, q, cache.rows(ints([3]), 3), 100, 5)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


# --- a serving step -----------------------------------------------------------------------

@pytest.mark.parametrize("type", TYPES)
def test_serving_steps(type):
    """Prompts in chunks beside single tokens: reserve, maps, append, bounds, dense and picked attention; a fork
    and a compaction between; against a plain copy of what was stored."""
    H, rep, ps = 2, 4, 16
    cache = PagedCache(2, 120, ps, H, 128, 5, 30, type=type)
    buf = cache.bounds_buffers()
    rng = np.random.RandomState(0)
    steps = [[40, 0, 100, 1, 0], [37, 3, 1, 1, 0], [1, 1, 1, 200, 0], [1, 30, 1, 1, 0], [1, 1, 5, 1, 7]]
    for step, counts in enumerate(steps):
        n = sum(counts)
        rows = n + 5
        c = ints(counts)
        start = cache.reserve(c)
        batch = cache.rows(c, rows, start=start)
        for layer in range(2):
            k, v, q = (ph.normal((rows, h, 128), 100 * step + 10 * layer + i, ph.DTYPE[type]).to(ph.DEV)
                       for i, h in ((0, H), (1, H), (2, H * rep)))
            cache.put(layer, k, v, batch)
            cache.renew(layer, batch, buf)
            out, lse = cache.attend_rows(layer, q, batch, window=60 * layer, sinks=2 * layer)
            want, wl, mag = expect(cache, q, starts(counts), 60 * layer, 2 * layer, start=start.tolist(), layer=layer)
            ph.close(out, want, mag, ph.HALF_STEP[type], weights=ph.HALF_STEP[type])
            ph.close_lse(lse, wl)
            assert (out[n:] == 0).all()
            # picked blocks: of every row with no more than 6, all; bounds are those of the whole cache done anew
            sel, n_sel = cache.pick(layer, q[:n], buf, 6, 1, 2, batch=_first(batch, n))
            anew = cache.bounds_buffers()
            lens = cache.lens.clone()
            cache.renew(layer, cache.rows(lens, int(lens.sum())), anew)
            used = cache.refs > 0
            assert torch.equal(buf[0][layer, used], anew[0][layer, used]) and torch.equal(buf[1][layer, used], anew[1][layer, used])
            out, lse = cache.attend_blocks(layer, q[:n], sel, n_sel, _first(batch, n))
            blocks = batch.pos[:n] // ps + 1
            assert torch.equal(n_sel, blocks.clamp(max=6)[:, None].expand(-1, H).int())
            few = (blocks <= 6).cpu().numpy()
            want, wl, mag = expect(cache, q[:n], starts(counts), 0, 0, start=start.tolist(), layer=layer)
            ph.close(out[few], want[few], mag[few], ph.HALF_STEP[type], weights=2.0 ** -16)
            ph.close_lse(lse[few], wl[few])
        if step == 2:
            cache.fork(ints([0]), ints([4]))         # shares full pages, copies the last one
            keep = torch.arange(0, 64, 2, dtype=torch.int32, device=ph.DEV).expand(2, 1, H, 32).contiguous()
            assert cache.compact(keep, ints([32]), seqs=ints([2])).tolist() == [1]
            for layer in range(2):
                cache.renew(layer, cache.rows(cache.lens[[2, 4]].contiguous(), int(cache.lens[2] + cache.lens[4]), seqs=ints([2, 4])), buf)
    assert _lib.mikv_wait_status() == 0


def _first(batch, n):
    return batch._replace(seq=batch.seq[:n].contiguous(), pos=batch.pos[:n].contiguous())


@pytest.mark.parametrize("type", TYPES)
def test_a_captured_step_follows_the_lengths(type):
    """A step of fixed row arrays, captured once, replayed while the sequences grow, next to the same calls made eagerly."""
    H, rep = 2, 3
    caches = [PagedCache(1, 64, 16, H, 128, 4, 16, type=type) for _ in range(2)]
    rows, step = 48, 6
    counts = torch.zeros(4, dtype=torch.int32, device=ph.DEV)
    k, v, q = (torch.zeros(rows, h, 128, dtype=ph.DTYPE[type], device=ph.DEV) for h in (H, H, H * rep))

    def run(cache, buf, out, ws, ws2):
        start = cache.reserve(counts, start=buf[2])
        batch = cache.rows(counts, rows, start=start)
        cache.put(0, k, v, batch)
        cache.renew(0, batch, buf[:2])
        cache.attend_rows(0, q, batch, out=out[0], lse=out[1], ws=ws)
        sel, n_sel = cache.pick(0, q, buf[:2], 4, 1, 1, batch=batch, ws=ws2)
        return cache.attend_blocks(0, q, sel, n_sel, batch, ws=ws2)

    state = []
    for cache in caches:
        out = (torch.zeros_like(q), torch.zeros(rows, H * rep, device=ph.DEV))
        buf = (*cache.bounds_buffers(), torch.zeros(4, dtype=torch.int32, device=ph.DEV))
        state.append((cache, buf, out, cache.chunk_workspace(4, rows, H * rep), cache.block_workspace(rows, H * rep, 4)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(*state[1])                               # nothing to add yet
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blocks = run(*state[1])
    for i, c in enumerate([[30, 0, 17, 1], [1, 40, 1, 1], [1, 1, 1, 1], [0, 0, 0, 45], [20, 1, 1, 1], [1, 1, 1, 1]][:step]):
        counts.copy_(ints(c))
        for j, t in enumerate((k, v, q)):
            t.copy_(ph.normal(t.shape, 50 * i + j, t.dtype))
        for s in state:
            s[2][0].fill_(3), s[2][1].fill_(3)
        want = run(*state[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state[0][2][0], state[1][2][0]) and torch.equal(state[0][2][1], state[1][2][1])
        assert torch.equal(state[0][1][0], state[1][1][0]) and torch.equal(state[0][1][1], state[1][1][1])
        n = sum(c)
        assert torch.equal(want[0][:n], blocks[0][:n]) and torch.equal(want[1][:n], blocks[1][:n])


def test_calls_on_another_stream():
    cache = ph.make([700, 300], 16, 2, "fp16")
    q = _rows(120, 8, "fp16")
    batch = cache.rows(ints([100, 20]), 120)
    want = cache.attend_rows(0, q, batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.zeros_like(q), torch.zeros(120, 8, device=ph.DEV)
    _lib.mikv_chunk_attention(q, cache, 0, batch.row_start, 0, 0, out, lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# --- the largest, and what goes on beside one another -------------------------------------

@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("ps", [5, 8, 24])
def test_single_tokens_and_chunks_in_one_part_under_windows(type, ps):
    """Items of one query tile and of two behind one another in a CTA, whose ring and barriers they share."""
    rng = np.random.RandomState(ps)
    counts = rng.choice([1, 1, 2, 30, 140, 260], 60).tolist()
    lens = [c + int(x) for c, x in zip(counts, rng.randint(0, 600, 60))]
    cache = ph.make(lens, ps, 3, type)
    for window, sinks in ((0, 0), (100, 7), (300, 150)):
        check(cache, _rows(sum(counts), 6, type), starts(counts), window, sinks)


def _plain(q, k, v, seen):
    """[rows][H][D] in 64 bits on the GPU, of k, v [keys][H][D]."""
    l = torch.einsum("qhd,khd->hqk", q.double(), k.double()) / 128 ** 0.5
    l = l.masked_fill(~seen, -float("inf"))
    w = l.softmax(-1)
    return (torch.einsum("hqk,khd->qhd", w, v.double()).cpu().numpy(), torch.logsumexp(l, -1).T.cpu().numpy(),
            torch.einsum("hqk,khd->qhd", w, v.double().abs()).cpu().numpy())


@pytest.mark.parametrize("type,ps", [("fp16", 16), ("bf16", 1), ("int8", 16)])
def test_a_pool_whose_offsets_pass_32_bits(type, ps):
    """Slots past 2^32 bytes of the keys' pool: rows appended there, their bounds, and both attentions."""
    slots = (1 << 25 if type == "int8" else 1 << 24) + 64 * ps
    n_pages, len0 = slots // ps, 300
    cache = PagedCache(1, n_pages, ps, 1, 128, 2, -(-len0 // ps) + 4, type=type)
    pages = -(-len0 // ps)
    last = torch.arange(n_pages - pages, n_pages, dtype=torch.int32, device=ph.DEV).flip(0)
    if ps == 1:                                      # the first 64 alone lie past the limit
        last[64:] -= 1 << 20
        last = last.roll(100)
    cache.table[1, :pages] = last
    cache.refs[last.long()] = 1
    cache.lens[1] = len0
    k, v, q = (ph.normal((len0, h, 128), 60 + i, ph.DTYPE[type]).to(ph.DEV) for i, h in ((0, 1), (1, 1), (2, 4)))
    batch = cache.rows(ints([len0]), len0, seqs=ints([1]))
    cache.put(0, k, v, batch)
    buf = cache.bounds_buffers()
    cache.renew(0, batch, buf)
    if type == "int8":
        k, v = (ph.values(*ph.quantize(t)) for t in (k, v))
    seen = torch.ones(len0, len0, dtype=torch.bool, device=ph.DEV).tril()
    want, wl, mag = _plain(q, k.expand(-1, 4, -1), v.expand(-1, 4, -1), seen)
    out, lse = cache.attend_rows(0, q, batch)
    ph.close(out, want, mag, ph.HALF_STEP[type], weights=ph.HALF_STEP[type])
    ph.close_lse(lse, wl)
    low, scale = ob.bounds(k[:ps, 0].float().cpu().numpy())
    at = int(last[0])
    assert float(buf[1][0, at, 0]) == scale and (buf[0][0, at, 0].cpu().numpy() == low).all()
    sel, n_sel = cache.pick(0, q, buf, pages, batch=batch)
    out, lse = cache.attend_blocks(0, q, sel, n_sel, batch)
    ph.close(out, want, mag, ph.HALF_STEP[type], weights=2.0 ** -16)
    ph.close_lse(lse, wl)
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", ["bf16", "int8"])
def test_the_most_requests_and_rows(type):
    """4096 requests of 256 rows each, 2^20 in all; then of single tokens."""
    n, c, H = 4096, 256, 2
    cache = PagedCache(1, n * c // 32, 32, 1, 128, n, c // 32, type=type)
    cache.table[:] = torch.randperm(n * c // 32, device=ph.DEV).int().view(n, c // 32)
    cache.refs.fill_(1)
    cache.lens.fill_(c)
    g = torch.Generator(device=ph.DEV).manual_seed(1)
    k, v, q = (torch.randn(n * c, h, 128, generator=g, device=ph.DEV).to(ph.DTYPE[type]) for h in (1, 1, H))
    counts = torch.full((n,), c, dtype=torch.int32, device=ph.DEV)
    batch = cache.rows(counts, n * c)
    cache.put(0, k, v, batch)
    out, lse = cache.attend_rows(0, q, batch, out=torch.full_like(q, float("nan")), lse=torch.full((n * c, H), float("nan"), device=ph.DEV))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    if type == "int8":
        k, v = (ph.values(*ph.quantize(t)) for t in (k, v))
    seen = torch.ones(c, c, dtype=torch.bool, device=ph.DEV).tril()
    for i in (0, 1, 777, 2048, 4094, 4095):
        at = slice(i * c, i * c + c)
        want, wl, mag = _plain(q[at], k[at].expand(-1, H, -1), v[at].expand(-1, H, -1), seen)
        ph.close(out[at], want, mag, ph.HALF_STEP[type], weights=ph.HALF_STEP[type])
        ph.close_lse(lse[at], wl)
    last = torch.arange(c - 1, n * c, c, device=ph.DEV)
    one, ones = cache.attend_rows(0, q[last], cache.rows(torch.ones_like(counts), n))
    other, others = cache.attend(0, q[last])
    # each is off by half a step of itself and, at most, the largest value times its weights' and fp32's share
    half, a, b, top = ph.HALF_STEP[type], one.double(), other.double(), float(v.abs().max())
    slack = top * (half + ph.FP32)
    assert ((a - b).abs() <= 2 * half * (torch.maximum(a.abs(), b.abs()) + slack) + 2 * slack).all()
    assert ((ones - others).abs() <= 4 * ph.FP32 + 2.0 ** -21 * others.abs()).all()
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", TYPES)
def test_two_calls_at_once(type):
    """On two streams, with a workspace each."""
    caches = [ph.make([900, 300, 5000], 16, 2, type, seed=s) for s in (1, 2)]
    qs = [_rows(420, 8, type, seed=s) for s in (3, 4)]
    counts = ints([300, 119, 1])
    batches = [c.rows(counts, 420) for c in caches]
    bufs = [c.bounds_buffers() for c in caches]
    for c, buf in zip(caches, bufs):
        lens = c.lens.clone()
        c.renew(0, c.rows(lens, int(lens.sum())), buf)

    def run(i):
        out = caches[i].attend_rows(0, qs[i], batches[i])
        sel, n_sel = caches[i].pick(0, qs[i], bufs[i], 5, batch=batches[i])
        return (*out, sel, n_sel, *caches[i].attend_blocks(0, qs[i], sel, n_sel, batches[i]))

    want = [run(0), run(1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for a, b in zip(g, want[i]):
                assert torch.equal(a, b)
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", TYPES)
def test_replays_with_a_workspace_that_others_used(type):
    """Two captured calls of different shapes share a workspace, which holds NaN at first."""
    cache = ph.make([2000, 700, 60], 16, 2, type)
    q = _rows(500, 8, type)
    shapes = ([400, 99, 1], [1, 1, 1])
    ws = torch.full((cache.chunk_workspace(3, 500, 8).numel(),), 255, dtype=torch.uint8, device=ph.DEV)
    outs = [(torch.zeros_like(q), torch.zeros(500, 8, device=ph.DEV)) for _ in shapes]
    batches = [cache.rows(ints(c), 500) for c in shapes]
    want = [tuple(t.clone() for t in cache.attend_rows(0, q, b, 900, 20)) for b in batches]
    graphs = []
    for b, o in zip(batches, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.attend_rows(0, q, b, 900, 20, out=o[0], lse=o[1], ws=ws)
        graphs.append(g)
    for _ in range(3):
        for g, o, w in zip(graphs, outs, want):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("depth", [15, 21, 25])
def test_many_small_weights_beside_a_large_one(type, rows, depth):
    """One key of weight 1 whose value is 0, and 40000 of 2^-depth whose values are 1: fp16 weights that small are
    subnormal numbers, and all of them count."""
    n = 40000 + rows
    cache = PagedCache(1, -(-n // 64), 64, 1, 128, 1, -(-n // 64), type=type)
    cache.table[0] = torch.randperm(cache.refs.numel(), device=ph.DEV).int()
    cache.refs.fill_(1)
    cache.lens.fill_(n)
    k, v = torch.zeros(n, 1, 128, device=ph.DEV), torch.ones(n, 1, 128, device=ph.DEV)
    k[..., 0] = -depth * float(np.log(2.0)) * 128 ** 0.5       # against queries that are 1 there and 0 elsewhere
    k[7] = 0
    v[7] = 0
    q = torch.zeros(rows, 4, 128, device=ph.DEV)
    q[..., 0] = 1
    k, v, q = (t.to(ph.DTYPE[type]) for t in (k, v, q))
    cache.put(0, k, v, cache.rows(ints([n]), n))
    check(cache, q, [0, rows])
    out, _ = cache.attend_rows(0, q, cache.rows(ints([rows]), rows))
    small = 30000 * 2.0 ** -depth                    # of 40000: the keys' rounding moves a weight by 2^-8 * 17.4 at most
    assert (out >= small / (1 + small)).all()


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 3)])
def test_parts_of_many_items(type, window, sinks):
    """Several items a CTA, those at its ends cut: joined in place or by the second kernel, the bits are the same."""
    H, c, past = 32, 1500, [1300, 0]
    cache = PagedCache(1, 200, 32, 8, 128, 2, 100, type=type)
    total = ints([p + c for p in past])
    cache.reserve(total)
    n = int(total.sum())
    k, v = (ph.normal((n, 8, 128), s, ph.DTYPE[type]).to(ph.DEV) for s in (1, 2))
    cache.put(0, k, v, cache.rows(total, n))
    q = ph.normal((2 * c, H, 128), 3, ph.DTYPE[type]).to(ph.DEV)
    batch = cache.rows(ints([c, c]), 2 * c)
    out, lse = cache.attend_rows(0, q, batch, window, sinks)
    if type == "int8":
        k, v = (ph.values(*ph.quantize(t)) for t in (k, v))
    at = 0
    for i, p in enumerate(past):
        pos, j = p + torch.arange(c, device=ph.DEV)[:, None], torch.arange(p + c, device=ph.DEV)[None]
        seen = (j <= pos) & ((j > pos - window) | (j < sinks)) if window else j <= pos
        rows, keys = slice(i * c, i * c + c), slice(at, at + p + c)
        for h in range(0, H, 8):
            kv = [t[keys, h // 4:h // 4 + 2].repeat_interleave(4, 1) for t in (k, v)]
            want, wl, mag = _plain(q[rows, h:h + 8], *kv, seen)
            ph.close(out[rows, h:h + 8], want, mag, ph.HALF_STEP[type], weights=ph.HALF_STEP[type])
            ph.close_lse(lse[rows, h:h + 8], wl)
        at += p + c
    side, beside = torch.cuda.Stream(), torch.randn(4096, 4096, device=ph.DEV)
    ws = cache.chunk_workspace(2, 2 * c, H)
    for i in range(12):
        with torch.cuda.stream(side):                # something else on the SMs, so that CTAs begin and end at other times
            beside = beside @ beside * 1e-3 if i % 3 else beside
        again = cache.attend_rows(0, q, batch, window, sinks, ws=ws)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("given", [False, True])
def test_a_batch_that_its_arrays_cut_off(given):
    """Maps and attention place the rows that are left of a request alike."""
    cache = ph.make([90, 70, 50], 16, 2, "fp16")
    counts, rows = ints([20, 30, 10]), 35
    start = ints([70, 40, 40]) if given else None
    batch = cache.rows(counts, rows, start=start)
    assert batch.row_start.tolist() == [0, 20, 35, 35]
    first = 40 if given else 70 - 15
    assert batch.pos.tolist() == list(range(70, 90)) + list(range(first, first + 15)) and batch.seq.tolist() == [0] * 20 + [1] * 15
    q = _rows(rows, 8, "fp16")
    want, wl, mag = expect(cache, q, [0, 20, 35, 35], 0, 0, start=None if start is None else start.tolist())
    out, lse = cache.attend_rows(0, q, batch)
    ph.close(out, want, mag, 2.0 ** -11, weights=2.0 ** -11)
    ph.close_lse(lse, wl)
    # and picked blocks, all of them, see the same slots
    buf = cache.bounds_buffers()
    lens = cache.lens.clone()
    cache.renew(0, cache.rows(lens, int(lens.sum())), buf)
    sel, n_sel = cache.pick(0, q, buf, 6, batch=batch)
    out, lse = cache.attend_blocks(0, q, sel, n_sel, batch)
    ph.close(out, want, mag, 2.0 ** -11, weights=2.0 ** -16)
    ph.close_lse(lse, wl)


FIRST_CAPTURED = """
import torch, sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import paged_helpers as ph
cache = ph.make([300, 40], 16, 2, {type!r})
q = ph.normal((60, 8, 128), 5, ph.DTYPE[{type!r}]).to(ph.DEV)
counts, buf = ph.ints([50, 10]), cache.bounds_buffers()
k, v = (ph.normal((60, 2, 128), i, ph.DTYPE[{type!r}]).to(ph.DEV) for i in (1, 2))
ws, ws2 = cache.chunk_workspace(2, 60, 8), cache.block_workspace(60, 8, 3)
def step():
    batch = cache.rows(counts, 60)
    cache.put(0, k, v, batch)
    cache.renew(0, batch, buf)
    out = cache.attend_rows(0, q, batch, ws=ws)
    return (*out, *cache.attend_blocks(0, q, *cache.pick(0, q, buf, 3, batch=batch, ws=ws2), batch=batch, ws=ws2))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
want = step()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("alike")
"""


@pytest.mark.parametrize("type", TYPES)
def test_first_calls_of_a_process_may_be_captured(type):
    from conftest import ROOT
    res = subprocess.run([sys.executable, "-c", FIRST_CAPTURED.format(root=ROOT, type=type)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "alike" in res.stdout, res.stdout + res.stderr


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("lens,ps,Hkv,rep,counts", [([300, 90], 16, 1, 130, [1, 70]), ([77, 140], 8, 2, 65, [2, 3]), ([40], 4, 1, 1024, [1]),
                                                    ([5000, 300], 2048, 1, 2, [200, 1]), ([900, 513], 256, 2, 4, [300, 9]), ([700], 12, 1, 4, [500])])
def test_wide_groups_and_long_pages(type, lens, ps, Hkv, rep, counts):
    cache = ph.make(lens, ps, Hkv, type)
    q = _rows(sum(counts), Hkv * rep, type)
    check(cache, q, starts(counts))
    check(cache, q, starts(counts), 150, 7)
    # the same rows over picked blocks, all of them
    batch = cache.rows(ints(counts), sum(counts))
    buf = cache.bounds_buffers()
    held_ = cache.lens.clone()
    cache.renew(0, cache.rows(held_, int(held_.sum())), buf)
    blocks = -(-max(lens) // ps)
    sel, n_sel = cache.pick(0, q, buf, blocks, batch=batch)
    out, lse = cache.attend_blocks(0, q, sel, n_sel, batch)
    want, wl, mag = expect(cache, q, starts(counts), 0, 0)
    ph.close(out, want, mag, ph.HALF_STEP[type], weights=2.0 ** -16)
    ph.close_lse(lse, wl)
    assert _lib.mikv_wait_status() == 0


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 2)])
def test_more_rows_than_slots_are_refused_by_maps_and_attention_alike(type, window, sinks):
    """Requests without a start: those that the maps refuse see nothing, as if their starts were -1."""
    cache = ph.make([8, 40, 0, 200, 300], 16, 2, type)
    counts = [10, 5, 3, 201, 300]
    n = sum(counts)
    q = _rows(n, 8, type)
    batch = cache.rows(ints(counts), n)
    refused = batch.seq < 0
    assert refused.nonzero()[:, 0].tolist() == list(range(10)) + list(range(15, 219))
    out, lse = (torch.full(s, 7.0, dtype=t, device=ph.DEV) for s, t in ((q.shape, q.dtype), (q.shape[:2], torch.float32)))
    cache.attend_rows(0, q, batch, window, sinks, out=out, lse=lse)
    assert (out[refused] == 0).all() and torch.isneginf(lse[refused]).all()
    want = check(cache, q, starts(counts), window, sinks, start=[-1, 35, -1, -1, 0])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    lens = cache.lens.clone()
    buf = cache.bounds_buffers()
    cache.renew(0, cache.rows(lens, int(lens.sum())), buf)
    out, lse = cache.attend_blocks(0, q, *cache.pick(0, q, buf, 4, batch=batch), batch)
    assert (out[refused] == 0).all() and torch.isneginf(lse[refused]).all() and torch.isfinite(lse[~refused]).all()
