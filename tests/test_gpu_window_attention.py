"""Prompt attention under a sliding window with sinks, against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import oracle.paged as op
import paged_helpers as ph
from mixed_precision_kv_balancer_gb300 import _lib

pytestmark = pytest.mark.gpu


def _make(B, H, T, dtype, layout, seed):
    if layout == "bthd":
        return ph.normal((B, T, H, 128), seed, dtype).to(ph.DEV).transpose(1, 2)
    if layout == "padded":
        return ph.normal((B, H + 1, T + 5, 136), seed, dtype).to(ph.DEV)[:, 1:, 2:T + 2, :128]
    if layout == "packed":            # q, k and v side by side, as one projection writes them
        return ph.normal((B, T, 3, H, 128), seed, dtype).to(ph.DEV)[:, :, 1].transpose(1, 2)
    return ph.normal((B, H, T, 128), seed, dtype).to(ph.DEV)


def _run(q, k, v, window, sinks, ql=None, kl=None):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=ph.DEV)
    lse = torch.full(q.shape[:3], 7.0, device=ph.DEV)
    _lib.mikv_window_attention(q, k, v, window, sinks, out, lse, q_lens=None if ql is None else ph.ints(ql),
                               k_lens=None if kl is None else ph.ints(kl))
    return out, lse


def _check(q, k, v, window, sinks, ql=None, kl=None):
    out, lse = _run(q, k, v, window, sinks, ql, kl)
    want, wl, mag = op.window_attention(ph.f64(q), ph.f64(k), ph.f64(v), window, sinks, ql, kl)
    name = "bf16" if q.dtype == torch.bfloat16 else "fp16"
    ph.close(out, want, mag, ph.HALF_STEP[name], weights=ph.HALF_STEP[name])    # weights rounded once
    ph.close_lse(lse, wl)
    left = np.isnan(wl)
    assert (ph.f64(out)[left] == 7).all() and (ph.f64(lse)[left] == 7).all()    # rows past q_lens
    assert _lib.mikv_wait_status() == 0
    return out, lse


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,Hkv,rep,Tq,Tk,layout", [
    (1, 1, 1, 1, 1, "bhtd"), (2, 1, 2, 1, 300, "bthd"), (1, 2, 4, 64, 64, "bhtd"), (3, 2, 1, 127, 127, "padded"),
    (1, 1, 8, 128, 128, "bthd"), (1, 2, 5, 129, 129, "packed"), (2, 1, 3, 257, 400, "bhtd"), (1, 1, 2, 511, 640, "padded"),
    (1, 1, 16, 300, 1200, "bthd"), (1, 4, 1, 1025, 1025, "bhtd"), (1, 1, 1, 17, 5, "bhtd"), (1, 1, 1, 600, 130, "bhtd")])
def test_causal(dtype, B, Hkv, rep, Tq, Tk, layout):
    q = _make(B, Hkv * rep, Tq, dtype, layout, 1)
    _check(q, _make(B, Hkv, Tk, dtype, layout, 2), _make(B, Hkv, Tk, dtype, layout, 3), 0, 0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Tq,Tk", [(700, 700), (300, 1500), (1, 1000), (130, 129)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 0), (64, 4), (128, 130), (200, 1), (513, 300), (5000, 9), (0, 5)])
def test_window_and_sinks(dtype, Tq, Tk, window, sinks):
    q, k, v = _make(1, 4, Tq, dtype, "bhtd", 1), _make(1, 2, Tk, dtype, "bhtd", 2), _make(1, 2, Tk, dtype, "bhtd", 3)
    _check(q, k, v, window, sinks)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,Hkv,rep,Tq,Tk", [(1, 1, 4, 1, 4000), (2, 2, 3, 5, 3000), (1, 1, 7, 18, 2500), (1, 2, 16, 8, 1500),
                                             (3, 1, 5, 33, 900), (1, 1, 2, 64, 5000), (1, 1, 2, 65, 2000), (1, 2, 1, 9, 6000),
                                             (1, 1, 40, 3, 2600), (1, 1, 3, 200, 4000)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5), (300, 400)])
def test_few_rows_over_many_keys(dtype, B, Hkv, rep, Tq, Tk, window, sinks):
    """Tiles that pack the rows of several heads, and items split over the keys; lengths of their own."""
    q = _make(B, Hkv * rep, Tq, dtype, "bthd", 1)
    k, v = _make(B, Hkv, Tk, dtype, "bhtd", 2), _make(B, Hkv, Tk, dtype, "bthd", 3)
    if window == 0 and Tk >= 2500:      # long enough to be split
        assert _lib.load().mikv_window_attention_workspace_bytes(B, Hkv * rep, Hkv, Tq, Tk, 0, 0) > 0
    _check(q, k, v, window, sinks)
    ql, kl = [max(0, Tq - 2 * b) for b in range(B)], [Tk - 131 * b for b in range(B)]
    kl[-1] = min(kl[-1], 200)                   # most parts see nothing
    _check(q, k, v, window, sinks, ql, kl)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,Hkv,rep,Tq,Tk,window,sinks", [
    (1, 9, 1, 2500, 2500, 0, 0), (1, 3, 5, 1300, 5000, 0, 0), (1, 3, 5, 1300, 5000, 4000, 200), (2, 40, 2, 130, 3500, 0, 0),
    (40, 2, 8, 40, 2000, 0, 0)])
def test_key_tiles_shared_out_as_one_line(dtype, B, Hkv, rep, Tq, Tk, window, sinks):
    """More items than half the SMs, cut where a CTA's equal part ends; ragged, empty and blind rows beside whole ones."""
    q = _make(B, Hkv * rep, Tq, dtype, "bthd", 1)
    k, v = _make(B, Hkv, Tk, dtype, "bhtd", 2), _make(B, Hkv, Tk, dtype, "bthd", 3)
    assert _lib.load().mikv_window_attention_workspace_bytes(B, Hkv * rep, Hkv, Tq, Tk, window, sinks) > 0
    _check(q, k, v, window, sinks)
    ql, kl = [max(0, Tq - 301 * (b % 7)) for b in range(B)], [max(0, Tk - 411 * (b % 9)) for b in range(B)]
    if B > 2:
        kl[1], ql[2], kl[5] = 10, 0, 0          # rows that see nothing, no rows, no keys
    _check(q, k, v, window, sinks, ql, kl)
    out, lse = _run(q, k, v, window, sinks, ql, kl)
    again = _run(q, k, v, window, sinks, ql, kl)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    _check(q, k, v, window, sinks, [0] * B, kl)          # nothing is asked: nothing is written
    _check(q, k, v, window, sinks, ql, [0] * B)          # no keys at all


@pytest.mark.parametrize("B,Hkv,rep,Tq,Tk,window,sinks", [(4, 3, 5, 700, 4000, 0, 0), (4, 3, 5, 700, 4000, 2000, 150), (2, 2, 3, 5, 3000, 0, 0),
                                                          (3, 2, 16, 70, 2500, 900, 5)])
def test_shared_out_keys_under_replay(B, Hkv, rep, Tq, Tk, window, sinks):
    """Lengths that change between the replays of one graph, whose workspace holds NaN before each."""
    q = _make(B, Hkv * rep, Tq, torch.float16, "bhtd", 1)
    k, v = _make(B, Hkv, Tk, torch.float16, "bthd", 2), _make(B, Hkv, Tk, torch.float16, "bhtd", 3)
    n = _lib.load().mikv_window_attention_workspace_bytes(B, Hkv * rep, Hkv, Tq, Tk, window, sinks)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device=ph.DEV)
    ql, kl = ph.ints([Tq] * B), ph.ints([Tk] * B)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=ph.DEV)
    go = lambda: _lib.mikv_window_attention(q, k, v, window, sinks, out, lse, q_lens=ql, k_lens=kl, ws=ws)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for turn in range(4):
        lens = [([Tq] * B, [Tk] * B), ([Tq - 3 * b for b in range(B)], [Tk - 700 * b for b in range(B)]), ([0] * (B - 1) + [1], [77] * B),
                ([Tq] * B, [Tq // 2] * B)][turn]
        ql.copy_(ph.ints(lens[0]))
        kl.copy_(ph.ints(lens[1]))
        ws.fill_(255)
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        want = _run(q, k, v, window, sinks, *lens)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        _check(q, k, v, window, sinks, *lens)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_padded_batches(dtype, window, sinks):
    """Lengths from none to all, more queries than keys; NaN behind every row's end."""
    ql, kl = [300, 0, 1, 130, 299, 5, 200, 0, 400, -3], [300, 0, 500, 131, 1, 0, 500, 20, 900, 7]
    q, k, v = (_make(10, H, T, dtype, "bhtd", s) for H, T, s in ((2, 300, 1), (1, 500, 2), (1, 500, 3)))
    for b in range(10):
        q[b, :, max(0, ql[b]):] = float("nan")
        k[b, :, kl[b]:] = float("nan")
        v[b, :, kl[b]:] = float("inf")
    _check(q, k, v, window, sinks, ql, kl)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rep", [1, 3])
@pytest.mark.parametrize("Tq,Tk,window,sinks", [(500, 500, 100, 200), (400, 900, 128, 400), (300, 700, 1, 257), (700, 700, 130, 140),
                                                (513, 513, 64, 513), (300, 3000, 600, 2500)])
def test_windows_that_begin_among_the_sinks(dtype, rep, Tq, Tk, window, sinks):
    """Odd groups: a CTA's two tiles are row blocks, and the second one's window begins later."""
    q, k, v = _make(1, rep, Tq, dtype, "bhtd", 1), _make(1, 1, Tk, dtype, "bhtd", 2), _make(1, 1, Tk, dtype, "bhtd", 3)
    _check(q, k, v, window, sinks)
    _check(q, k, v, window, sinks, [Tq - 130], [Tk - 7])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Tq,Tk,window,sinks", [(20, 900, 100, 5), (300, 700, 30, 0), (1, 400, 1, 130), (5, 300, 40, 64),
                                                (130, 1000, 513, 200)])
def test_rows_that_no_query_sees_hold_anything(dtype, Tq, Tk, window, sinks):
    """Between the sinks and the first query's window, and past the end, in tiles of every kind."""
    for k_len in (Tk, Tk - 37):
        q, k, v = (_make(1, H, T, dtype, "bhtd", s) for H, T, s in ((3, Tq, 1), (1, Tk, 2), (1, Tk, 3)))
        gap = slice(sinks, k_len - Tq - window + 1)
        for x, bad in ((k, float("nan")), (v, float("-inf"))):
            if gap.stop > gap.start:
                x[:, :, gap] = bad
            x[:, :, k_len:] = bad
        want, wl, mag = op.window_attention(*(ph.f64(torch.nan_to_num(x, 0, 0, 0)) for x in (q, k, v)), window, sinks, None, [k_len])
        out, lse = _run(q, k, v, window, sinks, None, [k_len])
        name = "bf16" if dtype == torch.bfloat16 else "fp16"
        ph.close(out, want, mag, ph.HALF_STEP[name], weights=ph.HALF_STEP[name])
        ph.close_lse(lse, wl)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("Hkv,rep,T,window,sinks", [(12, 2, 1200, 0, 0), (24, 1, 1900, 150, 3), (3, 5, 2500, 300, 140), (40, 2, 130, 0, 0)])
def test_many_items_of_one_cta(dtype, Hkv, rep, T, window, sinks):
    """Several items after one another in every CTA, of many lengths, empty ones among them."""
    q, k, v = (_make(4, H, T, dtype, "bthd", s) for H, s in ((Hkv * rep, 1), (Hkv, 2), (Hkv, 3)))
    _check(q, k, v, window, sinks, [T, T // 3, 0, T - 1], [T, T // 2, 9, T - 2])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("drop", [9.0, 10.5, 14.0])
def test_many_small_weights_beside_a_large_one(dtype, drop):
    q = torch.full((1, 1, 40, 128), 0.25, dtype=dtype, device=ph.DEV)
    k = torch.zeros(1, 1, 3000, 128, dtype=dtype, device=ph.DEV)
    k[0, 0, 1234] = drop / (0.25 * 128 ** 0.5)
    _check(q, k, _make(1, 1, 3000, dtype, "bhtd", 3), 0, 0)


def test_scores_that_grow_and_fall_along_the_keys():
    """The running maximum moves in every tile, by a little and by a lot."""
    for dtype in (torch.float16, torch.bfloat16):
        T = 1000
        q, k, v = (_make(1, 1, T, dtype, "bhtd", s) for s in (1, 2, 3))
        q[..., 0] = 8.0
        for sign in (1.0, -1.0):
            k[..., 0] = (sign * torch.linspace(-8, 8, T, device=ph.DEV)).to(dtype)
            _check(q, k, v, 0, 0)


def test_the_same_bits_every_time_and_in_a_graph():
    q, k, v = _make(2, 8, 700, torch.bfloat16, "bthd", 1), _make(2, 2, 900, torch.bfloat16, "bthd", 2), _make(2, 2, 900, torch.bfloat16, "bthd", 3)
    kl = ph.ints([900, 700])
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device=ph.DEV)
    call = lambda: _lib.mikv_window_attention(q, k, v, 100, 4, out, lse, k_lens=kl)
    call()
    want = out.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        lse.zero_()
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    kl.copy_(ph.ints([300, 900]))              # lengths are read when the graph runs
    graph.replay()
    again = out.clone()
    out.zero_()
    call()
    assert torch.equal(out, again) and not torch.equal(out, want[0])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_do_not_hang_on_rows_that_do_not_count(dtype):
    """The same bits whatever lies behind the queries' end, and beside them in a tile."""
    q, k, v = _make(1, 2, 40, dtype, "bhtd", 1), _make(1, 1, 3000, dtype, "bhtd", 2), _make(1, 1, 3000, dtype, "bhtd", 3)
    k[..., 0] = torch.linspace(-6, 6, 3000, device=ph.DEV).to(dtype)      # the maxima move along the keys
    out, lse = _run(q, k, v, 0, 0, [9], [2500])
    for fill in (100.0, float("inf"), float("nan"), 0.0):
        q[:, :, 9:] = fill
        o2, l2 = _run(q, k, v, 0, 0, [9], [2500])
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    want = [x[:, :, :1] for x in _run(q[:, :, :9].contiguous(), k, v, 0, 0, [9], [2500])]
    for n in range(20):                                                    # tiles that hold what the last call left
        _run(_make(1, 2, 128, dtype, "bhtd", n) * 30, k, v, 0, 0)
        got = _run(q[:, :, :9].contiguous(), k, v, 0, 0, [9], [2500])
        assert all(torch.equal(a[:, :, :1], b) for a, b in zip(got, want))


def test_two_calls_at_once_and_split_keys_in_a_graph():
    """Calls on two streams, one of them split over its keys, eager and replayed."""
    calls = [(_make(1, 8, 5, torch.float16, "bhtd", 1), _make(1, 2, 7000, torch.float16, "bhtd", 2), _make(1, 2, 7000, torch.float16, "bhtd", 3)),
             (_make(2, 6, 900, torch.bfloat16, "bthd", 4), _make(2, 3, 900, torch.bfloat16, "bthd", 5), _make(2, 3, 900, torch.bfloat16, "bthd", 6))]
    want = [_run(*c, 500, 3) for c in calls]
    outs = [(torch.empty_like(c[0]), torch.empty(c[0].shape[:3], device=ph.DEV)) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    sizes = [_lib.load().mikv_window_attention_workspace_bytes(c[0].shape[0], c[0].shape[1], c[1].shape[1], c[0].shape[2],
                                                               c[1].shape[2], 500, 3) for c in calls]
    ws = [torch.empty(max(n, 32), dtype=torch.uint8, device=ph.DEV) for n in sizes]
    go = lambda i: _lib.mikv_window_attention(*calls[i], 500, 3, *outs[i], ws=ws[i])
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                go(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(0)
        go(1)
    for _ in range(5):
        for o in outs:
            for x in o:
                x.zero_()
        graph.replay()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))


def test_rows_past_32_bit_offsets():
    """2.4e9 values a tensor; under a window of one every query answers with its own value row."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    H, T = 63, 301000
    k = torch.ones(1, 1, T, 128, dtype=torch.bfloat16, device=ph.DEV).expand(1, H, T, 128)
    v = torch.empty(1, H, T, 128, dtype=torch.bfloat16, device=ph.DEV).normal_()
    q = torch.empty_like(v).normal_()
    out = torch.empty_like(v)
    lse = torch.empty(1, H, T, device=ph.DEV)
    _lib.mikv_window_attention(q, k, v, 1, 0, out, lse)
    assert torch.equal(out, v)
    got, want = lse[0, -1, -9:], q[0, -1, -9:].double().sum(-1) / 128 ** 0.5
    assert (got.double() - want).abs().max() < 1e-3


def test_lse_may_be_left_out_and_rows_broadcast():
    q, k, v = (_make(2, 2, 90, torch.float16, "bhtd", s) for s in (1, 2, 3))
    k, v = k[:1].expand(2, 2, 90, 128), v[:, :1].expand(2, 2, 90, 128)
    out = torch.empty_like(q)
    _lib.mikv_window_attention(q, k, v, 0, 0, out)
    for qb in (q[:, :1].expand(2, 2, 90, 128), q[:, :1, :3].expand(2, 2, 3, 128)):    # repeated query heads
        ob = torch.empty(qb.shape, dtype=q.dtype, device=ph.DEV)
        _lib.mikv_window_attention(qb, k, v, 0, 0, ob)
        wb, _, mb = op.window_attention(ph.f64(qb), ph.f64(k), ph.f64(v), 0, 0)
        ph.close(ob, wb, mb, 2.0 ** -11, 2.0 ** -11)
    want, _, mag = op.window_attention(ph.f64(q), ph.f64(k), ph.f64(v), 0, 0)
    ph.close(out, want, mag, 2.0 ** -11, 2.0 ** -11)


def test_the_binding_refuses():
    q, k = _make(1, 4, 8, torch.float16, "bhtd", 1), _make(1, 2, 8, torch.float16, "bhtd", 2)
    out = torch.empty_like(q)
    wa = _lib.mikv_window_attention
    with pytest.raises(ValueError, match="q:"):
        wa(q.float(), k, k, 0, 0, out)
    with pytest.raises(ValueError, match="k:"):
        wa(q, k.bfloat16(), k, 0, 0, out)
    with pytest.raises(ValueError, match="v:"):
        wa(q, k, k[:, :, :7], 0, 0, out)
    with pytest.raises(ValueError, match="out:"):
        wa(q, k, k, 0, 0, out[:, :2])
    with pytest.raises(ValueError, match="lse"):
        wa(q, k, k, 0, 0, out, torch.empty(1, 4, 9, device=ph.DEV))
    with pytest.raises(ValueError, match="k_lens"):
        wa(q, k, k, 0, 0, out, k_lens=torch.tensor([3], dtype=torch.int32))
    for kw in (dict(window=-1, sinks=0), dict(window=0, sinks=-2)):
        with pytest.raises(_lib.MikvError) as e:
            wa(q, k, k, kw["window"], kw["sinks"], out)
        assert e.value.code == -1
    with pytest.raises(_lib.MikvError) as e:
        wa(q[..., :64].contiguous(), k[..., :64].contiguous(), k[..., :64].contiguous(), 0, 0, out[..., :64].contiguous())
    assert e.value.code == -4
    with pytest.raises(_lib.MikvError) as e:      # three query heads over two key heads
        wa(q[:, :3], k, k, 0, 0, out[:, :3])
    assert e.value.code == -2
    odd = ph.normal((1, 2, 8, 129), 1, torch.float16).to(ph.DEV)[..., :128]
    with pytest.raises(_lib.MikvError) as e:
        wa(q, odd, k, 0, 0, out)
    assert e.value.code == -3
