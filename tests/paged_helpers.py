"""Paged caches with random contents for the GPU tests, and their oracle copies."""
import numpy as np
import torch

import oracle.paged as op
from mixed_precision_kv_balancer_gb300.paged import PagedCache

DEV = "cuda"
DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.float16}
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "int8": 2.0 ** -11}   # of the outputs' type

# Errors of the fp32 work besides roundings to 16 bits, relative to sum_j w_j |v_j|.  A logit of 128
# products of N(0,1) values (sum |q k| / sqrt(128) below 16 with the outlier channels) is off by at
# most 16 * 128 * 2^-24 = 1.3e-4 if every product were rounded at the largest partial sum, which
# moves a weight by that share and the normalised one by twice it: 2.5e-4; exp2 adds 2^-22, the
# serial sums of at most 2^11 terms a thread 2^-13.  Together below 2^-11.
FP32 = 2.0 ** -11


def normal(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def raw(t):
    """The tensor's bytes as integers, for bitwise comparison."""
    t = t.detach().cpu().contiguous()
    if t.element_size() == 2:
        t = t.view(torch.int16)
    return t.numpy().copy()


def quantize(x):
    """codes uint8 and (scale, zero) fp16 of fp16 rows, per 64 channels (the definition, in fp32)."""
    x = x.float().unflatten(-1, (-1, 64))
    lo, hi = x.amin(-1), x.amax(-1)
    s, z = ((hi - lo) / torch.full_like(lo, 255.0)).half(), lo.half()
    c = (x - z.float().unsqueeze(-1)) / s.float().unsqueeze(-1)
    c = torch.where(s.float().unsqueeze(-1) > 0, c.round(), 0.0).clamp(0, 255).to(torch.uint8)
    return c.flatten(-2), torch.stack([s, z], -1)


def values(codes, meta):
    """What codes stand for, in 64 bits."""
    x = codes.double().unflatten(-1, (-1, 64))
    return (x * meta[..., :1].double() + meta[..., 1:].double()).flatten(-2)


def make(lens, ps, Hkv, type, seed=0, layers=1, spare=2, max_pages=None, poison=True):
    """A cache of sequences of these lengths over pages in random order.  Slots that no sequence
    owns hold NaN (INT8: NaN scales) if `poison`."""
    D = 128
    lens = np.asarray(lens, np.int32)
    need = -(-lens // ps)
    width = max(1, int(need.max())) if max_pages is None else max_pages
    n_pages = int(need.sum()) + spare
    rng = np.random.RandomState(seed)
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    at = 0
    live = np.zeros((n_pages, ps), bool)
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        refs[perm[at:at + n]] = 1
        for j in range(n):
            live[perm[at + j], :min(ps, lens[s] - j * ps)] = True
        at += n
    shape = (layers, n_pages, Hkv, ps, D)
    k, v = normal(shape, seed + 1, DTYPE[type]), normal(shape, seed + 2, DTYPE[type])
    k[..., 7::40] *= 3
    km = vm = None
    dead = torch.from_numpy(~live)[None, :, None, :, None]
    if type == "int8":
        (k, km), (v, vm) = quantize(k), quantize(v)
        if poison:
            km = torch.where(dead.unsqueeze(-1), torch.nan, km)
            vm = torch.where(dead.unsqueeze(-1), torch.nan, vm)
    elif poison:
        k, v = torch.where(dead, torch.nan, k), torch.where(dead, torch.nan, v)
    g = lambda t: None if t is None else t.to(DEV).contiguous()
    i32 = lambda a: torch.from_numpy(a).to(DEV)
    return PagedCache.over(k=g(k), v=g(v), k_meta=g(km), v_meta=g(vm), table=i32(table), lens=i32(lens), refs=i32(refs),
                           type=type)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def sequence(cache, layer, s):
    """Sequence s's keys and values in slot order, [Hkv][len][D] float64, from the device buffers."""
    L, ps = int(cache.lens[s]), cache.k.shape[3]
    j = torch.arange(L, device=DEV)
    page = cache.table[s].long()[j // ps]
    got = []
    for x, m in ((cache.k, cache.k_meta), (cache.v, cache.v_meta)):
        r = x[layer, page, :, j % ps]
        r = values(r, m[layer, page, :, j % ps]) if m is not None else r.double()
        got.append(r.transpose(0, 1).cpu().numpy())
    return got


def expect(cache, q, layer, window, sinks, seqs=None):
    """(out, lse, sum of weight * |value|) of every row, float64."""
    n, Hq, D = q.shape
    Hkv = cache.k.shape[2]
    out, lse, mag = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D))
    qn = f64(q)
    for i in range(n):
        s = i if seqs is None else seqs[i]
        if not 0 <= s < cache.lens.numel() or int(cache.lens[s]) == 0:
            continue
        k, v = sequence(cache, layer, s)
        seen = op.visible(k.shape[1] - 1, k.shape[1], window, sinks)
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            out[i, h], lse[i, h], mag[i, h] = op.attend_row(qn[i, h], k[hk], v[hk], seen)
    return out, lse, mag


def close(got, want, mag, half_step, weights=0.0):
    """|got - want| within half a step of the output's type plus the weights' and fp32's share."""
    got = f64(got)
    live = ~np.isnan(want)
    assert not np.isnan(got[live]).any()
    slack = mag * (weights + FP32)
    bad = np.abs(got - want) > half_step * (np.abs(want) + slack) + slack + 2.0 ** -25   # smallest fp16 half step
    bad &= live
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], mag[bad][:5])


def close_lse(got, want):
    """Within the logits' error above (twice FP32's share) and fp32's step; -inf exactly."""
    got = f64(got)
    live = ~np.isnan(want)
    got, want = got[live], want[live]
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= 2 * FP32 + 2.0 ** -22 * np.abs(want[fine])).all(), \
        np.abs(got[fine] - want[fine]).max()
