"""Measured cases of the packed-batch operators over the paged cache.

A serving step packs the new tokens of many requests, one after the other, into rows: chunks of
prompts beside single tokens.  Each case runs either in plain form (elementary torch operations, 32
bits) or, where ``own`` is true, through the package's calls.  Kinds:

  maps    which sequence, position and slot every packed row has, from the requests' lengths
          (mikv_batch_rows)
  store   the rows' keys and values into their slots, and the channel-wise bounds of the keys of the
          pages they touch (mikv_slot_append, mikv_page_bounds; 8-bit pages are read back as rows)
  chunk   attention of the packed rows over the pages (mikv_chunk_attention)
  sparse  each row picks blocks of its sequence by a score of their bounds, and attends to those
          (mikv_block_select, mikv_block_attention)
"""
import math

import torch

own = False

D = 128
GROUP = 64
DEV = "cuda"
_FLOAT = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.float16}


# --- cases ------------------------------------------------------------------------------

def _maps(name, n, T, past, ps, pad, refused):
    c = {"kind": "maps", "n": n, "chunks": n, "T": T, "past": past, "ps": ps, "pad": pad, "refused": refused, "Hkv": 1, "type": "fp16"}
    return c if name is None else {"name": name, **c}


def _store(name, n, chunks, T, past, Hkv, ps, type):
    c = {"kind": "store", "n": n, "chunks": chunks, "T": T, "past": past, "Hkv": Hkv, "ps": ps, "type": type}
    return c if name is None else {"name": name, **c}


def _chunk(name, n, chunks, T, past, Hkv, rep, ps, type, window=0, sinks=0):
    c = {"kind": "chunk", "n": n, "chunks": chunks, "T": T, "past": past, "Hkv": Hkv, "rep": rep, "ps": ps, "type": type,
         "window": window, "sinks": sinks}
    return c if name is None else {"name": name, **c}


def _sparse(name, n, each, len, Hkv, rep, ps, type, keep, first, recent, ragged):
    c = {"kind": "sparse", "n": n, "each": each, "len": len, "Hkv": Hkv, "rep": rep, "ps": ps, "type": type, "keep": keep,
         "first": first, "recent": recent, "ragged": ragged}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # a decode step of the full-depth workload's batch: a token each, nothing but latency
        _maps("maps_token", 64, 1, 8192, 16, 0, False),
        # chunks of very many requests, some refused for want of pages, rows padded to a fixed number
        _maps("maps_chunks", 700, 100, 2500, 16, 64, True),
        # a decode step's keys and values, a token each
        _store("store_token", 16, 0, 1, 4000, 8, 16, "bf16"),
        # a mixed step: some chunks of prompts and many single tokens
        _store("store_mixed", 64, 8, 1024, 4096, 8, 64, "fp16"),
        # fresh prompts stored in 8 bits
        _store("store_int8", 6, 6, 2000, 0, 4, 32, "int8"),
        # four drafted tokens and the one before them, checked behind short conversations
        _chunk("chunk_draft", 6, 6, 5, 700, 8, 4, 16, "bf16"),
        # a mixed step: four chunks of prompts and sixty single tokens
        _chunk("chunk_mixed", 64, 4, 512, 8192, 8, 4, 16, "fp16"),
        # a whole prompt of the full-depth workload's length, over the pages it was stored in
        _chunk("chunk_prompt", 1, 1, 8192, 0, 8, 4, 64, "bf16"),
        # chunks of long 8-bit prompts of a layer that sees a window and the first few tokens
        _chunk("chunk_window_int8", 3, 3, 1500, 20000, 4, 5, 32, "int8", window=2048, sinks=4),
        # one conversation of some length: nothing but latency
        _sparse("sparse_short", 1, 1, 5000, 8, 4, 16, "bf16", 64, 1, 2, False),
        # a decode batch of sequences up to 65536, an eighth of them read
        _sparse("sparse_batch", 24, 1, 65536, 8, 4, 16, "fp16", 512, 1, 4, True),
        # long 8-bit contexts, two tokens each, few large pages
        _sparse("sparse_int8", 8, 2, 131072, 4, 8, 64, "int8", 64, 1, 2, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["maps"] + ["store"] * 2 + ["chunk"] * 4 + ["sparse"] * 4)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    ps = rng.choice([1, 8, 16, 20, 32, 64, 100, 128])
    type = rng.choice(["fp16", "bf16", "int8"])
    if kind == "maps":
        n = _log(rng, 1, 1000)
        return _maps(None, n, _log(rng, 1, max(1, 70000 // n)), _log(rng, 1, min(16384, 2000000 // n)), ps, rng.choice([0, 0, 64]), rng.random() < 0.5)
    if kind == "store":
        n = _log(rng, 1, 64)
        chunks = rng.choice([0, 1, n // 8, n])
        T = _log(rng, 1, min(2048, max(1, 12000 // max(1, chunks))))
        return _store(None, n, chunks, T, 0 if type == "int8" else _log(rng, 1, 4096), Hkv, ps, type)
    if kind == "chunk":
        window = rng.choice([0, 0, 1]) * _log(rng, 1, 8192)
        sinks = rng.choice([0, 1]) * _log(rng, 1, 128)
        n = _log(rng, 1, 64)
        chunks = rng.choice([1, 1, max(1, n // 8), n])
        most = 16 * 8192 * 8192 // (Hkv * rep * chunks)           # pairs of a chunk and a head
        T = _log(rng, 1, min(8192, 2 * math.isqrt(most) // 2, max(1, 16384 // chunks)))
        room = min(16384, most // T - T // 2)
        past = _log(rng, 1, room) if room > 0 and rng.random() < 0.8 else 0
        return _chunk(None, n, chunks, T, past, Hkv, rep, ps, type, window, sinks)
    n = _log(rng, 1, 64)
    each = rng.choice([1, 1, 1, 2, 4])
    top = min(131072, 24 * 65536 * 8 // (n * Hkv), (1 << 20) * ps // (n * each * Hkv))
    len = _log(rng, max(1, each), max(each, top))
    first, recent = rng.choice([0, 1, 2]), rng.choice([1, 2, 4])
    keep = max(first + recent, _log(rng, 1, max(1, min(1024, (1 << 21) // (n * each * Hkv * ps)))))
    return _sparse(None, n, each, len, Hkv, rep, ps, type, keep, first, recent, rng.random() < 0.6)


def _lens(n, top, ragged=True):
    """n lengths up to `top`: all equal, or spread over 1 .. top with the first at the top."""
    if not ragged:
        return [top] * n
    return [max(1, int(top * (1.0 - (0.6180339887 * i) % 1.0))) for i in range(n)]


def _requests(case):
    """(rows, slots before them) of each request: chunks first, then single tokens; the last of more than
    three chunks is empty."""
    n, chunks = case["n"], case["chunks"]
    counts = _lens(chunks, case["T"]) + [1] * (n - chunks)
    if chunks > 3 and case["T"] > 1:
        counts[chunks - 1] = 0
    return counts, _lens(n, case["past"]) if case["past"] else [0] * n


def _refused(case):
    return [case["refused"] and i % 9 == 7 for i in range(case["n"])]


def _seen(p, window, sinks):
    """How many keys a query at position p sees."""
    if window == 0 or window >= p + 1:
        return p + 1
    return window + min(sinks, p + 1 - window)


def _token_bytes(type):
    return D * 2 if type != "int8" else D + D // GROUP * 4


def work(case):
    Hkv, rb, ps = case["Hkv"], _token_bytes(case["type"]), case["ps"]
    if case["kind"] == "maps":
        counts, past = _requests(case)
        pages = sum((p + c - 1) // ps - p // ps + 1 for c, p in zip(counts, past) if c)
        return {"bytes": case["n"] * 16 + pages * 4 + sum(counts) * 12}
    if case["kind"] == "store":
        counts, past = _requests(case)
        new = sum(counts)
        pages = sum((p + c - 1) // ps - p // ps + 1 for c, p in zip(counts, past) if c)
        before = sum(p % ps for c, p in zip(counts, past) if c)    # older keys of the pages touched
        back = new * 2 * (rb + 2 * D) if case["type"] == "int8" else 0
        return {"bytes": Hkv * (new * 2 * (2 * D + rb) + before * rb + pages * (2 * D + 4) + back) + new * 12}
    Hq = Hkv * case["rep"]
    if case["kind"] == "chunk":
        counts, past = _requests(case)
        w, s = case["window"], case["sinks"]
        pairs = sum(_seen(p + i, w, s) for c, p in zip(counts, past) for i in range(c))
        keys = sum(c + p - max(0, p + 1 - w) + min(s, max(0, p + 1 - w)) if w else c + p for c, p in zip(counts, past) if c)
        return {"bytes": sum(counts) * Hq * (4 * D + 4) + keys * Hkv * 2 * rb, "flops": 4 * D * Hq * pairs}
    lens = _lens(case["n"], case["len"], case["ragged"])
    blocks = [-(-max(0, L) // ps) for L in lens]
    read = [min(L, min(b, case["keep"]) * ps) for L, b in zip(lens, blocks)]
    rows = case["n"] * case["each"]
    return {"bytes": sum(blocks) * (Hkv * (2 * D + 4) + 4) + sum(read) * Hkv * 2 * rb + rows * (Hq * (4 * D + 4) + Hkv * 4 * (case["keep"] + 1)),
            "flops": case["each"] * Hq * (4 * D * sum(read) + 2 * D * sum(blocks))}


# --- inputs -----------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if dtype == torch.bfloat16 else dtype).to(dtype)


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _over(x, by):
    """x / by in 32 bits, one rounding."""
    return x / torch.full_like(x, float(by))


def _quantize(x):
    """Per row and 64 channels: codes uint8 and (scale, zero) fp16, x ~ scale * code + zero."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    s, z = _over(hi - lo, 255).half(), lo.half()
    sf, zf = s.float().unsqueeze(-1), z.float().unsqueeze(-1)
    code = torch.where(sf > 0, ((x - zf) / sf).round(), 0.0).clamp(0, 255).to(torch.uint8)
    return code.flatten(-2), torch.stack([s, z], -1)


def _values(codes, meta):
    """What codes and (scale, zero) stand for, in 32 bits."""
    x = codes.float().unflatten(-1, (-1, GROUP))
    return (x * meta[..., :1].float() + meta[..., 1:].float()).flatten(-2)


def _pool(g, n_pages, Hkv, ps, type):
    """Keys (those of a page alike in part, a few channels larger than the rest, as in trained models) and
    values of a whole pool."""
    shape = (1, n_pages, Hkv, ps, D)
    k, v = _normal(g, shape, _FLOAT[type]), _normal(g, shape, _FLOAT[type])
    k.mul_(0.8).add_(_normal(g, (1, n_pages, Hkv, 1, D), _FLOAT[type]), alpha=0.6)
    k[..., 5:D:37] *= 3
    if type != "int8":
        return {"k": k, "v": v, "k_meta": None, "v_meta": None}
    (kc, km), (vc, vm) = _quantize(k), _quantize(v)
    return {"k": kc, "v": vc, "k_meta": km, "v_meta": vm}


def _tables(g, lens, ps, extra_pages):
    """Tables of sequences of these lengths over pages in no order, and the references."""
    max_pages = max(1, -(-max(lens) // ps))
    lens = _int(lens)
    need = (lens + ps - 1) // ps
    total = int(need.sum())
    n_pages = total + extra_pages
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(max_pages, device=DEV)[None, :]
    first = (need.cumsum(0) - need)[:, None]
    table = torch.where(at < need[:, None], perm[(first + at).clamp(max=n_pages - 1)], -1).to(torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[perm[:total].long()] = 1
    return {"table": table.contiguous(), "lens": lens, "refs": refs}, n_pages


def _rows_of(counts, first):
    """(sequence, position) of packed rows, counts[i] of request i from position first[i] on."""
    c = torch.tensor(counts, device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(counts), device=DEV), c)
    at = torch.arange(seq.numel(), device=DEV) - (c.cumsum(0) - c)[seq]
    return seq.to(torch.int32), (at + torch.tensor(first, device=DEV)[seq]).to(torch.int32)


def _filled(pool, ps):
    """How many slots of each page its sequence fills."""
    rows, lens = pool["table"].long(), pool["lens"]
    at = torch.arange(rows.shape[1], device=DEV)
    fill = (lens[:, None] - at * ps).clamp(0, ps)
    got = torch.zeros(pool["refs"].numel(), dtype=torch.long, device=DEV)
    got[rows[rows >= 0]] = fill[rows >= 0].long()
    return got


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    ps, Hkv, dt = case["ps"], case["Hkv"], _FLOAT[case["type"]]
    if case["kind"] == "sparse":
        n, each = case["n"], case["each"]
        lens = _lens(n, case["len"], case["ragged"])
        t, n_pages = _tables(g, lens, ps, 3)
        s["pool"] = _pool(g, n_pages, Hkv, ps, case["type"]) | t
        s["bounds"] = torch.zeros(1, n_pages, Hkv, 2, D, dtype=torch.int8, device=DEV)
        s["scales"] = torch.zeros(1, n_pages, Hkv, dtype=torch.float32, device=DEV)
        fill = _filled(s["pool"], ps)
        step = max(1, (1 << 28) // (Hkv * ps * D))
        for p0 in range(0, n_pages, step):
            page = torch.arange(p0, min(n_pages, p0 + step), device=DEV)
            s["bounds"][0, page], s["scales"][0, page] = _plain_bounds(s["pool"], page, fill[page])
        # the sequence's last tokens, as far as it has any
        s["row_seq"] = torch.arange(n, device=DEV).repeat_interleave(each).to(torch.int32)
        s["row_pos"] = torch.tensor([max(0, L - each + i) for L in lens for i in range(each)], dtype=torch.int32, device=DEV)
        N, Hq = n * each, Hkv * case["rep"]
        s["q"] = _normal(g, (N, Hq, D), dt)
        s["q"][..., 5:D:37] *= 2
        s["sel"] = torch.empty(N, Hkv, case["keep"], dtype=torch.int32, device=DEV)
        s["n_sel"] = torch.empty(N, Hkv, dtype=torch.int32, device=DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(N, Hq, dtype=torch.float32, device=DEV)
        return s
    counts, past = _requests(case)
    t, n_pages = _tables(g, [max(0, p + c) for p, c in zip(past, counts)], ps, 3)
    N = sum(counts)
    s["start"] = _int(past)
    if case["kind"] == "maps":
        no = _refused(case)
        s["start"] = torch.where(torch.tensor(no, device=DEV), -1, s["start"]).contiguous()
        s["counts"] = _int(counts)
        rows = -(-N // case["pad"]) * case["pad"] if case["pad"] else N
        s["pool"] = _pool(g, n_pages, 1, ps, "fp16") | t
        s["row_start"] = torch.empty(case["n"] + 1, dtype=torch.int32, device=DEV)
        s["rows"] = torch.empty(3, rows, dtype=torch.int32, device=DEV)
        s["row_seq"], s["row_pos"], s["row_slot"] = s["rows"]
        return s
    s["pool"] = _pool(g, n_pages, Hkv, ps, case["type"]) | t
    if case["kind"] == "store":
        s["k"], s["v"] = _normal(g, (N, Hkv, D), dt), _normal(g, (N, Hkv, D), dt)
        s["row_seq"], s["row_pos"] = _rows_of(counts, past)
        page = s["pool"]["table"][s["row_seq"].long(), s["row_pos"].long() // ps]
        s["row_slot"] = (page * ps + s["row_pos"] % ps).contiguous()
        s["bounds"] = torch.zeros(1, n_pages, Hkv, 2, D, dtype=torch.int8, device=DEV)
        s["scales"] = torch.zeros(1, n_pages, Hkv, dtype=torch.float32, device=DEV)
        if case["type"] == "int8":
            s["k_out"] = torch.zeros(case["n"], Hkv, max(counts), D, dtype=dt, device=DEV)
            s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    Hq = Hkv * case["rep"]
    s["row_start"] = _int([0] + torch.tensor(counts).cumsum(0).tolist())
    s["q"] = _normal(g, (N, Hq, D), dt)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(N, Hq, dtype=torch.float32, device=DEV)
    return s


# --- plain forms ------------------------------------------------------------------------

def _plain_maps(s):
    pool, ps = s["pool"], s["case"]["ps"]
    counts, rows = s["counts"], s["rows"].shape[1]
    ends = counts.cumsum(0)
    row_start = torch.cat([torch.zeros_like(ends[:1]), ends]).clamp(max=rows).to(torch.int32)
    at = torch.arange(rows, device=DEV)
    req = torch.searchsorted(row_start[1:].contiguous(), at, right=True)
    live = req < counts.numel()
    req = req.clamp(max=counts.numel() - 1)
    live &= s["start"][req] >= 0
    pos = s["start"][req] + at - row_start[req]
    page = pool["table"][req, (pos // ps).clamp(0, pool["table"].shape[1] - 1)]
    slot = torch.where(live & (pos < pool["lens"][req]), page * ps + pos % ps, -1)
    s["row_start"].copy_(row_start)
    s["rows"][0].copy_(torch.where(live, req, -1))
    s["rows"][1].copy_(torch.where(live, pos, -1))
    s["rows"][2].copy_(slot)
    return {"row_start": s["row_start"], "rows": s["rows"]}


def _stored(pool, name, page):
    """Rows of whole pages, [pages][Hkv][ps][D] in 32 bits."""
    x = pool[name][0][page]
    return x.float() if pool["k_meta"] is None else _values(x, pool[name + "_meta"][0][page])


def _plain_bounds(pool, page, fill):
    """Codes int8 [pages][Hkv][2][D] and scales of the keys' channel-wise bounds over each page's filled slots."""
    x = _stored(pool, "k", page)
    there = (torch.arange(x.shape[2], device=DEV) < fill[:, None])[:, None, :, None]
    lo, hi = torch.where(there, x, math.inf).amin(2), torch.where(there, x, -math.inf).amax(2)
    some = (fill > 0)[:, None, None]
    lo, hi = torch.where(some, lo, 0.0), torch.where(some, hi, 0.0)
    scale = _over(torch.maximum(lo.abs(), hi.abs()).amax(-1), 127)
    by = scale.unsqueeze(-1)
    code = torch.stack([(lo / by).floor(), (hi / by).ceil()], 2)
    return torch.where(by.unsqueeze(2) > 0, code, 0.0).clamp(-127, 127).to(torch.int8), scale


def _plain_store(s):
    c, pool = s["case"], s["pool"]
    ps = c["ps"]
    page, r = s["row_slot"].long() // ps, s["row_slot"].long() % ps
    for x in ("k", "v"):
        new = s[x]
        if c["type"] == "int8":
            new, meta = _quantize(new)
            pool[x + "_meta"][0, page, :, r] = meta
        pool[x][0, page, :, r] = new
    touched = torch.zeros_like(pool["refs"], dtype=torch.bool)
    touched[page] = True
    touched = touched.nonzero()[:, 0]
    s["bounds"][0, touched], s["scales"][0, touched] = _plain_bounds(pool, touched, _filled(pool, ps)[touched])
    return _after_store(s, _plain_back(s) if c["type"] == "int8" else None)


def _plain_back(s):
    pool, T = s["pool"], s["k_out"].shape[2]
    at = pool["table"].clamp(min=0).long()
    got = {}
    there = (torch.arange(T, device=DEV) < pool["lens"][:, None])[:, None, :, None]
    for x in ("k", "v"):
        rows = _stored(pool, x, at.flatten()).unflatten(0, at.shape).transpose(1, 2).flatten(2, 3)[:, :, :T]
        got[x] = torch.where(there, rows.half(), s[x + "_out"])
    return got


def _after_store(s, rows):
    """What a store leaves: the pages (or 8-bit pages' rows), and the values of the bounds' codes."""
    return (rows or {"k": s["pool"]["k"], "v": s["pool"]["v"]}) | {"bounds": s["bounds"] * s["scales"][..., None, None]}


def _softmax_rows(s, vis):
    """Weights, their sum and log-sum-exp over the visible keys; zero weights where none is."""
    s = torch.where(vis, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p, l, (m + torch.log(l)).squeeze(-1)


def _plain_chunk(s):
    c, pool, q = s["case"], s["pool"], s["q"]
    Hkv, rep, ps, w, sinks = c["Hkv"], c["rep"], c["ps"], c["window"], c["sinks"]
    counts, past = _requests(c)
    out, lse = torch.zeros_like(q), torch.zeros_like(s["lse"])
    r = 0
    for i, (n, p0) in enumerate(zip(counts, past)):
        if n == 0:
            continue
        L = p0 + n
        page = pool["table"][i, :-(-L // ps)].long()
        k, v = (_stored(pool, x, page).transpose(0, 1).flatten(1, 2)[:, None, :L] for x in ("k", "v"))   # [Hkv][1][L][D]
        p, j = torch.arange(p0, L, device=DEV)[:, None], torch.arange(L, device=DEV)
        vis = j <= p
        if w:
            vis &= (j > p - w) | (j < sinks)
        x = q[r:r + n].float().unflatten(1, (Hkv, rep)).permute(1, 2, 0, 3)                              # [Hkv][rep][n][D]
        e, l, ls = _softmax_rows(x @ k.transpose(2, 3) / math.sqrt(D), vis)
        out[r:r + n] = (e @ v / l).flatten(0, 1).transpose(0, 1).to(q.dtype)
        lse[r:r + n] = ls.flatten(0, 1).transpose(0, 1)
        r += n
    return {"out": out, "lse": lse}


def _plain_select(s):
    """Blocks [N][Hkv][keep] that each row picks, ascending, -1 behind the last one, and how many."""
    c, pool = s["case"], s["pool"]
    Hkv, rep, ps, keep = c["Hkv"], c["rep"], c["ps"], c["keep"]
    q = s["q"].float()
    q_scale = _over(q.abs().amax(-1), 127)
    by = q_scale.unsqueeze(-1)
    code = torch.where(by > 0, (q / by).round(), 0.0).clamp(-127, 127).unflatten(1, (Hkv, rep))           # [N][Hkv][rep][D]
    table = pool["table"][s["row_seq"].long()].clamp(min=0).long()
    b, scale = s["bounds"][0][table].float(), s["scales"][0][table]                                     # [N][blocks][Hkv][2][D]
    b = b.permute(0, 2, 3, 4, 1)
    dot = code.clamp(max=0) @ b[:, :, 0] + code.clamp(min=0) @ b[:, :, 1]                               # whole numbers below 2^24
    score = dot * scale.transpose(1, 2)[:, :, None] * q_scale.view(-1, Hkv, rep, 1)
    score = torch.where(score.isnan(), math.inf, score).amax(2)
    blocks = s["row_pos"][:, None, None] // ps + 1
    j = torch.arange(score.shape[-1], device=DEV)
    there, forced = j < blocks, (j < c["first"]) | (j >= blocks - c["recent"])
    count = torch.minimum(blocks, torch.full_like(blocks, keep))
    # first those that are always read, then by score, then the others; equal ones by their number
    order = torch.sort(torch.where(there & ~forced, score, -math.inf), dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, torch.sort((~(there & forced)).int().expand_as(order).gather(-1, order), dim=-1, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    taken = there & ((blocks <= keep) | (rank < count))
    sel = torch.where(taken, j, score.shape[-1]).sort(-1).values
    sel = torch.cat([sel, torch.full((*sel.shape[:2], keep), score.shape[-1], device=DEV)], -1)[..., :keep]
    return torch.where(sel < score.shape[-1], sel, -1).to(torch.int32), count.expand(-1, Hkv, -1)[..., 0].to(torch.int32)


def _plain_sparse(s):
    c, pool, q = s["case"], s["pool"], s["q"]
    Hkv, rep, ps = c["Hkv"], c["rep"], c["ps"]
    sel, n_sel = _plain_select(s)
    N = q.shape[0]
    slot = (sel.long().unsqueeze(-1) * ps + torch.arange(ps, device=DEV)).flatten(2)                     # [N][Hkv][keep ps]
    vis = (slot >= 0) & (slot <= s["row_pos"].long()[:, None, None])
    slot = torch.where(vis, slot, 0)
    page = pool["table"][s["row_seq"].long()[:, None, None], slot // ps].long()
    head = torch.arange(Hkv, device=DEV)[:, None]
    kv = []
    for x in ("k", "v"):
        rows = pool[x][0][page, head, slot % ps]
        kv.append(rows.float() if pool["k_meta"] is None else _values(rows, pool[x + "_meta"][0][page, head, slot % ps]))
    w = q.float().view(N, Hkv, rep, D) @ kv[0].transpose(2, 3) / math.sqrt(D)
    e, l, lse = _softmax_rows(w, vis[:, :, None])
    return {"sel": sel, "n_sel": n_sel, "out": (e @ kv[1] / l).view(N, -1, D).to(q.dtype), "lse": lse.view(N, -1)}


# --- the framework's calls --------------------------------------------------------------

def _cache(s):
    """The handle a user's program keeps beside its pool."""
    if "cache" not in s:
        from mixed_precision_kv_balancer_gb300.paged import PagedCache
        s["cache"] = PagedCache.over(type=s["case"]["type"], **s["pool"])
    return s["cache"]


def _own(s):
    import mixed_precision_kv_balancer_gb300 as pkg
    lib, c, cache = pkg.load(), s["case"], _cache(s)
    if c["kind"] == "maps":
        lib.mikv_batch_rows(cache, s["counts"], s["row_start"], s["row_seq"], s["row_pos"], s["row_slot"], start=s["start"])
        return {"row_start": s["row_start"], "rows": s["rows"]}
    if c["kind"] == "store":
        lib.mikv_slot_append(cache, 0, s["k"], s["v"], s["row_slot"])
        lib.mikv_page_bounds(cache, 0, s["row_seq"], s["row_pos"], s["bounds"], s["scales"])
        if c["type"] != "int8":
            return _after_store(s, None)
        lib.mikv_paged_gather(cache, 0, s["k_out"], s["v_out"])
        return _after_store(s, {"k": s["k_out"], "v": s["v_out"]})
    if c["kind"] == "chunk":
        if "ws" not in s:
            s["ws"] = cache.chunk_workspace(c["n"], s["q"].shape[0], s["q"].shape[1])
        lib.mikv_chunk_attention(s["q"], cache, 0, s["row_start"], c["window"], c["sinks"], s["out"], s["lse"], start=s["start"],
                                 ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if "ws" not in s:
        s["ws"] = cache.block_workspace(s["q"].shape[0], s["q"].shape[1], c["keep"])
    lib.mikv_block_select(s["q"], cache, 0, s["bounds"], s["scales"], c["first"], c["recent"], s["sel"], s["n_sel"],
                          row_seq=s["row_seq"], row_pos=s["row_pos"], ws=s["ws"])
    lib.mikv_block_attention(s["q"], cache, 0, s["sel"], s["n_sel"], s["out"], s["lse"], row_seq=s["row_seq"], row_pos=s["row_pos"],
                             ws=s["ws"])
    return {"sel": s["sel"], "n_sel": s["n_sel"], "out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"maps": _plain_maps, "store": _plain_store, "chunk": _plain_chunk, "sparse": _plain_sparse}[state["case"]["kind"]](state)


# --- the definition in 64 bits ----------------------------------------------------------

def _slots64(pool, name, seq, at):
    """Stored rows of one sequence's slots `at`, [slots][Hkv][D] in 64 bits."""
    ps = pool["k"].shape[3]
    page = pool["table"][seq].long()[at // ps]
    x = pool[name][0, page, :, at % ps].double()
    if pool["k_meta"] is None:
        return x
    m = pool[name + "_meta"][0, page, :, at % ps].double().repeat_interleave(GROUP, 2)
    return x * m[..., 0] + m[..., 1]


def _attention64(q, k, v, seen):
    """Rows q of one head over its keys under a mask that gives each row's keys."""
    a = (q @ k.T) * D ** -0.5
    a.masked_fill_(~seen, -math.inf)
    lse = torch.logsumexp(a, 1)
    return torch.exp(a - lse.nan_to_num(neginf=0.0)[:, None]) @ v, lse


def _quantized64(x):
    """The value of each row's stored 8-bit codes, scale and zero in fp16."""
    grp = x.double().unflatten(-1, (-1, GROUP))
    z = grp.amin(-1, keepdim=True)
    span = (grp.amax(-1, keepdim=True) - z).float()
    sc = (span / torch.full_like(span, 255.0)).half().double()
    code = torch.where(sc > 0, ((grp - z).float() / sc.float()).round().double(), 0.0).clamp(0, 255)
    return (code * sc + z).view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    pool, ps = s["pool"], case["ps"]
    if case["kind"] == "maps":
        counts, past = _requests(case)
        rows = s["rows"].shape[1]
        starts, seq, pos, slot = [0], [], [], []
        table = pool["table"].tolist()
        for i, (c, p0, no) in enumerate(zip(counts, past, _refused(case))):
            starts.append(starts[-1] + c)
            seq += [-1 if no else i] * c
            pos += [-1 if no else p0 + t for t in range(c)]
            slot += [-1 if no else table[i][(p0 + t) // ps] * ps + (p0 + t) % ps for t in range(c)]
        end = [-1] * (rows - len(seq))
        return {"row_start": _int(starts), "rows": _int([seq + end, pos + end, slot + end])}
    if case["kind"] == "store":
        counts, past = _requests(case)
        k, v = (pool[x].double() if case["type"] != "int8" else None for x in ("k", "v"))
        bounds = torch.zeros(s["bounds"].shape, dtype=torch.float64, device=DEV)
        back = {x: s[x + "_out"].double() for x in ("k", "v")} if case["type"] == "int8" else None
        r = 0
        for i, (c, p0) in enumerate(zip(counts, past)):
            if c == 0:
                continue
            new = {x: (_quantized64(s[x][r:r + c]) if case["type"] == "int8" else s[x][r:r + c].double()) for x in ("k", "v")}
            r += c
            if back:
                for x in ("k", "v"):
                    back[x][i, :, :c] = new[x].transpose(0, 1)
            else:
                at = p0 + torch.arange(c, device=DEV)
                page = pool["table"][i].long()[at // ps]
                k[0, page, :, at % ps], v[0, page, :, at % ps] = new["k"], new["v"]
            keys = torch.cat([_slots64(pool, "k", i, torch.arange(p0 // ps * ps, p0, device=DEV)), new["k"]]).float()
            for b in range(p0 // ps, (p0 + c - 1) // ps + 1):
                mine = keys[max(0, b * ps - p0 // ps * ps):(b + 1) * ps - p0 // ps * ps]
                lo, hi = mine.amin(0), mine.amax(0)
                top = torch.maximum(lo.abs(), hi.abs()).amax(-1, keepdim=True)
                scale = top / torch.full_like(top, 127.0)
                code = torch.stack([torch.floor(lo / scale), torch.ceil(hi / scale)], 1).clamp(-127, 127).nan_to_num(0.0)
                bounds[0, int(pool["table"][i, b])] = code.double() * scale.double().unsqueeze(-1)
        return (back or {"k": k, "v": v}) | {"bounds": bounds}
    Hkv, rep = case["Hkv"], case["rep"]
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    if case["kind"] == "chunk":
        w, sinks = case["window"], case["sinks"]
        r = 0
        for i, (c, p0) in enumerate(zip(*_requests(case))):
            j = torch.arange(p0 + c, device=DEV)
            if c:
                k, v = _slots64(pool, "k", i, j), _slots64(pool, "v", i, j)
            step = max(1, (1 << 26) // (p0 + c + 1))
            for a in range(0, c, step):
                m = min(step, c - a)
                p = p0 + a + torch.arange(m, device=DEV)[:, None]
                seen = (p >= j) if w == 0 else (p >= j) & ((p - j < w) | (j < sinks))
                for h in range(Hkv * rep):
                    out[r + a:r + a + m, h], lse[r + a:r + a + m, h] = _attention64(
                        s["q"][r + a:r + a + m, h].double(), k[:, h // rep], v[:, h // rep], seen)
            r += c
        return {"out": out, "lse": lse}
    # sparse: one row and key head at a time
    keep, first, recent = case["keep"], case["first"], case["recent"]
    sel, n_sel = torch.full(s["sel"].shape, -1, dtype=torch.int32), torch.zeros(s["n_sel"].shape, dtype=torch.int32)
    if s["q"].shape[0] * Hkv > 1024:
        return None
    for i, (seq, p) in enumerate(zip(s["row_seq"].tolist(), s["row_pos"].tolist())):
        nb = p // ps + 1
        page = pool["table"][seq, :nb].long()
        for h in range(Hkv):
            q = s["q"][i, h * rep:(h + 1) * rep]
            if nb <= keep:
                got = list(range(nb))
            else:
                top = q.float().abs().amax(-1, keepdim=True)
                qs = top / torch.full_like(top, 127.0)
                code = torch.where(qs > 0, torch.round(q.float() / qs), 0.0).clamp(-127, 127).double()
                lo, hi = s["bounds"][0, page, h, 0].double(), s["bounds"][0, page, h, 1].double()
                dot = torch.where(code > 0, code, 0.0) @ hi.T + torch.where(code < 0, code, 0.0) @ lo.T
                # two roundings to 32 bits, as the score is defined
                score = ((dot * s["scales"][0, page, h].double()).float().double() * qs.double()).float().amax(0)
                always = sorted(set(range(first)) | set(range(nb - recent, nb)))
                score[always] = -math.inf
                best = torch.argsort(score, descending=True, stable=True)[:keep - len(always)]
                got = sorted(always + best.tolist())
            n_sel[i, h] = len(got)
            sel[i, h, :len(got)] = torch.tensor(got, dtype=torch.int32)
            b = torch.tensor(got, device=DEV)
            j = (b[:, None] * ps + torch.arange(ps, device=DEV)).flatten()
            j = j[j <= p]
            k, v = _slots64(pool, "k", seq, j)[:, h], _slots64(pool, "v", seq, j)[:, h]
            at = slice(h * rep, (h + 1) * rep)
            out[i, at], lse[i, at] = _attention64(q.double(), k, v, torch.ones(rep, j.numel(), dtype=torch.bool, device=DEV))
    return {"sel": sel.to(DEV), "n_sel": n_sel.to(DEV), "out": out, "lse": lse}
