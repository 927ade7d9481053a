"""Measured cases of the paged-cache and windowed-attention operators.

Each case runs either in plain form (elementary torch operations, 32 bits) or, where ``own`` is
true, through the package's calls.  Kinds:

  attend   one new token per sequence over a paged cache (mikv_paged_attention)
  prompt   a prompt, or a chunk of one, under a sliding window with sinks (mikv_window_attention)
  chunk    a chunk's keys and values into the pages, and the sequences so far read back as rows
           (mikv_paged_append, mikv_paged_gather)
  pages    children released, forked anew from their parents, cut down to their kept tokens and
           given room for new ones, and some pages copied to pages held aside (mikv_page_free,
           mikv_page_fork, mikv_page_compact, mikv_page_reserve, mikv_page_copy)
"""
import math

import torch

own = False

D = 128
GROUP = 64
DEV = "cuda"
_FLOAT = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.float16}


# --- cases ------------------------------------------------------------------------------

def _attend(name, n, len, Hkv, rep, ps, type, window=0, sinks=0, ragged=True):
    c = {"kind": "attend", "n": n, "len": len, "Hkv": Hkv, "rep": rep, "ps": ps, "type": type,
         "window": window, "sinks": sinks, "ragged": ragged}
    return c if name is None else {"name": name, **c}


def _prompt(name, B, Tq, past, Hkv, rep, type, window=0, sinks=0, ragged=False, layout="bhtd"):
    c = {"kind": "prompt", "B": B, "Tq": Tq, "past": past, "Hkv": Hkv, "rep": rep, "type": type,
         "window": window, "sinks": sinks, "ragged": ragged, "layout": layout}
    return c if name is None else {"name": name, **c}


def _chunk(name, n, T, past, Hkv, ps, type, ragged=True):
    c = {"kind": "chunk", "n": n, "T": T, "past": past, "Hkv": Hkv, "ps": ps, "type": type, "ragged": ragged}
    return c if name is None else {"name": name, **c}


def _pages(name, parents, children, len, keep_pct, add, copies, layers, Hkv, ps, type):
    c = {"kind": "pages", "parents": parents, "children": children, "len": len, "keep_pct": keep_pct, "add": add,
         "copies": copies, "layers": layers, "Hkv": Hkv, "ps": ps, "type": type}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # the first tokens of one short conversation: nothing but latency
        _attend("attend_short", 1, 77, 8, 4, 16, "bf16", ragged=False),
        # an ordinary serving batch, sequences of all lengths up to 4096, small pages
        _attend("attend_ragged", 24, 4096, 8, 4, 16, "fp16"),
        # the full-depth workload's batch and length
        _attend("attend_full", 64, 8192, 8, 4, 64, "fp16", ragged=False),
        # long 8-bit contexts of a model whose layer sees a window and the first few tokens
        _attend("attend_window_int8", 48, 65536, 4, 8, 32, "int8", window=4096, sinks=4),
        # a few short prompts of different lengths in one padded batch
        _prompt("prompt_short", 4, 131, 0, 8, 4, "fp16", ragged=True),
        # a whole prompt of the full-depth workload's length, causal
        _prompt("prompt_full", 1, 8192, 0, 8, 4, "bf16"),
        # a long prompt under a window with sinks, as its projection lays it out
        _prompt("prompt_window", 2, 16384, 0, 2, 2, "bf16", window=1024, sinks=4, layout="bthd"),
        # the next chunk of some half-read prompts
        _prompt("prompt_chunk", 4, 500, 7680, 8, 5, "fp16", ragged=True),
        # a decode step's keys and values stored 16-bit, short sequences read back
        _chunk("chunk_token", 16, 1, 200, 8, 16, "bf16", ragged=False),
        # a chunk of each prompt stored 8-bit, and the sequences so far read back
        _chunk("chunk_int8", 8, 512, 4096, 8, 16, "int8"),
        # one conversation branched, in one layer: nothing but latency
        _pages("pages_small", 1, 1, 300, 50, 1, 1, 1, 8, 16, "fp16"),
        # two branches of each of a few long prompts, evicted to a 20 % budget in all layers
        _pages("pages_budget", 3, 2, 8190, 20, 3, 16, 16, 8, 16, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["attend"] * 4 + ["prompt"] * 4 + ["chunk"] * 2 + ["pages"] * 2)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    ps = rng.choice([1, 8, 16, 20, 32, 64, 100, 128])
    any_type = rng.choice(["fp16", "bf16", "int8"])
    window = rng.choice([0, 0, 1]) * _log(rng, 1, 8192)
    sinks = rng.choice([0, 1]) * _log(rng, 1, 128)
    if kind == "attend":
        n = _log(rng, 1, 128)
        top = min(65536, 64 * 8192 * 8 // (n * Hkv))
        return _attend(None, n, _log(rng, 1, top), Hkv, rep, ps, any_type, window, sinks, rng.random() < 0.7)
    if kind == "prompt":
        B = _log(rng, 1, 8)
        most = 32 * 8192 * 8192 // (B * Hkv * rep)
        Tq = _log(rng, 1, min(16384, math.isqrt(most)))
        room = min(16384, (most // Tq - Tq) // 2)           # the past's pairs count whole, the chunk's own half
        past = _log(rng, 1, room) if room > 0 and rng.random() < 0.5 else 0
        return _prompt(None, B, Tq, past, Hkv, rep, rng.choice(["fp16", "bf16"]), window, sinks,
                       rng.random() < 0.5, rng.choice(["bhtd", "bthd"]))
    if kind == "chunk":
        return _chunk(None, _log(rng, 1, 16), _log(rng, 1, 1024), _log(rng, 1, 4096), Hkv, ps, any_type,
                      rng.random() < 0.5)
    return _pages(None, _log(rng, 1, 3), _log(rng, 1, 3), _log(rng, 1, 4096), rng.choice([10, 20, 25, 40, 90]),
                  _log(rng, 1, 64), _log(rng, 1, 16), _log(rng, 1, 16), Hkv, ps, rng.choice(["fp16", "bf16"]))


def _lens(case, n, top, ragged):
    """n lengths up to `top`: all equal, or spread over 1 .. top with the first at the top."""
    if not ragged:
        return [top] * n
    return [max(1, int(top * (1.0 - (0.6180339887 * i) % 1.0))) for i in range(n)]


def _prompt_lens(case):
    """(q_len, k_len) of each row; a ragged batch's last row is empty."""
    B, Tq, past = case["B"], case["Tq"], case["past"]
    ql = _lens(case, B, Tq, case["ragged"])
    kl = [q + p for q, p in zip(ql, _lens(case, B, past, case["ragged"]) if past else [0] * B)]
    if case["ragged"] and B > 2:
        ql[-1] = kl[-1] = 0
    return ql, kl


def _pages_lens(case):
    """The parents' lengths, and how many tokens their children keep."""
    L = [max(1, case["len"] - 5 * i) for i in range(case["parents"])]
    return L, max(1, min(L) * case["keep_pct"] // 100)


def _seen(p, window, sinks):
    """How many keys a query at position p sees."""
    if p < 0:
        return 0
    if window == 0 or window >= p + 1:
        return p + 1
    return window + min(sinks, p + 1 - window)


def _token_bytes(type):
    return D * 2 if type != "int8" else D + D // GROUP * 4


def work(case):
    Hkv, rb = case["Hkv"], _token_bytes(case["type"])
    if case["kind"] == "attend":
        n, Hq = case["n"], case["Hkv"] * case["rep"]
        vis = sum(_seen(L - 1, case["window"], case["sinks"]) for L in _lens(case, n, case["len"], case["ragged"]))
        return {"bytes": vis * Hkv * 2 * rb + n * Hq * (2 * D * 2 + 4) + vis * 4 // case["ps"],
                "flops": 4 * D * Hq * vis}
    if case["kind"] == "prompt":
        Hq = case["Hkv"] * case["rep"]
        ql, kl = _prompt_lens(case)
        pairs = sum(_seen(k - q + i, case["window"], case["sinks"]) for q, k in zip(ql, kl) for i in range(q))
        return {"bytes": sum(ql) * Hq * (2 * D * 2 + 4) + sum(kl) * Hkv * 2 * D * 2, "flops": 4 * D * Hq * pairs}
    if case["kind"] == "chunk":
        new = sum(_lens(case, case["n"], case["T"], case["ragged"]))
        total = new + case["n"] * case["past"]
        return {"bytes": Hkv * 2 * (new * (D * 2 + rb) + total * (D * 2 + rb))}
    L, keep = _pages_lens(case)
    c, ps = case["children"], case["ps"]
    rows = c * sum(x % ps + keep for x in L) + case["copies"] * ps
    entries = c * sum(-(-x // ps) + -(-(keep + case["add"]) // ps) for x in L)   # of tables, and their references
    return {"bytes": rows * case["layers"] * Hkv * 2 * rb * 2 + c * len(L) * case["layers"] * Hkv * keep * 4 + entries * 12}


# --- inputs -----------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if dtype == torch.bfloat16 else dtype).to(dtype)


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _quantize(x):
    """Per row and 64 channels: codes uint8 and (scale, zero) fp16, x ~ scale * code + zero."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    s, z = ((hi - lo) / torch.full_like(lo, 255.0)).half(), lo.half()
    sf, zf = s.float().unsqueeze(-1), z.float().unsqueeze(-1)
    code = torch.where(sf > 0, ((x - zf) / sf).round(), 0.0).clamp(0, 255).to(torch.uint8)
    return code.flatten(-2), torch.stack([s, z], -1)


def _values(codes, meta):
    """What codes and (scale, zero) stand for, in 32 bits."""
    x = codes.float().unflatten(-1, (-1, GROUP))
    return (x * meta[..., :1].float() + meta[..., 1:].float()).flatten(-2)


def _pool(g, layers, n_pages, Hkv, ps, type):
    """Keys (a few channels larger than the rest, as in trained models) and values of a whole pool."""
    shape = (layers, n_pages, Hkv, ps, D)
    k, v = _normal(g, shape, _FLOAT[type]), _normal(g, shape, _FLOAT[type])
    k[..., 5:D:37] *= 3
    if type != "int8":
        return {"k": k, "v": v, "k_meta": None, "v_meta": None}
    (kc, km), (vc, vm) = _quantize(k), _quantize(v)
    return {"k": kc, "v": vc, "k_meta": km, "v_meta": vm}


def _tables(g, lens, ps, max_pages, extra_seqs, extra_pages):
    """Tables of sequences of these lengths over pages in no order, and the references."""
    lens = _int(lens)
    n = lens.numel()
    need = (lens + ps - 1) // ps
    total = int(need.sum())
    n_pages = total + extra_pages
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(max_pages, device=DEV)[None, :]
    first = (need.cumsum(0) - need)[:, None]
    table = torch.where(at < need[:, None], perm[(first + at).clamp(max=n_pages - 1)], -1).to(torch.int32)
    table = torch.cat([table, torch.full((extra_seqs, max_pages), -1, dtype=torch.int32, device=DEV)])
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[perm[:total].long()] = 1
    lens = torch.cat([lens, torch.zeros(extra_seqs, dtype=torch.int32, device=DEV)])
    return {"table": table.contiguous(), "lens": lens, "refs": refs}, n_pages


def prepare(case, seed):
    g = _gen(seed)
    Hkv = case["Hkv"]
    dt = _FLOAT[case["type"]]
    s = {"case": case}
    if case["kind"] == "prompt":
        B, Tq, Hq = case["B"], case["Tq"], Hkv * case["rep"]
        Tk = Tq + case["past"]
        ql, kl = _prompt_lens(case)

        def rows(H, T):
            return (_normal(g, (B, H, T, D), dt) if case["layout"] == "bhtd"
                    else _normal(g, (B, T, H, D), dt).transpose(1, 2))

        s |= {"q": rows(Hq, Tq), "k": rows(Hkv, Tk), "v": rows(Hkv, Tk)}
        s["k"][..., 5:D:37] *= 3
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, Hq, Tq, dtype=torch.float32, device=DEV)
        s["q_lens"], s["k_lens"] = (_int(ql), _int(kl)) if case["ragged"] else (None, None)
        return s
    ps = case["ps"]
    if case["kind"] == "attend":
        n, Hq = case["n"], Hkv * case["rep"]
        t, n_pages = _tables(g, _lens(case, n, case["len"], case["ragged"]), ps, -(-case["len"] // ps), 0, 3)
        s |= {"pool": _pool(g, 1, n_pages, Hkv, ps, case["type"]) | t, "q": _normal(g, (n, Hq, D), dt)}
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, Hq, dtype=torch.float32, device=DEV)
        return s
    if case["kind"] == "chunk":
        n, T, past = case["n"], case["T"], case["past"]
        counts = _lens(case, n, T, case["ragged"])
        t, n_pages = _tables(g, [past + c for c in counts], ps, -(-(past + T) // ps), 0, 3)
        s |= {"pool": _pool(g, 1, n_pages, Hkv, ps, case["type"]) | t}
        s |= {"k": _normal(g, (n, Hkv, T, D), dt), "v": _normal(g, (n, Hkv, T, D), dt), "counts": _int(counts),
              "start": torch.full((n,), past, dtype=torch.int32, device=DEV)}
        s["k_out"] = torch.zeros(n, Hkv, past + T, D, dtype=dt, device=DEV)
        s["v_out"] = torch.zeros_like(s["k_out"])
        return s
    L, keep = _pages_lens(case)
    m, n = len(L), len(L) * case["children"]
    most = -(-(case["len"] + case["add"]) // ps)
    t, n_pages = _tables(g, L, ps, most, n, n * (-(-keep // ps) + -(-case["add"] // ps) + 2) + case["copies"] + 3)
    s["parent"] = torch.arange(m, dtype=torch.int32, device=DEV).repeat_interleave(case["children"])
    s["child"] = torch.arange(m, m + n, dtype=torch.int32, device=DEV)
    score = torch.rand(case["layers"], n, Hkv, min(L), generator=g, device=DEV)
    s["keep_pos"] = score.topk(keep, dim=-1).indices.sort(-1).values.to(torch.int32)
    s["keep_n"] = torch.full((n,), keep, dtype=torch.int32, device=DEV)
    s["add"] = torch.full((n,), case["add"], dtype=torch.int32, device=DEV)
    held = (t["refs"] == 0).nonzero()[:case["copies"], 0]
    t["refs"][held] = 1
    s["dst"] = held.to(torch.int32)
    s["src"] = t["table"][0, torch.arange(case["copies"], device=DEV) % -(-L[0] // ps)].contiguous()
    s["pool"] = _pool(g, case["layers"], n_pages, Hkv, ps, case["type"]) | t
    s["start"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    s["ok"] = torch.zeros(4, max(n, case["copies"]), dtype=torch.int32, device=DEV)
    return s


# --- plain forms ------------------------------------------------------------------------

def _visible(pos, k_len, S, window, sinks):
    """Which of S keys a query at `pos` (any shape) sees."""
    j = torch.arange(S, device=DEV)
    p = pos.unsqueeze(-1)
    seen = (j <= p) & (j < k_len.unsqueeze(-1))
    return seen & ((j > p - window) | (j < sinks)) if window else seen


def _softmax_rows(s, vis):
    """Weights, their sum and log-sum-exp over the visible keys; zero weights where none is."""
    s = torch.where(vis, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p, l, (m + torch.log(l)).squeeze(-1)


def _sequence_rows(pool, name, layer, table):
    """Rows of whole sequences, [n][Hkv][max_pages * ps][D] in 32 bits."""
    at = table.clamp(min=0).long()
    x = pool[name][layer][at]                                       # [n][max_pages][Hkv][ps][row]
    x = x.float() if pool["k_meta"] is None else _values(x, pool[name + "_meta"][layer][at])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    c, pool, q = s["case"], s["pool"], s["q"]
    n, Hkv = c["n"], c["Hkv"]
    lens = pool["lens"][:n]
    k, v = (_sequence_rows(pool, x, 0, pool["table"][:n]) for x in ("k", "v"))
    vis = _visible(lens - 1, lens, k.shape[2], c["window"], c["sinks"])[:, None, None, :]
    w = q.float().view(n, Hkv, c["rep"], D) @ k.transpose(2, 3) / math.sqrt(D)
    p, l, lse = _softmax_rows(w, vis)
    o = p @ torch.where(vis.transpose(2, 3), v, 0.0) / torch.where(l > 0, l, 1.0)
    return {"out": o.view(n, -1, D).to(q.dtype), "lse": lse.view(n, -1)}


def _plain_prompt(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    B, Hq, Tq, _ = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    ql = torch.full((B,), Tq, device=DEV) if s["q_lens"] is None else s["q_lens"]
    kl = torch.full((B,), Tk, device=DEV) if s["k_lens"] is None else s["k_lens"]
    i = torch.arange(Tq, device=DEV)
    vis = _visible((kl - ql)[:, None] + i, kl[:, None], Tk, c["window"], c["sinks"])[:, None, None]
    there = torch.arange(Tk, device=DEV) < kl[:, None]
    w = q.float().unflatten(1, (Hkv, -1)) @ k.float().transpose(2, 3)[:, :, None] / math.sqrt(D)
    p, l, lse = _softmax_rows(w, vis)
    del w
    vz = torch.where(there[:, None, :, None], v.float(), 0.0)
    o = (p @ vz[:, :, None] / torch.where(l > 0, l, 1.0)).flatten(1, 2)
    row = (i < ql[:, None])[:, None]
    return {"out": torch.where(row.unsqueeze(-1), o.to(q.dtype), s["out"]),
            "lse": torch.where(row, lse.flatten(1, 2), s["lse"])}


def _plain_chunk(s):
    c, pool = s["case"], s["pool"]
    n, T, ps = c["n"], c["T"], c["ps"]
    t = torch.arange(T, device=DEV)
    live = t < s["counts"][:, None]
    row, tok = live.nonzero(as_tuple=True)
    slot = (s["start"][row] + tok).long()
    page = pool["table"][row, slot // ps].long()
    got = {}
    for x in ("k", "v"):
        new = s[x][row, :, tok]                                     # [tokens][Hkv][D]
        if c["type"] == "int8":
            new, meta = _quantize(new)
            pool[x + "_meta"][0, page, :, slot % ps] = meta
        pool[x][0, page, :, slot % ps] = new
        rows = _sequence_rows(pool, x, 0, pool["table"][:n])[:, :, :s["k_out"].shape[2]]
        j = torch.arange(rows.shape[2], device=DEV)
        there = (j < pool["lens"][:n, None])[:, None, :, None]
        got[x] = torch.where(there, rows.to(s["k_out"].dtype), s[x + "_out"])
    return got


def _used(pool, seqs, ps):
    """Pages of the sequences and which entries of their table rows are theirs."""
    at = torch.arange(pool["table"].shape[1], device=DEV)
    rows = pool["table"][seqs.long()].long()
    return rows, at < ((pool["lens"][seqs.long()] + ps - 1) // ps)[:, None], at


def _plain_free(pool, seqs, ps):
    rows, mine, _ = _used(pool, seqs, ps)
    pool["refs"].index_add_(0, rows.clamp(min=0).flatten(), -mine.int().flatten())
    pool["table"][seqs.long()] = -1
    pool["lens"][seqs.long()] = 0


def _free_order(pool):
    """All pages, the free ones first, each part in ascending order."""
    return torch.argsort((pool["refs"] != 0).int(), stable=True)


def _plain_fork(pool, parent, child, ps):
    rows, mine, at = _used(pool, parent, ps)
    L = pool["lens"][parent.long()]
    full, rest = L // ps, L % ps
    shared = at < full[:, None]
    part = rest > 0
    fresh = _free_order(pool)[(part.int().cumsum(0) - 1).clamp(min=0)]
    old = rows.gather(1, full.clamp(max=rows.shape[1] - 1).long()[:, None])[:, 0]
    pool["refs"].index_add_(0, rows.clamp(min=0).flatten(), shared.int().flatten())
    pool["refs"].index_add_(0, fresh, part.int())
    new = torch.where(shared, rows, -1)
    new = torch.where((at == full[:, None]) & part[:, None], fresh[:, None], new)
    pool["table"][child.long()] = new.int()
    pool["lens"][child.long()] = L
    dst, src = fresh[part], old[part]
    take = (torch.arange(ps, device=DEV) < rest[part][:, None])[None, :, None, :]
    for x in (pool["k"], pool["v"]):
        x[:, dst] = torch.where(take.unsqueeze(-1), x[:, src], x[:, dst])


def _plain_reserve(pool, seqs, add, ps):
    L = pool["lens"][seqs.long()]
    have, want = (L + ps - 1) // ps, (L + add + ps - 1) // ps
    at = torch.arange(pool["table"].shape[1], device=DEV)
    new = (at >= have[:, None]) & (at < want[:, None])
    need = want - have
    rank = ((need.cumsum(0) - need)[:, None] + at - have[:, None]).clamp(0, pool["refs"].numel() - 1)
    fresh = _free_order(pool)[rank.long()]
    pool["table"][seqs.long()] = torch.where(new, fresh, pool["table"][seqs.long()]).int()
    pool["refs"].index_add_(0, fresh.flatten(), new.int().flatten())
    pool["lens"][seqs.long()] = L + add
    return L


def _plain_compact(pool, seqs, keep_pos, keep_n, ps):
    rows, mine, at = _used(pool, seqs, ps)
    keep = keep_pos.shape[-1]
    need = (keep_n + ps - 1) // ps
    rank = ((need.cumsum(0) - need)[:, None] + at).clamp(max=pool["refs"].numel() - 1)
    new = at < need[:, None]
    fresh = _free_order(pool)[rank.long()]
    layers, n, Hkv, _ = keep_pos.shape
    li = torch.arange(layers, device=DEV)[:, None, None, None]
    hi = torch.arange(Hkv, device=DEV)[:, None]
    ni = torch.arange(n, device=DEV)[:, None, None]
    kp = keep_pos.long()
    j = torch.arange(keep, device=DEV)
    for x in (pool["k"], pool["v"]):
        x[li, fresh[ni, j // ps], hi, j % ps] = x[li, rows[ni, kp // ps], hi, kp % ps]
    pool["refs"].index_add_(0, rows.clamp(min=0).flatten(), -mine.int().flatten())
    pool["refs"].index_add_(0, fresh.flatten(), new.int().flatten())
    pool["table"][seqs.long()] = torch.where(new, fresh, -1).int()
    pool["lens"][seqs.long()] = keep_n


def _stored(s):
    return {x: s[x] for x in ("ok", "start")} | {x: s["pool"][x] for x in ("k", "v", "table", "lens", "refs")}


def _plain_pages(s):
    pool, ps = s["pool"], s["case"]["ps"]
    n, copies = s["child"].numel(), s["src"].numel()
    _plain_free(pool, s["child"], ps)
    _plain_fork(pool, s["parent"], s["child"], ps)
    _plain_compact(pool, s["child"], s["keep_pos"], s["keep_n"], ps)
    s["start"].copy_(_plain_reserve(pool, s["child"], s["add"], ps))
    for x in (pool["k"], pool["v"]):
        x[:, s["dst"].long()] = x[:, s["src"].long()]
    s["ok"][:3, :n] = 1
    s["ok"][3, :copies] = 1
    return _stored(s)


# --- the framework's calls --------------------------------------------------------------

def _calls():
    import mixed_precision_kv_balancer_gb300 as pkg
    return pkg.load()


def _cache(s):
    """The handle a user's program keeps beside its pool."""
    if "cache" not in s:
        from mixed_precision_kv_balancer_gb300.paged import PagedCache
        s["cache"] = PagedCache.over(type=s["case"]["type"], **s["pool"])
    return s["cache"]


def _own(s):
    c, lib = s["case"], _calls()
    if c["kind"] == "prompt":
        lib.mikv_window_attention(s["q"], s["k"], s["v"], c["window"], c["sinks"], s["out"], s["lse"],
                                  q_lens=s["q_lens"], k_lens=s["k_lens"])
        return {"out": s["out"], "lse": s["lse"]}
    cache = _cache(s)
    if c["kind"] == "attend":
        if "ws" not in s:
            s["ws"] = cache.attention_workspace(c["n"], c["Hkv"] * c["rep"])
        lib.mikv_paged_attention(s["q"], cache, 0, c["window"], c["sinks"], s["out"], s["lse"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["kind"] == "chunk":
        lib.mikv_paged_append(cache, 0, s["k"], s["v"], start=s["start"], counts=s["counts"])
        lib.mikv_paged_gather(cache, 0, s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    n, ok = s["child"].numel(), s["ok"]
    if "ws" not in s:
        s["ws"] = cache.page_workspace(n)
    lib.mikv_page_free(cache, s["child"], ok[0, :n])
    lib.mikv_page_fork(cache, s["parent"], s["child"], ok[1, :n], ws=s["ws"])
    lib.mikv_page_compact(cache, s["child"], s["keep_pos"], s["keep_n"], ok[2, :n], ws=s["ws"])
    lib.mikv_page_reserve(cache, s["child"], s["add"], s["start"], ws=s["ws"])
    lib.mikv_page_copy(cache, s["src"], s["dst"], ok[3, :s["src"].numel()])
    return _stored(s)


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "prompt": _plain_prompt,
            "chunk": _plain_chunk}.get(state["case"]["kind"], _plain_pages)(state)


# --- the definition in 64 bits ----------------------------------------------------------

def _attention64(q, k, v, first, window, sinks):
    """Rows q (positions first, first + 1, ...) of one key head over its keys, row by row of the mask."""
    outs, lses = [], []
    step = max(1, (1 << 26) // max(1, k.shape[0]))
    j = torch.arange(k.shape[0], device=q.device)
    for r in range(0, q.shape[0], step):
        p = first[r:r + step, None]
        ok = (p >= j) if window == 0 else (p >= j) & ((p - j < window) | (j < sinks))
        a = (q[r:r + step] @ k.T) * D ** -0.5
        a[~ok] = -math.inf
        lse = torch.logsumexp(a, 1) if k.shape[0] else torch.full((a.shape[0],), -math.inf, dtype=a.dtype, device=a.device)
        w = torch.exp(a - lse.nan_to_num(neginf=0.0)[:, None])
        outs.append(w @ v)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


def _slots64(pool, name, layer, seq, type):
    """One sequence's stored rows in slot order, [len][Hkv][D] in 64 bits."""
    L, ps = int(pool["lens"][seq]), pool["k"].shape[3]
    j = torch.arange(L, device=DEV)
    page = pool["table"][seq].long()[j // ps]
    x = pool[name][layer, page, :, j % ps].double()
    if type != "int8":
        return x
    m = pool[name + "_meta"][layer, page, :, j % ps].double().repeat_interleave(GROUP, 2)
    return x * m[..., 0] + m[..., 1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attend":
        n, rep = case["n"], case["rep"]
        q = s["q"].double()
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=q.dtype, device=DEV)
        for i in range(n):
            k, v = (_slots64(s["pool"], x, 0, i, case["type"]) for x in ("k", "v"))
            last = torch.full((rep,), k.shape[0] - 1, device=DEV)
            for h in range(case["Hkv"]):
                at = slice(h * rep, h * rep + rep)
                out[i, at], lse[i, at] = _attention64(q[i, at], k[:, h], v[:, h], last, case["window"], case["sinks"])
        return {"out": out, "lse": lse}
    if case["kind"] == "prompt":
        rep = case["rep"]
        out, lse = s["out"].double(), s["lse"].double()
        for b, (ql, kl) in enumerate(zip(*_prompt_lens(case))):
            pos = kl - ql + torch.arange(ql, device=DEV)
            for h in range(out.shape[1]):
                if ql:
                    out[b, h, :ql], lse[b, h, :ql] = _attention64(
                        s["q"][b, h, :ql].double(), s["k"][b, h // rep, :kl].double(),
                        s["v"][b, h // rep, :kl].double(), pos, case["window"], case["sinks"])
        return {"out": out, "lse": lse}
    if case["kind"] == "chunk":
        got = {}
        for x in ("k", "v"):
            rows = s[x + "_out"].double()
            for i in range(case["n"]):
                past, c = case["past"], int(s["counts"][i])
                rows[i, :, :past + c] = _slots64(s["pool"], x, 0, i, case["type"]).transpose(0, 1)
                new = s[x][i, :, :c].double()
                if case["type"] == "int8":       # the stored code's value, scale and zero in fp16
                    grp = new.view(*new.shape[:2], -1, GROUP)
                    z = grp.amin(-1, keepdim=True)
                    span = (grp.amax(-1, keepdim=True) - z).float()
                    sc = (span / torch.full_like(span, 255.0)).half().double()
                    code = torch.where(sc > 0, ((grp - z).float() / sc.float()).round().double(), 0.0).clamp(0, 255)
                    new = (code * sc + z).view_as(new)
                rows[i, :, past:past + c] = new
            got[x] = rows
        return got
    # pages: one page at a time, by the book
    pool, ps = s["pool"], case["ps"]
    table, lens, refs = (pool[x].tolist() for x in ("table", "lens", "refs"))
    k, v = pool["k"].double(), pool["v"].double()
    start = []                                       # of the new tokens

    def take():
        page = refs.index(0)
        refs[page] = 1
        return page

    def pages(seq):
        return -(-lens[seq] // ps)

    moves = []                                       # (parent's pages, child's pages) before the children are cut down
    for a, c in zip(s["parent"].tolist(), s["child"].tolist()):
        lens[c] = lens[a]
        for i in range(pages(a)):
            if (i + 1) * ps <= lens[a]:
                table[c][i] = table[a][i]
                refs[table[a][i]] += 1
            else:
                table[c][i] = take()
                moves.append((table[a][i], table[c][i], lens[a] % ps))
    for a, c, rest in moves:
        for x in (k, v):
            x[:, c, :, :rest] = x[:, a, :, :rest]
    old = [table[c][:pages(c)] for c in s["child"].tolist()]
    new = [[take() for _ in range(-(-keep // ps))] for keep in s["keep_n"].tolist()]
    for i, c in enumerate(s["child"].tolist()):
        keep = int(s["keep_n"][i])
        was, now = torch.tensor(old[i], device=DEV), torch.tensor(new[i], device=DEV)
        j = torch.arange(keep, device=DEV)
        for layer in range(case["layers"]):
            for h in range(case["Hkv"]):
                at = s["keep_pos"][layer, i, h, :keep].long()
                for x in (k, v):
                    x[layer, now[j // ps], h, j % ps] = x[layer, was[at // ps], h, at % ps]
        for page in old[i]:
            refs[page] -= 1
        table[c] = new[i] + [-1] * (len(table[c]) - len(new[i]))
        lens[c] = keep
    for c, add in zip(s["child"].tolist(), s["add"].tolist()):
        start.append(lens[c])
        for i in range(pages(c), -(-(lens[c] + add) // ps)):
            table[c][i] = take()
        lens[c] = start[-1] + add
    for a, c in zip(s["src"].tolist(), s["dst"].tolist()):
        for x in (k, v):
            x[:, c] = x[:, a]
    ok = s["ok"].clone()
    ok[:3, :len(start)] = 1
    ok[3, :s["src"].numel()] = 1
    return {"ok": ok, "start": _int(start), "k": k, "v": v, "table": _int(table), "lens": _int(lens), "refs": _int(refs)}
