"""ctypes binding of libmikv.so: the C ABI calls under the same names, taking torch tensors.

Argument marshalling only: every computation runs in the library's CUDA kernels.
There is no fallback; if the library is missing or a call fails, this raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmikv.so")

MIKV_PREFILL, MIKV_DECODE = 0, 1
MIKV_H2O, MIKV_CRITICALKV, MIKV_DEMOTE = 0, 1, 2
MIKV_TIER_HI, MIKV_TIER_LO, MIKV_TIER_DEMOTE = 0, 1, 2
MIKV_KEYS_PER_TOKEN, MIKV_KEYS_PER_CHANNEL = 0, 1
MIKV_PAGES_FP16, MIKV_PAGES_BF16, MIKV_PAGES_INT8 = 0, 1, 2

EXPORTS = (
    "mikv_balance_prefill", "mikv_balance_workspace_bytes", "mikv_balance_prefill_noalloc",
    "mikv_score_update", "mikv_score_workspace_bytes",
    "mikv_select", "mikv_select_workspace_bytes",
    "mikv_quantize_append",
    "mikv_decode_attention", "mikv_decode_workspace_bytes",
    "mikv_decode_step", "mikv_decode_step_workspace_bytes",
    "mikv_output_perturbation", "mikv_output_perturbation_workspace_bytes",
    "mikv_topk_attention", "mikv_topk_attention_workspace_bytes",
    "mikv_channel_quantize",
    "mikv_page_reserve", "mikv_page_fork", "mikv_page_free", "mikv_page_copy", "mikv_page_compact",
    "mikv_page_workspace_bytes", "mikv_paged_append", "mikv_paged_gather",
    "mikv_paged_attention", "mikv_paged_attention_workspace_bytes",
    "mikv_window_attention", "mikv_window_attention_workspace_bytes",
    "mikv_set_attention_events", "mikv_wait_status", "mikv_wait_probe", "mikv_last_error",
)


class MikvError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


class mikv_cache(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("Hq", ctypes.c_int32), ("D", ctypes.c_int32),
        ("hi_bits", ctypes.c_int32), ("lo_bits", ctypes.c_int32),
        ("cap_hi", ctypes.c_int32), ("cap_lo", ctypes.c_int32),
        ("n_hi", ctypes.c_int32), ("n_lo", ctypes.c_int32),
        ("k_hi", ctypes.c_void_p), ("v_hi", ctypes.c_void_p),
        ("k_hi_meta", ctypes.c_void_p), ("v_hi_meta", ctypes.c_void_p),
        ("k_lo", ctypes.c_void_p), ("v_lo", ctypes.c_void_p),
        ("k_lo_meta", ctypes.c_void_p), ("v_lo_meta", ctypes.c_void_p),
        ("pos_hi", ctypes.c_void_p), ("pos_lo", ctypes.c_void_p),
        ("balancer", ctypes.c_void_p), ("scores", ctypes.c_void_p),
        ("key_mode", ctypes.c_int32), ("k_pend", ctypes.c_void_p), ("v_pend", ctypes.c_void_p),
    ]


class mikv_pages(ctypes.Structure):
    _fields_ = [
        ("layers", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("type", ctypes.c_int32),
        ("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_meta", ctypes.c_void_p), ("v_meta", ctypes.c_void_p),
        ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
    ]


class mikv_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_t", ctypes.c_int64)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libmikv.so (built in-tree by build()); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() or "
                           "python -m mixed_precision_kv_balancer_gb300.build")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    CP, GP, RP = ctypes.POINTER(mikv_cache), ctypes.POINTER(mikv_pages), ctypes.POINTER(mikv_rows)
    sig = {
        "mikv_balance_prefill": (I, [P, P, I, I, I, I, I, P, P, S, P]),
        "mikv_balance_workspace_bytes": (S, [I, I, I]),
        "mikv_balance_prefill_noalloc": (I, [P, P, I, I, I, I, I, P, P]),
        "mikv_score_update": (I, [I, P, P, I, P, P, CP, P, P, P, S, P]),
        "mikv_score_workspace_bytes": (S, [I, I, I]),
        "mikv_select": (I, [I, CP, I, I, I, F, P, P, P, P, I, P, P, P, P, P, S, P]),
        "mikv_select_workspace_bytes": (S, [I, I, I, I, I, I]),
        "mikv_quantize_append": (I, [I, P, P, I, P, I, I, P, CP, P]),
        "mikv_decode_attention": (I, [P, CP, P, P, P, P, S, P]),
        "mikv_decode_workspace_bytes": (S, [CP]),
        "mikv_decode_step": (I, [P, P, P, I, I, I, I, CP, P, P, P, S, P]),
        "mikv_decode_step_workspace_bytes": (S, [CP]),
        "mikv_output_perturbation": (I, [P, P, P, I, I, I, I, P, P, P, S, P]),
        "mikv_output_perturbation_workspace_bytes": (S, [I, I, I]),
        "mikv_topk_attention": (I, [P, CP, I, P, P, P, P, S, P]),
        "mikv_topk_attention_workspace_bytes": (S, [CP, I]),
        "mikv_channel_quantize": (I, [P, I, I, I, I, P, P, P]),
        "mikv_page_reserve": (I, [GP, P, P, I, P, P, S, P]),
        "mikv_page_fork": (I, [GP, P, P, I, P, P, S, P]),
        "mikv_page_free": (I, [GP, P, I, P, P]),
        "mikv_page_copy": (I, [GP, P, P, I, P, P]),
        "mikv_page_compact": (I, [GP, P, P, P, I, I, P, P, S, P]),
        "mikv_page_workspace_bytes": (S, [GP, I]),
        "mikv_paged_append": (I, [GP, I, RP, RP, I, I, P, P, P, P]),
        "mikv_paged_gather": (I, [GP, I, P, I, I, RP, RP, P]),
        "mikv_paged_attention": (I, [P, GP, I, P, I, I, I, I, P, P, P, S, P]),
        "mikv_paged_attention_workspace_bytes": (S, [GP, I, I, I, I]),
        "mikv_window_attention": (I, [RP, RP, RP, I, I, I, I, I, I, I, P, P, I, I, RP, P, P, S, P]),
        "mikv_window_attention_workspace_bytes": (S, [I, I, I, I, I, I, I]),
        "mikv_set_attention_events": (I, [P, P]),
        "mikv_wait_status": (I, [ctypes.POINTER(ctypes.c_uint), I]),
        "mikv_wait_probe": (I, [ctypes.c_int64, I, P]),
        "mikv_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


def _ptr(t):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors"
    return t.data_ptr()


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(name: str, rc: int):
    if rc != 0:
        raise MikvError(name, rc, load().mikv_last_error().decode())


def _ws(nbytes: int, device, ws):
    if ws is not None:
        return ws, ws.numel() * ws.element_size()
    if nbytes == 0:
        return None, 0
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, nbytes


# --- the C ABI calls -----------------------------------------------------------------

def mikv_balance_prefill(q, k, b_out, ws=None, stream=None):
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    lib = load()
    w, nb = _ws(lib.mikv_balance_workspace_bytes(B, Hkv, D), q.device, ws)
    _check("mikv_balance_prefill", lib.mikv_balance_prefill(
        _ptr(q), _ptr(k), B, Hq, Hkv, T, D, _ptr(b_out), _ptr(w), nb, _stream(stream)))


def mikv_balance_prefill_noalloc(q, k, b_out, stream=None):
    """Balancer without a workspace: scratch is the library's static device array."""
    B, Hq, T, D = q.shape
    _check("mikv_balance_prefill_noalloc", load().mikv_balance_prefill_noalloc(
        _ptr(q), _ptr(k), B, Hq, k.shape[1], T, D, _ptr(b_out), _stream(stream)))


def mikv_score_update(mode, cache, q=None, k=None, T=0, hi_logits=None, lse=None,
                      scores_full=None, scores_head=None, ws=None, stream=None):
    lib = load()
    c = cache.struct if hasattr(cache, "struct") else cache
    w, nb = None, 0
    if mode == MIKV_PREFILL:
        dev = q.device
        w, nb = _ws(lib.mikv_score_workspace_bytes(c.B, c.Hq, T), dev, ws)
    _check("mikv_score_update", lib.mikv_score_update(
        mode, _ptr(q), _ptr(k), T, _ptr(hi_logits), _ptr(lse), ctypes.byref(c),
        _ptr(scores_full), _ptr(scores_head), _ptr(w), nb, _stream(stream)))


def mikv_select(policy, cache, L, budget_pct, window, alpha=0.5, scores=None, scores_head=None,
                v=None, w_o=None, hidden=0, vwo_norm=None, keep_pos=None, evict_pos=None,
                keep_scores=None, ws=None, stream=None):
    lib = load()
    c = cache.struct if hasattr(cache, "struct") else cache
    dev = (scores if scores is not None else evict_pos).device
    w, nb = _ws(lib.mikv_select_workspace_bytes(policy, c.B, c.Hkv, c.Hq, L, hidden), dev, ws)
    _check("mikv_select", lib.mikv_select(
        policy, ctypes.byref(c), L, budget_pct, window, float(alpha), _ptr(scores),
        _ptr(scores_head), _ptr(v), _ptr(w_o), hidden, _ptr(vwo_norm), _ptr(keep_pos),
        _ptr(evict_pos), _ptr(keep_scores), _ptr(w), nb, _stream(stream)))


def mikv_quantize_append(tier, cache, k, v, src_pos, n_tokens, pos_base=0, src_scores=None,
                         stream=None):
    lib = load()
    c = cache.struct if hasattr(cache, "struct") else cache
    src_len = 0 if k is None else k.shape[2]
    _check("mikv_quantize_append", lib.mikv_quantize_append(
        tier, _ptr(k), _ptr(v), src_len, _ptr(src_pos), n_tokens, pos_base, _ptr(src_scores),
        ctypes.byref(c), _stream(stream)))


def mikv_decode_attention(q, cache, out, lse, hi_logits=None, ws=None, stream=None):
    lib = load()
    c = cache.struct if hasattr(cache, "struct") else cache
    w, nb = _ws(lib.mikv_decode_workspace_bytes(ctypes.byref(c)), q.device, ws)
    _check("mikv_decode_attention", lib.mikv_decode_attention(
        _ptr(q), ctypes.byref(c), _ptr(out), _ptr(lse), _ptr(hi_logits), _ptr(w), nb,
        _stream(stream)))


def mikv_decode_step(q, k_new, v_new, pos, budget_pct, window, policy, cache, out, lse, ws=None,
                     stream=None):
    lib = load()
    c = cache.struct if hasattr(cache, "struct") else cache
    w, nb = _ws(lib.mikv_decode_step_workspace_bytes(ctypes.byref(c)), q.device, ws)
    _check("mikv_decode_step", lib.mikv_decode_step(
        _ptr(q), _ptr(k_new), _ptr(v_new), pos, budget_pct, window, policy, ctypes.byref(c),
        _ptr(out), _ptr(lse), _ptr(w), nb, _stream(stream)))


def mikv_output_perturbation(o, o_hat=None, w_o_t=None, y=None, pert=None, ws=None, stream=None):
    """o, o_hat fp32 [B][Hq][D]; w_o_t fp16 [hidden][Hq*D] (W_O transposed, nn.Linear layout);
    y fp32 [B][hidden] and / or pert fp32 [B][Hq] are written."""
    lib = load()
    B, Hq, D = o.shape
    hidden = 0 if w_o_t is None else w_o_t.shape[0]
    w, nb = (None, 0) if w_o_t is None else _ws(lib.mikv_output_perturbation_workspace_bytes(B, Hq, hidden),
                                                o.device, ws)
    _check("mikv_output_perturbation", lib.mikv_output_perturbation(
        _ptr(o), _ptr(o_hat), _ptr(w_o_t), B, Hq, D, hidden, _ptr(y), _ptr(pert), _ptr(w), nb,
        _stream(stream)))


def mikv_topk_attention(q, cache, budget_pct, out, lse=None, keep_idx=None, ws=None, stream=None):
    """Post-attention top-k over a full FP16 cache (all tokens in the important tier)."""
    lib = load()
    c = cache.struct if hasattr(cache, "struct") else cache
    w, nb = _ws(lib.mikv_topk_attention_workspace_bytes(ctypes.byref(c), budget_pct), q.device, ws)
    _check("mikv_topk_attention", lib.mikv_topk_attention(
        _ptr(q), ctypes.byref(c), budget_pct, _ptr(out), _ptr(lse), _ptr(keep_idx), _ptr(w), nb,
        _stream(stream)))


def mikv_channel_quantize(k, bits, codes, meta, stream=None):
    """k fp16 [units, n, D]; codes uint8 [units, n, D*bits/8]; meta fp16 [units, n//64, D, 2]."""
    units, n, D = k.shape
    _check("mikv_channel_quantize", load().mikv_channel_quantize(
        _ptr(k), units, n, D, bits, _ptr(codes), _ptr(meta), _stream(stream)))


# --- the paged cache and windowed attention --------------------------------------------

_PAGE_DTYPE = {MIKV_PAGES_FP16: torch.float16, MIKV_PAGES_BF16: torch.bfloat16, MIKV_PAGES_INT8: torch.float16}


def _launch(dev, stream, call, *args):
    """call(*args, stream) on CUDA device `dev` (its number), where the tensors are: on that device's
    current stream unless one is given, with the device made current for the launch.  The
    status is checked under the call's name."""
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        rc = call(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, st)
    if rc != 0:
        raise MikvError(call.__name__, rc, load().mikv_last_error().decode())


def _need(t, name, dtype, shape, dev):
    """Pointer of a contiguous tensor of this dtype and shape on device `dev`; None for None."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _rows(t, name, dtype, shape, dev):
    """mikv_rows of a [B][H][T][D] tensor whose last dimension is contiguous."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        sb, sh, st, sd = t.stride()
        if sd == 1 or shape[3] <= 1:
            # a dimension of one element is never stepped along: its stride may be anything
            return mikv_rows(t.data_ptr(), sb if shape[0] > 1 else 0, sh if shape[1] > 1 else 0, st if shape[2] > 1 else 0)
    raise ValueError(f"{name}: expected a {dtype} tensor of shape {tuple(shape)} on cuda:{dev} with a contiguous "
                     f"last dimension, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _ws_given(ws, dev):
    """(pointer, bytes, tensor to keep) of a workspace that the caller keeps."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on cuda:{dev}, got one on {ws.device}")
    return ws.data_ptr(), ws.nbytes, ws


def _ws_new(n, dev, stream):
    """The same of a new one of n bytes, which belongs to the stream of the call: freed on return,
    it is not handed out again before that stream has come past the call."""
    if n == 0:
        return None, 0, None
    if stream is None:
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        with torch.cuda.stream(stream):
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    return ws.data_ptr(), n, ws


def _page_ws(pages, n, ws, stream):
    if ws is not None:
        return _ws_given(ws, pages.index)
    return _ws_new(load().mikv_page_workspace_bytes(pages.ref, n), pages.index, stream)


def mikv_page_reserve(pages, seqs, add, start, ws=None, stream=None):
    """Room for add int32 [n] more tokens behind sequences seqs (int32 [n], None: 0 .. n - 1);
    start int32 [n] receives each one's first new slot, or -1 where it was refused."""
    lib, dev, n = load(), pages.index, add.shape[0]
    w, nb, _keep = _page_ws(pages, n, ws, stream)
    _launch(dev, stream, lib.mikv_page_reserve, pages.ref, _need(seqs, "seqs", torch.int32, (n,), dev),
            _need(add, "add", torch.int32, (n,), dev), n, _need(start, "start", torch.int32, (n,), dev), w, nb)


def mikv_page_fork(pages, parent, child, ok, ws=None, stream=None):
    """child[i] becomes a copy of parent[i] (int32 [n] each); ok int32 [n] receives 1, or 0 where refused."""
    lib, dev, n = load(), pages.index, parent.shape[0]
    w, nb, _keep = _page_ws(pages, n, ws, stream)
    _launch(dev, stream, lib.mikv_page_fork, pages.ref, _need(parent, "parent", torch.int32, (n,), dev),
            _need(child, "child", torch.int32, (n,), dev), n, _need(ok, "ok", torch.int32, (n,), dev), w, nb)


def mikv_page_free(pages, seqs, ok, stream=None):
    """Sequences seqs (int32 [n], None: 0 .. n - 1) give their pages back; ok int32 [n]."""
    lib, dev, n = load(), pages.index, ok.shape[0]
    _launch(dev, stream, lib.mikv_page_free, pages.ref, _need(seqs, "seqs", torch.int32, (n,), dev), n,
            _need(ok, "ok", torch.int32, (n,), dev))


def mikv_page_copy(pages, src, dst, ok, stream=None):
    """Page dst[i] takes what page src[i] holds, in all layers (int32 [n] each); ok int32 [n]."""
    lib, dev, n = load(), pages.index, src.shape[0]
    _launch(dev, stream, lib.mikv_page_copy, pages.ref, _need(src, "src", torch.int32, (n,), dev),
            _need(dst, "dst", torch.int32, (n,), dev), n, _need(ok, "ok", torch.int32, (n,), dev))


def mikv_page_compact(pages, seqs, keep_pos, keep_n, ok, ws=None, stream=None):
    """Sequence seqs[i] keeps keep_n[i] slots per key head: keep_pos int32 [layers][n][Hkv][max_keep],
    keep_n and ok int32 [n]."""
    lib, dev, n, s = load(), pages.index, keep_n.shape[0], pages.struct
    w, nb, _keep = _page_ws(pages, n, ws, stream)
    most = keep_pos.shape[-1]
    _launch(dev, stream, lib.mikv_page_compact, pages.ref, _need(seqs, "seqs", torch.int32, (n,), dev),
            _need(keep_pos, "keep_pos", torch.int32, (s.layers, n, s.Hkv, most), dev),
            _need(keep_n, "keep_n", torch.int32, (n,), dev), n, most, _need(ok, "ok", torch.int32, (n,), dev), w, nb)


def mikv_paged_append(pages, layer, k, v, seqs=None, start=None, counts=None, stream=None):
    """Rows k, v [n][Hkv][T][D] (strided; fp16, bf16 for BF16 pages) into one layer: counts int32 [n]
    tokens each (None: T), from slot start int32 [n] (None: each sequence's last slots)."""
    lib, dev, s = load(), pages.index, pages.struct
    n, _, T, _ = k.shape
    shape, dt = (n, s.Hkv, T, s.D), _PAGE_DTYPE[s.type]
    _launch(dev, stream, lib.mikv_paged_append, pages.ref, layer, _rows(k, "k", dt, shape, dev),
            _rows(v, "v", dt, shape, dev), n, T, _need(seqs, "seqs", torch.int32, (n,), dev),
            _need(start, "start", torch.int32, (n,), dev), _need(counts, "counts", torch.int32, (n,), dev))


def mikv_paged_gather(pages, layer, k_out, v_out, seqs=None, stream=None):
    """The first T slots of each sequence of one layer as rows k_out, v_out [n][Hkv][T][D] (strided)."""
    lib, dev, s = load(), pages.index, pages.struct
    n, _, T, _ = k_out.shape
    shape, dt = (n, s.Hkv, T, s.D), _PAGE_DTYPE[s.type]
    _launch(dev, stream, lib.mikv_paged_gather, pages.ref, layer, _need(seqs, "seqs", torch.int32, (n,), dev), n, T,
            _rows(k_out, "k_out", dt, shape, dev), _rows(v_out, "v_out", dt, shape, dev))


def mikv_paged_attention(q, pages, layer, window, sinks, out, lse=None, seqs=None, ws=None, stream=None):
    """One new token per sequence: q, out [n][Hq][D] fp16 (bf16 for BF16 pages), lse fp32 [n][Hq]."""
    lib, dev, s = load(), pages.index, pages.struct
    n, Hq, _ = q.shape
    shape, dt = (n, Hq, s.D), _PAGE_DTYPE[s.type]
    w, nb, _keep = _ws_given(ws, dev) if ws is not None else _ws_new(
        lib.mikv_paged_attention_workspace_bytes(pages.ref, n, Hq, window, sinks), dev, stream)
    _launch(dev, stream, lib.mikv_paged_attention, _need(q, "q", dt, shape, dev), pages.ref, layer,
            _need(seqs, "seqs", torch.int32, (n,), dev), n, Hq, window, sinks, _need(out, "out", dt, shape, dev),
            _need(lse, "lse", torch.float32, (n, Hq), dev), w, nb)


@functools.lru_cache(maxsize=1024)
def _window_workspace_bytes(*dims):   # a function of the dimensions alone
    return load().mikv_window_attention_workspace_bytes(*dims)


def mikv_window_attention(q, k, v, window, sinks, out, lse=None, q_lens=None, k_lens=None, ws=None, stream=None):
    """A prompt's or a chunk's attention: q, out [B][Hq][Tq][D], k, v [B][Hkv][Tk][D] (strided; all fp16 or
    all bf16), lse fp32 [B][Hq][Tq], q_lens, k_lens int32 [B] (None: Tq, Tk)."""
    lib, dev, dt = load(), q.get_device(), q.dtype
    B, Hq, Tq, D = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    if dev < 0 or dt not in (torch.float16, torch.bfloat16):
        raise ValueError(f"q: expected fp16 or bf16 on a CUDA device, got {dt} on {q.device}")
    qs, ks = (B, Hq, Tq, D), (B, Hkv, Tk, D)
    w, nb, _keep = _ws_given(ws, dev) if ws is not None else _ws_new(
        _window_workspace_bytes(B, Hq, Hkv, Tq, Tk, window, sinks), dev, stream)
    _launch(dev, stream, lib.mikv_window_attention, _rows(q, "q", dt, qs, dev), _rows(k, "k", dt, ks, dev),
            _rows(v, "v", dt, ks, dev), B, Hq, Hkv, Tq, Tk, D,
            MIKV_PAGES_BF16 if dt is torch.bfloat16 else MIKV_PAGES_FP16, _need(q_lens, "q_lens", torch.int32, (B,), dev),
            _need(k_lens, "k_lens", torch.int32, (B,), dev), window, sinks, _rows(out, "out", dt, qs, dev),
            _need(lse, "lse", torch.float32, (B, Hq, Tq), dev), w, nb)


def mikv_set_attention_events(begin=None, end=None):
    """Record two torch.cuda.Event objects around the split-K attention launch of every
    following decode call of this thread (None, None clears).  Each event must have been
    recorded once through torch, so that its CUDA event exists."""
    lib = load()
    h = lambda e: None if e is None else e.cuda_event
    _check("mikv_set_attention_events", lib.mikv_set_attention_events(h(begin), h(end)))


WAIT_BITS = {1: "K3 pass 1 (row log-sum-exp)", 2: "K3 pass 2 (column sums)", 4: "K6 (V.W_O norms)",
             8: "K9 (output perturbation)", 16: "mikv_wait_probe", 32: "mikv_window_attention",
             64: "a page outside the pool", 128: "an append into a shared page"}


def mikv_wait_status(clear=True) -> int:
    """OR of the wait-status bits the tensor-core kernels set since the last clear (0 when no
    bounded mbarrier wait gave up).  Synchronous: call after the work has completed."""
    v = ctypes.c_uint(0)
    _check("mikv_wait_status", load().mikv_wait_status(ctypes.byref(v), int(bool(clear))))
    return v.value


def mikv_wait_probe(polls, arrive, stream=None):
    """One bounded mbarrier wait that gives up (sets wait-status bit 16) unless `arrive`."""
    _check("mikv_wait_probe", load().mikv_wait_probe(int(polls), int(bool(arrive)), _stream(stream)))
