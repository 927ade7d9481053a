"""Inputs on which the outputs' own rounding does not hide how exact softmax weights and sums are, and
the bounds that attention with fp32 statistics keeps on them.

Queries are multiples of 1/16 up to 1/8, keys multiples of 1/8 up to 1/4: every score is a multiple of
2^-7 below 4, exact in fp32 in any order of its sum, and all logits lie within 0.36 of zero.  Values are
1 and -1, as many of each in a channel, so an output is what the weights differ by: small beside the
weights' sum of |weight * value|, which is 1.
"""
import numpy as np
import torch

HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "int8": 2.0 ** -11}    # of the outputs' type


def rows(n_keys, heads, key_heads, seed):
    """q [heads][128], k and v [key_heads][n_keys][128] float64; n_keys even."""
    rng = np.random.RandomState(seed)
    q = rng.randint(-2, 3, size=(heads, 128)) / 16.0
    k = rng.randint(-2, 3, size=(key_heads, n_keys, 128)) / 8.0
    v = np.ones((key_heads, n_keys, 128))
    v[:, n_keys // 2:] = -1
    order = rng.rand(key_heads, n_keys, 128).argsort(1)
    return q, k, np.take_along_axis(v, order, 1)


# Errors of a weight besides its rounding to 16 bits, relative to it: the scale log2(e) / sqrt(128) is a
# product of two rounded numbers and multiplies the score (4 roundings of 2^-24, times a logit of 0.52 in
# log2 units), a factor up to 2^15 enters as a sum with a number below 16 (two roundings of 2^-21 of a
# log2, times ln 2), exp2 is within 2^-22: together below 2^-20.  Sums over n keys in fp32, in products
# that may cut what they add at 2^-23 of it: 16 keys a product, both parts of the weights, and a few
# joins: below (n / 8 + 4) 2^-22 of sum w |v|.
def fp32_share(n_keys):
    return 2.0 ** -20 + (n_keys / 8 + 4) * 2.0 ** -22


def out_error(got, want, half_step, weights, n_keys):
    """The largest share of its bound that an output is off by; sum w |v| is 1."""
    s = weights + fp32_share(n_keys)
    return float(np.max(np.abs(got - want) / (half_step * (np.abs(want) + s) + s + 2.0 ** -25)))


# log2 of a sum below 2^24 is off by a step of 2^-19 at most and added to numbers below 32 (three
# roundings of 2^-20), times ln 2; the sum by its weights' and additions' share.
def lse_error(got, want, n_keys):
    return float(np.max(np.abs(got - want) / (2.0 ** -18 + fp32_share(n_keys) + 2.0 ** -22 * np.abs(want))))


def softmax64(q, k, v):
    """out [heads][128] and lse [heads] in 64 bits, rep query heads a key head in order."""
    rep = q.shape[0] // k.shape[0]
    out, lse = np.zeros(q.shape), np.zeros(q.shape[0])
    for h in range(q.shape[0]):
        l = k[h // rep] @ q[h] / np.sqrt(128.0)
        w = np.exp(l - l.max())
        out[h], lse[h] = w @ v[h // rep] / w.sum(), l.max() + np.log(w.sum())
    return out, lse


def to16(x, type):
    dt = torch.bfloat16 if type == "bf16" else torch.float16
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dt).float().numpy()


def emulated(q, k, v, type, parts, rounded_sum):
    """The same in fp32 with weights of `parts` 16-bit parts; their sum of the weights before that, or
    (`rounded_sum`) after.  Outputs are rounded to 16 bits."""
    rep = q.shape[0] // k.shape[0]
    factor = np.float32(1 if type == "bf16" else 2.0 ** 15)
    out, lse = np.zeros(q.shape), np.zeros(q.shape[0])
    for h in range(q.shape[0]):
        s = (k[h // rep] @ q[h]).astype(np.float32) * np.float32(1.4426950408889634 / np.sqrt(128.0))
        p = np.exp2(s - s.max()) * factor
        w = to16(p, type)
        if parts == 2:
            w = w + to16(p - w, type)
        total = (w if rounded_sum else p).sum(dtype=np.float32)
        out[h] = to16((w @ v[h // rep].astype(np.float32)) / total, type)
        lse[h] = (s.max() + np.log2(total / factor)) * np.float32(np.log(2.0))
    return out, lse


def codes_beyond_16_bits(n_keys, heads, key_heads, seed):
    """q [heads][128], and 8-bit keys and values (codes [key_heads][n_keys][128] and (scale, zero) [...][2][2]) whose values no 16-bit
    number holds.  Queries are 1/16 or -1/16 in four channels, the keys of a head all alike (roundings of many would average
    out), spread over -16 .. 16 by channels: sum |q k| is at most 4.  Values are 1 + 2^-12 or -1 in turn."""
    rng = np.random.RandomState(seed)
    q = np.zeros((heads, 128))
    for h in range(heads):
        q[h, rng.permutation(128)[:4]] = rng.choice([-1, 1], 4) / 16.0
    k = rng.randint(0, 256, (key_heads, 1, 128)).astype(np.uint8).repeat(n_keys, 1)
    km = np.empty((key_heads, n_keys, 2, 2), np.float16)
    km[..., 0], km[..., 1] = rng.uniform(0.1, 0.125, (key_heads, 1, 2)), -16
    v = np.zeros(k.shape, np.uint8)
    vm = np.zeros_like(km)
    v[:, ::2], vm[:, ::2, :, 0], vm[:, ::2, :, 1], vm[:, 1::2, :, 1] = 1, 2.0 ** -12, 1, -1
    return q, (k, km), (v, vm)


def code_values(codes, meta):
    """What 8-bit rows stand for, in 64 bits."""
    x = codes.reshape(*codes.shape[:-1], 2, 64).astype(np.float64)
    return (x * meta[..., :1].astype(np.float64) + meta[..., 1:].astype(np.float64)).reshape(codes.shape)
