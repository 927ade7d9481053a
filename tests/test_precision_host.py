"""The bounds of the precision tests, against emulations: fp32 statistics and weights of two 16-bit parts
keep them, weights of one part and sums of rounded weights do not."""
import numpy as np
import pytest

import precision_cases as pc

SIZES = [2, 4, 16, 18, 40, 64, 200]


@pytest.mark.parametrize("type", ["fp16", "bf16"])
@pytest.mark.parametrize("n", SIZES)
def test_bounds_tell_weights_and_sums_apart(type, n):
    q, k, v = pc.rows(n, 32, 2, n)
    assert ((k @ np.ones(128)) * 8 == np.rint((k @ np.ones(128)) * 8)).all() and (v.sum(1) == 0).all()
    want, wl = pc.softmax64(q, k, v)
    two = pc.HALF_STEP[type] ** 2
    good, gl = pc.emulated(q, k, v, type, 2, False)
    assert pc.out_error(good, want, pc.HALF_STEP[type], two, n) < 1 and pc.lse_error(gl, wl, n) < 1
    one, ol = pc.emulated(q, k, v, type, 1, True)
    assert pc.out_error(one, want, pc.HALF_STEP[type], two, n) > 2
    assert pc.lse_error(ol, wl, n) > 1
    assert pc.out_error(pc.emulated(q, k, v, type, 1, False)[0], want, pc.HALF_STEP[type], two, n) > 2
    # one rounding, where it is what the operator says, keeps the bound that counts it
    assert pc.out_error(one, want, pc.HALF_STEP[type], pc.HALF_STEP[type], n) < 1


def test_bounds_tell_the_weights_types_apart():
    """fp16 outputs from weights rounded to bf16; over more keys their errors average out below fp16's bound."""
    for n in SIZES[:5]:
        q, k, v = pc.rows(n, 32, 2, n)
        want, _ = pc.softmax64(q, k, v)
        coarse, _ = pc.emulated(q, k, v, "bf16", 1, False)
        assert pc.out_error(coarse, want, pc.HALF_STEP["fp16"], pc.HALF_STEP["fp16"], n) > 1


@pytest.mark.parametrize("n", [2, 18, 64, 200])
def test_bounds_tell_codes_of_one_16_bit_number(n):
    """8-bit keys that enter the products as one fp16 number miss the lse's bound, as two they keep it; values that do miss the
    outputs' where all weights are alike."""
    q, k, v = pc.codes_beyond_16_bits(n, 8, 2, n)
    kv, vv = pc.code_values(*k), pc.code_values(*v)
    assert np.abs(kv).max() <= 16 and (np.abs(q) @ np.abs(kv[0]).T).max() <= 4
    want, wl = pc.softmax64(q, kv, vv)
    share = 2.0 ** -20
    one = pc.to16(kv, "fp16").astype(np.float64)
    two = one + pc.to16(kv - one, "fp16")
    for keys, keeps in ((one, False), (two, True)):
        err = np.abs(pc.emulated(q, keys, vv, "fp16", 1, False)[1] - wl) - share
        assert (pc.lse_error(wl + err, wl, n) < 1) == keeps
    # no query: all weights are alike, and outputs are 2^-13
    want, _ = pc.softmax64(0 * q, kv, vv)
    assert (want == 2.0 ** -13).all()
    one = pc.to16(vv, "fp16").astype(np.float64)
    assert pc.out_error(pc.softmax64(0 * q, kv, one)[0], want, 2.0 ** -11, 2.0 ** -22, n) > 1
    two = one + pc.to16(vv - one, "fp16")
    assert pc.out_error(pc.softmax64(0 * q, kv, two)[0], want, 2.0 ** -11, 2.0 ** -22, n) < 1
