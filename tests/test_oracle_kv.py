"""Pins of the cache oracle: e4m3's table against its published limits, quantised rows
worked by hand, and the attention against a closed form."""
import math

import numpy as np
import pytest

from oracle import kv_cache as okv


def test_e4m3_table():
    v = okv.e4m3_values()
    assert v[0x7E] == 448.0 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x38] == 1.0
    assert math.isnan(v[0x7F]) and math.isnan(v[0xFF]) and v[0xFE] == -448.0 and len(set(v[:0x7F])) == 0x7F


@pytest.mark.parametrize("row,codes,scale", [
    ([448.0, 1.0, -3.0, 0.0], [448.0, 1.0, -3.0, 0.0], 1.0),
    ([450.0, 34.0, 38.0, 2.0 ** -10], [224.0, 16.0, 20.0, 0.0], 2.0),  # 225 -> 224, 17 -> 16, 19 -> 20
    ([0.875, 0.25, -0.0625, 0.0], [448.0, 128.0, -32.0, 0.0], 2.0 ** -9),
    ([0.0, 0.0, 0.0, 0.0], [0.0, 0.0, 0.0, 0.0], 2.0 ** -126),
    ([2.0 ** -133, 0.0, 0.0, 0.0], [2.0 ** -7, 0.0, 0.0, 0.0], 2.0 ** -126),
])
def test_e4m3_rows(row, codes, scale):
    c, s = okv.quantise(np.array(row), okv.E4M3)
    assert s == scale and np.array_equal(c, codes)


def test_int8_rows():
    c, s = okv.quantise(np.array([127.0, 63.5, 0.5, -126.5]), okv.INT8)
    assert s == 1.0 and np.array_equal(c, [127, 64, 0, -126])
    c, s = okv.quantise(np.array([-2.0, 1.0, 0.0, 0.015625]), okv.INT8)
    assert abs(s * 127 - 2.0) <= 2.0 ** -22 and c[0] == -127 and c[2] == 0 and c[3] == 1


@pytest.mark.parametrize("dtype", [okv.E4M3, okv.INT8])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_that_are_not_finite(dtype, bad):
    c, s = okv.quantise(np.array([[1.0, bad], [1.0, 0.5]]), dtype)
    assert math.isnan(s[0]) and not c[0].any() and s[1] > 0 and c[1].all()


def test_quantisation_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 128)).astype(np.float32).astype(np.float64)
    for dtype, step in ((okv.E4M3, None), (okv.INT8, 1.0)):
        c, s = okv.quantise(x, dtype)
        y = x / s[:, None]
        half = 0.5 * (step if step else 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3))
        assert np.all(np.abs(c - y) <= half * (1 + 1e-6)) and np.max(np.abs(c)) <= (448 if dtype == okv.E4M3 else 127)


def test_attention_closed_form():
    # equal scores: the mean of v; lse = s + ln n
    k, v = np.ones((5, 4)), np.arange(20.0).reshape(5, 4)
    o, l, _ = okv.attend(np.full(4, 0.25), k, v, 2.0)
    assert np.allclose(o, v.mean(0)) and math.isclose(l, 2.0 + math.log(5))
    o, l, _ = okv.attend(np.ones(4), k[:0], v[:0], 1.0)
    assert not o.any() and l == -math.inf
