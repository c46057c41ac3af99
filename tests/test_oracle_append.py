"""Pins of the append oracle: closed forms and invariances, none through the CUDA path."""
import math

import numpy as np
import pytest

from oracle import append_rows as ora

FREQ = 10000.0 ** (-np.arange(0, 64, 2) / 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn_closed_forms(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 64))
    # position 0 turns nothing; a turn keeps every pair's length; turns add up
    assert np.array_equal(ora.turn(x, np.zeros(5), FREQ, interleaved), x)
    a = ora.turn(x, np.arange(5) * 1000, FREQ, interleaved)
    pair = (lambda v: v.reshape(5, 3, 32, 2)) if interleaved else (lambda v: v.reshape(5, 3, 2, 32).swapaxes(-1, -2))
    assert np.allclose(np.linalg.norm(pair(a), axis=-1), np.linalg.norm(pair(x), axis=-1), rtol=1e-12)
    assert np.allclose(ora.turn(a, np.full(5, 17), FREQ, interleaved),
                       ora.turn(x, np.arange(5) * 1000 + 17, FREQ, interleaved), rtol=0, atol=1e-9)
    # a quarter turn of pair 0: (x, y) -> (-y, x)
    f = np.zeros(32)
    f[0] = math.pi / 2
    q = ora.turn(x, np.ones(5), f, interleaved)
    j = 1 if interleaved else 32
    assert np.allclose(q[..., 0], -x[..., j]) and np.allclose(q[..., j], x[..., 0])
    # the product of a turned query and a turned key goes by the distance alone
    k = rng.standard_normal((5, 3, 64))
    d = [np.sum(ora.turn(x, np.full(5, p + 9), FREQ, interleaved) * ora.turn(k, np.full(5, p), FREQ, interleaved), -1)
         for p in (0, 1 << 20)]
    assert np.allclose(d[0], d[1], atol=1e-7)


def test_norm_closed_forms():
    z = np.full((1, 512), -3.0)
    assert np.allclose(ora.norm(z, np.ones(512), 0.0), -1.0)
    assert np.allclose(ora.norm(z, np.full(512, 2.0), 7.0), -6.0 / 4.0)
    assert np.array_equal(ora.norm(np.zeros((1, 512)), np.ones(512), 1e-6), np.zeros((1, 512)))


def test_formats():
    v = ora.e4m3_value(np.arange(256, dtype=np.uint8))
    assert np.nanmax(v) == 448.0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0xb8] == -1.0
    assert np.isnan(v[127]) and np.isnan(v[255]) and np.isnan(v).sum() == 2
    z = np.zeros((1, 512))
    z[0, 128:256] = np.linspace(-2, 1, 128)
    z[0, 300] = 1e-44
    assert np.allclose(ora.scales(z), [[1.0, 2.0 / 448, 2.0 ** -126, 1.0]], rtol=1e-15)
    assert ora.bf16_value(np.array([0x3f80, 0xc000], np.uint16)).tolist() == [1.0, -2.0]
