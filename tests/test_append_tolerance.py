"""The bound on the latents of a 656-byte row, and that mistakes in such rows do not pass it.

In units of the row's own scale sc (an fp32 number, taken as it stands): the kernel encodes y' = z' / sc, where z' is the
latent, off by less than `rel` of itself (0 without a norm, 2^-14 with one), and the quotient by less than 2^-22 of itself (two
roundings of a reciprocal and one of a product, each 2^-24). The nearest e4m3 value is off by 2^-4 of y' at most, or by
2^-10, half a step of 2^-9, below the normal range, and values are at most 448 (1 + 2^-22), where 448 is the largest code. So
    |code - z / sc| <= max(2^-4 |z / sc|, 2^-10) (1 + rel + 2^-22) + (rel + 2^-22) |z / sc|.
No term of it is absolute but the half step. The scale itself is off by less than rel + 2^-23 of max |z| / 448.
"""
import numpy as np
import pytest

from oracle import append_rows as ora


def latents_within(row, z, rel):
    """Whether rows' first 528 bytes [n][528] hold the latents z [n][512]: every scale, then every code."""
    row = np.ascontiguousarray(row[:, :528])
    sc = np.ascontiguousarray(row[:, 512:]).view(np.float32).astype(np.float64)
    ref = ora.scales(z)
    code = ora.e4m3_value(row[:, :512]).reshape(-1, 4, 128)
    y = np.abs(np.asarray(z, np.float64).reshape(-1, 4, 128) / sc[..., None])
    slack = rel + 2.0 ** -22
    off = np.abs(code - np.asarray(z, np.float64).reshape(-1, 4, 128) / sc[..., None])
    bound = np.maximum(2.0 ** -4 * y, 2.0 ** -10) * (1 + slack) + slack * y
    return bool((np.abs(sc - ref) <= (rel + 2.0 ** -23) * ref).all() and (off <= bound).all())


def spread_latents(n, seed=0):
    """Latents whose groups of 128 reach from their largest value down past the format's smallest: a third of the codes are
    below the normal range, some of them zero."""
    g = np.random.default_rng(seed)
    z = g.choice([-1.0, 1.0], (n, 4, 128)) * 2.0 ** g.uniform(-20, 0, (n, 4, 128))
    z[..., g.integers(128)] = 1.0
    return (z * 2.0 ** g.uniform(-3, 3, (n, 4, 1))).reshape(n, 512)


VALUES = ora.e4m3_value(np.arange(256))


def encode(z):
    """Rows' first 528 bytes by a search for the nearest code."""
    z = np.asarray(z, np.float64)
    sc = ora.scales(z).astype(np.float32)
    y = z.reshape(-1, 4, 128) / sc[..., None].astype(np.float64)
    order = np.argsort(np.where(np.isnan(VALUES), np.inf, VALUES), kind="stable")[:254]
    v = VALUES[order]
    at = np.clip(np.searchsorted(v, y), 1, len(v) - 1)
    at = np.where(y - v[at - 1] <= v[at] - y, at - 1, at)
    return np.concatenate([order[at].astype(np.uint8).reshape(-1, 512), sc.view(np.uint8)], axis=1)


def test_the_nearest_codes_pass():
    z = spread_latents(50)
    row = encode(z)
    code = ora.e4m3_value(row[:, :512])
    assert 0.2 < (np.abs(code) < 2.0 ** -6).mean() < 0.5 and (code == 0).any() and (np.abs(code) == 448).any()
    assert latents_within(row, z, 0.0)
    assert latents_within(row, z * (1 + 2.0 ** -15), 2.0 ** -14)
    assert not latents_within(row, z * (1 + 2.0 ** -12), 2.0 ** -14)


@pytest.mark.parametrize("mistake", ["flush", "subnormals", "sign", "neighbour", "truncated", "scale"])
def test_planted_mistakes_do_not(mistake):
    z = spread_latents(50)
    row = encode(z)
    codes, v = row[:, :512], np.abs(ora.e4m3_value(row[:, :512]))
    if mistake == "flush":
        codes[v < 0.109] = 0
    elif mistake == "subnormals":
        codes[v < 2.0 ** -6] = 0
    elif mistake == "sign":
        codes[(v < 0.05) & (v > 2.0 ** -9)] ^= 0x80
    elif mistake == "neighbour":
        codes[(v < 400) & (v > 0.02)] += 1
    elif mistake == "truncated":  # towards zero instead of to the nearest
        y = np.abs(z.reshape(-1, 4, 128) / ora.scales(z)[..., None]).reshape(-1, 512)
        codes[(v > y) & (v > 0)] -= 1
    else:
        sc = np.ascontiguousarray(row[:, 512:]).view(np.float32) * np.float32(1 + 2.0 ** -12)
        row[:, 512:] = sc.view(np.uint8)
    assert not latents_within(row, z, 2.0 ** -14)
