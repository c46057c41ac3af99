"""The oracle of the 4-bit rows: closed forms, and planted mistakes that do not pass them."""
import numpy as np
import pytest

from oracle import int4_rows as ora


def test_scale_codes_are_the_upper_bits_of_a_half():
    codes = np.arange(256, dtype=np.uint8)
    half = (codes.astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(ora.scale_value(codes)[:248], half[:248])
    assert np.isnan(ora.scale_value(255)) and np.isnan(half[255])
    assert ora.scale_value(1) == 2.0 ** -17 and ora.scale_value(215) == 3840


@pytest.mark.parametrize("amax,code", [(0.0, 1), (7 * 2.0 ** -17, 1), (1e-9, 1), (7.0, 120), (26880.0, 215), (1e30, 215),
                                       (7 * 1.0625, 120), (7 * 1.1875, 122), (7 * 1.07, 121), (7 * 2.0 ** -14, 8),
                                       (7 * 2.5 * 2.0 ** -17, 2), (7 * 3.5 * 2.0 ** -17, 4)])
def test_nearest_scale_and_ties(amax, code):
    assert ora.scale_code(amax) == code


def test_numbers_and_places():
    z = np.zeros((1, 512))
    z[0, 0:16] = [7, -7, 6.5, 5.5, -6.5, 0.5, 1.5, -0.5, 0.49, -0.51, 1, 2, 3, -3, 7, 0]
    q, codes, _ = ora.unpack(np.concatenate([ora.pack(z), np.zeros((1, 128), np.uint8)], 1))
    assert codes[0, 0] == 120 and (codes[0, 1:] == 1).all()
    assert q[0, :16].tolist() == [7, -7, 6, 6, -6, 0, 2, 0, 0, -1, 1, 2, 3, -3, 7, 0] and not q[0, 16:].any()
    word = int(ora.pack(z)[0, :4].view("<u4")[0])
    assert [(word >> at & 15) - 8 for at in (0, 16, 4, 20, 8, 24, 12, 28)] == q[0, :8].tolist()


def test_a_row_is_within_half_a_step_of_its_latents():
    g = np.random.default_rng(3)
    z = (g.standard_normal((200, 512)) * np.exp(g.standard_normal((200, 1)) * 3)).astype(np.float32)
    rows = np.concatenate([ora.pack(z), np.zeros((200, 128), np.uint8)], 1)
    s = np.repeat(ora.scale_value(rows[:, 256:288]), 16, axis=1)
    off = np.abs(ora.values(rows)[:, :512] - z)
    # The scale was rounded down: the largest are cut off, by 7 times what it lost. That is at most half a step of an eighth,
    # a sixteenth of it, or below 2^-14 half of 2^-17; where the scale is the largest there is, it may be anything.
    cut, most = np.abs(z) > 7 * s, s == 3840
    assert (off[~cut] <= s[~cut] * (0.5 + 2.0 ** -20)).all()
    assert (off <= np.maximum(np.abs(z) / 15, 7.01 * 2.0 ** -18))[cut & ~most].all()
    assert np.array_equal(np.abs(ora.values(rows)[:, :512])[cut], 7 * s[cut])


def test_planted_mistakes_are_seen():
    g = np.random.default_rng(4)
    z = g.standard_normal((50, 512)).astype(np.float32)
    good = ora.pack(z)
    rows = lambda b: np.concatenate([b, np.zeros((50, 128), np.uint8)], 1)  # noqa: E731
    s = np.repeat(ora.scale_value(good[:, 256:288]), 16, axis=1)

    def fine(b):
        return (np.abs(ora.values(rows(b))[:, :512] - z) <= np.maximum(0.5 * s, np.abs(z) / 15) + 1e-6).all()

    assert fine(good)
    swapped = good.copy()
    swapped[:, :256] = (good[:, :256] >> 4) | (good[:, :256] << 4)
    shifted = good.copy()
    shifted[:, 256:288] = np.roll(good[:, 256:288], 1, axis=1)
    truncated = good.copy()
    truncated[:, 256:288] -= 1
    plain = good.copy()
    plain[:, :256] = good.reshape(50, -1)[:, :256].reshape(50, 64, 4)[:, :, [0, 2, 1, 3]].reshape(50, 256)
    for bad in (swapped, shifted, truncated, plain):
        assert not fine(bad)
