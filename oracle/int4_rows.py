"""Oracle of the 4-bit row format in plain numpy, written from the definition; it shares no code with the CUDA path.

A row of 416 bytes: 64 words of 32 bits with eight latents each, 32 scale codes, 64 bf16 of the rotary key. Scale code c
stands for (c % 8 / 8) 2^-14 where c < 8, else (1 + c % 8 / 8) 2^(c // 8 - 15); 255 for NaN. A latent is its number times its
scale.
"""
from __future__ import annotations

import numpy as np

from oracle.append_rows import bf16_value

SCALE_CODES = 216  # codes 0 .. 215 stand for 0 .. 3840


def scale_value(code):
    c = np.asarray(code, np.uint8).astype(np.int64)
    v = np.where(c < 8, c % 8 * 2.0 ** -17, (8 + c % 8) * 2.0 ** (c // 8 - 18.0))
    return np.where(c == 255, np.nan, v)


def scale_code(amax):
    """The code nearest to amax / 7 of those from 1 on, ties to the even code."""
    every = scale_value(np.arange(1, SCALE_CODES))
    a = np.clip(np.asarray(amax, np.float64) / 7, every[0], every[-1])
    i = np.clip(np.searchsorted(every, a), 1, len(every) - 1)  # every[i - 1] < a <= every[i]
    low, up = a - every[i - 1], every[i] - a
    return (np.where((up < low) | ((up == low) & (i % 2 == 1)), i, i - 1) + 1).astype(np.uint8)  # entry i has code i + 1


def numbers(z, codes):
    """The whole numbers of latents [n][512] over the scales of codes [n][32]; the quotient in 32 bits, ties to even."""
    s = np.repeat(scale_value(codes), 16, axis=-1).astype(np.float32)
    return np.clip(np.rint(np.asarray(z, np.float32) / s), -7, 7).astype(np.int64)


def pack(z):
    """The first 288 bytes of the rows of latents [n][512] that are 32-bit numbers."""
    z = np.asarray(z, np.float64)
    codes = scale_code(np.abs(z.reshape(len(z), 32, 16)).max(-1))
    u = (numbers(z, codes) + 8).reshape(len(z), 64, 8)
    word = sum(u[..., e] << (4 * (e // 2) + 16 * (e % 2)) for e in range(8)).astype("<u4")
    return np.concatenate([np.ascontiguousarray(word).view(np.uint8).reshape(len(z), 256), codes], axis=1)


def unpack(rows):
    """(numbers [n][512], scale codes [n][32], rotary keys [n][64] in 64 bits) of rows [n][416]."""
    rows = np.ascontiguousarray(np.asarray(rows, np.uint8))
    word = np.ascontiguousarray(rows[:, :256]).view("<u4").astype(np.int64)
    q = np.stack([word >> (4 * (e // 2) + 16 * (e % 2)) & 15 for e in range(8)], -1).reshape(len(rows), 512) - 8
    return q, rows[:, 256:288], bf16_value(np.ascontiguousarray(rows[:, 288:]).view(np.uint16))


def values(rows):
    """The 576 values of rows [n][416], in 64 bits."""
    q, codes, key = unpack(rows)
    return np.concatenate([q * np.repeat(scale_value(codes), 16, axis=-1), key], axis=1)
