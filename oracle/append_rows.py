"""Float64 oracle of appending KV rows: the latent's norm, the rotation of the key's and the queries' pairs, and the two
row formats, in plain numpy and written from the formulas; it shares no code with the CUDA path.

Token i at position p: z = kv[0:512], with a norm z * weight / sqrt(mean(z^2) + eps); pair j of kv[512:576], (j, j + 32) or
(2j, 2j + 1), turns by p * inv_freq[j]. A row is 576 bf16 values, or 512 e4m3 values with one scale for each 128 (largest
magnitude / 448, 1 where all are zero) and 64 bf16 values.
"""
from __future__ import annotations

import numpy as np

LATENT, ROPE = 512, 64


def norm(z, weight, eps):
    z = np.asarray(z, dtype=np.float64)
    return z * np.asarray(weight, np.float64) / np.sqrt(np.mean(z * z, axis=-1, keepdims=True) + eps)


def turn(x, positions, inv_freq, interleaved):
    """x [n][...][64] at positions [n]: every pair turned."""
    x = np.asarray(x, dtype=np.float64)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :]
    angle = angle.reshape(len(x), *([1] * (x.ndim - 2)), ROPE // 2)
    first = slice(0, None, 2) if interleaved else slice(0, ROPE // 2)
    second = slice(1, None, 2) if interleaved else slice(ROPE // 2, None)
    out = np.empty_like(x)
    out[..., first] = x[..., first] * np.cos(angle) - x[..., second] * np.sin(angle)
    out[..., second] = x[..., first] * np.sin(angle) + x[..., second] * np.cos(angle)
    return out


def rows(kv, positions, inv_freq, interleaved, weight=None, eps=0.0):
    """The unrounded rows [n][576]."""
    kv = np.asarray(kv, dtype=np.float64)
    z = kv[:, :LATENT] if weight is None else norm(kv[:, :LATENT], weight, eps)
    return np.concatenate([z, turn(kv[:, LATENT:], positions, inv_freq, interleaved)], axis=1)


def scales(z):
    """The fp8 format's scale of each 128 latents [n][4]."""
    m = np.abs(np.asarray(z, np.float64).reshape(-1, 4, 128)).max(-1)
    return np.where(m > 0, np.maximum(m / 448.0, 2.0 ** -126), 1.0)


def e4m3_value(bits):
    """The value of e4m3 bit patterns: 1 sign, 4 exponent (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    b = np.asarray(bits, np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b & 127 == 127, np.nan, np.where(b >= 128, -v, v))


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
