"""Float64 oracle of the latent cache store and the latent attention -- TEST
INFRASTRUCTURE ONLY (see the package's header).

Plain numpy: the rotation, the pool's two forms, and the attention of query
columns over a list of keys, from their definitions.
"""
from __future__ import annotations

import numpy as np

import oracle

LATENT, ROPE = 512, 64


def rotate(x, cos_sin, positions, interleaved: bool):
    """x [T, ..., 64] float64 rotated by its token's position: pairs
    (2i, 2i + 1) or (i, 32 + i), angles' cosines and sines from the table."""
    x = np.asarray(x, np.float64)
    cs = np.asarray(cos_sin, np.float64)[np.asarray(positions)]
    cs = cs.reshape(cs.shape[:1] + (1,) * (x.ndim - 2) + (ROPE,))
    cos, sin = cs[..., : ROPE // 2], cs[..., ROPE // 2:]
    out = np.empty_like(x)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    a, b = x[..., first], x[..., second]
    out[..., first] = a * cos - b * sin
    out[..., second] = b * cos + a * sin
    return out


def quantise(c):
    """(codes [T, 512] uint8, scales [T] float32) of latent rows c (float32
    values): s = max(max |c|, 1e-4) / 448 and codes of c / s, both in float32;
    a row that holds a NaN has the scale NaN."""
    c = np.asarray(c, np.float32)
    top = np.max(np.abs(c), axis=1, initial=0.0)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.where(np.isnan(top), np.float32("nan"), np.maximum(top, np.float32(1e-4)) / np.float32(448.0)).astype(np.float32)
        y = (c / s[:, None]).astype(np.float32)
    codes = oracle.e4m3_encode(np.where(np.isnan(y), 0.0, y).astype(np.float64)).reshape(c.shape)
    codes[np.isnan(y)] = 0x7F
    return codes, s


def keys_of(kv, s=None, pe=None):
    """Pool rows as float64 keys [slots, 576]: bf16 rows as they are, or codes x scale next to the rotated part."""
    if s is None:
        return np.asarray(kv, np.float64)
    c = oracle.e4m3_decode(np.asarray(kv, np.uint8)).reshape(-1, LATENT) * np.asarray(s, np.float64)[:, None]
    return np.concatenate([c, np.asarray(pe, np.float64)], axis=1)


def attend(q, keys, scale: float):
    """Columns q [n, 576] over keys [m, 576]: (out [n, 512], lse [n]); no key gives 0 and -inf."""
    q = np.asarray(q, np.float64)
    if len(keys) == 0:
        return np.zeros((len(q), LATENT)), np.full(len(q), -np.inf)
    x = scale * (q @ keys.T)
    top = x.max(axis=1, keepdims=True)
    p = np.exp(x - top)
    total = p.sum(axis=1, keepdims=True)
    return (p @ keys[:, :LATENT]) / total, (top + np.log(total))[:, 0]


def limits(q, keys, scale: float, fp8: bool):
    """How far a kernel may be from attend(): (out [n, 512], lse [n]).

    With A = sum_j p_j |v_j| (p normalised), half steps u = 2^-8 (bf16),
    2^-11 (fp16), 2^-24 (fp32):
      scores    576 products are exact and summed in fp32, then two or three
                more operations: |dx| <= 580 u32 scale max_j sum_d |q_d k_jd|,
                and |x| u32 for the reference maximum and the change to base 2
                (twice), and 2^-22 relative for exp2;
      weights   rounded to bf16, or to fp16 against a reference that leaves
                2^-24 of 2^7 as the smallest: n 2^-32 of the largest weight;
      sums      at most n / 16 + 64 additions in a row in fp32;
      result    one rounding to bf16.
    """
    q, keys = np.asarray(q, np.float64), np.asarray(keys, np.float64)
    n = len(keys)
    if n == 0:
        return np.zeros((len(q), LATENT)), np.zeros(len(q))
    u32, ub, uh = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
    x = scale * (q @ keys.T)
    dx = 580 * u32 * scale * (np.abs(q) @ np.abs(keys).T).max(axis=1) + 4 * u32 * np.abs(x).max(axis=1) + 2.0 ** -22
    p = np.exp(x - x.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    v = np.abs(keys[:, :LATENT])
    A = p @ v
    out, _ = attend(q, keys, scale)
    sums = (n / 16 + 64) * u32
    lse = dx + sums + 4 * u32 * np.abs(x).max(axis=1) + 2.0 ** -22
    weight = uh + 4 * u32 if fp8 else ub
    tol = A * (weight + 2 * dx + sums)[:, None]
    if fp8:
        tol = tol + n * 2.0 ** -32 * v.max(axis=0)
    return tol * (1 + ub) + ub * np.abs(out) + 1e-30, lse
