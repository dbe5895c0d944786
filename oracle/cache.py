"""Oracle for the cache formats and what writes them: plain numpy in 64 bits.

The 4-bit page (mla_decode.h, MLA_CACHE_FP4) decoded and encoded value by
value, the prologue's norm and rotation, and page copies.  Like the rest of
this package it shares no code with the CUDA path; tests/test_cache_oracle.py
pins it.
"""
from __future__ import annotations

import numpy as np

LATENT, ROPE, DIM, PAGE, BLOCK = 512, 64, 576, 32, 32
FP4_PAGE = 10752
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round_to(x, min_exp: int, bits: int, high: float):
    """x rounded to `bits` fraction bits (ties to even), steps no finer than
    2^(min_exp - bits), magnitudes saturating at `high`; also returns half the
    step at x."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
    step = np.ldexp(1.0, np.maximum(e - 1, min_exp) - bits)
    r = np.where(np.isfinite(x), np.rint(np.where(np.isfinite(x), x, 0.0) / step) * step, x)
    return np.clip(r, -high, high), step / 2


def e4m3_values() -> np.ndarray:
    """The 256 E4M3 values, from the format's definition."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_codes(x) -> np.ndarray:
    """Codes of the nearest E4M3 values (ties to even, saturating; NaN 0x7F)."""
    x = np.asarray(x, dtype=np.float64)
    r, _ = round_to(x, -6, 3, 448.0)
    mag = np.abs(np.where(np.isnan(r), 0.0, r))
    code = np.searchsorted(e4m3_values()[:127], mag)
    code = np.where(np.signbit(x), code | 128, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def _sign_bit(j: int) -> int:
    return 8 * j + 7 if j < 4 else 8 * (j - 4) + 3


def fp4_decode(pages) -> np.ndarray:
    """uint8 [P, 10752] -> float64 [P, 32, 576] (before kv_scale)."""
    pages = np.asarray(pages, dtype=np.uint8)
    n = pages.shape[0]
    words = pages[:, :8192].reshape(n, PAGE, 64, 4).astype(np.uint32)
    words = words[..., 0] | words[..., 1] << 8 | words[..., 2] << 16 | words[..., 3] << 24
    lat = np.zeros((n, PAGE, 64, 8))
    for j in range(8):
        mag = E2M1[(words >> np.uint32(4 * j)) & 7]
        neg = (words >> np.uint32(_sign_bit(j))) & 1
        lat[..., j] = np.where(neg == 1, -mag, mag)
    sc = (pages[:, 8192:8704].reshape(n, 16, PAGE) & 15).transpose(0, 2, 1)
    step = np.where(sc == 15, np.nan, np.exp2(sc - 8.0))
    lat = lat.reshape(n, PAGE, 16, BLOCK) * step[..., None]
    rope = e4m3_values()[pages[:, 8704:].reshape(n, PAGE, ROPE)]
    return np.concatenate([lat.reshape(n, PAGE, LATENT), rope], axis=2)


def fp4_scale_codes(amax) -> np.ndarray:
    sc = np.zeros(amax.shape, dtype=np.int64)
    for k in range(14):
        sc += np.nan_to_num(amax, nan=0.0, posinf=1e30) > 7.0 * 2.0 ** (k - 8)
    return np.where(np.isnan(amax), 15, sc)


def fp4_encode_rows(x):
    """float64 [n, 576] (over kv_scale) -> (codes [n, 256], scales [n, 16], rope [n, 64])."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x[:, :LATENT].reshape(-1, 16, BLOCK)
    amax = np.where(np.isnan(blocks).any(-1), np.nan, np.abs(np.nan_to_num(blocks, posinf=np.inf, neginf=-np.inf)).max(-1))
    sc = fp4_scale_codes(amax)
    with np.errstate(invalid="ignore"):
        r, _ = round_to(blocks * np.exp2(8.0 - sc)[..., None], 0, 1, 6.0)
    mag = np.searchsorted(E2M1, np.abs(np.nan_to_num(r)))
    neg = np.signbit(blocks)
    dead = (sc == 15)[..., None]
    mag, neg = np.where(dead, 0, mag), np.where(dead, False, neg)
    mag = mag.reshape(-1, 64, 8).astype(np.uint64)
    neg = neg.reshape(-1, 64, 8).astype(np.uint64)
    words = np.zeros(mag.shape[:2], dtype=np.uint64)
    for j in range(8):
        words |= mag[..., j] << np.uint64(4 * j) | neg[..., j] << np.uint64(_sign_bit(j))
    codes = np.stack([(words >> np.uint64(8 * b)) & np.uint64(255) for b in range(4)], axis=-1)
    return (codes.reshape(-1, 256).astype(np.uint8), sc.astype(np.uint8),
            e4m3_codes(x[:, LATENT:]))


def fp4_put(pool, page, slot, parts) -> None:
    """Writes one encoded row (the i-th of fp4_encode_rows) into a page pool."""
    codes, sc, rope = parts
    pool[page, :8192].reshape(PAGE, 256)[slot] = codes
    pool[page, 8192:8704].reshape(16, PAGE)[:, slot] = sc
    pool[page, 8704:].reshape(PAGE, ROPE)[slot] = rope


def prologue_rows(rows, weight, eps, cos_sin, positions, halves):
    """Normed (weight None: not) and rotated (cos_sin None: not) key rows."""
    x = np.asarray(rows, dtype=np.float64).copy()
    if weight is not None:
        lat = x[:, :LATENT]
        x[:, :LATENT] = lat / np.sqrt((lat ** 2).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return rotate(x, cos_sin, positions, halves)


def rotate(x, cos_sin, positions, halves):
    """Rotates values 512..575 of rows [n, ..., 576] by their positions' table rows."""
    x = np.asarray(x, dtype=np.float64).copy()
    if cos_sin is None:
        return x
    cs = np.asarray(cos_sin, dtype=np.float64)[np.asarray(positions)]
    cs = cs.reshape(cs.shape[0], *([1] * (x.ndim - 2)), ROPE)
    c, s = cs[..., :32], cs[..., 32:]
    ia, ib = (np.arange(32), np.arange(32) + 32) if halves else (2 * np.arange(32), 2 * np.arange(32) + 1)
    a, b = x[..., LATENT + ia], x[..., LATENT + ib]
    x[..., LATENT + ia], x[..., LATENT + ib] = a * c - b * s, b * c + a * s
    return x
