"""Shared helpers of the 4-bit cache's GPU tests."""
from __future__ import annotations

import numpy as np
import torch

import split_kv_mla_paged_gb300 as mla
from oracle import cache
from synth import decode_inputs


def fp4_case(batch, heads, q_len, lens, seed, extra_pages=2):
    """decode_inputs with its cache re-encoded in 4 bits: (inputs with the
    expanded E4M3 cache, 4-bit pool).  Rows behind a sequence's end stay NaN in
    the 4-bit pool (scale bytes 0xFF, rope 0x7F)."""
    inp = decode_inputs(batch, heads, q_len, lens, seed, extra_pages=extra_pages)
    host = inp.kv.numpy()
    vals = cache.e4m3_values()[host].reshape(-1, 576)
    rng = np.random.default_rng(seed)
    spread = np.exp2(rng.integers(-9, 6, (vals.shape[0], 18)).repeat(32, 1) * (rng.random((vals.shape[0], 1)) < 0.1))
    stale = np.isnan(vals).any(1)
    vals = np.where(stale[:, None], np.nan, np.nan_to_num(vals) * spread)
    codes, sc, rope = cache.fp4_encode_rows(vals)
    sc[stale], codes[stale] = 255, 255
    pool = np.zeros((host.shape[0], mla.FP4_PAGE_BYTES), np.uint8)
    n = host.shape[0]
    pool[:, :8192] = codes.reshape(n, 8192)
    pool[:, 8192:8704] = sc.reshape(n, 32, 16).transpose(0, 2, 1).reshape(n, 512)
    pool[:, 8704:] = rope.reshape(n, 2048)
    inp.kv = torch.from_numpy(cache.e4m3_codes(cache.fp4_decode(pool)))
    return inp, torch.from_numpy(pool)


def same_outputs(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def equal_outputs(a, b, rows):
    """Outputs (bf16, lse, fp32) of the 4-bit and the E4M3 decode of `rows` rows a request."""
    if rows > 16:
        return same_outputs(a, b)
    (o, l, f), (ob, lb, fb) = a, b
    assert ((f - fb).abs() <= 2.0 ** -15 * fb.abs()).all()
    assert ((l - lb).abs() <= 2.0 ** -15).all()
    assert ((o.float() - ob.float()).abs() <= 2.0 ** -7 * ob.float().abs()).all()  # one BF16 step
