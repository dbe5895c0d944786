"""GPU: how exactly key weights hold scores, their scale and the LSE.

A weight is sum_r 2^x, x = c s - l log2(e), c = softmax_scale log2(e).  Bounds:
* c and l log2(e) are held in two fp32 terms each, so that x is off by the rounding of
  c s - l log2(e) and of the sum with the low terms, 2^-24 |x| each, and by 2^-30 for what the
  low terms leave out (their own rounding, for scores up to 2^13);
* 2^-22 for the exponential (ex2.approx), 2^-24 for each row's addition and two more;
* a score is formed in several accumulators, each over its share of the row's blocks, which
  the epilogue adds in fp32, half a step of the result each.  An instruction that adds to an
  accumulator (32 values of E4M3, 16 of BF16) drops less than two steps of the largest of the
  accumulator before and after it and its products: one where the products are aligned, one
  where the sum is cut to fp32.
An exponent off by d changes its weight by the factor 2^d."""
import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE
from test_key_weights_gpu import _case

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634
# Rows of a request by the forms that the kernel has, and their accumulators.
ROWS = {"fp8": {12: 4, 64: 4, 96: 2, 200: 2}, "fp4": {12: 4, 64: 4, 96: 2, 200: 2}, "bf16": {12: 8, 32: 8, 48: 4, 96: 4, 200: 4}}
FORMS = [(kind, rows) for kind in ROWS for rows in ROWS[kind]]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _pool(kind, keys):
    """Keys of exact values -> a pool of their pages."""
    n = -(-len(keys) // 32)
    rows = np.zeros((32 * n, 576))
    rows[:len(keys)] = keys
    if kind == "bf16":
        pool = torch.from_numpy(rows).bfloat16().view(n, 32, 576)
        held = pool.double().numpy()
    elif kind == "fp8":
        pool = torch.from_numpy(cache.e4m3_codes(rows)).view(n, 32, 576)
        held = cache.e4m3_values()[pool.numpy()]
    else:
        codes, sc, rope = cache.fp4_encode_rows(rows)
        raw = np.zeros((n, mla.FP4_PAGE_BYTES), np.uint8)
        raw[:, :8192] = codes.reshape(n, 8192)
        raw[:, 8192:8704] = sc.reshape(n, 32, 16).transpose(0, 2, 1).reshape(n, 512)
        raw[:, 8704:] = rope.reshape(n, 2048)
        pool = torch.from_numpy(raw)
        held = cache.fp4_decode(raw)
    assert np.array_equal(held.reshape(-1, 576), rows)
    return pool


def _instructions(kind, sums):
    """(first dim, last dim + 1, accumulator) of the instructions of a score in order."""
    k, blocks = (16, [64] * 9) if kind == "bf16" else (32, [128] * 4 + [64])
    at = 0
    for d, width in enumerate(blocks):
        for i in range(0, width, k):
            yield at + i, at + i + k, d * sums // len(blocks)
        at += width


def _weights(kind, q, pool, n, lse, scale, table=None):
    rows = q.shape[0]
    heads = next(h for h in range(min(rows, 128), 0, -1) if rows % h == 0)
    q = torch.from_numpy(q)
    q = q.bfloat16() if kind == "bf16" else torch.from_numpy(cache.e4m3_codes(q.numpy()))
    table = torch.arange(pool.shape[0], dtype=torch.int32)[None] if table is None else table
    return mla.key_weights(q.view(1, rows // heads, heads, 576).cuda(), pool.cuda(), table.cuda(), [n], lse.view(1, rows // heads, heads).cuda(),
                           num_heads=heads, q_len=rows // heads, causal=False, softmax_scale=scale)[0, :n].cpu().double().numpy()


def _large_scores(kind, rows, sums, tiny):
    """Scores of 4,096 and a few units, the 4,096 from the first instruction, all exact in
    fp32; `tiny`: besides, three quarters of a step of 4,096 (2^-11) from every instruction of
    the accumulators behind the first one."""
    rng = np.random.default_rng(rows)
    n = 300
    q, k = np.zeros((rows, 576)), np.zeros((n, 576))
    q[:, :16], k[:, :16] = 16.0, 16.0
    q[:, 40], k[:, 40] = 4.0, 4.0  # (none below 4,096)
    q[:, 32:40] = rng.integers(-1, 2, (rows, 8)) * 0.25
    k[:, 32:40] = rng.integers(-3, 4, (n, 8)) * 0.5
    others = [a for a, _, acc in _instructions(kind, sums) if acc > 0]
    if tiny:
        for a in others:
            q[:, a] = 2.0 ** -6
            k[:, a] = np.where(rng.random(n) < 0.7, 1.5 * 2.0 ** -6, 0.0)
    return q, k, n, len(others)


def _bound(x, rows):
    return np.log(2.0) * (2.0 ** -23 * np.abs(x).max() + 2.0 ** -30) + 2.0 ** -22 + 2.0 ** -24 * (rows + 2)


@pytest.mark.parametrize("kind,rows", FORMS)
def test_large_scores_with_exact_products(kind, rows):
    # The scale's or the LSE's low term left out: 4,096 * 2^-25 * ln 2 or more, 5e-5.
    q, k, n, _ = _large_scores(kind, rows, ROWS[kind][rows], False)
    s = q @ k.T
    lse = torch.from_numpy(np.log(np.exp(s - 4096.0).sum(1)) + 4096.0).float()
    z = s - lse.double().numpy()[:, None]
    ref = np.exp(z).sum(0)
    bound = _bound(z * LOG2E, rows)
    l = lse.double().numpy()[:, None]
    for c, low in ((float(np.float32(LOG2E)), l * LOG2E), (LOG2E, (lse * np.float32(LOG2E)).double().numpy()[:, None])):
        assert (np.abs(np.exp2(c * s - low).sum(0) - ref) > 2 * bound * ref).any()  # one term each would be seen
    assert (np.abs(_weights(kind, q, _pool(kind, k), n, lse, 1.0) - ref) <= bound * ref).all()


@pytest.mark.parametrize("kind,rows", FORMS)
def test_accumulators_keep_small_sums(kind, rows):
    # Added to the accumulator that holds 4,096, each would be cut off: with half of the
    # accumulators at least four of them, three steps, more than the epilogue's roundings.
    sums = ROWS[kind][rows]
    q, k, n, count = _large_scores(kind, rows, sums, True)
    s = q @ k.T
    assert count >= 4 and s.min() > 4096.0
    lse = torch.from_numpy(np.log(np.exp(s - 4096.0).sum(1)) + 4096.0).float()
    z = s - lse.double().numpy()[:, None]
    ref = np.exp(z).sum(0)
    bound = _bound(z * LOG2E, rows) + np.expm1(sums / 2 * 2.0 ** -12)  # (sums / 2 additions to the 4,096)
    assert (np.abs(_weights(kind, q, _pool(kind, k), n, lse, 1.0) - ref) <= bound * ref).all()


def _step(x):
    """The step of fp32 numbers of this magnitude."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 23)


@pytest.mark.parametrize("kind,rows", FORMS)
def test_ordinary_scores(kind, rows):
    n, sums = 500, ROWS[kind][rows]
    heads = next(h for h in range(min(rows, 128), 0, -1) if rows % h == 0)
    inp, pool, q, keys = _case(kind, heads, rows // heads, [n], rows)
    q, k = q.reshape(rows, 576), keys[0]
    s = q @ k.T * SOFTMAX_SCALE
    top = s.max(1, keepdims=True)
    lse = torch.from_numpy((top + np.log(np.exp(s - top).sum(1, keepdims=True)))[:, 0]).float()
    held, off = [np.zeros((rows, n)) for _ in range(sums)], np.zeros((rows, n))
    for a, b, acc in _instructions(kind, sums):
        product = np.abs(q[:, a:b]).max(1)[:, None] * np.abs(k[:, a:b]).max(1)[None]
        after = held[acc] + q[:, a:b] @ k[:, a:b].T
        off += 2.0 * _step(np.maximum(np.maximum(np.abs(held[acc]), np.abs(after)), product))
        held[acc] = after
    off += (sums - 1) * 0.5 * _step(sum(np.abs(h) for h in held))
    z = s - lse.double().numpy()[:, None]
    w = np.exp(z)
    ref = w.sum(0)
    d = SOFTMAX_SCALE * LOG2E * off + 2.0 ** -23 * np.abs(z * LOG2E) + 2.0 ** -30
    bound = (w * np.expm1(np.log(2.0) * d)).sum(0) + (2.0 ** -22 + 2.0 ** -24 * (rows + 2)) * ref
    error = np.abs(_weights(kind, q, pool, n, lse, SOFTMAX_SCALE, inp.page_table) - ref)
    print(kind, rows, "largest error of its bound", (error / bound).max(), "of the weight", (error / ref).max())
    assert (error <= bound).all()
