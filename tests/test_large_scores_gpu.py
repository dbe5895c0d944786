"""GPU: rows whose scores are millions of log2 units from zero, next to ordinary rows.

fp32 holds such a score to half a unit or better up to 2^23, to one unit up to
2^24, and the softmax only depends on differences of scores: the outputs are
those of the definition.  Scores are built exactly: a query row has two values
that are not zero, q0 in {448, -448, 0} against key value 0 (256 or 384) and q1 =
2^-m against key value 32 (0..6), and softmax_scale * log2(e) is 1 in fp32, so that
with q_scale = 2^m a score in log2 units is the integer 2^m q0 k0 + k1.

Tolerances.  softmax_scale is within 2^-25 (relative) of ln 2; the weights that
are not zero differ by at most 6 log2 units, so this moves them by less than
2^-22.  A weight enters the product as two E4M3 terms, each off by at most half
a step, 2^-4 relative: 2^-8 together, and up to 2^-11 more where it goes through
halves; it is 4 or more, so no term is subnormal before 2^-10.  O is a mean of the
values under these weights: |err| <= (2^-8 + 2^-11 + 2^-12) max_j |v_jd| < 2^-7 max_j
|v_jd| before the BF16 store.  LSE = ln2 (m + log2 l) carries the score's 2^-25, the
sum's, the product's and ln2's rounding, 2^-24 each: below 2^-21 |LSE|; and in l
2^-22 for each ex2 and 16 roundings of 2^-24: below 2^-18 with log2's own.
"""
import numpy as np
import pytest
import torch

import oracle
import split_kv_mla_paged_gb300 as mla
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build

pytestmark = pytest.mark.gpu

LN2 = float(np.float32(np.log(2.0)))
LENS = [700, 131, 9]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _inputs(heads, q_len, m, seed):
    """(q codes, 4-bit pool, E4M3 pool with the same values, page table)."""
    rng = np.random.default_rng(seed)
    pages = [(n + 31) // 32 for n in LENS]
    order = rng.permutation(sum(pages))
    table = np.full((len(LENS), max(pages)), -1, np.int32)
    x = np.zeros((sum(pages), 32, 576))
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
        n = 32 * k
        v = rng.choice([-3.0, -2, -1.5, -1, 0, 0.5, 1, 2, 3], (n, 576))
        # Both classes of keys, and within a class scores that rise along the
        # request, so that the reference rises by little and by much.
        v[:, 0] = np.where(rng.random(n) < 0.5, 384.0, 256.0)
        v[:min(n, 40), 0] = rng.choice([384.0, 256.0])
        v[:, 1:32] = rng.choice([-128.0, -64, 0, 64, 192], (n, 31))  # (value 0's scale is 64)
        steps = np.array([0.0, 1, 2, 3, 4, 6])
        v[:, 32] = steps[np.minimum(rng.integers(0, 3, n) + np.arange(n) // 160, 5)]
        x[table[b, :k]] = v.reshape(k, 32, 576)
    codes, sc, rope = cache.fp4_encode_rows(x.reshape(-1, 576))
    pool = np.zeros((x.shape[0], mla.FP4_PAGE_BYTES), np.uint8)
    for i in range(codes.shape[0]):
        cache.fp4_put(pool, i // 32, i % 32, (codes[i], sc[i], rope[i]))
    assert np.array_equal(cache.fp4_decode(pool), x)
    q = np.zeros((len(LENS), q_len, heads, 576))
    row = np.arange(q_len)[:, None] + np.arange(heads)[None, :]
    q[..., 0] = np.array([448.0, -448.0, 0.0])[row % 3]
    q[..., 32] = 2.0 ** -m
    return tuple(torch.from_numpy(a) for a in (cache.e4m3_codes(q), pool, cache.e4m3_codes(x), table))


@pytest.mark.parametrize("kind", ["fp4", "fp8"])
@pytest.mark.parametrize("m", [4, 5, 6])  # |scores| up to 2.8e6, 5.6e6 and 1.1e7 log2 units
@pytest.mark.parametrize("heads, q_len", [(12, 1), (12, 2), (12, 4), (12, 8), (33, 3)])
def test_far_scores_match_oracle(heads, q_len, m, kind):
    q, pool, wide, table = _inputs(heads, q_len, m, seed=7 * m + heads + q_len)
    rows = len(LENS) * q_len * heads
    ref_o, ref_l = oracle.decode_rows(q, wide, table, torch.tensor(LENS, dtype=torch.int32), q_len=q_len, num_heads=heads,
                                      causal=q_len > 1, softmax_scale=LN2, q_scale=2.0 ** m)
    assert np.abs(ref_l).max() > 2 ** 21 * LN2
    vmax = np.empty((len(LENS), 512))
    values = cache.e4m3_values()[wide.numpy()]
    for b, n in enumerate(LENS):
        vmax[b] = np.abs(values[table[b, :(n + 31) // 32].numpy()].reshape(-1, 576)[:n, :512]).max(0)
    tol = np.repeat(vmax, q_len * heads, 0) * 2.0 ** -7
    # One and several splits, and the variants with windows and with device scales.
    # (E4M3: and CTAs that go from one item to the next).
    for kw in (dict(target_ctas=1), dict(target_ctas=9), dict(kv_bounds=[[0, n] for n in LENS]), dict(device_scales=True),
               dict(target_ctas=9, persistent_ctas=2 if kind == "fp8" else 0)):
        _, lse, out = mla.decode(q.cuda(), (pool if kind == "fp4" else wide).cuda(), table.cuda(), LENS, num_heads=heads,
                                 q_len=q_len, causal=q_len > 1, softmax_scale=LN2, q_scale=2.0 ** m, want_f32=True, **kw)
        torch.cuda.synchronize()
        o, l = out.double().cpu().numpy().reshape(rows, 512), lse.double().cpu().numpy().reshape(rows)
        assert (np.abs(l - ref_l.reshape(-1)) <= 2.0 ** -21 * np.abs(ref_l.reshape(-1)) + 2.0 ** -18).all(), kw
        assert (np.abs(o - ref_o.reshape(rows, 512)) <= tol).all(), kw


@pytest.mark.parametrize("heads, q_len", [(12, 1), (12, 2), (12, 8)])
def test_far_scores_over_selected_pages(heads, q_len):
    m = 5
    q, pool, wide, table = _inputs(heads, q_len, m, seed=3 + q_len)
    sel = np.array([[0, 3, 4, 9, 15, 21], [1, 4, -1, -1, -1, -1], [0, -1, -1, -1, -1, -1]], np.int32)
    ref_o, ref_l = oracle.decode_rows(q, wide, table, torch.tensor(LENS, dtype=torch.int32), q_len=q_len, num_heads=heads,
                                      causal=q_len > 1, softmax_scale=LN2, q_scale=2.0 ** m, block_idx=sel)
    got = [mla.decode(q.cuda(), kv.cuda(), table.cuda(), LENS, num_heads=heads, q_len=q_len, causal=q_len > 1,
                      softmax_scale=LN2, q_scale=2.0 ** m, want_f32=True, block_idx=torch.from_numpy(sel)) for kv in (pool, wide)]
    torch.cuda.synchronize()
    for _, lse, out in got:
        o, l = out.double().cpu().numpy().reshape(-1, 512), lse.double().cpu().numpy().reshape(-1)
        assert (np.abs(l - ref_l.reshape(-1)) <= 2.0 ** -21 * np.abs(ref_l.reshape(-1)) + 2.0 ** -18).all()
        vmax = np.where(np.arange(512) < 32, 192.0, 6.0)
        vmax[0] = 384.0
        assert (np.abs(o - ref_o.reshape(-1, 512)) <= 2.0 ** -7 * vmax).all()
