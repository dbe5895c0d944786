"""GPU: decode of requests that share prefixes (mla_decode_shared).

What it computes is mla_decode on the same arguments, so the oracle runs on the
whole page tables.  Tolerances: the decode's (mla_testutil) against the oracle;
against mla_decode in fp32 the two-plan tolerance, as prefix and suffix are one
more way to split the keys: the weights are the same numbers up to exact powers
of two as long as the CTAs form and round them alike.  CTAs of 96 rows round a
weight p to halves before its two E4M3 terms, the smaller ones do not.  Either is
p (1 + e) with |e| <= 2^-8 (the second term, at most 2^-4 p, is rounded by at most
2^-4 of itself), so between them an output, a mean of values with those weights,
moves by at most 2 * 2^-8 max|v|.  BF16 CTAs of 16 rows take Q as the other operand
of the product than the wider ones, so that their scores differ in the last bits
and a weight next to a border is rounded to the other side: p (1 + e) with
|e| <= 2^-9 on either side, at most 2 * 2^-9 max|v|.  The 4-bit inputs have values
and scores so far apart that weights reach the range where E4M3 steps no longer
shrink with them, and the step then depends on the part's own maximum: the E4M3
bound for all of them.
"""
import numpy as np
import pytest
import torch

import oracle
import split_kv_mla_paged_gb300 as mla
from fp4_testutil import fp4_case
from mla_testutil import PLAN_ABS, assert_parity
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE, decode_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _case(kind, heads, q_len, sizes, prefixes, suffixes, seed):
    """Inputs whose groups' page tables begin with the same pages, and the pool."""
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    of = np.repeat(np.arange(len(sizes)), sizes)
    lens = [prefixes[of[b]] + suffixes[b] for b in range(len(of))]
    if kind == "fp4":
        inp, pool = fp4_case(len(of), heads, q_len, lens, seed)
    else:
        inp = decode_inputs(len(of), heads, q_len, lens, seed, extra_pages=2, dtype="bf16" if kind == "bf16" else "e4m3")
        pool = inp.kv
    for g in range(len(sizes)):
        first, k = offsets[g], prefixes[g] // 32
        inp.page_table[first:offsets[g + 1], :k] = inp.page_table[first, :k].clone()
    return inp, pool, offsets, np.asarray(prefixes, dtype=np.int32)


def _run(inp, pool, causal, **kw):
    out = mla.decode(inp.q.cuda(), pool.cuda(), inp.page_table.cuda(), inp.kv_lens, num_heads=inp.num_heads,
                     q_len=inp.q_len, causal=causal, softmax_scale=SOFTMAX_SCALE, want_f32=True, **kw)
    torch.cuda.synchronize()
    return out


KIND = {"fp8": mla.CACHE_FP8, "fp4": mla.CACHE_FP4, "bf16": mla.CACHE_BF16}


def _largest_value(inp):
    if inp.kv.dtype == torch.bfloat16:
        return float(torch.nan_to_num(inp.kv.float()).abs().max())
    return float(np.nanmax(np.abs(oracle.e4m3_decode(np.unique(inp.kv.numpy())))))


SHAPES = [
    # heads, q_len, group sizes, prefixes, suffixes, causal
    (12, 1, [1], [32], [1], False),
    (12, 1, [2], [64], [0, 5], False),            # one request is its prefix
    (12, 1, [4], [1024], [23, 1, 32, 33], False),
    (1, 1, [3], [96], [1, 1, 1], False),
    (12, 1, [8], [4096], [200] * 8, False),       # 96 rows in one CTA
    (12, 1, [9, 1, 2], [512, 0, 2048], [7, 300, 129, 128, 127, 1, 2, 3, 4, 700, 31, 64], False),
    (12, 8, [2], [320], [8, 200], True),
    (12, 8, [3, 2], [1280, 32], [9, 8, 500, 8, 64], True),
    (12, 3, [2, 2], [96, 0], [3, 77, 40, 3], True),
    (48, 1, [2], [640], [130, 1], False),
    (33, 3, [2], [160], [300, 5], True),          # 99 rows a request: row groups inside requests
    (128, 8, [1], [128], [260], True),            # 1024 rows
    (16, 1, [20], [1536], [3] * 20, False),       # 320 rows
    (12, 1, [3], [9984], [5000, 10, 1000], False),
]


@pytest.mark.parametrize("kind", ["fp8", "fp4", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}q{s[1]}g{'-'.join(map(str, s[2]))}")
def test_matches_the_oracle_and_the_plain_decode(kind, shape):
    heads, q_len, sizes, prefixes, suffixes, causal = shape
    inp, pool, offsets, pl = _case(kind, heads, q_len, sizes, prefixes, suffixes, 11)
    out, lse, f32 = _run(inp, pool, causal, group_offsets=offsets, prefix_lens=pl)
    ref, ref_lse = oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=q_len, num_heads=heads, causal=causal,
                                      softmax_scale=SOFTMAX_SCALE)
    assert_parity(out, lse, ref, ref_lse, str(shape))
    plain = _run(inp, pool, causal)
    plan = mla.mla_shared_plan(inp.kv_lens.tolist(), offsets, pl, heads, q_len, causal=causal, cache_kind=KIND[kind]).info
    forms = {n > (16 if kind == "bf16" else 48) for n in (heads * q_len, plan.suffix_nr, plan.prefix_nr)}
    tol = PLAN_ABS if len(forms) == 1 and kind != "fp4" else (2.0 ** -8 if kind == "bf16" else 2.0 ** -7) * _largest_value(inp)
    assert float((f32 - plain[2]).abs().max()) <= tol
    assert float((lse - plain[1]).abs().max()) <= PLAN_ABS
