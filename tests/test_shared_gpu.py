"""GPU: decode of requests that share prefixes (mla_decode_shared).

What it computes is mla_decode on the same arguments, so the oracle runs on the
whole page tables.  Tolerances: the decode's (mla_testutil) against the oracle;
against mla_decode in fp32 the two-plan tolerance, as prefix and suffix are one
more way to split the keys: the weights are the same numbers up to exact powers
of two as long as the CTAs form and round them alike.  CTAs of 96 rows round a
weight p to halves before its two E4M3 terms, the smaller ones do not.  Either is
p (1 + e) with |e| <= 2^-8 (the second term, at most 2^-4 p, is rounded by at most
2^-4 of itself), so between them an output, a mean of values with those weights,
moves by at most 2 * 2^-8 max|v|.  mla_decode's BF16 CTAs of more than 16 rows take Q
as the other operand of the product than these, so that scores differ in the last
bits and a weight next to a border is rounded to the other side: p (1 + e) with
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
    (12, 1, [8, 1], [512, 2048], [9000, 8000, 7000, 9001, 33, 9002, 5, 4000, 9000], False),  # two launches
    (4, 8, [3], [256], [20000, 19000, 8], True),                                          # likewise
    # Prefixes so long that the plan attends them once for their group on one SM.
    (12, 8, [3, 2], [3200, 32], [9, 8, 500, 8, 64], True),
    (12, 3, [5, 2], [2080, 0], [3, 77, 40, 3, 500, 9, 10], True),
    (48, 1, [3], [6400], [130, 1, 0], False),
    (33, 3, [4], [1600], [300, 5, 3, 64], True),
    (128, 8, [3], [2048], [260, 8, 9], True),
    (12, 1, [8, 1], [16384, 2048], [9000, 8000, 7000, 9001, 33, 9002, 5, 4000, 9000], False),  # two launches
    (4, 8, [6], [8192], [20000, 19000, 8, 9, 10, 5000], True),                             # likewise
]


@pytest.mark.parametrize("kind", ["fp8", "fp4", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}q{s[1]}g{'-'.join(map(str, s[2]))}")
@pytest.mark.parametrize("sms", [152, 1])  # one SM: plans that share short prefixes as well
def test_matches_the_oracle_and_the_plain_decode(kind, shape, sms):
    heads, q_len, sizes, prefixes, suffixes, causal = shape
    inp, pool, offsets, pl = _case(kind, heads, q_len, sizes, prefixes, suffixes, 11)
    out, lse, f32 = _run(inp, pool, causal, group_offsets=offsets, prefix_lens=pl, sm_count=sms)
    ref, ref_lse = oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=q_len, num_heads=heads, causal=causal,
                                      softmax_scale=SOFTMAX_SCALE)
    assert_parity(out, lse, ref, ref_lse, str(shape))
    plain = _run(inp, pool, causal)
    plan = mla.mla_shared_plan(inp.kv_lens.tolist(), offsets, pl, heads, q_len, causal=causal, cache_kind=KIND[kind], sm_count=sms).info
    assert sms > 1 or plan.prefix_ctas > 0 or max(prefixes) < 8000 or kind == "bf16"
    forms = {heads * q_len > 16, False} if kind == "bf16" else {n > 48 for n in (heads * q_len, plan.suffix_nr, plan.prefix_nr)}
    tol = PLAN_ABS if len(forms) == 1 and kind != "fp4" else (2.0 ** -8 if kind == "bf16" else 2.0 ** -7) * _largest_value(inp)
    assert float((f32 - plain[2]).abs().max()) <= tol
    assert float((lse - plain[1]).abs().max()) <= PLAN_ABS


def _oracle(inp, causal, **kw):
    return oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=inp.q_len, num_heads=inp.num_heads, causal=causal,
                              softmax_scale=SOFTMAX_SCALE, **kw)


KINDS = ["fp8", "fp4", "bf16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sms", [152, 1])
def test_sinks_output_scale_and_scales(kind, sms):
    inp, pool, offsets, pl = _case(kind, 12, 2, [3, 1], [640, 96], [2, 200, 5, 300], 5)
    sinks = np.linspace(-2.0, 3.0, 12).astype(np.float32)
    scales = {} if kind == "bf16" else dict(q_scale=1.5, kv_scale=0.37)
    for device_scales in (False, True):
        out, lse, _ = _run(inp, pool, True, group_offsets=offsets, prefix_lens=pl, sinks=sinks, output_scale=0.5, device_scales=device_scales,
                           sm_count=sms, **scales)
        ref, ref_lse = _oracle(inp, True, sinks=sinks, output_scale=0.5, **scales)
        assert_parity(out, lse, ref, ref_lse)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sms", [152, 1])
def test_ragged_query_counts(kind, sms):
    inp, pool, offsets, pl = _case(kind, 12, 8, [4], [320], [8, 100, 9, 8], 6)
    ql = [1, 8, 3, 5]
    for sinks in (None, np.zeros(12, np.float32)):
        out, lse, _ = _run(inp, pool, True, group_offsets=offsets, prefix_lens=pl, query_lens=ql, sinks=sinks, sm_count=sms)
        ref, ref_lse = _oracle(inp, True, query_lens=ql, sinks=sinks)
        empty = np.isinf(ref_lse)
        assert empty.any() == (sinks is None)
        l = lse.cpu().numpy().reshape(ref_lse.shape)
        assert (l[empty] == -np.inf).all()
        assert_parity(out, torch.from_numpy(np.where(empty, 0.0, l)), ref, np.where(empty, 0.0, ref_lse))
        assert (out[0, 1:] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_stale_plans_are_reported(kind):
    inp, pool, offsets, pl = _case(kind, 12, 1, [2], [3200], [100, 5], 7)
    kw = dict(group_offsets=offsets, prefix_lens=pl, sm_count=1)
    for row, entry in ((0, 1), (1, 100)):
        table = inp.page_table.clone()
        inp.page_table[row, entry] = 10 ** 6
        with pytest.raises(mla.MlaError) as err:
            _run(inp, pool, False, **kw)
        assert err.value.status == mla.MLA_ERR_INVALID_ARG
        inp.page_table = table
    # Lengths that have left the plan: below the prefix, and past the suffix's splits.
    plan = mla.mla_shared_plan(inp.kv_lens.tolist(), offsets, pl, 12, 1, cache_kind=KIND[kind], sm_count=1)
    assert plan.info.prefix_ctas > 0
    data = torch.from_numpy(plan.data).cuda()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 1, 12, 512, dtype=torch.bfloat16, device="cuda")
    wide = torch.cat([inp.page_table, torch.zeros(2, 8, dtype=torch.int32)], 1).clamp(min=0).cuda()  # valid ids behind the ends
    for lens, good in (([3300, 3205], True), ([3300, 3328], True), ([3199, 3205], False), ([3300, 3329], False), ([-5, 3205], False)):
        mla.mla_decode_shared(inp.q.cuda(), pool.cuda(), pool.shape[0], wide, wide.shape[1], torch.tensor(lens, dtype=torch.int32).cuda(), plan, data,
                              2, 1, 12, False, 1.0, 1.0, SOFTMAX_SCALE, ws, plan.workspace_bytes, out)
        if good:
            mla.mla_decode_status(ws)
        else:
            with pytest.raises(mla.MlaError) as err:
                mla.mla_decode_status(ws)
            assert err.value.status == mla.MLA_ERR_INVALID_ARG
    out, lse, _ = _run(inp, pool, False, **kw)
    assert_parity(out, lse, *_oracle(inp, False))


@pytest.mark.parametrize("kind", KINDS)
def test_plan_data_that_does_not_fit_is_reported(kind):
    # The plan's arrays of another call, or overwritten: nothing outside the batch, its
    # pages and the workspace is read or written, and the status says so.
    inp, pool, offsets, pl = _case(kind, 12, 1, [8], [4096], [200] * 8, 4)
    plan = mla.mla_shared_plan(inp.kv_lens.tolist(), offsets, pl, 12, 1, cache_kind=KIND[kind], sm_count=20)
    n, info = plan.info.num_segments, plan.info
    assert info.prefix_ctas > 0
    q, kv, pt, lens = inp.q.cuda(), pool.cuda(), inp.page_table.cuda(), inp.kv_lens.to(torch.int32).cuda()
    ws = torch.zeros(plan.workspace_bytes + 4096, dtype=torch.uint8, device="cuda")
    out = torch.full((9, 1, 12, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    FIRST, ROWS, IN_REQ, REQUEST, KEY0, LEN, SPLITS, CHUNK = range(8)
    last = n - 1  # a suffix; segment 0 is a prefix
    bad = [(last, REQUEST, 8), (last, REQUEST, -1), (last, FIRST, 96), (last, FIRST, -1), (last, ROWS, 97), (last, ROWS, 0), (last, IN_REQ, 5),
           (last, IN_REQ, -1), (last, KEY0, 16), (last, KEY0, -32), (last, SPLITS, 0), (last, CHUNK, 100), (0, REQUEST, 8), (0, FIRST, 90),
           (0, LEN, 1 << 20), (0, KEY0, 1 << 30), (0, SPLITS, 0), (0, ROWS, 1000)]
    for seg, field, value in [(None, None, None)] + bad:
        data = plan.data.copy()
        if seg is not None:
            data[8 * seg + field] = value
        ws[:plan.workspace_bytes].zero_()
        mla.mla_decode_shared(q, kv, kv.shape[0], pt, pt.shape[1], lens, plan, torch.from_numpy(data).cuda(), 8, 1, 12, False, 1.0, 1.0,
                              SOFTMAX_SCALE, ws, plan.workspace_bytes, out)
        if seg is None:
            mla.mla_decode_status(ws)
            continue
        torch.cuda.synchronize()
        code = int(ws[:4].view(torch.int32))
        assert code == mla.MLA_ERR_INVALID_ARG, (seg, field, value)
    # Numbers of partials: at most the workspace's slots are merged.
    data = plan.data.copy()
    data[8 * n:8 * n + 16] = 1 << 20
    ws[:plan.workspace_bytes].zero_()
    mla.mla_decode_shared(q, kv, kv.shape[0], pt, pt.shape[1], lens, plan, torch.from_numpy(data).cuda(), 8, 1, 12, False, 1.0, 1.0,
                          SOFTMAX_SCALE, ws, plan.workspace_bytes, out)
    torch.cuda.synchronize()
    assert (out[8] == 7.0).all() and (ws[plan.workspace_bytes:] == 0).all()
    # One request's arrays behind a call for eight.
    small = mla.mla_shared_plan([300], [0, 1], [0], 12, 1, cache_kind=KIND[kind])
    data = np.resize(small.data, plan.data.shape)
    mla.mla_decode_shared(q, kv, kv.shape[0], pt, pt.shape[1], lens, plan, torch.from_numpy(data).cuda(), 8, 1, 12, False, 1.0, 1.0,
                          SOFTMAX_SCALE, ws, plan.workspace_bytes, out)
    with pytest.raises(mla.MlaError):
        mla.mla_decode_status(ws)
    assert (out[8] == 7.0).all() and (ws[plan.workspace_bytes:] == 0).all()


# Every row group of the segments' kernels: heads, q_len, group size, suffix.
WIDTHS = {16: (12, 1, 1, 300), 32: (12, 2, 1, 300), 48: (12, 1, 4, 300), 96: (12, 8, 1, 300), "two": (12, 1, 8, 9000)}
ROLES = [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("kind,width", [(k, w) for k in KINDS for w in WIDTHS if k != "bf16" or w in (16, 32)])
def test_expired_waits_end_the_call(kind, width):
    heads, q_len, size, suffix = WIDTHS[width]
    inp, pool, offsets, pl = _case(kind, heads, q_len, [size], [6400], [suffix] * size, 8)
    kw = dict(group_offsets=offsets, prefix_lens=pl, sm_count=4)  # few CTAs, many tiles each
    info = mla.mla_shared_plan(inp.kv_lens.tolist(), offsets, pl, heads, q_len, causal=True, cache_kind=KIND[kind], sm_count=4).info
    assert (info.prefix_nr, info.suffix_nr) == ((96, 16) if width == "two" else (width, width if width != 32 or kind != "bf16" else info.suffix_nr))
    ref = _oracle(inp, True)
    for role in ROLES:
        if role == 4 and (kind == "bf16" or width == 16):
            continue  # P^T lives in the KV stages: no such wait
        mla.mla_debug_set_expire(role, 0 if role == 5 else 2)
        try:
            with pytest.raises(mla.MlaError) as err:
                _run(inp, pool, True, **kw)
            assert err.value.status == mla.MLA_ERR_TIMEOUT, role
        finally:
            mla.mla_debug_set_expire(-1)
        out, lse, _ = _run(inp, pool, True, **kw)
        assert_parity(out, lse, *ref, what=f"after role {role}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("suffix", [40, 9000])
def test_graph_replays_on_another_stream(kind, suffix):
    inp, pool, offsets, pl = _case(kind, 12, 1, [8], [4096], [suffix] * 8, 9)
    plan = mla.mla_shared_plan(inp.kv_lens.tolist(), offsets, pl, 12, 1, cache_kind=KIND[kind], sm_count=20)
    assert plan.info.prefix_ctas > 0
    data, lens = torch.from_numpy(plan.data).cuda(), inp.kv_lens.to(torch.int32).cuda()
    q, kv, pt = inp.q.cuda(), pool.cuda(), inp.page_table.cuda()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros(8, 1, 12, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 1, 12, device="cuda")
    args = (q, kv, kv.shape[0], pt, pt.shape[1], lens, plan, data, 8, 1, 12, False, 1.0, 1.0, SOFTMAX_SCALE, ws, plan.workspace_bytes, out, lse)
    mla.mla_decode_shared(*args)
    first = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):  # calls that follow each other in one workspace
            mla.mla_decode_shared(*args)
    for _ in range(20):
        out.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    mla.mla_decode_status(ws)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    q.copy_(q.flip(2))  # the heads in the opposite order
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0].flip(2)) and torch.equal(lse, first[1].flip(2))
    assert_parity(first[0], first[1], *_oracle(inp, False))


def test_decode_refuses_what_has_no_shared_form():
    inp, pool, offsets, pl = _case("fp8", 12, 1, [2], [64], [100, 5], 7)
    for kw in (dict(kv_bounds=np.array([[0, 5], [0, 5]])), dict(block_idx=np.array([[0], [0]])), dict(persistent_ctas=4), dict(use_items=True), dict(target_ctas=4),
               dict(kv_split=2)):
        with pytest.raises(ValueError):
            _run(inp, pool, False, group_offsets=offsets, prefix_lens=pl, **kw)
    with pytest.raises(ValueError):
        _run(inp, pool, False, group_offsets=offsets)


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    rng = np.random.default_rng(seed)
    kind = KINDS[seed % 3]
    heads, q_len = int(rng.choice([1, 4, 8, 12, 16, 33])), int(rng.choice([1, 1, 2, 3, 8]))
    sizes = [int(n) for n in rng.integers(1, 9, rng.integers(1, 4))]
    prefixes = [int(p) * 32 for p in rng.integers(0, 60, len(sizes))]
    causal = bool(rng.integers(0, 2))
    suffixes = [int(n) for n in rng.integers(q_len, 700, sum(sizes))]
    inp, pool, offsets, pl = _case(kind, heads, q_len, sizes, prefixes, suffixes, 100 + seed)
    ql = None if rng.random() < 0.6 else rng.integers(1, q_len + 1, sum(sizes)).tolist()
    sinks = None if rng.random() < 0.6 else rng.standard_normal(heads).astype(np.float32)
    out, lse, _ = _run(inp, pool, causal, group_offsets=offsets, prefix_lens=pl, query_lens=ql, sinks=sinks, sm_count=int(rng.choice([3, 40, 152])))
    ref, ref_lse = _oracle(inp, causal, query_lens=ql, sinks=sinks)
    empty = np.isinf(ref_lse)
    l = lse.cpu().numpy().reshape(ref_lse.shape)
    assert (np.isinf(l) == empty).all()
    assert_parity(out, torch.from_numpy(np.where(empty, 0.0, l)), ref, np.where(empty, 0.0, ref_lse), f"{kind} {heads} {q_len} {sizes} {prefixes}")
