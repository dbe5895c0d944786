"""GPU: decode over the 4-bit cache.

Every value of a 4-bit page times its block's scale is an E4M3 number, so the
kernel's tensor-core operands are those of the E4M3 cache that the pages expand
to: with the same plan its outputs equal mla_decode's, bit for bit from 17 rows
on.  Up to 16 rows only the row sums differ, which are added
in another order: at most 128 tiles of a split, one after the other, then a tree
over 128 tokens, 136 roundings on either side, 2 * 136 * 2^-24 < 2^-15 relative
(and as much, absolute, in the natural logarithm).  The oracle runs on that
expanded cache (expanded by oracle.cache, not by the kernel under test), with the
decode tests' tolerances.
"""
import numpy as np
import pytest
import torch

import oracle
import split_kv_mla_paged_gb300 as mla
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE
from fp4_testutil import equal_outputs as _equal, fp4_case as _case, same_outputs as _same
from mla_testutil import assert_parity

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _decode(inp, kv, causal, **kw):
    out = mla.decode(inp.q.cuda(), kv.cuda(), inp.page_table.cuda(), inp.kv_lens, num_heads=inp.num_heads, q_len=inp.q_len,
                     causal=causal, softmax_scale=SOFTMAX_SCALE, want_f32=True, **kw)
    torch.cuda.synchronize()
    return out


SHAPES = [
    # batch, heads, q_len, lens, causal
    (1, 12, 1, [1], False),
    (1, 1, 1, [31], False),
    (1, 12, 1, [33], False),
    (3, 12, 1, [128, 129, 127], False),
    (2, 12, 1, [4096, 1], False),
    (2, 16, 1, [1000, 5000], False),
    (1, 12, 2, [2, ], True),
    (2, 12, 2, [515, 2049], True),   # 24 rows
    (2, 32, 1, [700, 64], False),
    (2, 12, 4, [4, 3333], True),     # 48 rows
    (1, 48, 1, [1500], False),
    (2, 12, 8, [8, 1000], True),     # 96 rows: two groups
    (1, 33, 3, [300], True),         # 99 rows: three groups of 33
    (1, 128, 8, [260], True),        # 1024 rows
    (5, 12, 1, [20000, 9000, 333, 64, 2], False),
]


@pytest.mark.parametrize("batch, heads, q_len, lens, causal", SHAPES)
def test_matches_oracle(batch, heads, q_len, lens, causal):
    inp, pool = _case(batch, heads, q_len, lens, seed=50 + heads + sum(lens) % 7)
    out, lse, _ = _decode(inp, pool, causal, kv_scale=0.5, q_scale=2.0)
    ref_o, ref_l = oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=q_len, num_heads=heads, causal=causal,
                                      softmax_scale=SOFTMAX_SCALE, kv_scale=0.5, q_scale=2.0)
    assert_parity(out, lse, ref_o, ref_l)


@pytest.mark.parametrize("batch, heads, q_len, lens, causal", [s for s in SHAPES if s[1] * s[2] <= 48])
@pytest.mark.parametrize("target", [0, 7, 40])
def test_equals_the_e4m3_decode(batch, heads, q_len, lens, causal, target):
    inp, pool = _case(batch, heads, q_len, lens, seed=60 + heads)
    plan = mla.mla_decode_plan(lens, heads, q_len, sm_count=152, target_ctas=target)
    _equal(_decode(inp, pool, causal, plan=plan), _decode(inp, inp.kv, causal, plan=plan), heads * q_len)


def test_long_request_over_every_sm():
    inp, pool = _case(1, 12, 1, [70001], seed=71)
    got = _decode(inp, pool, False)
    _equal(got, _decode(inp, inp.kv, False), 12)
    ref_o, ref_l = oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=1, num_heads=12, causal=False,
                                      softmax_scale=SOFTMAX_SCALE)
    assert_parity(got[0], got[1], ref_o, ref_l)


@pytest.mark.parametrize("heads, q_len", [(12, 1), (12, 2), (12, 4), (12, 8)])
def test_options_match_oracle(heads, q_len):
    lens = [900, 64, 3000]
    inp, pool = _case(3, heads, q_len, lens, seed=80 + q_len)
    sinks = np.linspace(-2, 3, heads).astype(np.float32)
    qlens = [q_len, 1, max(1, q_len - 1)]
    bounds = [[100, 777], [0, 10], [0, 3000]]
    for kw in (dict(sinks=sinks), dict(output_scale=0.25, device_scales=True), dict(query_lens=qlens),
               dict(kv_bounds=bounds), dict(kv_bounds=[[5, 5], [64, 90], [2990, 3000]], sinks=sinks),
               dict(use_items=True), dict(use_items=True, kv_bounds=bounds)):
        causal = q_len > 1
        out, lse, f32 = _decode(inp, pool, causal, **kw)
        kw = {k: (np.asarray(v, np.int32) if k in ("query_lens", "kv_bounds") else v) for k, v in kw.items()
              if k not in ("use_items", "device_scales")}
        ref_o, ref_l = oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=q_len, num_heads=heads,
                                          causal=causal, softmax_scale=SOFTMAX_SCALE, **kw)
        empty = np.isneginf(ref_l).reshape(-1)
        got_l = lse.cpu().numpy().reshape(-1)
        assert np.array_equal(np.isneginf(got_l), empty)
        o = out.float().cpu().numpy().reshape(ref_o.shape)
        assert (o[empty] == 0).all()
        lse_f = lse.clone().reshape(-1)
        lse_f[torch.from_numpy(empty).cuda()] = 0
        assert_parity(out, lse_f, ref_o, np.where(empty, 0.0, ref_l.reshape(-1)), what=str(kw))


@pytest.mark.parametrize("heads, q_len", [(12, 1), (12, 4), (12, 8)])
def test_selected_pages(heads, q_len):
    lens = [4000, 70, 9000]
    inp, pool = _case(3, heads, q_len, lens, seed=90 + q_len)
    rng = np.random.default_rng(3)
    topk = 37
    sel = np.full((3, topk), -1, np.int32)
    for b, n in enumerate(lens):
        pages = (n + 31) // 32
        k = min(topk - 2, pages)
        sel[b, :k] = np.sort(rng.permutation(pages)[:k])
        sel[b, k - 1] = pages - 1
        sel[b, :k] = np.sort(sel[b, :k])
    sel[2, 10] = -1  # an unused slot in between
    out, lse, f32 = _decode(inp, pool, q_len > 1, block_idx=torch.from_numpy(sel))
    ref_o, ref_l = oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=q_len, num_heads=heads, causal=q_len > 1,
                                      softmax_scale=SOFTMAX_SCALE, block_idx=sel)
    assert_parity(out, lse, ref_o, ref_l)
    if heads * q_len <= 48:
        _equal((out, lse, f32), _decode(inp, inp.kv, q_len > 1, block_idx=torch.from_numpy(sel)), heads * q_len)


def test_nans_reach_only_the_rows_that_see_them():
    inp, pool = _case(2, 12, 1, [200, 200], seed=95)
    want = _decode(inp, pool, False)
    page = int(inp.page_table[1, 2])
    pool[page, 8192 + 32 * 4 + 7] = 15  # block 4 of request 1's token 71
    got = _decode(inp, pool, False)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    # Behind a key window they have no effect at all.
    bounds = [[0, 200], [72, 200]]
    clean = _decode(inp, _case(2, 12, 1, [200, 200], seed=95)[1], False, kv_bounds=bounds)
    _same(_decode(inp, pool, False, kv_bounds=bounds), clean)


def test_bad_page_id_and_bad_plan_are_reported():
    inp, pool = _case(1, 12, 1, [6000], seed=96)
    inp.page_table[0, 40] = inp.num_pages + 9
    with pytest.raises(mla.MlaError) as e:
        _decode(inp, pool, False)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG
    inp, pool = _case(1, 12, 1, [6000], seed=96)
    plan = mla.mla_decode_plan([3000], 12, 1, sm_count=152)
    with pytest.raises(mla.MlaError) as e:
        _decode(inp, pool, False, plan=plan)
    assert e.value.status == mla.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("q_len", [1, 2, 4, 8])  # 16, 32, 48 and 96-row CTAs
@pytest.mark.parametrize("role", range(6))
def test_expired_waits_end_the_call_with_a_status(role, q_len):
    # The hook makes one wait read as expired without any stall; the kernel
    # stops its other roles, drains its copies and MMAs and returns.
    inp, pool = _case(1, 12, q_len, [5000], seed=97)
    want = _decode(inp, pool, q_len > 1)
    for tile in (0, 3):
        mla.mla_debug_set_expire(role, tile)
        try:
            if role == 4 and q_len == 1 or role == 5 and tile > 0:
                _same(_decode(inp, pool, q_len > 1, target_ctas=2), _decode(inp, pool, q_len > 1, target_ctas=2))
            else:
                with pytest.raises(mla.MlaError) as e:
                    _decode(inp, pool, q_len > 1, target_ctas=2)
                assert e.value.status == mla.MLA_ERR_TIMEOUT
        finally:
            mla.mla_debug_set_expire(-1)
    _same(want, _decode(inp, pool, q_len > 1))


def test_graphs_and_streams():
    inp, pool = _case(4, 12, 1, [3000, 700, 5000, 33], seed=98)
    want = _decode(inp, pool, False)
    plan = mla.mla_decode_plan(inp.kv_lens.tolist(), 12, 1, sm_count=152)
    d = [t.cuda() for t in (inp.q, pool, inp.page_table, inp.kv_lens, torch.from_numpy(plan.splits), torch.from_numpy(plan.chunks))]
    size = mla.mla_decode_workspace_size(4, 1, 12, plan.max_splits)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mla.mla_decode_workspace_init(ws, size)
    out = torch.zeros(4, 1, 12, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(4, 1, 12, device="cuda")

    def call(stream=None):
        mla.mla_decode_fp4(d[0], d[1], inp.num_pages, d[2], inp.max_pages, d[3], d[4], d[5], plan.max_splits, plan.kv_split, 4, 1, 12,
                           False, 1.0, 1.0, SOFTMAX_SCALE, ws, size, out, lse, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    call(side)
    side.synchronize()
    assert torch.equal(out, want[0])
    mla.mla_decode_status(ws)


def test_phases_are_the_whole_call():
    inp, pool = _case(2, 12, 1, [9000, 500], seed=99)
    whole = _decode(inp, pool, False)
    plan = mla.mla_decode_plan([9000, 500], 12, 1, sm_count=152)
    d = [t.cuda() for t in (inp.q, pool, inp.page_table, inp.kv_lens, torch.from_numpy(plan.splits), torch.from_numpy(plan.chunks))]
    size = mla.mla_decode_workspace_size(2, 1, 12, plan.max_splits)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mla.mla_decode_workspace_init(ws, size)
    out = torch.zeros(2, 1, 12, 512, dtype=torch.bfloat16, device="cuda")
    for phase in (mla.PHASE_SPLIT, mla.PHASE_MERGE):
        mla.mla_decode_fp4(d[0], d[1], inp.num_pages, d[2], inp.max_pages, d[3], d[4], d[5], plan.max_splits, plan.kv_split, 2, 1, 12,
                           False, 1.0, 1.0, SOFTMAX_SCALE, ws, size, out, phases=phase)
    torch.cuda.synchronize()
    assert torch.equal(out, whole[0])


def test_prologue_pages_and_decode_run_together():
    """A request is written by the prologue, forked, extended by its forks,
    compacted, and decoded: each step against the oracle's cache."""
    g = torch.Generator().manual_seed(5)
    heads, total = 12, 64
    pool_h, pool = mla.PagePool(total), mla.fp4_pool(total)
    host = pool.cpu().numpy()
    scratch = pool_h.alloc(7)                       # pages below the request, freed later
    first = pool_h.alloc(4)
    n0 = 3 * 32 + 17
    ang = torch.rand(256, 32, generator=g, dtype=torch.float64) * 6.28
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    kv_scale = 0.5

    def write(tables, req, pos, rows):
        width = max(len(t) for t in tables)
        table = torch.full((len(tables), width), -1, dtype=torch.int32)
        for k, t in enumerate(tables):
            table[k, :len(t)] = torch.from_numpy(np.asarray(t, np.int32))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.mla_prologue(len(pos), positions=torch.tensor(pos, dtype=torch.int32).cuda(), cos_sin=cs.cuda(), kv_rows=rows.cuda(),
                         req_idx=torch.tensor(req, dtype=torch.int32).cuda(), page_table=table.cuda(), max_pages_per_req=width,
                         batch=len(tables), kv_pages=pool, num_pages=total, cache_kind=mla.CACHE_FP4, kv_scale=kv_scale, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        y = cache.rotate(rows.double().numpy(), cs.numpy(), pos, False)
        parts = cache.fp4_encode_rows(y / kv_scale)
        for k in range(len(pos)):
            cache.fp4_put(host, tables[req[k]][pos[k] // 32], pos[k] % 32, [q[k] for q in parts])

    def decode(tables, lens):
        width = max(len(t) for t in tables)
        table = torch.full((len(tables), width), -1, dtype=torch.int32)
        for k, t in enumerate(tables):
            table[k, :len(t)] = torch.from_numpy(np.asarray(t, np.int32))
        q = torch.randn(len(tables), 1, heads, 576, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
        out, lse, _ = mla.decode(q.cuda(), pool, table.cuda(), lens, num_heads=heads, q_len=1, causal=False,
                                 softmax_scale=SOFTMAX_SCALE, kv_scale=kv_scale)
        # The oracle reads the 4-bit pool as the device holds it; that it is the
        # host model's is checked on its values (rotated values may round to
        # neighbouring E4M3 codes: fp32 against 64 bits).
        dev = cache.fp4_decode(pool.cpu().numpy())
        mine = cache.fp4_decode(host)
        for k, t in enumerate(tables):
            rows = dev[np.asarray(t)].reshape(-1, 576)[:lens[k]], mine[np.asarray(t)].reshape(-1, 576)[:lens[k]]
            assert np.array_equal(rows[0][:, :512], rows[1][:, :512])
            assert (np.abs(rows[0] - rows[1]) <= np.abs(rows[1]) * 2.0 ** -3 + 2.0 ** -9).all()
        ref_o, ref_l = oracle.decode_rows(q, torch.from_numpy(cache.e4m3_codes(dev)), table, torch.tensor(lens, dtype=torch.int32),
                                          q_len=1, num_heads=heads, causal=False, softmax_scale=SOFTMAX_SCALE, kv_scale=kv_scale)
        assert_parity(out, lse, ref_o, ref_l)

    write([first], [0] * n0, list(range(n0)), torch.randn(n0, 576, generator=g).bfloat16())
    decode([first], [n0])
    forks, src, dst, rows = pool_h.fork(first, n0, 2)
    mla.copy_pages(pool, pool, src, dst, rows)
    for s, d, r in zip(src, dst, rows):
        for a, b, w in ((0, 8192, 256), (8704, 10752, 64)):
            host[d, a:a + r * w] = host[s, a:a + r * w]
        host[d, 8192:8704].reshape(16, 32)[:, :r] = host[s, 8192:8704].reshape(16, 32)[:, :r]
    tables = [first, forks[0], forks[1]]
    write(tables, [0, 1, 2, 1, 2], [n0, n0, n0, n0 + 1, n0 + 1], torch.randn(5, 576, generator=g).bfloat16())
    decode(tables, [n0 + 1, n0 + 2, n0 + 2])
    pool_h.release(scratch)
    src, dst, page_map = pool_h.compact()
    assert len(src) > 0
    mla.copy_pages(pool, pool, src, dst)
    host[dst] = host[src]
    t = torch.tensor(np.stack(tables), dtype=torch.int32, device="cuda")
    mla.mla_pages_remap(t, t.numel(), torch.from_numpy(page_map).cuda(), total)
    torch.cuda.synchronize()
    tables = list(t.cpu().numpy())
    assert max(x.max() for x in tables) < total - pool_h.free_pages
    decode(tables, [n0 + 1, n0 + 2, n0 + 2])
