"""GPU: a decode over shared prefixes gives the same bits every time, whatever the
workspace held before and whatever else the GPU does."""
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


@pytest.mark.parametrize("kind", [mla.CACHE_FP8, mla.CACHE_BF16, mla.CACHE_FP4])
@pytest.mark.parametrize("batch,q_len,prefix,own,sms", [(4, 1, 1024, 23, 152), (16, 1, 16384, 2001, 152), (8, 8, 4096, 517, 20), (15, 1, 8192, 700, 152)])
def test_the_same_bits(kind, batch, q_len, prefix, own, sms):
    heads, g = 12, torch.Generator().manual_seed(batch)
    each, shared = (own + 31) // 32, prefix // 32
    pages = shared + batch * each
    if kind == mla.CACHE_FP4:
        pool = torch.randint(0, 256, (pages, mla.FP4_PAGE_BYTES), generator=g, dtype=torch.uint8)
        pool[:, 8192:8704] &= 7
        pool[:, 8704:] = (torch.randn(pages, 2048, generator=g) * 0.5).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        pool = torch.randn(pages, 32, 576, generator=g) * 0.5
        pool = pool.bfloat16() if kind == mla.CACHE_BF16 else pool.to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(batch, q_len, heads, 576, generator=g)
    q = (q.bfloat16() if kind == mla.CACHE_BF16 else q.to(torch.float8_e4m3fn).view(torch.uint8)).cuda()
    order = torch.randperm(pages, generator=g).int()
    table = torch.cat([order[:shared].expand(batch, -1), order[shared:].reshape(batch, each)], 1).contiguous().cuda()
    lens = [prefix + own - 5 * b % 16 for b in range(batch)]
    plan = mla.mla_shared_plan(lens, [0, batch], [prefix], heads, q_len, causal=q_len > 1, cache_kind=kind, sm_count=sms)
    data, lens_d, pool = torch.from_numpy(plan.data).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), pool.cuda()
    side, noise = torch.cuda.Stream(), torch.rand(1 << 24, device="cuda")
    first = None
    for turn in range(12):
        ws = torch.full((plan.workspace_bytes,), [0, 255, 127][turn % 3], dtype=torch.uint8, device="cuda")  # (255: NaN)
        mla.mla_decode_workspace_init(ws, plan.workspace_bytes)
        out = torch.empty(batch, q_len, heads, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(batch, q_len, heads, device="cuda")
        torch.cuda.synchronize()
        if turn % 2:
            with torch.cuda.stream(side):
                for _ in range(5):
                    noise.mul_(1.0)
        mla.mla_decode_shared(q, pool, pages, table, table.shape[1], lens_d, plan, data, batch, q_len, heads, q_len > 1, 1.0, 1.0, SOFTMAX_SCALE, ws,
                              plan.workspace_bytes, out, lse)
        mla.mla_decode_status(ws)
        torch.cuda.synchronize()
        if first is None:
            first = (out, lse)
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse, first[1])
    assert torch.isfinite(first[1]).all()


@pytest.mark.parametrize("kind", [mla.CACHE_FP8, mla.CACHE_BF16, mla.CACHE_FP4])
def test_two_launches_read_what_was_written_just_before(kind):
    # The second launch starts before the first one ends, on SMs that the first leaves free
    # and that have read other page tables, lengths and queries before.
    heads, g = 12, torch.Generator().manual_seed(7)
    batch, prefix, own, sms = (8, 16384, 9000, 152) if kind != mla.CACHE_BF16 else (8, 6400, 9000, 4)
    each, shared = (own + 31) // 32, prefix // 32
    pages = shared + batch * each
    if kind == mla.CACHE_FP4:
        pool = torch.randint(0, 256, (pages, mla.FP4_PAGE_BYTES), generator=g, dtype=torch.uint8)
        pool[:, 8192:8704] &= 7
        pool[:, 8704:] = (torch.randn(pages, 2048, generator=g) * 0.5).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        pool = torch.randn(pages, 32, 576, generator=g) * 0.5
        pool = pool.bfloat16() if kind == mla.CACHE_BF16 else pool.to(torch.float8_e4m3fn).view(torch.uint8)
    pool = pool.cuda()
    lens = [prefix + own - 5 * b for b in range(batch)]
    plan = mla.mla_shared_plan(lens, [0, batch], [prefix], heads, 1, cache_kind=kind, sm_count=sms)
    assert plan.info.prefix_ctas > 0 and plan.info.prefix_nr != plan.info.suffix_nr
    data = torch.from_numpy(plan.data).cuda()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(batch, 1, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(batch, 1, heads, device="cuda")

    def variant(shift):
        q = torch.randn(batch, 1, heads, 576, generator=g)
        q = q.bfloat16() if kind == mla.CACHE_BF16 else q.to(torch.float8_e4m3fn).view(torch.uint8)
        order = torch.randperm(pages, generator=g).int()
        table = torch.cat([order[:shared].expand(batch, -1), order[shared:].reshape(batch, each)], 1).contiguous()
        return [q.cuda(), table.cuda(), torch.tensor([n - shift for n in lens], dtype=torch.int32).cuda()]

    variants = [variant(0), variant(7), variant(19)]
    current = [t.clone() for t in variants[0]]

    def run():
        mla.mla_decode_shared(current[0], pool, pages, current[1], current[1].shape[1], current[2], plan, data, batch, 1, heads, False, 1.0, 1.0,
                              SOFTMAX_SCALE, ws, plan.workspace_bytes, out, lse)

    want = []
    for v in variants:
        for c, x in zip(current, v):
            c.copy_(x)
        torch.cuda.synchronize()
        run()
        mla.mla_decode_status(ws)
        want.append((out.clone(), lse.clone()))
    assert not torch.equal(want[0][1], want[1][1])
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for turn in range(120):
        v, (o, s) = variants[turn % 3], want[turn % 3]
        for c, x in zip(current, v):
            c.copy_(x)
        run()
        wrong += (out.view(torch.int16) != o.view(torch.int16)).sum() + (lse != s).sum()
    assert int(wrong) == 0
    mla.mla_decode_status(ws)
