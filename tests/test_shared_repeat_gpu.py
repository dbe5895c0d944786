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
