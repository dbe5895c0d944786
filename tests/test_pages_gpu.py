"""GPU: page copies, conversions between the E4M3 and 4-bit pools, table rewrites,
and the pool's forks and compactions run through them."""
import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build

pytestmark = pytest.mark.gpu
KINDS = {"fp8": mla.CACHE_FP8, "bf16": mla.CACHE_BF16, "fp4": mla.CACHE_FP4}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _pool(kind, pages, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "bf16":
        return torch.randn(pages, 32, 576, generator=g).bfloat16().cuda()
    shape = (pages, mla.FP4_PAGE_BYTES) if kind == "fp4" else (pages, 32, 576)
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()  # every code, NaN and rubbish scales among them


def _rows_of(pool, kind):
    """Views of a host pool's rows: list of [pages, 32, bytes] arrays."""
    p = pool.cpu()
    if kind == "fp4":
        p = p.numpy()
        return [p[:, :8192].reshape(-1, 32, 256), p[:, 8192:8704].reshape(-1, 16, 32).transpose(0, 2, 1), p[:, 8704:].reshape(-1, 32, 64)]
    return [p.view(torch.uint8).numpy().reshape(-1, 32, 576 * p.element_size())]


def _copy(src, sk, dst, dk, si, di, rows=None):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = [None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda") for x in (si, di, rows)]
    mla.mla_pages_copy(src, src.shape[0], KINDS[sk], dst, dst.shape[0], KINDS[dk], t[0], t[1], len(si), rows=t[2], status=status)
    torch.cuda.synchronize()
    return int(status.item())


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
@pytest.mark.parametrize("rows", [None, [32, 1, 0, 31, 13]])
@pytest.mark.parametrize("same", [True, False])
def test_copies_are_exact_and_leave_the_rest(kind, rows, same):
    src = _pool(kind, 23, 1)
    dst = src if same else _pool(kind, 11, 2)
    before, to = src.clone(), dst.clone()
    si, di = [22, 0, 5, 17, 5], [1, 10, 3, 9, 4]
    assert _copy(src, kind, dst, kind, si, di, rows) == 0
    want = _rows_of(to, kind)
    for got, w, s in zip(_rows_of(dst, kind), want, _rows_of(before, kind)):
        w = w.copy()
        for k in range(5):
            n = 32 if rows is None else rows[k]
            w[di[k], :n] = s[si[k], :n]
        assert np.array_equal(got, w)
    if not same:
        assert torch.equal(src, before)


def _demoted(page_rows):
    v = cache.e4m3_values()[page_rows]
    parts = list(cache.fp4_encode_rows(v))
    parts[2] = page_rows[:, 512:]  # the rope codes go over as they are, NaN signs included
    return parts


@pytest.mark.parametrize("rows", [None, [32, 1, 0, 31, 13]])
def test_demotion_bytes(rows):
    src, dst = _pool("fp8", 9, 3), _pool("fp4", 8, 4)
    # Two pages of ordinary values (random codes have a NaN in every tenth block).
    g = torch.Generator().manual_seed(5)
    src[3:5] = (torch.randn(2, 32, 576, generator=g) * torch.exp2(torch.randint(-8, 7, (2, 32, 18), generator=g).float())
                .repeat_interleave(32, dim=2)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    want = dst.cpu().numpy().copy()
    si, di = [3, 8, 0, 4, 1], [7, 0, 5, 2, 3]
    assert _copy(src, "fp8", dst, "fp4", si, di, rows) == 0
    host = src.cpu().numpy()
    for k in range(5):
        parts = _demoted(host[si[k]])
        for r in range(32 if rows is None else rows[k]):
            cache.fp4_put(want, di[k], r, [p[r] for p in parts])
    assert np.array_equal(dst.cpu().numpy(), want)


@pytest.mark.parametrize("rows", [None, [32, 1, 0, 31, 13]])
def test_promotion_is_exact(rows):
    src, dst = _pool("fp4", 9, 6), _pool("fp8", 8, 7)
    want = dst.cpu().numpy().copy()
    si, di = [3, 8, 0, 4, 1], [7, 0, 5, 2, 3]
    assert _copy(src, "fp4", dst, "fp8", si, di, rows) == 0
    host = src.cpu().numpy()
    codes = cache.e4m3_codes(cache.fp4_decode(host))
    for k in range(5):
        n = 32 if rows is None else rows[k]
        want[di[k], :n] = codes[si[k], :n]
        want[di[k], :n, 512:] = host[si[k], 8704:].reshape(32, 64)[:n]  # rope codes as they are
    got = dst.cpu().numpy()
    # NaN codes may carry a sign; everything else is equal bit for bit.
    nan = np.isnan(cache.e4m3_values()[want]) & np.isnan(cache.e4m3_values()[got])
    assert np.array_equal(got[~nan], want[~nan])
    assert np.array_equal(got[:, :, 512:], want[:, :, 512:])


def test_promote_then_demote_keeps_the_values():
    g = torch.Generator().manual_seed(8)
    fp8 = (torch.randn(6, 32, 576, generator=g) * 2).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    fp4, back, again = mla.fp4_pool(6), torch.zeros_like(fp8), mla.fp4_pool(6)
    ids = list(range(6))
    mla.copy_pages(fp8, fp4, ids, ids)
    mla.copy_pages(fp4, back, ids, ids)
    mla.copy_pages(back, again, ids, ids)
    torch.cuda.synchronize()
    a, b = cache.fp4_decode(fp4.cpu().numpy()), cache.fp4_decode(again.cpu().numpy())
    assert np.array_equal(a, b)
    assert np.array_equal(cache.e4m3_values()[back.cpu().numpy()], a)


@pytest.mark.parametrize("sk, dk", [("fp8", "fp8"), ("bf16", "bf16"), ("fp4", "fp4"), ("fp8", "fp4"), ("fp4", "fp8")])
def test_bad_entries_are_reported_and_padding_skipped(sk, dk):
    src, dst = _pool(sk, 5, 9), _pool(dk, 6, 10)
    before = dst.clone()
    assert _copy(src, sk, dst, dk, [-1, 2, -1], [0, -1, -1]) == 0
    assert torch.equal(dst, before)
    for si, di, rows in (([5], [0], None), ([0], [6], None), ([-2], [0], None), ([0], [-2], None), ([0], [1], [33]), ([0], [1], [-1])):
        assert _copy(src, sk, dst, dk, si, di, rows) == mla.MLA_ERR_INVALID_ARG
        assert torch.equal(dst, before)


def test_remap():
    g = torch.Generator().manual_seed(11)
    table = torch.randint(-1, 40, (7, 301), generator=g).int().cuda()
    m = torch.randperm(40, generator=g).int().cuda()
    want = torch.where(table >= 0, m[table.clamp(min=0).long()], table)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_pages_remap(table, table.numel(), m, 40, status)
    torch.cuda.synchronize()
    assert torch.equal(table, want) and int(status.item()) == 0
    table[3, 200] = 40
    want = torch.where((table >= 0) & (table < 40), m[table.clamp(0, 39).long()], table)
    mla.mla_pages_remap(table, table.numel(), m, 40, status)
    torch.cuda.synchronize()
    assert torch.equal(table, want) and int(status.item()) == mla.MLA_ERR_INVALID_ARG


def test_side_stream_and_capture():
    src, dst = _pool("fp8", 40, 12), mla.fp4_pool(40)
    ids = torch.arange(40, dtype=torch.int32, device="cuda")
    mla.mla_pages_copy(src, 40, mla.CACHE_FP8, dst, 40, mla.CACHE_FP4, ids, ids, 40)
    torch.cuda.synchronize()
    other, side = mla.fp4_pool(40), torch.cuda.Stream()
    torch.cuda.synchronize()
    mla.copy_pages(src, other, list(range(40)), list(range(40)), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other, dst)
    other.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.mla_pages_copy(src, 40, mla.CACHE_FP8, other, 40, mla.CACHE_FP4, ids, ids, 40)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(other, dst)
