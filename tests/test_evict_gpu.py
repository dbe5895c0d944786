"""GPU: eviction (mla_evict_select, mla_rows_move, evict) against plain numpy.

Positions, copied weights and copied bytes: everything has to be equal."""
import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _plain(weights, length, keep, first, last):
    """Positions that stay, ascending."""
    w = weights[:length].astype(np.float64) + 0.0
    rank = np.where(np.isnan(w), -np.inf, w)
    guard = np.zeros(length, bool)
    guard[:first] = True
    guard[max(0, length - last):] = True
    # lexsort's last key counts most: protected, then not a NaN, then the weight, then the position.
    order = np.lexsort((np.arange(length), -np.where(guard, 0.0, rank), np.isnan(w) & ~guard, ~guard))
    return np.sort(order[:min(length, keep)]).astype(np.int32)


def _select(weights, lens, keep, first=0, last=0, room=None):
    batch = len(lens)
    room = max(1, max(keep)) if room is None else room
    kept = torch.full((batch, room), -7, dtype=torch.int32, device="cuda")
    new_w = torch.full((batch, room), -7.0, device="cuda")
    out = torch.full((batch,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mla.mla_evict_select(torch.from_numpy(weights).cuda(), i32(lens), i32(keep), kept, out, first=first, last=last, new_weights=new_w,
                         status=status)
    return kept.cpu().numpy(), out.cpu().numpy(), new_w.cpu().numpy(), int(status)


def _check(weights, lens, keep, first=0, last=0):
    kept, out, new_w, status = _select(weights, lens, keep, first, last)
    assert status == 0
    for b, n in enumerate(lens):
        ref = _plain(weights[b], n, keep[b], first, last)
        k = len(ref)
        assert out[b] == k
        assert np.array_equal(kept[b, :k], ref)
        assert np.array_equal(new_w[b, :k], weights[b][ref], equal_nan=True)
        assert (kept[b, k:] == -7).all() and (new_w[b, k:] == -7.0).all()


def _weights(batch, width, seed, kind):
    rng = np.random.default_rng(seed)
    w = np.exp(2.5 * rng.standard_normal((batch, width)) - 8.0).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, (batch, width)).astype(np.float32) / 8
    elif kind == "equal":
        w[:] = 0.0
    elif kind == "wild":
        w = rng.standard_normal((batch, width)).astype(np.float32)
        for v in (np.nan, np.inf, -np.inf, -0.0, 0.0, 1e-42, -1e-42, np.finfo(np.float32).min):
            w[rng.random((batch, width)) < 0.05] = v
    return w


@pytest.mark.parametrize("kind", ["tail", "ties", "equal", "wild"])
@pytest.mark.parametrize("lens,keep", [([1], [1]), ([0, 1, 2], [5, 0, 1]), ([31, 32, 33, 100], [7, 32, 40, 99]),
                                       ([1000, 1024, 1025, 8192], [1, 1000, 512, 8191]), ([8193, 300], [1000, 200]),
                                       ([20000, 0, 65537], [4096, 3, 20001])])
def test_select(lens, keep, kind):
    _check(_weights(len(lens), max(lens) + 3, sum(lens), kind), lens, keep)


@pytest.mark.parametrize("first,last", [(4, 0), (0, 64), (4, 64), (300, 300), (5000, 0), (0, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_protected_keys(first, last):
    lens, keep = [1000, 2111, 64, 3], [500, 700, 30, 3]
    _check(_weights(4, 2111, 9, "tail"), lens, keep, first, last)
    _check(_weights(4, 2111, 9, "wild"), lens, keep, first, last)


def test_long_requests_in_larger_clusters():
    w = _weights(2, 1 << 20, 21, "tail")
    w[0, ::7] = 0.0
    _check(w, [1 << 20, 700001], [131072, 650000], 4, 4096)
    _check(_weights(1, 400000, 22, "ties"), [399999], [123456])


@pytest.mark.parametrize("lens,keep", [([3000, 200, 8192], [1500, 120, 5000]), ([20000, 9000], [11000, 3000]), ([400000], [170000])])
@pytest.mark.parametrize("low", [np.nan, -np.inf, 0.0])
def test_ties_of_the_lowest_weights(lens, keep, low):
    # The last kept one is among many equal lowest weights (NaNs rank below all).
    w = _weights(len(lens), max(lens) + 1, 31, "tail")
    w[np.random.default_rng(5).random(w.shape) < 0.8] = low
    _check(w, lens, keep, 3, 17)


def test_bad_lengths_keep_nothing():
    w = _weights(4, 50, 3, "tail")
    kept, out, _, status = _select(w, [51, -1, 50, 50], [5, 5, -2, 5])
    assert status == mla.MLA_ERR_INVALID_ARG and out.tolist() == [0, 0, 0, 5]
    assert np.array_equal(kept[3], _plain(w[3], 50, 5, 0, 0)) and (kept[:3] == -7).all()


def test_the_width_of_kept_bounds_the_budget():
    w = _weights(2, 500, 4, "tail")
    kept, out, _, status = _select(w, [500, 80], [400, 60], room=100)
    assert status == 0 and out.tolist() == [100, 60]
    assert np.array_equal(kept[0], _plain(w[0], 500, 100, 0, 0))


KINDS = {mla.CACHE_FP8: ((32, 576), torch.uint8), mla.CACHE_BF16: ((32, 576), torch.bfloat16), mla.CACHE_FP4: ((10752,), torch.uint8)}


def _pool(kind, pages, seed):
    shape, dtype = KINDS[kind]
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (pages, 10752 if kind == mla.CACHE_FP4 else 32 * 576 * (2 if kind == mla.CACHE_BF16 else 1)), generator=g,
                        dtype=torch.uint8)
    return raw.view(dtype).view(pages, *shape) if dtype != torch.uint8 else raw.view(pages, *shape)


def _rows(kind, page_bytes):
    """A page's bytes -> its 32 rows' bytes, and back."""
    if kind != mla.CACHE_FP4:
        return page_bytes.reshape(32, -1)
    return np.concatenate([page_bytes[:8192].reshape(32, 256), page_bytes[8192:8704].reshape(16, 32).T, page_bytes[8704:].reshape(32, 64)], 1)


def _bytes(pool):
    return pool.cpu().contiguous().view(torch.uint8).numpy().reshape(pool.shape[0], -1)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("counts", [[0], [1], [33, 0, 32], [31, 7, 250, 64]])
def test_rows_move(kind, counts):
    rng = np.random.default_rng(sum(counts))
    batch, room, src_n = len(counts), max(counts) + 5, 12
    src, dst = _pool(kind, batch * src_n, 1), _pool(kind, 40, 2)
    src_table = rng.permutation(batch * src_n).reshape(batch, src_n).astype(np.int32)
    width = (room + 31) // 32
    dst_table = rng.permutation(40)[:batch * width].reshape(batch, width).astype(np.int32)
    kept = np.full((batch, room), -1, np.int32)
    for b, n in enumerate(counts):
        kept[b, :n] = np.sort(rng.choice(src_n * 32, n, replace=False))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dst.cuda()
    cuda = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    mla.mla_rows_move(src.cuda(), src.shape[0], cuda(src_table), out, 40, cuda(dst_table), cuda(kept), cuda(counts), cache_kind=kind,
                      status=status)
    assert int(status) == 0
    s, got = _bytes(src), _bytes(out)
    want = [_rows(kind, p).copy() for p in _bytes(dst)]
    for b, n in enumerate(counts):
        for i in range(n):
            want[dst_table[b, i // 32]][i % 32] = _rows(kind, s[src_table[b, kept[b, i] // 32]])[kept[b, i] % 32]
    for p in range(40):
        assert np.array_equal(_rows(kind, got[p]), want[p])


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_rows_move_reports_what_is_out_of_range(kind):
    src, dst = _pool(kind, 4, 1), _pool(kind, 4, 2)
    base = dict(src=[[0, 1]], dst=[[2, 3]], kept=[[0, 40, 63]], counts=[3])
    for bad in (dict(src=[[0, 4]]), dict(src=[[0, -1]]), dict(dst=[[4, 3]]), dict(dst=[[-1, 3]]), dict(kept=[[0, 64, 63]]),
                dict(kept=[[0, -1, 63]]), dict(counts=[4]), dict(counts=[-1])):
        c = {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in {**base, **bad}.items()}
        status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), dst.cuda()
        mla.mla_rows_move(src.cuda(), 4, c["src"], out, 4, c["dst"], c["kept"], c["counts"], cache_kind=kind, status=status)
        assert int(status) == mla.MLA_ERR_INVALID_ARG, bad
        if "counts" in bad:
            assert np.array_equal(_bytes(out), _bytes(dst))


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_evict_through_the_pool(kind):
    lens, keep = [100, 0, 33, 700], [40, 10, 33, 200]
    pool = mla.PagePool(64)
    lists = [pool.alloc((n + 31) // 32) for n in lens]
    shared = pool.fork(lists[3], 700, 1)[0][0]  # another request holds the last one's full pages
    data = _pool(kind, 64, 5)
    dev = data.cuda()
    w = _weights(4, 700, 6, "tail")
    new_lists, new_lens, new_w = mla.evict(pool, dev, lists, lens, torch.from_numpy(w).cuda(), keep, first=2, last=5)
    s, got = _bytes(data), _bytes(dev)
    assert new_lens.tolist() == [40, 0, 33, 200]
    for b, n in enumerate(lens):
        ref = _plain(w[b], n, keep[b], 2, 5)
        assert np.array_equal(new_w[b, :len(ref)].cpu().numpy(), w[b][ref])
        for i, pos in enumerate(ref):
            a = _rows(kind, got[new_lists[b][i // 32]])[i % 32]
            assert np.array_equal(a, _rows(kind, s[lists[b][pos // 32]])[pos % 32])
        for p in new_lists[b]:
            assert pool.references(p) == 1
    for p in shared[:21]:
        assert pool.references(p) == 1 and np.array_equal(got[p], s[p])
    assert pool.free_pages == 64 - sum((n + 31) // 32 for n in new_lens) - len(shared)
    held = pool.alloc(pool.free_pages - 3)
    with pytest.raises(mla.MlaError):
        mla.evict(pool, dev, [shared], [700], torch.from_numpy(w[3:]).cuda(), 3 * 32 + 1)
    assert pool.free_pages == 3 and len(held) > 0 and np.array_equal(_bytes(dev), got)


@pytest.mark.parametrize("kind", KINDS)
def test_refused_evictions_take_no_pages(kind):
    pool = mla.PagePool(16)
    lists = [pool.alloc(3)]
    dev = _pool(kind, 16, 5).cuda()
    w = torch.rand(1, 96, device="cuda")
    for bad, kw in ((w.double(), {}), (w.cpu(), {}), (w.t(), {}), (w, dict(first=-1)), (w, dict(last=-1))):
        with pytest.raises((ValueError, mla.MlaError)):
            mla.evict(pool, dev, lists, [90], bad, 40, **kw)
        assert pool.free_pages == 13 and all(pool.references(int(p)) == 1 for p in lists[0])


def test_another_stream_waits_for_the_current_one():
    # The zeroed outputs and the status of a call are made on the current stream.
    side = torch.cuda.Stream()
    pool = mla.PagePool(64)
    lists = [pool.alloc(20)]
    dev = _pool(mla.CACHE_FP8, 64, 5).cuda()
    w = torch.from_numpy(_weights(1, 640, 6, "tail")).cuda()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    lists, lens, new_w = mla.evict(pool, dev, lists, [640], w, 100, stream=side)
    ref = _plain(w[0].cpu().numpy(), 640, 100, 0, 0)
    assert np.array_equal(new_w[0].cpu().numpy(), w[0, ref].cpu().numpy())
    probs = torch.rand(1, 2, 64, device="cuda")
    torch.cuda._sleep(50_000_000)
    with pytest.raises(mla.MlaError):
        mla.verify_drafts(probs, torch.full((1, 1), 64, dtype=torch.int32, device="cuda"), torch.rand(1, 2, device="cuda"), stream=side.cuda_stream)
