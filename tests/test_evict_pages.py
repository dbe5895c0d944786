"""CPU: the page bookkeeping of evict, with the kernels stood in for."""
import contextlib

import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build


@pytest.fixture(autouse=True)
def moves(monkeypatch):
    """The kernels' calls as they are made, on the host; the row counts that were to move."""
    mla_build.build()
    mla.load_library()
    made = []

    def select(weights, kv_lens, keep, kept, new_lens, *, first=0, last=0, new_weights=None, status=None, stream=None):
        for b in range(kv_lens.shape[0]):
            n, k = int(kv_lens[b]), min(int(kv_lens[b]), int(keep[b]))
            pos = np.sort(np.argsort(-weights[b, :n].numpy(), kind="stable")[:k])
            kept[b, :k] = torch.from_numpy(pos.astype(np.int32))
            new_weights[b, :k] = weights[b, pos]
            new_lens[b] = k

    def move(src, src_pages, src_table, dst, dst_pages, dst_table, kept, counts, *, cache_kind, status=None, stream=None):
        made.append(counts.tolist())
        for b in range(counts.shape[0]):
            for i in range(int(counts[b])):
                pos = int(kept[b, i])
                dst[int(dst_table[b, i // 32]), i % 32] = src[int(src_table[b, pos // 32]), pos % 32]

    monkeypatch.setattr(mla, "mla_evict_select", select)
    monkeypatch.setattr(mla, "mla_rows_move", move)
    monkeypatch.setattr(mla, "_ordered", lambda stream, dev: contextlib.nullcontext())
    return made


def _data(pages):
    return torch.randint(0, 256, (pages, 32, 576), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))


def _rows(data, pages, n):
    return data[torch.from_numpy(np.asarray(pages, np.int64))].reshape(-1, 576)[:n]


def test_an_error_at_the_release_takes_and_gives_no_page():
    pool, data, w = mla.PagePool(16), _data(16), torch.rand(2, 96)
    good = pool.alloc(3)
    for bad in ([12, 13, 14], [good[0], 13, 14], good):  # not held, in part, not held so often
        with pytest.raises(mla.MlaError):
            mla.evict(pool, data, [good, bad], [96, 96], w, 40)
        assert pool.free_pages == 13 and all(pool.references(int(p)) == 1 for p in good)


def test_what_stays_is_moved_and_the_old_pages_are_free():
    pool, data, w = mla.PagePool(16), _data(16), torch.rand(2, 96)
    lists, before = [pool.alloc(3), pool.alloc(2)], data.clone()
    new, lens, new_w = mla.evict(pool, data, lists, [96, 50], w, [40, 20])
    assert lens.tolist() == [40, 20] and pool.free_pages == 16 - 3
    for b, n in enumerate([96, 50]):
        pos = np.sort(np.argsort(-w[b, :n].numpy(), kind="stable")[:lens[b]])
        assert torch.equal(_rows(data, new[b], lens[b]), _rows(before, lists[b], n)[pos])
        assert torch.equal(new_w[b, :lens[b]], w[b, pos])


def test_a_request_that_loses_nothing_keeps_its_pages(moves):
    # 96 and 50 keys stay; of the third's 96 keys 40; the second's unused page is given back.
    pool, data, w = mla.PagePool(16), _data(16), torch.rand(3, 96)
    lists, before = [pool.alloc(3), pool.alloc(3), pool.alloc(3)], data.clone()
    new, lens, new_w = mla.evict(pool, data, lists, [96, 50, 96], w, [96, 200, 40])
    assert lens.tolist() == [96, 50, 40] and moves == [[0, 0, 40]]
    assert new[0].tolist() == lists[0].tolist() and new[1].tolist() == lists[1][:2].tolist()
    assert pool.free_pages == 16 - 3 - 2 - 2 and not set(new[2]) & set(lists[2])
    for b in range(2):
        assert torch.equal(_rows(data, new[b], lens[b]), _rows(before, lists[b], lens[b])) and torch.equal(new_w[b, :lens[b]], w[b, :lens[b]])
    # All within their budgets, without a free page.
    held = pool.alloc(pool.free_pages)
    again, lens, _ = mla.evict(pool, data, new, lens, new_w, 96)
    assert [p.tolist() for p in again] == [p.tolist() for p in new] and pool.free_pages == 0 and len(moves) == 1 and len(held) == 9


def test_a_shared_partly_filled_page_does_not_stay(moves):
    # 50 keys in pages that another request holds as well: what is appended next is the request's own.
    pool, data = mla.PagePool(16), _data(16)
    pages = pool.alloc(2)
    other = pool.fork(pages, 64, 1)[0][0]
    for lens, private in (([50], True), ([64], False)):
        new, _, _ = mla.evict(pool, data, [pages], lens, torch.rand(1, 64), 64)
        assert (set(new[0]).isdisjoint(other)) == private and pool.references(other[0]) == (1 if private else 2)
        if private:  # (back to the start)
            pool.release(new[0])
            pages = pool.fork(other, 64, 1)[0][0]


def test_pages_that_stay_have_to_be_held():
    pool, data, w = mla.PagePool(16), _data(16), torch.rand(2, 96)
    good = pool.alloc(3)
    for lists, keep in (([good, [12, 13, 14]], 96), ([good, good], 96), ([good, good], [96, 40])):
        with pytest.raises(mla.MlaError):
            mla.evict(pool, data, lists, [96, 96], w, keep)
        assert pool.free_pages == 13 and all(pool.references(int(p)) == 1 for p in good)
