"""Host page pool: allocation, sharing, forks, compaction (CPU), against a model
of the pool as a list of reference counts."""
import random
import threading

import numpy as np
import pytest

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def test_alloc_is_lowest_first_and_all_or_nothing():
    p = mla.PagePool(5)
    assert p.alloc(3).tolist() == [0, 1, 2] and p.free_pages == 2
    with pytest.raises(mla.MlaError) as e:
        p.alloc(3)
    assert e.value.status == mla.MLA_ERR_NO_PAGES and p.free_pages == 2
    p.release([1])
    assert p.alloc(2).tolist() == [1, 3]
    assert p.alloc(0).tolist() == []


def test_release_is_all_or_nothing():
    p = mla.PagePool(4)
    p.alloc(3)
    for bad in ([0, 3], [0, 0], [0, -1], [2, 4]):
        with pytest.raises(mla.MlaError):
            p.release(bad)
        assert [p.references(k) for k in range(4)] == [1, 1, 1, 0] and p.free_pages == 1
    p.release([])
    p.release([2, 0, 1])
    assert p.free_pages == 4


@pytest.mark.parametrize("kv_len", [0, 1, 31, 32, 33, 64, 95])
def test_fork_shares_full_pages_and_copies_the_rest(kv_len):
    p = mla.PagePool(12)
    n = (kv_len + 31) // 32
    ids = p.alloc(n)
    out, src, dst, rows = p.fork(ids, kv_len, 3)
    full, rest = kv_len // 32, kv_len % 32
    assert out.shape == (3, n)
    assert (out[:, :full] == ids[:full]).all()
    assert [p.references(k) for k in ids[:full]] == [4] * full
    if rest:
        assert src.tolist() == [ids[-1]] * 3 and rows.tolist() == [rest] * 3
        assert out[:, -1].tolist() == dst.tolist() == [n, n + 1, n + 2]
        assert p.references(ids[-1]) == 1
    else:
        assert src.size == dst.size == rows.size == 0
    for f in range(3):
        p.release(out[f])
    p.release(ids)
    assert p.free_pages == 12


def test_fork_refusals():
    p = mla.PagePool(4)
    ids = p.alloc(2)
    with pytest.raises(mla.MlaError) as e:
        p.fork(ids, 40, 3)
    assert e.value.status == mla.MLA_ERR_NO_PAGES
    with pytest.raises(mla.MlaError):
        p.fork([0, 3], 40, 1)  # page 3 is free
    with pytest.raises(ValueError):
        p.fork(ids, 65, 1)
    with pytest.raises(mla.MlaError):
        p.fork(ids, 64, -1)
    assert [p.references(k) for k in range(4)] == [1, 1, 0, 0]
    out, src, _, _ = p.fork(ids, 64, 0)
    assert out.shape == (0, 2) and src.size == 0


def test_create_refusals():
    for n in (0, -3, 1 << 31):
        with pytest.raises(mla.MlaError):
            mla.PagePool(n)
    lib = mla.load_library()
    assert lib.mla_pool_alloc(None, 1, None) == mla.MLA_ERR_INVALID_ARG
    assert lib.mla_pool_free_pages(None) == -1 and lib.mla_pool_references(None, 0) == -1
    p = mla.PagePool(2)
    assert p.references(2) == -1 and p.references(-1) == -1 and p.references(1) == 0


@pytest.mark.parametrize("seed", range(6))
def test_against_a_model(seed):
    rng = random.Random(seed)
    n = rng.choice([1, 7, 40, 200])
    pool, refs, reqs = mla.PagePool(n), [0] * n, []
    for _ in range(300):
        act = rng.choice(["alloc", "release", "fork", "compact"])
        if act == "alloc":
            k = rng.randint(0, 6)
            free = [i for i, r in enumerate(refs) if r == 0]
            if k > len(free):
                with pytest.raises(mla.MlaError):
                    pool.alloc(k)
            else:
                got = pool.alloc(k).tolist()
                assert got == free[:k]
                for i in got:
                    refs[i] = 1
                reqs.append(got)
        elif act == "release" and reqs:
            got = reqs.pop(rng.randrange(len(reqs)))
            pool.release(got)
            for i in got:
                refs[i] -= 1
        elif act == "fork" and reqs:
            got = rng.choice(reqs)
            kv_len = rng.randint(max(0, 32 * len(got) - 31), 32 * len(got)) if got else 0
            free = [i for i, r in enumerate(refs) if r == 0]
            need = 2 if kv_len % 32 else 0
            if need > len(free):
                with pytest.raises(mla.MlaError):
                    pool.fork(got, kv_len, 2)
                continue
            out, src, dst, rows = pool.fork(got, kv_len, 2)
            for row in out.tolist():
                reqs.append(row)
            for i in got[:kv_len // 32]:
                refs[i] += 2
            assert dst.tolist() == free[:need]
            for i in dst:
                refs[i] = 1
        elif act == "compact":
            cap = rng.choice([None, 0, 1, 3])
            src, dst, m = pool.compact(cap)
            used = sum(r > 0 for r in refs)
            above = [i for i in range(used, n) if refs[i] > 0]
            holes = [i for i in range(used) if refs[i] == 0]
            k = len(above) if cap is None else min(cap, len(above))
            assert src.tolist() == above[:k] and dst.tolist() == holes[:k]
            want = list(range(n))
            for a, b in zip(above[:k], holes[:k]):
                want[a] = b
                refs[b], refs[a] = refs[a], 0
            assert m.tolist() == want
            reqs = [[want[i] for i in r] for r in reqs]
        assert [pool.references(i) for i in range(n)] == refs
        assert pool.free_pages == sum(r == 0 for r in refs)


def test_threads_do_not_share_pages():
    p, got = mla.PagePool(4000), []

    def take():
        got.append(np.concatenate([p.alloc(5) for _ in range(100)]))
    threads = [threading.Thread(target=take) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert np.array_equal(np.sort(np.concatenate(got)), np.arange(4000))


def test_ids_are_not_truncated_and_pools_not_copied():
    import copy
    import pickle
    p = mla.PagePool(4)
    p.alloc(2)
    for bad in ([1 << 32], [0.0], [-(1 << 40)]):
        with pytest.raises(ValueError):
            p.release(bad)
        with pytest.raises(ValueError):
            p.fork(bad, 32, 1)
    assert p.free_pages == 2
    for f in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(TypeError):
            f(p)
    assert p.alloc(1).tolist() == [2]


def test_single_ids_are_not_truncated():
    p = mla.PagePool(4)
    p.alloc(2)
    for bad in (1 << 32, (1 << 32) + 1, -(1 << 32), 1 << 70, 0.0, 1.5):
        with pytest.raises(ValueError):
            p.references(bad)
    assert [p.references(k) for k in (0, 1, 2, np.int64(3), 4, -1)] == [1, 1, 0, 0, -1, -1]
    for bad in (1 << 64, (1 << 64) + 3):
        with pytest.raises(ValueError):
            mla.PagePool(bad)
