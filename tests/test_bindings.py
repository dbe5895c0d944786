"""CPU: what the bindings of the prologue and the page operators check before
they hand addresses to the library.

Stand-ins of CUDA tensors: CPU tensors that report a device.  Every call here
is refused, so no address of theirs is used."""
import contextlib
import random

import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


@pytest.fixture(autouse=True)
def _no_launch(monkeypatch):
    def refused(*args, **kw):
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(mla, "_call_on", refused)


class On:
    """A CPU tensor that says it is on CUDA device `index`."""

    def __init__(self, t, index):
        self._t, self._index = t, index

    is_cuda = True

    def get_device(self):
        return self._index

    def __getattr__(self, name):
        return getattr(self._t, name)


def _tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(positions=i32(2), cos_sin=torch.zeros(8, 64), rope_positions=i32(2), norm_weight=torch.zeros(512), req_idx=i32(2),
                page_table=i32(1, 1), kv_pages=torch.zeros(1, 32, 576, dtype=torch.uint8), status=i32(1),
                q_rows=torch.zeros(2, 3, 576, dtype=torch.bfloat16), q_out=torch.zeros(2, 3, 576, dtype=torch.uint8),
                kv_rows=torch.zeros(2, 576, dtype=torch.bfloat16))


def _prologue(**moved):
    t = {k: moved.get(k, On(v, 0)) for k, v in _tensors().items()}
    mla.mla_prologue(2, max_pages_per_req=1, batch=1, num_pages=1, num_heads=3, **t)


def test_the_prologue_call_itself_is_sound():
    with pytest.raises(AssertionError):
        _prologue()


@pytest.mark.parametrize("name", sorted(_tensors()))
def test_prologue_tensors_share_a_device(name):
    t = _tensors()[name]
    for other in (On(t, 1), t):
        with pytest.raises(ValueError):
            _prologue(**{name: other})


def _copy(**moved):
    pool = torch.zeros(4, 32, 576, dtype=torch.uint8)
    ids = torch.zeros(2, dtype=torch.int32)
    t = {k: moved.get(k, On(v, 0)) for k, v in dict(src=pool, dst=pool.clone(), src_ids=ids, dst_ids=ids + 1, rows=ids, status=ids).items()}
    mla.mla_pages_copy(t["src"], 4, mla.CACHE_FP8, t["dst"], 4, mla.CACHE_FP8, t["src_ids"], t["dst_ids"], 2, rows=t["rows"],
                       status=t["status"])


@pytest.mark.parametrize("name", ["src", "dst", "src_ids", "dst_ids", "rows", "status"])
def test_page_copies_share_a_device(name):
    with pytest.raises(AssertionError):
        _copy()
    t = torch.zeros(4, 32, 576, dtype=torch.uint8) if name in ("src", "dst") else torch.zeros(2, dtype=torch.int32)
    for other in (On(t, 1), t):
        with pytest.raises(ValueError):
            _copy(**{name: other})


@pytest.mark.parametrize("name", ["page_table", "page_map", "status"])
def test_remaps_share_a_device(name):
    def call(**moved):
        t = {k: moved.get(k, On(torch.zeros(3, dtype=torch.int32), 0)) for k in ("page_table", "page_map", "status")}
        mla.mla_pages_remap(t["page_table"], 3, t["page_map"], 3, status=t["status"])
    with pytest.raises(AssertionError):
        call()
    t = torch.zeros(3, dtype=torch.int32)
    for other in (On(t, 1), t):
        with pytest.raises(ValueError):
            call(**{name: other})


@pytest.mark.parametrize("sparse", [False, True])
def test_the_four_bit_pool_is_on_the_queries_device(sparse):
    def call(pool):
        q = On(torch.zeros(1, 1, 12, 576, dtype=torch.uint8), 0)
        one = On(torch.zeros(1, 1, dtype=torch.int32), 0)
        tail = (one, one, 1, 1, 1, 1, 12, False, 1.0, 1.0, 0.1, On(torch.zeros(1 << 16, dtype=torch.uint8), 0), 1 << 16, q)
        if sparse:
            mla.mla_decode_fp4_sparse(q, pool, 1, one, 1, one, one, 1, *tail)
        else:
            mla.mla_decode_fp4(q, pool, 1, one, 1, one, *tail)
    pool = torch.zeros(1, mla.FP4_PAGE_BYTES, dtype=torch.uint8)
    with pytest.raises(AssertionError):
        call(On(pool, 0))
    for other in (On(pool, 1), pool):
        with pytest.raises(ValueError):
            call(other)


def _views():
    big = torch.zeros(200, 32, 576, dtype=torch.uint8)
    return big, On(big[:100], 0), On(big[50:150], 0)


@pytest.mark.parametrize("src, dst", [([50], [0]), ([0, 99], [7, 49]), ([60, 70], [20, 5])])
def test_page_copies_see_through_views_of_one_pool(src, dst):
    # Page 50 + k of the first view is page k of the second.
    _, a, b = _views()
    with pytest.raises(ValueError, match="both a source"):
        mla.copy_pages(a, b, src, dst)
    with pytest.raises(ValueError, match="both a source"):
        mla.copy_pages(b, a, dst, src)


def test_page_copies_see_through_views_of_other_kinds():
    # E4M3 pages are 18,432 bytes and 4-bit pages 10,752: page 7 of one
    # buffer's 4-bit view lies in E4M3 pages 4 (73,728 .. 92,160) and no other.
    buf = torch.zeros(20 * 18432 + 16, dtype=torch.uint8)
    wide = On(buf[:20 * 18432].view(20, 32, 576), 0)
    slim = On(buf[:20 * 10752].view(20, mla.FP4_PAGE_BYTES), 0)
    with pytest.raises(ValueError, match="both a source"):
        mla.copy_pages(wide, slim, [0, 4], [0, 7])
    with pytest.raises(ValueError, match="both a source"):
        mla.copy_pages(slim, wide, [7], [4])
    shifted = On(buf[16:16 + 19 * 18432].view(19, 32, 576), 0)  # 16 bytes on: page 3 ends in page 4
    with pytest.raises(ValueError, match="both a source"):
        mla.copy_pages(shifted, wide, [3], [4])


def test_page_copies_between_disjoint_parts_go_on(monkeypatch):
    went = []
    monkeypatch.setattr(mla, "mla_pages_copy", lambda *a, **k: went.append(a))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: None)
    big, a, b = _views()
    mla.copy_pages(a, b, [0, 49], [50, 99])      # pages 0 and 49 of the pool to 100 and 149
    mla.copy_pages(a, b, [50, 51], [2, 3])       # 50 and 51 to 52 and 53
    mla.copy_pages(a, a, [1, 2], [3, 4])
    mla.copy_pages(a, On(big[100:], 0), [0, 99], [0, 99])
    assert len(went) == 4


def test_clashes_against_a_plain_search():
    rng = random.Random(3)
    sizes = {mla.CACHE_FP8: 18432, mla.CACHE_FP4: 10752, mla.CACHE_BF16: 36864}
    seen = set()
    for _ in range(2000):
        sk, dk = rng.choice(list(sizes)), rng.choice(list(sizes))
        sa, da = (rng.choice([0, 16, 18432, 10752 * 3, 1 << 20, 16 * rng.randrange(30000)]) for _ in range(2))
        src = np.array([rng.randrange(12) for _ in range(rng.randint(1, 5))], np.int32)
        dst = np.array(rng.sample(range(12), len(src)), np.int32)
        want = any(max(sa + int(i) * sizes[sk], da + int(j) * sizes[dk]) < min(sa + (int(i) + 1) * sizes[sk], da + (int(j) + 1) * sizes[dk])
                   for i in src for j in dst)
        assert mla._pages_clash(sa, sk, src, da, dk, dst) == want
        seen.add(want)
    assert seen == {True, False}
