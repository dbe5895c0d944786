"""CPU: the planner of decodes over shared prefixes, the groups of a batch, and the
refusals of mla_decode_shared that need no GPU."""
import ctypes

import numpy as np
import pytest

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build

KINDS = (mla.CACHE_FP8, mla.CACHE_BF16, mla.CACHE_FP4)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _parts(plan):
    n = plan.info.num_segments
    segs = plan.data[:8 * n].reshape(n, 8)
    slots = plan.data[8 * n:8 * n + 2 * plan.info.batch].reshape(-1, 2)
    return segs, slots, plan.data[8 * n + 2 * plan.info.batch:]


CASES = [
    # heads, q_len, group sizes, prefixes, suffixes, causal
    (12, 1, [1], [0], [1], False),
    (12, 1, [4], [1024], [23, 0, 5, 128], False),
    (12, 1, [16], [131072], [2000] * 16, False),
    (12, 8, [3, 1, 4], [32, 0, 65536], [8, 300, 9, 1000, 8, 8, 16, 8], True),
    (128, 8, [2], [4096], [2000, 8], True),
    (33, 3, [5], [320], [3, 4, 5, 6, 7], True),
    (16, 1, [400, 1], [32, 64], [1] * 401, False),
    (12, 1, [2], [32], [1 << 20, 1], False),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"h{c[0]}q{c[1]}g{len(c[2])}b{len(c[4])}")
@pytest.mark.parametrize("sms", [152, 2])
def test_segments_cover_every_row_and_key_once(case, kind, sms):
    heads, q_len, sizes, prefixes, suffixes, causal = case
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    of = np.repeat(np.arange(len(sizes)), sizes)
    lens = [prefixes[of[b]] + suffixes[b] for b in range(len(of))]
    if min(lens) < 1:
        lens = [max(1, n) for n in lens]
    plan = mla.mla_shared_plan(lens, offsets, prefixes, heads, q_len, causal=causal, cache_kind=kind, sm_count=sms)
    info, (segs, slots, items) = plan.info, _parts(plan)
    shared = info.prefix_ctas > 0  # else every request has all of its keys in its own segments
    if max(prefixes) == 0 or max(sizes) == 1:
        assert not shared
    per = heads * q_len
    cap = 32 if kind == mla.CACHE_BF16 else 96
    seen = np.zeros((len(lens) * per, 2), int)  # rows covered by prefix and suffix segments
    for first, n, row_in, req, key0, length, splits, chunk in segs:
        suffix = length < 0
        assert 1 <= n <= min(cap, info.suffix_nr if suffix else info.prefix_nr)
        assert chunk >= 128 and chunk % 128 == 0
        keys = lens[req] - key0 if suffix else length
        assert splits * chunk >= keys and (splits == 1 or (splits - 1) * chunk < keys)
        seen[first:first + n, int(suffix)] += 1
        g = of[req]
        if suffix:
            assert key0 == (prefixes[g] if shared else 0) and row_in == first - req * per and first // per == (first + n - 1) // per == req
            assert slots[req, 1] == splits <= info.suffix_slots
        else:
            assert key0 == 0 and length == prefixes[g] and req == offsets[g] and row_in == 0
            assert first >= offsets[g] * per and first + n <= offsets[g + 1] * per
            assert (slots[offsets[g]:offsets[g + 1], 0] == splits).all() and splits <= info.prefix_slots
    has = np.repeat([shared and prefixes[g] > 0 for g in of], per)
    assert (seen[:, 1] == 1).all() and (seen[:, 0] == has).all()
    # Items: every split of every segment once, prefixes first.
    want = {(s, i) for s in range(len(segs)) for i in range(segs[s, 6])}
    got = [(int(e) >> 14, (int(e) >> 5) & 511) for e in items]
    assert len(got) == len(want) and set(got) == want and all(int(e) & 31 == 0 for e in items)
    n_prefix = int((segs[:, 5] >= 0).sum())
    assert [s < n_prefix for s, _ in got] == sorted([s < n_prefix for s, _ in got], reverse=True)
    assert info.prefix_ctas + info.suffix_ctas == len(got) and info.prefix_slots + info.suffix_slots <= mla.MAX_SPLITS
    assert len(got) <= max(2 * sms, len(segs))
    assert plan.workspace_bytes == mla.mla_decode_workspace_size(len(lens), q_len, heads, info.prefix_slots + info.suffix_slots)


def test_long_prefixes_fill_one_wave():
    info = mla.mla_shared_plan([131072 + 2000] * 16, [0, 16], [131072], 12, 1, sm_count=152).info
    assert 130 <= info.prefix_ctas + info.suffix_ctas <= 152 and info.prefix_nr == 96


def test_long_suffixes_have_ctas_of_their_own_size():
    # Suffixes as long as the prefix: in 96-row CTAs they would take twice as long.
    for kind, wide in ((mla.CACHE_FP8, 96), (mla.CACHE_FP4, 96)):
        info = mla.mla_shared_plan([40000] * 8, [0, 8], [20000 // 32 * 32], 12, 1, cache_kind=kind).info
        assert info.prefix_nr == wide and info.suffix_nr == 16
    middle = mla.mla_shared_plan([32800] * 4, [0, 4], [32768], 12, 1).info
    assert middle.prefix_ctas > 0 and middle.prefix_nr == middle.suffix_nr == 48  # one launch


def test_short_prefixes_are_attended_by_every_request():
    for batch, prefix, shared in ((4, 1024, False), (30, 64, False), (16, 4096, False), (16, 8192, True), (8, 32768, True), (2, 131072, True)):
        info = mla.mla_shared_plan([prefix + 100] * batch, [0, batch], [prefix], 12, 1).info
        assert (info.prefix_ctas > 0) == shared, (batch, prefix)


@pytest.mark.parametrize("bad", [
    dict(offsets=[1, 2]), dict(offsets=[0, 1]), dict(offsets=[0, 2, 2], prefixes=[32, 32]), dict(offsets=[0, 3, 2], prefixes=[32, 32]),
    dict(prefixes=[33]), dict(prefixes=[-32]), dict(prefixes=[128]), dict(lens=[0, 100], prefixes=[0]), dict(lens=[97, 100], causal=True, q_len=2),
    dict(heads=0), dict(q_len=0), dict(sm=0), dict(kind=3), dict(kind=-1), dict(lens=[2 ** 31 - 1, 100])])
def test_bad_plans_are_refused(bad):
    a = dict(lens=[100, 100], offsets=[0, 2], prefixes=[96], heads=12, q_len=1, causal=False, kind=0, sm=152)
    a.update(bad)
    with pytest.raises(mla.MlaError) as err:
        mla.mla_shared_plan(a["lens"], a["offsets"], a["prefixes"], a["heads"], a["q_len"], causal=a["causal"], cache_kind=a["kind"],
                            sm_count=a["sm"])
    assert err.value.status == mla.MLA_ERR_INVALID_ARG


def test_too_many_rows_and_short_buffers():
    with pytest.raises(mla.MlaError) as err:
        mla.mla_shared_plan([100], [0, 1], [0], 129, 8)
    assert err.value.status == mla.MLA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        mla.mla_shared_plan([100], [0, 1], [0, 0], 12, 1)
    lib, info = mla.load_library(), mla.mla_shared_plan([100], [0, 1], [0], 12, 1).info
    arr = [np.array(v, np.int32) for v in ([100], [0, 1], [0])]
    out = np.zeros(64, np.int32)
    assert lib.mla_shared_plan(*[x.ctypes.data for x in arr], 1, 1, 12, 1, 0, 0, 152, out.ctypes.data, info.data_len - 1,
                               ctypes.byref(info)) == mla.MLA_ERR_INVALID_ARG


def test_groups_of_a_batch():
    pool = mla.PagePool(500)
    a = pool.alloc(10)
    forks = pool.fork(a, 300, 3)[0]  # 9 full pages shared, the tenth of their own
    b = pool.alloc(3)
    lists = [a, *forks, b, pool.alloc(1)]
    offsets, prefixes = mla.shared_groups(lists, [300, 300, 310, 320, 90, 5])
    assert offsets.tolist() == [0, 4, 5, 6] and prefixes.tolist() == [288, 0, 0]
    # A fork that has not grown past the shared pages keeps its last q_len keys to itself.
    offsets, prefixes = mla.shared_groups([a[:9], forks[0]], [288, 300], q_len=8)
    assert offsets.tolist() == [0, 2] and prefixes.tolist() == [256]
    offsets, prefixes = mla.shared_groups(lists[:4], [300, 300, 310, 320], least=289)
    assert offsets.tolist() == [0, 1, 2, 3, 4] and prefixes.tolist() == [0] * 4
    # One that shares little with a group that shares much stays by itself.
    long = list(range(100))
    offsets, prefixes = mla.shared_groups([long + [200], long + [201], long[:2] + [202], long[:2] + [203]], [3210, 3220, 90, 90])
    assert offsets.tolist() == [0, 2, 4] and prefixes.tolist() == [3200, 64]
    offsets, prefixes = mla.shared_groups([long + [200], long + [201], long[:60] + [202]], [3210, 3220, 1930])
    assert offsets.tolist() == [0, 3] and prefixes.tolist() == [1920]


@pytest.mark.parametrize("seed", range(30))
def test_groups_against_a_plain_search(seed):
    rng = np.random.default_rng(seed)
    q_len, lists, lens = int(rng.integers(1, 40)), [], []
    for _ in range(rng.integers(1, 9)):
        base = lists[-1] if lists and rng.random() < 0.7 else []
        cut = int(rng.integers(0, len(base) + 1))
        lists.append(list(base[:cut]) + list(rng.integers(0, 400, rng.integers(1, 6))))
        lens.append(int(rng.integers(max(1, q_len), 32 * len(lists[-1]) + 1)) if 32 * len(lists[-1]) >= q_len else q_len)
    offsets, prefixes = mla.shared_groups(lists, lens, q_len=q_len)
    assert offsets[0] == 0 and offsets[-1] == len(lists) and (np.diff(offsets) > 0).all() and len(prefixes) == len(offsets) - 1
    for g, p in enumerate(prefixes):
        members = range(offsets[g], offsets[g + 1])
        assert p % 32 == 0 and (p > 0) == (len(members) > 1)
        for m in members:
            assert lists[m][:p // 32] == lists[offsets[g]][:p // 32] and lens[m] - p >= (q_len if p else 0)


def _decode_shared(plan, **over):
    """A call with addresses that are never used: every one of these is refused."""
    a = dict(q=4096, kv=4096, pages=4, table=4096, width=8, lens=4096, data=4096, batch=1, q_len=1, heads=12, causal=0, qs=1.0, ks=1.0, ss=0.1,
             ws=4096, ws_bytes=1 << 30, out=4096, opts=None)
    a.update(over)
    return mla.load_library().mla_decode_shared(a["q"], a["kv"], a["pages"], a["table"], a["width"], a["lens"],
                                                ctypes.byref(plan) if plan is not None else None, a["data"], a["batch"], a["q_len"], a["heads"],
                                                a["causal"], a["qs"], a["ks"], a["ss"], a["ws"], a["ws_bytes"], a["out"], None, None,
                                                ctypes.byref(a["opts"]) if a["opts"] else None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(kv=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(data=None), 1), (dict(ws=None), 1), (dict(out=None), 1),
    (dict(q=4097), 1), (dict(kv=4104), 1), (dict(data=4104), 1), (dict(ws=4112), 1), (dict(batch=2), 1), (dict(q_len=2), 1), (dict(heads=11), 1),
    (dict(causal=1), 1), (dict(qs=float("nan")), 1), (dict(ws_bytes=1000), 3), (dict(pages=1 << 27), 2),
    (dict(opts=mla.DecodeOptions(output_scale=1.0, kv_bounds=4096)), 2), (dict(opts=mla.DecodeOptions(output_scale=1.0, cta_items=4096)), 2),
    (dict(opts=mla.DecodeOptions(output_scale=1.0, persistent_ctas=1)), 2), (dict(opts=mla.DecodeOptions(output_scale=1.0, phases=1)), 2),
    (dict(opts=mla.DecodeOptions(output_scale=float("inf"))), 1)])
def test_decode_refusals(bad, status):
    plan = mla.mla_shared_plan([100], [0, 1], [0], 12, 1).info
    assert _decode_shared(plan, **bad) == status


def test_decode_refuses_foreign_plans_and_bf16_scales():
    assert _decode_shared(None) == mla.MLA_ERR_INVALID_ARG
    for name, value in (("cache_kind", 3), ("num_segments", 0), ("suffix_ctas", 0), ("prefix_slots", -1), ("suffix_slots", 257), ("data_len", 3),
                        ("kv_split", 3)):
        plan = mla.mla_shared_plan([100], [0, 1], [0], 12, 1).info
        setattr(plan, name, value)
        assert _decode_shared(plan) == mla.MLA_ERR_INVALID_ARG
    plan = mla.mla_shared_plan([100], [0, 1], [0], 12, 1, cache_kind=mla.CACHE_BF16).info
    assert _decode_shared(plan, ks=0.5) == mla.MLA_ERR_INVALID_ARG
    assert _decode_shared(plan, opts=mla.DecodeOptions(output_scale=1.0, q_scale_dev=4096)) == mla.MLA_ERR_UNSUPPORTED
