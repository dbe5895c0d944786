"""GPU: key weights over the steps of a serving loop: rejected drafts whose places are
written again."""
import ctypes

import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE
from test_key_weights_gpu import _case

pytestmark = pytest.mark.gpu

KINDS = {"fp8": mla.CACHE_FP8, "bf16": mla.CACHE_BF16, "fp4": mla.CACHE_FP4}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(kind, inp, pool, lens, lse, out, previous, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_key_weights(inp.q.cuda(), pool.cuda(), pool.shape[0], inp.page_table.cuda(), inp.page_table.shape[1], _i32(lens), lse, out, len(lens),
                        inp.q_len, inp.num_heads, inp.q_len > 1, 1.0, 1.0, SOFTMAX_SCALE, cache_kind=KINDS[kind], previous=previous, decay=0.7,
                        status=status, **kw)
    return int(status)


@pytest.mark.parametrize("kind", sorted(KINDS))
@pytest.mark.parametrize("heads,q_len", [(12, 1), (12, 8), (128, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_keys_behind_the_previous_lengths_had_nothing(kind, heads, q_len, in_place):
    lens, had = [700, 131, 128, 300, 40], [696, 128, 200, 0, 39]
    inp, pool, _, _ = _case(kind, heads, q_len, lens, 6)
    lse = torch.full((len(lens), q_len, heads), 5.0, device="cuda")
    prev = torch.rand(len(lens), 705, generator=torch.Generator().manual_seed(2)).cuda()
    clean = prev.clone()
    for b, n in enumerate(had):
        clean[b, n:] = 0.0
        prev[b, n:lens[b]] = float("nan")  # never read
    want, got = torch.full_like(prev, -7.0), prev if in_place else torch.full_like(prev, -7.0)
    assert _run(kind, inp, pool, lens, lse, want, clean) == 0
    assert _run(kind, inp, pool, lens, lse, got, prev, previous_lens=_i32(had)) == 0
    for b, n in enumerate(lens):
        assert torch.equal(got[b, :n], want[b, :n]) and torch.isfinite(got[b, :n]).all()
        if not in_place:
            assert (got[b, n:] == -7.0).all()
    # Previous weights in a tensor that holds only those that count.
    narrow = clean[:, :696].contiguous()
    got = torch.full_like(prev, -7.0)
    assert _run(kind, inp, pool, lens, lse, got, narrow, previous_lens=_i32(had)) == 0
    assert torch.equal(got, want)


def test_bad_previous_lengths_are_reported():
    lens = [200, 100, 300]
    inp, pool, _, _ = _case("fp8", 12, 1, lens, 4)
    lse, prev = torch.full((3, 1, 12), 5.0, device="cuda"), torch.rand(3, 300, device="cuda")
    good = torch.full((3, 300), -7.0, device="cuda")
    assert _run("fp8", inp, pool, lens, lse, good, prev, previous_lens=_i32([200, 90, 300])) == 0
    for had, width in (([200, -1, 300], 300), ([90, 91, 90], 90)):
        out, p = torch.full((3, 300), -7.0, device="cuda"), prev[:, :width].contiguous()
        assert _run("fp8", inp, pool, lens, lse, out, p, previous_lens=_i32(had)) == mla.MLA_ERR_INVALID_ARG
        clean = prev.clone()
        for b, n in enumerate(had):  # the nearest length that is possible counts
            clean[b, min(max(n, 0), width):] = 0.0
        assert torch.equal(out, _once(inp, pool, lens, lse, clean))
    out = torch.full((3, 300), -7.0, device="cuda")
    assert _run("fp8", inp, pool, lens, lse, out, prev[:, :299].contiguous()) == mla.MLA_ERR_INVALID_ARG  # (as without previous_lens)
    assert torch.equal(out[0, :200], _once(inp, pool, lens, lse, prev)[0, :200]) and (out[2] == -7.0).all()


def _once(inp, pool, lens, lse, prev):
    out = torch.full((len(lens), 300), -7.0, device="cuda")
    assert _run("fp8", inp, pool, lens, lse, out, prev) == 0
    return out


def test_a_structure_without_previous_weights_ignores_the_rest():
    inp, pool, _, _ = _case("fp8", 12, 1, [100], 4)
    lse, out = torch.full((1, 1, 12), 5.0, device="cuda"), torch.zeros(1, 100, device="cuda")
    qd, kvd, pt, lens, status = inp.q.cuda(), pool.cuda(), inp.page_table.cuda(), _i32([100]), _i32([0])
    a = mla.KeyWeightsArgs(q=qd.data_ptr(), kv_pages=kvd.data_ptr(), num_pages=kvd.shape[0], page_table=pt.data_ptr(), kv_lens=lens.data_ptr(),
                           lse=lse.data_ptr(), weights=out.data_ptr(), weights_stride=100, previous_stride=-5, status=status.data_ptr(),
                           max_pages_per_req=pt.shape[1], batch=1, q_len=1, num_heads=12, q_scale=1.0, kv_scale=1.0, softmax_scale=SOFTMAX_SCALE)
    assert mla.load_library().mla_key_weights(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert int(status) == 0 and (out > 0).all()
