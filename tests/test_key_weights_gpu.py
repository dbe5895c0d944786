"""GPU: the attention weight that cached keys received (mla_key_weights).

Against the definition in 64 bits on the values that the caches hold.  Tolerance
per key: a weight is 2^(c s - l) with c, s and l = lse log2(e) rounded to fp32 and
the difference rounded once more.  With T the largest |c s| + |l| of the case in
log2 units, the exponent is off by at most 4 * 2^-24 T (c, the product's scaling,
l, the difference) plus the fp32 sum of 576 products, 2^-24 * 576 times the sum of
their magnitudes at worst; 2^-22 for the exponential itself, and 2^-24 per added
row and for decay * previous.  The relative error of the sum is ln 2 times the
exponent's plus these."""
import ctypes

import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from fp4_testutil import fp4_case
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE, decode_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _case(kind, heads, q_len, lens, seed):
    """(inputs, pool, values of q [B, q, H, 576] and of each request's keys, 64 bits)."""
    if kind == "fp4":
        inp, pool = fp4_case(len(lens), heads, q_len, [max(1, n) for n in lens], seed)
    else:
        inp = decode_inputs(len(lens), heads, q_len, [max(1, n) for n in lens], seed, extra_pages=2, dtype="bf16" if kind == "bf16" else "e4m3")
        pool = inp.kv
    if kind == "bf16":
        q, kv = inp.q.double().numpy(), inp.kv.double().numpy()
    else:
        q, kv = (cache.e4m3_values()[t.numpy()] for t in (inp.q, inp.kv))
    keys = [kv[inp.page_table[b].numpy()].reshape(-1, 576)[:n] for b, n in enumerate(lens)]
    return inp, pool, q, keys


def _scores(q, keys, b, n, q_b, causal, scale):
    """[q_b, H, n] scores, -inf where a key is not seen, and the largest |s| sum of magnitudes."""
    s = np.einsum("ihd,jd->ihj", q[b, :q_b], keys[b]) * scale
    if causal:
        limit = n - q_b + np.arange(q_b)
        s = np.where(np.arange(n)[None, None] <= limit[:, None, None], s, -np.inf)
    return s


def _lse(q, keys, lens, query_lens, q_len, causal, scale):
    out = np.full((len(lens), q_len, q.shape[2]), -np.inf)
    for b, n in enumerate(lens):
        if n:
            s = _scores(q, keys, b, n, query_lens[b], causal, scale)
            m = s.max(-1, keepdims=True)
            out[b, :query_lens[b]] = (m + np.log(np.exp(s - m).sum(-1, keepdims=True)))[..., 0]
    return out


def _check(kind, heads, q_len, lens, causal, *, seed=3, query_lens=None, previous=True, decay=0.9, kv_scale=1.0, q_scale=1.0, in_place=False,
           device_scales=False):
    inp, pool, q, keys = _case(kind, heads, q_len, lens, seed)
    scale = SOFTMAX_SCALE * q_scale * kv_scale
    ql = [q_len] * len(lens) if query_lens is None else query_lens
    lse = torch.from_numpy(_lse(q, keys, lens, ql, q_len, causal, scale)).float()
    width = max(lens) + 3
    rng = np.random.default_rng(seed)
    prev = torch.from_numpy(rng.random((len(lens), width), dtype=np.float32)).cuda()
    before = prev.clone()
    out = prev if in_place else torch.full((len(lens), width), -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = torch.tensor([q_scale, kv_scale, SOFTMAX_SCALE], device="cuda")
    dev = dict(q_scale_dev=one[0:1], kv_scale_dev=one[1:2], softmax_scale_dev=one[2:3]) if device_scales else {}
    host = (99.0, 99.0, 99.0) if device_scales else (q_scale, kv_scale, SOFTMAX_SCALE)
    mla.mla_key_weights(inp.q.cuda(), pool.cuda(), pool.shape[0], inp.page_table.cuda(), inp.page_table.shape[1],
                        torch.tensor(lens, dtype=torch.int32).cuda(), lse.cuda(), out, len(lens), q_len, heads, causal, *host,
                        cache_kind={"fp8": 0, "bf16": 1, "fp4": 2}[kind], previous=prev if previous else None, decay=decay, status=status,
                        query_lens=None if query_lens is None else torch.tensor(query_lens, dtype=torch.int32).cuda(), **dev)
    assert int(status) == 0
    got, had = out.cpu().double().numpy(), before.cpu().double().numpy()
    c = scale * np.log2(np.e)
    for b, n in enumerate(lens):
        behind = had if in_place else np.full_like(had, -7.0)
        assert (got[b, n:] == behind[b, n:]).all()
        if not n:
            continue
        s = _scores(q, keys, b, n, ql[b], causal, scale)
        l = lse[b, :ql[b]].double().numpy()[..., None]
        with np.errstate(invalid="ignore"):
            w = np.where(np.isfinite(l) & np.isfinite(s), np.exp(s - l), 0.0)
        ref = w.sum((0, 1)) + (decay * had[b, :n] if previous else 0.0)
        seen = np.isfinite(s) & np.isfinite(l)
        size = (np.abs(np.where(seen, s, 0.0)).max() + np.abs(np.where(np.isfinite(l), l, 0.0)).max()) * np.log2(np.e)
        products = np.abs(c) * np.einsum("ihd,jd->ihj", np.abs(q[b, :ql[b]]), np.abs(keys[b])).max()
        exponent = 2.0 ** -24 * (4 * size + 576 * products)
        tol = np.log(2.0) * exponent + 2.0 ** -22 + 2.0 ** -24 * (heads * q_len + 2)
        assert (np.abs(got[b, :n] - ref) <= tol * ref + 1e-37).all(), (b, np.max(np.abs(got[b, :n] - ref) / ref), tol)
    return got


SHAPES = [
    (12, 1, [1], False),
    (12, 1, [31, 0, 129, 128, 127], False),
    (1, 1, [33], False),
    (12, 8, [8, 1000, 515], True),
    (16, 1, [4096, 1], False),
    (12, 3, [3, 257], True),
    (33, 3, [300, 128], True),
    (64, 2, [700], True),        # 128 rows
    (100, 2, [513, 40], False),  # 200 rows
    (128, 8, [2100, 260], True),  # 1024 rows: row groups in turn
    (12, 1, [20000, 9000, 333, 64, 2], False),
]


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s[0]}q{s[1]}n{max(s[2])}")
def test_matches_the_definition(kind, shape):
    _check(kind, *shape)


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
def test_without_a_previous_sum_and_in_place(kind):
    _check(kind, 12, 2, [300, 77], True, previous=False)
    _check(kind, 12, 2, [300, 77], True, in_place=True)
    _check(kind, 128, 8, [1500, 8], True, in_place=True, decay=1.0)


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
def test_ragged_query_counts(kind):
    _check(kind, 12, 8, [1000, 500, 64], True, query_lens=[1, 8, 3])
    _check(kind, 128, 4, [300, 200], True, query_lens=[1, 4])  # groups that are padding only


@pytest.mark.parametrize("device_scales", [False, True])
def test_scales(device_scales):
    _check("fp8", 12, 2, [300, 700], True, kv_scale=0.37, q_scale=1.5, device_scales=device_scales)


def test_many_short_requests():
    rng = np.random.default_rng(1)
    _check("fp8", 4, 1, rng.integers(0, 300, 700).tolist(), False)


def test_the_divisions_among_ctas_give_the_same_bits():
    # The same request alone and in a batch, where other CTAs take other runs of its tiles.
    inp, pool, q, keys = _case("fp8", 12, 1, [9000, 4000, 600], 5)
    lse = torch.from_numpy(_lse(q, keys, [9000, 4000, 600], [1] * 3, 1, False, SOFTMAX_SCALE)).float().cuda()
    kw = dict(num_heads=12, q_len=1, causal=False, softmax_scale=SOFTMAX_SCALE)
    qd, kvd, pt = inp.q.cuda(), pool.cuda(), inp.page_table.cuda()
    both = mla.key_weights(qd, kvd, pt, [9000, 4000, 600], lse, **kw)
    again = mla.key_weights(qd, kvd, pt, [9000, 4000, 600], lse, **kw)
    assert torch.equal(both, again)
    for b, n in enumerate([9000, 4000, 600]):
        one = mla.key_weights(qd[b:b + 1], kvd, pt[b:b + 1], [n], lse[b:b + 1].contiguous(), **kw)
        assert torch.equal(one[0, :n], both[b, :n])


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
def test_weights_of_a_decode_sum_to_its_rows(kind):
    inp, pool, _, _ = _case(kind, 12, 4, [1000, 40], 8)
    args = dict(num_heads=12, q_len=4, causal=True, softmax_scale=SOFTMAX_SCALE)
    qd, kvd, pt = inp.q.cuda(), pool.cuda(), inp.page_table.cuda()
    _, lse, _ = mla.decode(qd, kvd, pt, inp.kv_lens, **args)
    w = mla.key_weights(qd, kvd, pt, inp.kv_lens, lse, **args)
    assert torch.allclose(w.sum(1), torch.full((2,), 48.0, device="cuda"), rtol=1e-4)


def _args(inp, pool, lens, lse, out, status, **kw):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    mla.mla_key_weights(inp.q.cuda(), pool.cuda(), kw.pop("pages", pool.shape[0]), kw.pop("table", inp.page_table).cuda(), inp.page_table.shape[1],
                        i32(lens), lse, out, len(lens), inp.q_len, inp.num_heads, False, 1.0, 1.0, SOFTMAX_SCALE, cache_kind=0, status=status, **kw)


def test_bad_requests_are_skipped_and_reported():
    inp, pool, q, keys = _case("fp8", 12, 1, [200, 100, 300], 4)
    lse = torch.from_numpy(_lse(q, keys, [200, 100, 300], [1] * 3, 1, False, SOFTMAX_SCALE)).float().cuda()
    good = torch.full((3, 300), -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _args(inp, pool, [200, 100, 300], lse, good, status)
    assert int(status) == 0
    for lens, kw in (([200, -1, 300], {}), ([200, 301, 300], {}), ([200, 100, 300], dict(query_lens=torch.tensor([1, 2, 1], dtype=torch.int32).cuda()))):
        out = torch.full((3, 300), -7.0, device="cuda")
        status.zero_()
        _args(inp, pool, lens, lse, out, status, **kw)
        assert int(status) == mla.MLA_ERR_INVALID_ARG
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and (out[1] == -7.0).all()
    # A length that 32-bit tile positions cannot hold, within strides that claim as much.
    out = torch.full((300,), -7.0, device="cuda")
    status.zero_()
    lens = torch.tensor([200, 2 ** 31 - 1], dtype=torch.int32).cuda()
    qd, kvd, pt = inp.q.cuda(), pool.cuda(), inp.page_table[0].contiguous().cuda()
    a = mla.KeyWeightsArgs(q=qd.data_ptr(), kv_pages=kvd.data_ptr(), num_pages=kvd.shape[0], page_table=pt.data_ptr(), kv_lens=lens.data_ptr(),
                           lse=lse.data_ptr(), weights=out.data_ptr(), weights_stride=2 ** 31, status=status.data_ptr(), max_pages_per_req=1 << 26,
                           batch=2, q_len=1, num_heads=12, q_scale=1.0, kv_scale=1.0, softmax_scale=SOFTMAX_SCALE)
    assert mla.load_library().mla_key_weights(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    assert int(status) == mla.MLA_ERR_INVALID_ARG and torch.equal(out, good[0])
    table = inp.page_table.clone()
    table[0, 1] = 10 ** 6
    status.zero_()
    out = torch.full((3, 300), -7.0, device="cuda")
    _args(inp, pool, [200, 100, 300], lse, out, status, table=table)
    assert int(status) == mla.MLA_ERR_INVALID_ARG and torch.equal(out[1:], good[1:])


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
@pytest.mark.parametrize("role,tile", [(0, 0), (0, 3), (1, 0), (1, 2), (3, 0), (3, 1)])
def test_expired_waits_end_the_call(kind, role, tile):
    # One request over few CTAs' runs: every CTA's own steps count from 0.
    inp, pool, q, keys = _case(kind, 12, 8, [152 * 128 * 5], 2)
    lens = [152 * 128 * 5]
    lse = torch.zeros(1, 8, 12, device="cuda")
    kw = dict(num_heads=12, q_len=8, causal=True, softmax_scale=SOFTMAX_SCALE)
    qd, kvd, pt = inp.q.cuda(), pool.cuda(), inp.page_table.cuda()
    ref = mla.key_weights(qd, kvd, pt, lens, lse, **kw)
    mla.mla_debug_set_expire(role, tile)
    try:
        with pytest.raises(mla.MlaError) as err:
            mla.key_weights(qd, kvd, pt, lens, lse, **kw)
        assert err.value.status == mla.MLA_ERR_TIMEOUT
    finally:
        mla.mla_debug_set_expire(-1)
    assert torch.equal(mla.key_weights(qd, kvd, pt, lens, lse, **kw), ref)
