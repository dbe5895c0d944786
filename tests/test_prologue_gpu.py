"""GPU: the prologue (norm, rotation, quantisation, scatter) against the 64-bit oracle.

Tolerances.  A stored value v stands for a 64-bit y: |v - y| <= half a step of
the stored type at y, plus the fp32 error of y itself.  That error: the sum of
512 squares carries at most 16 + 5 + 1 roundings along any path, halved by the
reciprocal square root, and the root, the three products and the scale add 5 of
2^-24 each: 16 * 2^-24 = 2^-20 relative for the latent part (2^-19 is taken).
A rotated value is two rounded products and a rounded sum, then a product with
the scale's rounded reciprocal: below 5 * 2^-24 (|a| + |b|) <= 2^-21 (|a| + |b|).
"""
import numpy as np
import pytest
import torch

import oracle
import split_kv_mla_paged_gb300 as mla
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build

pytestmark = pytest.mark.gpu
EPS = 1e-6
KINDS = {"fp8": mla.CACHE_FP8, "bf16": mla.CACHE_BF16, "fp4": mla.CACHE_FP4}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _pool(kind, pages, device="cuda"):
    if kind == "fp4":
        return torch.full((pages, mla.FP4_PAGE_BYTES), 0x5A, dtype=torch.uint8, device=device)
    if kind == "fp8":
        return torch.full((pages, 32, 576), 0x5A, dtype=torch.uint8, device=device)
    return torch.full((pages, 32, 576), 7.0, dtype=torch.bfloat16, device=device)


def _values(pool, kind):
    p = pool.cpu()
    if kind == "fp4":
        return cache.fp4_decode(p.numpy())
    if kind == "fp8":
        return cache.e4m3_values()[p.numpy()]
    return p.double().numpy()


def _inputs(n_req, tokens, heads, seed, start=0, spread=True):
    g = torch.Generator().manual_seed(seed)
    n = n_req * tokens
    rows = torch.randn(n, 576, generator=g)
    if spread:
        rows = rows * torch.exp2(torch.randint(-4, 4, (n, 18), generator=g).float()).repeat_interleave(32, dim=1)
    pos = torch.cat([torch.arange(start + 5 * i, start + 5 * i + tokens, dtype=torch.int32) for i in range(n_req)])
    req = torch.arange(n_req, dtype=torch.int32).repeat_interleave(tokens)
    max_pages = int(pos.max()) // 32 + 1
    table = torch.randperm(n_req * max_pages, generator=g).int().reshape(n_req, max_pages)
    ang = torch.rand(int(pos.max()) + 3, 32, generator=g, dtype=torch.float64) * 6.28
    return dict(rows=rows.bfloat16(), pos=pos, req=req, table=table, pages=n_req * max_pages + 1,
                cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(),
                weight=1.0 + 0.3 * torch.randn(512, generator=g),
                q=torch.randn(n, heads, 576, generator=g).bfloat16() if heads else None)


def _run(i, kind, halves=False, norm=True, rope=True, kv_scale=1.0, q_kind="fp8", q_scale=1.0, pool=None, stream=None, **kw):
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in i.items()}
    pool = _pool(kind, i["pages"]) if pool is None else pool
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(positions=d["pos"], cos_sin=d["cos_sin"] if rope else None, rope_halves=halves, kv_rows=d["rows"],
                norm_weight=d["weight"] if norm else None, norm_eps=EPS, req_idx=d["req"], page_table=d["table"],
                max_pages_per_req=d["table"].shape[1], batch=d["table"].shape[0], kv_pages=pool, num_pages=i["pages"],
                cache_kind=KINDS[kind], kv_scale=kv_scale, status=status)
    q_out = None
    if i["q"] is not None:
        q_out = torch.full(i["q"].shape, 3, device="cuda", dtype=torch.bfloat16 if q_kind == "bf16" else torch.uint8)
        args.update(q_rows=d["q"], num_heads=i["q"].shape[1], q_out=q_out, q_kind=KINDS[q_kind], q_scale=q_scale)
    args.update(kw)
    torch.cuda.synchronize()  # the test's uploads are done before another stream reads them
    mla.mla_prologue(i["pos"].shape[0], stream=stream, **args)
    torch.cuda.synchronize()
    return pool, q_out, int(status.item())


def _slots(i):
    page = i["table"][i["req"].long(), (i["pos"] // 32).long()].long().numpy()
    return page, (i["pos"] % 32).numpy()


def _half_step(y, kind):
    if kind == "bf16":
        return cache.round_to(y, -126, 7, 3.4e38)[1]
    return cache.round_to(y, -6, 3, 448.0)[1]


def _check_rows(got, y, err, kind, sc=None):
    """got, y, err: [n, 576] stored values, 64-bit values and fp32 error bounds (over kv_scale)."""
    if kind != "fp4":
        high = 448.0 if kind == "fp8" else np.inf
        assert (np.abs(got - np.clip(y, -high, high)) <= _half_step(np.abs(y) + err, kind) + err).all()
        return
    _check_rows(got[:, 512:], y[:, 512:], err[:, 512:], "fp8")
    lat, e = y[:, :512].reshape(-1, 16, 32), err[:, :512].reshape(-1, 16, 32)
    amax, aerr = np.abs(lat).max(-1), e.max(-1)
    lo, hi = cache.fp4_scale_codes(amax - aerr), cache.fp4_scale_codes(amax + aerr)
    assert ((sc >= lo) & (sc <= hi)).all()
    unit = np.exp2(sc - 8.0)[..., None]
    u, ue = np.abs(lat) / unit, e / unit
    half = cache.round_to(u + ue, 0, 1, 6.0)[1]
    want = np.clip(lat / unit, -6, 6)
    ok = np.abs(got[:, :512].reshape(-1, 16, 32) / unit - want) <= np.where(u + ue > 6, 1.0, half) + ue
    assert ok.all()


@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
@pytest.mark.parametrize("n_req, tokens, heads, start, halves, norm, rope, scale", [
    (1, 1, 1, 0, False, True, True, 1.0),
    (3, 7, 12, 29, False, True, True, 0.37),
    (2, 65, 5, 1000, True, True, True, 0.5),
    (1, 33, 16, 31, True, False, True, 1.0),
    (4, 9, 3, 12, False, True, False, 3.0),
    (2, 17, 0, 500, False, True, True, -0.25),
])
def test_prologue_matches_oracle(kind, n_req, tokens, heads, start, halves, norm, rope, scale):
    i = _inputs(n_req, tokens, heads, seed=7 * n_req + tokens, start=start)
    if kind == "bf16":
        scale = 1.0
    q_kind, q_scale = ("bf16", 1.0) if kind == "bf16" else ("fp8", 0.3)
    pool, q_out, st = _run(i, kind, halves, norm, rope, scale, q_kind, q_scale)
    assert st == 0
    page, slot = _slots(i)
    cs = i["cos_sin"].numpy() if rope else None
    y = cache.prologue_rows(i["rows"].double().numpy(), i["weight"].double().numpy() if norm else None, EPS, cs,
                            i["pos"].numpy(), halves) / scale
    mag = np.abs(i["rows"].double().numpy()[:, 512:])
    pair = mag[:, :32] + mag[:, 32:] if halves else mag[:, 0::2] + mag[:, 1::2]
    pair = np.concatenate([pair, pair], 1) if halves else pair.repeat(2, 1)
    err = np.concatenate([np.abs(y[:, :512]) * 2.0 ** -19, pair * 2.0 ** -21 / abs(scale)], 1)
    sc = pool.cpu().numpy()[:, 8192:8704].reshape(-1, 16, 32)[page, :, slot] if kind == "fp4" else None
    _check_rows(_values(pool, kind)[page, slot], y, err, kind, sc)
    # Rows that no token went to are as they were.
    fresh, after = _pool(kind, i["pages"]).cpu(), pool.cpu()
    if kind == "fp4":
        keep = torch.ones(i["pages"], 32, dtype=torch.bool)
        keep[page, slot] = False
        for view in (lambda p: p[:, :8192].reshape(-1, 32, 256), lambda p: p[:, 8704:].reshape(-1, 32, 64),
                     lambda p: p[:, 8192:8704].reshape(-1, 16, 32).transpose(1, 2)):
            assert torch.equal(view(after)[keep], view(fresh)[keep])
    else:
        after[page, slot] = fresh[page, slot]
        assert torch.equal(after, fresh)
    if heads:
        qd = i["q"].double().numpy()
        yq = cache.rotate(qd, cs, i["pos"].numpy(), halves) / q_scale
        m = np.abs(qd[..., 512:])
        pair = m[..., :32] + m[..., 32:] if halves else m[..., 0::2] + m[..., 1::2]
        pair = np.concatenate([pair, pair], -1) if halves else pair.repeat(2, -1)
        err = np.concatenate([np.abs(yq[..., :512]) * 2.0 ** -22, pair * 2.0 ** -21 / q_scale], -1)
        got = cache.e4m3_values()[q_out.cpu().numpy()] if q_kind == "fp8" else q_out.cpu().double().numpy()
        _check_rows(got, yq, err, q_kind)


@pytest.mark.parametrize("kv_scale", [1.0, 4.0, -0.125])
def test_without_norm_and_rotation_it_is_the_append(kv_scale):
    # Powers of two: reciprocal and division give the same numbers.
    i = _inputs(3, 41, 0, seed=5, start=17)
    pool, _, st = _run(i, "fp8", norm=False, rope=False, kv_scale=kv_scale)
    want, _ = oracle.kv_append(i["rows"], i["req"].numpy(), i["pos"].numpy(), i["table"].numpy(),
                               _pool("fp8", i["pages"], "cpu").numpy(), kv_scale)
    assert st == 0 and np.array_equal(pool.cpu().numpy(), want)


@pytest.mark.parametrize("kv_scale", [1.0, 2.0 ** -6, -8.0])
def test_fp4_bytes_match_oracle(kv_scale):
    # Every BF16 pattern among the latent values, NaN, infinities and signed zeros included.
    bits = np.zeros(130 * 512, dtype=np.uint16)
    bits[:65536] = np.random.default_rng(6).permutation(65536).astype(np.uint16)
    rng = np.random.default_rng(8)
    small = (rng.standard_normal((130, 512)) * np.exp2(rng.integers(-12, 9, (130, 16)).repeat(32, 1))).astype(np.float32)
    for lat in (torch.from_numpy(bits.view(np.int16).reshape(130, 512)).view(torch.bfloat16), torch.from_numpy(small).bfloat16()):
        i = _inputs(1, 130, 0, seed=9, start=3)
        i["rows"][:, :512] = lat
        pool, _, st = _run(i, "fp4", norm=False, rope=False, kv_scale=kv_scale)
        with np.errstate(invalid="ignore"):
            parts = cache.fp4_encode_rows(i["rows"].float().numpy().astype(np.float64) / kv_scale)
        want = _pool("fp4", i["pages"], "cpu").numpy()
        page, slot = _slots(i)
        for k in range(130):
            cache.fp4_put(want, page[k], slot[k], [p[k] for p in parts])
        assert st == 0 and np.array_equal(pool.cpu().numpy(), want)


def test_strided_rows_and_rope_positions():
    i = _inputs(2, 6, 4, seed=11, start=40)
    ref, qref, _ = _run(i, "fp4")
    # The same rows as slices of wider buffers.
    wide = torch.zeros(12, 600, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:592] = i["rows"].cuda()
    qw = torch.zeros(4, 12, 584, dtype=torch.bfloat16, device="cuda")
    qw[:, :, :576] = i["q"].cuda().transpose(0, 1)
    got, qgot, st = _run(i, "fp4", kv_rows=wide[:, 16:592], q_rows=qw[:, :, :576].transpose(0, 1))
    assert st == 0 and torch.equal(got, ref) and torch.equal(qgot, qref)
    # Rotation rows of their own.
    rp = (i["pos"] - 40).cuda()
    cs = i["cos_sin"][40:].contiguous().cuda()
    got, qgot, st = _run(i, "fp4", cos_sin=cs, rope_positions=rp)
    assert st == 0 and torch.equal(got, ref) and torch.equal(qgot, qref)


def test_padding_tokens_and_bad_targets():
    i = _inputs(3, 4, 2, seed=12, start=30)
    ref, qref, _ = _run(i, "fp8")
    page, slot = _slots(i)
    keep = torch.ones(12, dtype=torch.bool)
    # Padding: neither row written, nothing reported, whatever its position.
    pad = dict(i, req=i["req"].clone(), pos=i["pos"].clone())
    pad["req"][[1, 7]] = -1
    pad["pos"][7] = 1 << 30
    keep[[1, 7]] = False
    got, qgot, st = _run(pad, "fp8")
    want = ref.clone()
    want[page[~keep], slot[~keep]] = 0x5A
    assert st == 0 and torch.equal(got, want)
    assert torch.equal(qgot[keep], qref[keep]) and (qgot[~keep] == 3).all()
    # Bad request, negative position, position past the table, bad page id: reported and skipped.
    for change in ("req", "neg", "far", "page"):
        b = dict(i, req=i["req"].clone(), pos=i["pos"].clone(), table=i["table"].clone())
        if change == "req":
            b["req"][5] = 3
        elif change == "neg":
            b["pos"][5] = -1
        elif change == "far":
            b["pos"][5] = 32 * b["table"].shape[1]
        else:
            b["table"][1, b["pos"][5] // 32] = b["pages"]
        got, qgot, st = _run(b, "fp8")
        assert st == mla.MLA_ERR_INVALID_ARG, change
        want = ref.clone()
        lost = (i["table"][i["req"].long(), (i["pos"] // 32).long()] == i["table"][1, i["pos"][5] // 32]) if change == "page" \
            else torch.arange(12) == 5
        want[page[lost], slot[lost]] = 0x5A
        assert torch.equal(got, want), change
        q_keep = torch.arange(12) != 5 if change in ("neg", "far") else torch.ones(12, dtype=torch.bool)
        assert torch.equal(qgot[q_keep], qref[q_keep]), change


def test_nan_and_infinity_rows():
    i = _inputs(1, 4, 1, seed=13)
    i["rows"][1, 100] = float("nan")
    i["rows"][2, 530] = float("nan")
    i["rows"][3, 7] = float("inf")
    for kind in ("fp8", "bf16", "fp4"):
        pool, _, st = _run(i, kind, kv_scale=1.0, q_kind="bf16" if kind == "bf16" else "fp8")
        page, slot = _slots(i)
        v = _values(pool, kind)[page, slot]
        assert st == 0 and np.isfinite(v[0]).all()
        assert np.isnan(v[1, :512]).all() and np.isfinite(v[1, 512:]).all()  # the norm carries it to the whole row
        # the NaN's pair (530, 531) and nothing else
        assert np.flatnonzero(np.isnan(v[2])).tolist() == [530, 531]
        # infinite mean: every other value 0 * x = 0, the infinity itself 0 * inf
        assert np.isnan(v[3, 7]) and (v[3, 32:512] == 0).all()


def test_queries_alone_and_keys_alone():
    i = _inputs(2, 5, 3, seed=14, start=9)
    ref, qref, _ = _run(i, "fp8", q_scale=0.5)
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in i.items()}
    q_out = torch.zeros_like(qref)
    mla.mla_prologue(10, positions=d["pos"], cos_sin=d["cos_sin"], q_rows=d["q"], num_heads=3, q_out=q_out, q_scale=0.5)
    torch.cuda.synchronize()
    assert torch.equal(q_out, qref)
    got, none, _ = _run(dict(i, q=None), "fp8")
    assert none is None and torch.equal(got, ref)


def test_empty_batch():
    i = _inputs(1, 3, 2, seed=18)
    empty = {k: (v[:0] if k in ("rows", "q", "pos", "req") else v) for k, v in i.items()}
    pool, q_out, st = _run(empty, "fp4")
    assert st == 0 and q_out.numel() == 0 and torch.equal(pool, _pool("fp4", i["pages"]))


def test_side_stream_and_graph_replay():
    i = _inputs(2, 8, 4, seed=15, start=100)
    ref, qref, _ = _run(i, "fp4")
    side = torch.cuda.Stream()
    got, qgot, _ = _run(i, "fp4", stream=side)
    assert torch.equal(got, ref) and torch.equal(qgot, qref)
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in i.items()}
    pool, q_out = _pool("fp4", i["pages"]), torch.zeros_like(qref)

    def call():
        mla.mla_prologue(16, positions=d["pos"], cos_sin=d["cos_sin"], kv_rows=d["rows"], norm_weight=d["weight"], norm_eps=EPS,
                         req_idx=d["req"], page_table=d["table"], max_pages_per_req=d["table"].shape[1], batch=2, kv_pages=pool,
                         num_pages=i["pages"], cache_kind=mla.CACHE_FP4, q_rows=d["q"], num_heads=4, q_out=q_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool, ref) and torch.equal(q_out, qref)
    # New inputs in the same buffers.
    j = _inputs(2, 8, 4, seed=16, start=100)
    for k in ("rows", "q", "weight", "cos_sin", "table"):
        d[k].copy_(j[k])
    pool.fill_(0x5A)
    graph.replay()
    want, qwant, _ = _run(j, "fp4")
    assert torch.equal(pool, want) and torch.equal(q_out, qwant)


def test_binding_refuses_what_an_address_cannot_carry():
    i = _inputs(1, 4, 2, seed=17)
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in i.items()}
    pool, q_out = _pool("fp8", i["pages"]), torch.zeros(4, 2, 576, dtype=torch.uint8, device="cuda")
    good = dict(positions=d["pos"], cos_sin=d["cos_sin"], kv_rows=d["rows"], req_idx=d["req"], page_table=d["table"],
                max_pages_per_req=d["table"].shape[1], batch=1, kv_pages=pool, num_pages=i["pages"], q_rows=d["q"], num_heads=2, q_out=q_out)
    for n, bad in ((5, {}), (4, dict(num_heads=3)), (4, dict(kv_rows=d["rows"][:1].expand(4, 576))), (4, dict(kv_rows=d["rows"].float())),
                   (4, dict(q_rows=d["q"][:, :1].expand(4, 2, 576))), (4, dict(q_rows=d["q"].transpose(1, 2).contiguous().transpose(1, 2))),
                   (4, dict(positions=d["pos"].long())), (4, dict(page_table=d["table"].cpu())), (4, dict(q_out=q_out[:2])),
                   (4, dict(cos_sin=d["cos_sin"].double())), (4, dict(norm_weight=d["weight"].bfloat16())),
                   (4, dict(norm_weight=d["weight"][:511].contiguous())), (4, dict(positions=d["pos"][:3].contiguous())),
                   (4, dict(num_pages=i["pages"] + 1)), (4, dict(cache_kind=mla.CACHE_BF16)), (4, dict(rope_rows=d["cos_sin"].shape[0] + 1)),
                   (4, dict(batch=2)), (4, dict(q_kind=mla.CACHE_BF16))):
        with pytest.raises(ValueError):
            mla.mla_prologue(n, **dict(good, **bad))
    mla.mla_prologue(4, **good)
    torch.cuda.synchronize()
