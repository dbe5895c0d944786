"""GPU: key weights over the steps of a serving loop: caches that grow, rejected drafts
whose places are written again, and evictions in between.

Tolerances as in test_key_weights_gpu: the weights of a step are within its relative
bound of the definition in 64 bits with the device's LSE; all terms are positive, so that
the sum over steps is within the largest of those bounds and 2^-24 for each step's
rounding of decay * previous and of the addition."""
import ctypes

import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from oracle import cache
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


def test_widths_of_new_and_narrow_weights():
    lens = [200, 100]
    inp, pool, _, _ = _case("fp8", 12, 1, lens, 4)
    args = (inp.q.cuda(), pool.cuda(), inp.page_table.cuda())
    lse, kw = torch.full((2, 1, 12), 5.0, device="cuda"), dict(num_heads=12, q_len=1, causal=False, softmax_scale=SOFTMAX_SCALE)
    assert mla.key_weights(*args, lens, lse, **kw).shape == (2, 200)
    w = mla.key_weights(*args, lens, lse, capacity=300, **kw)
    assert w.shape == (2, 300) and not w[0, 200:].any() and not w[1, 100:].any()
    assert mla.key_weights(*args, lens, lse, previous=w, **kw) is w
    narrow = torch.ones(2, 150, device="cuda")
    wide = mla.key_weights(*args, lens, lse, previous=narrow, decay=0.5, capacity=256, **kw)
    alone = mla.key_weights(*args, lens, lse, **kw)
    want = torch.zeros(2, 256, device="cuda")
    want[:, :200] = alone
    want[0, :150] += 0.5
    want[1, :100] += 0.5
    assert wide.shape == (2, 256) and torch.equal(wide, want) and (narrow == 1.0).all()
    with pytest.raises(ValueError):
        mla.key_weights(*args, lens, lse, previous=torch.ones(300, device="cuda"), **kw)


@pytest.mark.parametrize("kind", sorted(KINDS))
def test_a_loop_over_steps(kind):
    heads, q_len, vocab, decay, total, batch, steps = 12, 4, 501, 0.8, 160, 3, 7
    g = torch.Generator().manual_seed(40)
    bf16 = kind == "bf16"
    pages = mla.PagePool(total)
    pool = mla.fp4_pool(total) if kind == "fp4" else torch.zeros(total, 32, 576, dtype=torch.bfloat16 if bf16 else torch.uint8, device="cuda")
    kv_lens = [400, 333, 64]
    lists = [pages.alloc((n + 31) // 32) for n in kv_lens]

    def table():
        out = torch.zeros(batch, max(len(p) for p in lists), dtype=torch.int32)
        for b, p in enumerate(lists):
            out[b, :len(p)] = torch.from_numpy(np.asarray(p, np.int32))
        return out.cuda()

    def write(starts, ends):
        at = [(b, j) for b in range(batch) for j in range(starts[b], ends[b])]
        t, status = table(), torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.mla_prologue(len(at), positions=_i32([j for _, j in at]), kv_rows=torch.randn(len(at), 576, generator=g).bfloat16().cuda(),
                         req_idx=_i32([b for b, _ in at]), page_table=t, max_pages_per_req=t.shape[1], batch=batch, kv_pages=pool, num_pages=total,
                         cache_kind=KINDS[kind], status=status)
        assert int(status) == 0

    def values():
        host = pool.cpu()
        if kind == "fp4":
            return cache.fp4_decode(host.numpy())
        return host.double().numpy() if bf16 else cache.e4m3_values()[host.numpy()]

    write([0] * batch, kv_lens)
    weights, ref, bound, rejected, evicted = None, [np.zeros(n) for n in kv_lens], 0.0, 0, 0
    for step in range(steps):
        # The block of the next token and three drafts behind what is cached.
        ends = [n + q_len for n in kv_lens]
        lists = [np.concatenate([p, pages.alloc((n + 31) // 32 - len(p))]) if (n + 31) // 32 > len(p) else p for p, n in zip(lists, ends)]
        write(kv_lens, ends)
        seen, kv_lens = kv_lens, ends
        q = torch.randn(batch, q_len, heads, 576, generator=g) * 0.5
        q = q.bfloat16() if bf16 else q.to(torch.float8_e4m3fn).view(torch.uint8)
        args = dict(num_heads=heads, q_len=q_len, causal=True, softmax_scale=SOFTMAX_SCALE)
        _, lse, _ = mla.decode(q.cuda(), pool, table(), kv_lens, **args)
        weights = mla.key_weights(q.cuda(), pool, table(), kv_lens, lse, previous=weights, previous_lens=None if weights is None else seen,
                                  decay=decay, capacity=410, **args)
        held, qv = values(), q.double().numpy() if bf16 else cache.e4m3_values()[q.numpy()]
        for b, n in enumerate(kv_lens):
            k = held[lists[b]].reshape(-1, 576)[:n]
            s = np.einsum("ihd,jd->ihj", qv[b], k) * SOFTMAX_SCALE
            limit = n - q_len + np.arange(q_len)
            s = np.where(np.arange(n)[None, None] <= limit[:, None, None], s, -np.inf)
            l = lse[b].cpu().double().numpy()[..., None]
            new = np.exp(s - l).sum((0, 1))
            new[:len(ref[b])] += decay * ref[b]
            ref[b] = new
            size = (np.abs(s[np.isfinite(s)]).max() + np.abs(l).max()) * np.log2(np.e)
            products = SOFTMAX_SCALE * np.log2(np.e) * np.einsum("ihd,jd->ihj", np.abs(qv[b]), np.abs(k)).max()
            bound = max(bound, np.log(2.0) * 2.0 ** -24 * (4 * size + 576 * products) + 2.0 ** -22 + 2.0 ** -24 * (heads * q_len + 2))
            got = weights[b, :n].cpu().double().numpy()
            assert (np.abs(got - ref[b]) <= (bound + 2 * (step + 1) * 2.0 ** -24) * ref[b]).all()
        target = torch.softmax(2 * torch.randn(batch, q_len, vocab, generator=g), -1)
        drafts, u = target[:, :q_len - 1].argmax(-1).int(), torch.rand(batch, q_len, generator=g) * 0.1
        _, accepted, lens_d = mla.verify_drafts(target.cuda(), drafts.cuda(), u.cuda(), kv_lens=_i32(kv_lens))
        kv_lens = lens_d.tolist()
        rejected += int((q_len - 1 - accepted).sum())
        ref = [r[:n] for r, n in zip(ref, kv_lens)]
        if step in (2, 4):
            lists, kept, weights = mla.evict(pages, pool, lists, kv_lens, weights, [300, 200, 500], first=4, last=16)
            ref = [r[:0] if n == 0 else w[:n].cpu().double().numpy() for r, n, w in zip(ref, kept.tolist(), weights)]
            kv_lens = kept.tolist()
            evicted += 1
    assert rejected > 0 and evicted == 2 and weights.shape[1] >= max(kv_lens)
