"""GPU: the operators of a speculative serving step run together, as a serving loop
uses them: forks of one prompt, the prologue that writes the drafted block, the
decode over the shared prefix, verification, key weights of the block's rows, and
an eviction after which the requests decode on.  Each step against the oracle or a
plain form on what the device holds."""
import numpy as np
import pytest
import torch

import oracle
import split_kv_mla_paged_gb300 as mla
from mla_testutil import assert_parity
from oracle import cache
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE

pytestmark = pytest.mark.gpu

HEADS, Q, VOCAB = 12, 4, 3001


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _values(kind, dev):
    """The pool's values as a tensor that the oracle takes."""
    host = dev.cpu()
    if kind == mla.CACHE_FP4:
        return torch.from_numpy(cache.e4m3_codes(cache.fp4_decode(host.numpy())))
    return host


def _table(lists):
    out = torch.zeros(len(lists), max(len(p) for p in lists), dtype=torch.int32)
    for b, p in enumerate(lists):
        out[b, :len(p)] = torch.from_numpy(np.asarray(p, np.int32))
    return out


@pytest.mark.parametrize("kind", [mla.CACHE_FP8, mla.CACHE_BF16, mla.CACHE_FP4])
def test_step(kind):
    g = torch.Generator().manual_seed(17 + kind)
    total, prompt, forks = 120, 1000, 3
    bf16 = kind == mla.CACHE_BF16
    pool_h = mla.PagePool(total)
    pool = (mla.fp4_pool(total) if kind == mla.CACHE_FP4
            else torch.zeros(total, 32, 576, dtype=torch.bfloat16 if bf16 else torch.uint8, device="cuda"))

    def write(lists, starts, count):
        n = len(lists) * count
        pos = [s + i for s in starts for i in range(count)]
        req = [b for b in range(len(lists)) for _ in range(count)]
        table = _table(lists).cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.mla_prologue(n, positions=torch.tensor(pos, dtype=torch.int32).cuda(), kv_rows=torch.randn(n, 576, generator=g).bfloat16().cuda(),
                         req_idx=torch.tensor(req, dtype=torch.int32).cuda(), page_table=table, max_pages_per_req=table.shape[1],
                         batch=len(lists), kv_pages=pool, num_pages=total, cache_kind=kind, status=status)
        assert int(status) == 0

    # A prompt, its forks, and the block of drafts that each writes behind it.
    base = pool_h.alloc((prompt + 31) // 32)
    write([base], [0], prompt)
    forked, src, dst, rows = pool_h.fork(base, prompt, forks)
    mla.copy_pages(pool, pool, src, dst, rows)
    lists = [np.concatenate([p, pool_h.alloc(1)]) for p in [base, *forked]]
    lens = [prompt + Q] * 4
    write(lists, [prompt] * 4, Q)
    offsets, prefixes = mla.shared_groups(lists, lens, q_len=Q)
    assert offsets.tolist() == [0, 4] and prefixes.tolist() == [992]

    q = torch.randn(4, Q, HEADS, 576, generator=g) * 0.5
    q = q.bfloat16() if bf16 else q.to(torch.float8_e4m3fn).view(torch.uint8)
    table = _table(lists)
    args = dict(num_heads=HEADS, q_len=Q, causal=True, softmax_scale=SOFTMAX_SCALE)
    out, lse, _ = mla.decode(q.cuda(), pool, table.cuda(), lens, group_offsets=offsets, prefix_lens=prefixes, sm_count=1, **args)
    held = _values(kind, pool)
    ref, ref_lse = oracle.decode_rows(q, held, table, torch.tensor(lens, dtype=torch.int32), **args)
    assert_parity(out, lse, ref, ref_lse)

    # The weight that every key received: each request's sum to its rows.
    weights = mla.key_weights(q.cuda(), pool, table.cuda(), lens, lse, **args)
    assert torch.allclose(weights.sum(1).cpu(), torch.full((4,), float(HEADS * Q)), rtol=1e-4)

    # Drafts against the target's probabilities: what is rejected leaves the cache.
    target = torch.softmax(3 * torch.randn(4, Q, VOCAB, generator=g), -1)
    drafts = target[:, :Q - 1].argmax(-1).int()
    u = torch.rand(4, Q, generator=g)
    u[0, :Q - 1] = 0.0  # all of the first request's are accepted
    u[1, :Q - 1] = 0.99999
    tokens, accepted, new_lens = mla.verify_drafts(target.cuda(), drafts.cuda(), u.cuda(),
                                                   kv_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    accepted, new_lens, tokens = accepted.tolist(), new_lens.tolist(), tokens.cpu()
    assert accepted[:2] == [Q - 1, 0] and new_lens == [prompt + 1 + a for a in accepted]
    for b in range(4):
        assert tokens[b, :accepted[b]].tolist() == drafts[b, :accepted[b]].tolist()
        assert 0 <= int(tokens[b, accepted[b]]) < VOCAB and (tokens[b, accepted[b] + 1:] == -1).all()

    # Evict down to half; shared pages stay with whom they are shared until all have gone.
    free = pool_h.free_pages
    new_lists, kept_lens, kept_w = mla.evict(pool_h, pool, lists, new_lens, weights, [500, 500, 2000, 333], first=4, last=8)
    assert kept_lens.tolist() == [500, 500, new_lens[2], 333]
    assert pool_h.free_pages == free + len(base) + 3 + 4 - sum(len(p) for p in new_lists)
    now = _values(kind, pool)
    w = weights.cpu().numpy()
    for b in range(4):
        n, k = new_lens[b], int(kept_lens[b])
        rank = w[b, :n].astype(np.float64).copy()
        rank[:4] = rank[n - 8:] = np.inf
        pos = np.sort(np.lexsort((np.arange(n), -rank))[:k])
        assert np.array_equal(kept_w[b, :k].cpu().numpy(), w[b, pos])
        was = held[torch.from_numpy(lists[b].astype(np.int64))].reshape(-1, 576)[torch.from_numpy(pos)]
        new = now[torch.from_numpy(new_lists[b].astype(np.int64))].reshape(-1, 576)[:k]
        assert torch.equal(was.view(torch.uint8), new.view(torch.uint8))

    # The next step on what is left, every request by itself now.
    q1 = q[:, :1].contiguous()
    args = dict(num_heads=HEADS, q_len=1, causal=False, softmax_scale=SOFTMAX_SCALE)
    table = _table(new_lists)
    out, lse, _ = mla.decode(q1.cuda(), pool, table.cuda(), kept_lens, **args)
    ref, ref_lse = oracle.decode_rows(q1, now, table, torch.from_numpy(kept_lens), **args)
    assert_parity(out, lse, ref, ref_lse)
    again = mla.key_weights(q1.cuda(), pool, table.cuda(), kept_lens, lse, previous=kept_w.clone(), decay=0.5, **args)
    for b in range(4):
        k = int(kept_lens[b])
        added = (again[b, :k] - 0.5 * kept_w[b, :k]).sum()
        assert abs(float(added) - HEADS) <= 1e-3 * HEADS


def _step(kind, seed, batch=6, prefix=4096, own=700, sms=16):
    """A step's calls on tensors of their own, as one function without allocations,
    and those tensors by name."""
    g = torch.Generator().manual_seed(seed)
    bf16, rows = kind == mla.CACHE_BF16, batch * Q * HEADS
    each, shared = (own + 31) // 32, prefix // 32
    pages = shared + batch * each
    if kind == mla.CACHE_FP4:
        pool = torch.randint(0, 256, (pages, mla.FP4_PAGE_BYTES), generator=g, dtype=torch.uint8)
        pool[:, 8192:8704] &= 7
        pool[:, 8704:] = (torch.randn(pages, 2048, generator=g) * 0.5).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        pool = torch.randn(pages, 32, 576, generator=g) * 0.5
        pool = pool.bfloat16() if bf16 else pool.to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn(batch, Q, HEADS, 576, generator=g) * 0.5
    q = q.bfloat16() if bf16 else q.to(torch.float8_e4m3fn).view(torch.uint8)
    order = torch.randperm(pages, generator=g).int()
    table = torch.cat([order[:shared].expand(batch, -1), order[shared:].reshape(batch, each)], 1).contiguous().cuda()
    lens = [prefix + own - 9 * b for b in range(batch)]
    plan = mla.mla_shared_plan(lens, [0, batch], [prefix], HEADS, Q, causal=True, cache_kind=kind, sm_count=sms)
    assert plan.info.prefix_ctas > 0
    data = torch.from_numpy(plan.data).cuda()
    q, pool, lens_d = q.cuda(), pool.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty(batch, Q, HEADS, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(batch, Q, HEADS, device="cuda")
    weights = torch.rand(batch, lens[0], generator=g).cuda()
    target = torch.softmax(3 * torch.randn(batch, Q, VOCAB, generator=g), -1).cuda()
    drafts, u = target[:, :Q - 1].argmax(-1).int(), torch.rand(batch, Q, generator=g).cuda()
    tokens, accepted, left = (torch.empty(batch, n, dtype=torch.int32, device="cuda") for n in (Q, 1, 1))
    keep = torch.tensor([500 + 40 * b for b in range(batch)], dtype=torch.int32).cuda()
    most = 32 * ((500 + 40 * batch) // 32 + 1)
    kept, kept_w = torch.full((batch, most), -1, dtype=torch.int32, device="cuda"), torch.zeros(batch, most, device="cuda")
    counts, status = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    moved = torch.zeros((batch * most // 32, *pool.shape[1:]), dtype=pool.dtype, device="cuda")
    to = torch.randperm(moved.shape[0], generator=g).int().reshape(batch, -1).cuda()

    def run():
        mla.mla_decode_shared(q, pool, pages, table, table.shape[1], lens_d, plan, data, batch, Q, HEADS, True, 1.0, 1.0, SOFTMAX_SCALE, ws,
                              plan.workspace_bytes, out, lse)
        mla.mla_key_weights(q, pool, pages, table, table.shape[1], lens_d, lse, weights, batch, Q, HEADS, True, 1.0, 1.0, SOFTMAX_SCALE,
                            cache_kind=kind, previous=weights, decay=0.5, status=status)
        mla.mla_verify_drafts(target, drafts, u, tokens, accepted, kv_lens=lens_d, new_lens=left, status=status)
        mla.mla_evict_select(weights, left, keep, kept, counts, first=4, last=8, new_weights=kept_w, status=status)
        mla.mla_rows_move(pool, pages, table, moved, moved.shape[0], to, kept, counts, cache_kind=kind, status=status)

    return run, dict(q=q, pool=pool, out=out, lse=lse, weights=weights, tokens=tokens, accepted=accepted, left=left, kept=kept, kept_w=kept_w,
                     counts=counts, moved=moved, decode_status=ws[:4], status=status)


RESULTS = ("out", "lse", "weights", "tokens", "accepted", "left", "kept", "kept_w", "counts", "moved")


@pytest.mark.parametrize("kind", [mla.CACHE_FP8, mla.CACHE_BF16, mla.CACHE_FP4])
def test_two_captured_steps_at_once(kind):
    # Two steps in graphs of their own, replayed on two streams at a time: the bits of
    # the steps called one after the other.
    times, want, graphs = 8, [], []
    for seed in (1, 2):
        run, t = _step(kind, seed)
        for _ in range(times + 1):
            run()
        torch.cuda.synchronize()
        assert int(t["status"]) == 0 and not t["decode_status"].any()
        want.append([t[n] for n in RESULTS])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed, stream in zip((1, 2), streams):
        run, t = _step(kind, seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            run()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run()
        graphs.append((graph, t))
    for _ in range(times):
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, t), ref in zip(graphs, want):
        assert int(t["status"]) == 0 and not t["decode_status"].any()
        for a, b in zip((t[n] for n in RESULTS), ref):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _alternate(run, current, variants, results, times=30):
    """Every call right behind the copies that write its inputs, on one stream: the
    results of each variant's first call, made after a wait."""
    want = []
    for v in variants:
        for c, x in zip(current, v):
            c.copy_(x)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        want.append([r.clone() for r in results])
    assert not all(torch.equal(a, b) for a, b in zip(*want))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(times):
        for v, w in zip(variants, want):
            for c, x in zip(current, v):
                c.copy_(x)
            run()
            for r, x in zip(results, w):
                wrong += (r.contiguous().view(torch.uint8) != x.contiguous().view(torch.uint8)).sum()
    assert int(wrong) == 0


@pytest.mark.parametrize("kind", [mla.CACHE_FP8, mla.CACHE_BF16, mla.CACHE_FP4])
def test_inputs_written_just_before_decode_and_weights(kind):
    run, t = _step(kind, 5, batch=4, prefix=16384, own=900)
    current = [t[n] for n in ("q", "pool", "weights")]
    _alternate(run, current, [[c.clone() for c in current], [c.flip(0) for c in current]], [t[n] for n in RESULTS])


def test_inputs_written_just_before_selection_and_verification():
    # Sizes whose launches are programmatic dependents of the copies before them.
    n, keep = 600_000, 5000
    w, lens = torch.rand(1, n, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    kept, counts = torch.empty(1, keep, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    budget, kept_w = torch.tensor([keep], dtype=torch.int32, device="cuda"), torch.empty(1, keep, device="cuda")
    _alternate(lambda: mla.mla_evict_select(w, lens, budget, kept, counts, new_weights=kept_w), [w, lens],
               [[torch.rand(1, n, device="cuda"), lens.clone()], [torch.rand(1, n, device="cuda"), lens - 100_000]], [kept, kept_w, counts])
    batch, vocab = 72, 65536
    p, u = torch.empty(batch, 2, vocab, device="cuda"), torch.empty(batch, 2, device="cuda")
    x = torch.empty(batch, 1, dtype=torch.int32, device="cuda")
    tokens, accepted = torch.empty(batch, 2, dtype=torch.int32, device="cuda"), torch.empty(batch, dtype=torch.int32, device="cuda")

    def inputs():
        t = torch.softmax(2 * torch.randn_like(p), -1)
        return [t, torch.rand_like(u), t[:, :1].argmax(-1).int()]

    _alternate(lambda: mla.mla_verify_drafts(p, x, u, tokens, accepted), [p, u, x], [inputs(), inputs()], [tokens, accepted])


def _ops():
    """The calls that can start while the kernel before them ends, each with an input
    that decides its result and its results, at sizes where it does."""
    run, t = _step(mla.CACHE_FP8, 9, batch=4, prefix=16384, own=900)  # (its own eviction is small)
    yield run, t["q"], [t[n] for n in RESULTS]
    n, keep = 600_000, 5000
    w, lens = torch.rand(1, n, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    kept, counts = torch.empty(1, keep, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    budget = torch.tensor([keep], dtype=torch.int32, device="cuda")
    yield (lambda: mla.mla_evict_select(w, lens, budget, kept, counts)), w, [kept, counts]
    p, u = torch.softmax(2 * torch.randn(72, 2, 65536, device="cuda"), -1), torch.rand(72, 2, device="cuda")
    x, tokens = p[:, :1].argmax(-1).int(), torch.empty(72, 2, dtype=torch.int32, device="cuda")
    accepted = torch.empty(72, dtype=torch.int32, device="cuda")
    yield (lambda: mla.mla_verify_drafts(p, x, u, tokens, accepted)), u, [tokens, accepted]


@pytest.mark.parametrize("before", ["nothing", "copy", "zero", "kernel", "join"])
def test_captured_behind_other_work(before):
    for run, inp, results in _ops():
        good, blank = inp.clone(), [r.clone() for r in results]
        run()
        torch.cuda.synchronize()
        want = [r.clone() for r in results]
        side, other = torch.cuda.Stream(), torch.empty_like(inp)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if before in ("copy", "join"):
                inp.copy_(good)
            elif before == "zero":
                other.view(torch.uint8).zero_()
            elif before == "kernel":
                torch.bitwise_or(good.view(torch.uint8), 0, out=inp.view(torch.uint8))
            if before == "join":  # behind the nodes of two streams
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    other.copy_(good)
                torch.cuda.current_stream().wait_stream(side)
            run()
        for _ in range(3):
            if before in ("copy", "join", "kernel"):
                inp.view(torch.uint8).zero_()
            for r, x in zip(results, blank):
                r.copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            for r, x in zip(results, want):
                assert torch.equal(r.view(torch.uint8), x.view(torch.uint8))
