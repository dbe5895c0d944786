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
    out, lse, _ = mla.decode(q.cuda(), pool, table.cuda(), lens, group_offsets=offsets, prefix_lens=prefixes, **args)
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
