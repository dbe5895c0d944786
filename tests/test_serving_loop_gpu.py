"""GPU: the serving loop of the user's documentation, run as it stands there."""
import os
import re

import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build

pytestmark = pytest.mark.gpu

DOCUMENT = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_the_serving_loop():
    mla_build.build()
    blocks = re.findall(r"```python\n(.*?)```", open(DOCUMENT).read(), re.S)
    code = [b for b in blocks if "for step in range(steps)" in b]
    assert len(code) == 1
    q_len, heads, vocab, total, prompt, steps = 4, 12, 777, 4000, 18985, 12
    g = torch.Generator().manual_seed(3)
    pool, kv_pages = mla.PagePool(total), torch.zeros(total, 32, 576, dtype=torch.uint8, device="cuda")
    seen_lens = []

    def table_of(lists):
        out = torch.zeros(len(lists), max(len(p) for p in lists), dtype=torch.int32)
        for b, p in enumerate(lists):
            out[b, :len(p)] = torch.from_numpy(np.asarray(p, np.int32))
        return out.cuda()

    def write(table, starts, ends):
        at = [(b, j) for b in range(len(starts)) for j in range(starts[b], ends[b])]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        mla.mla_prologue(len(at), positions=i32([j for _, j in at]), kv_rows=torch.randn(len(at), 576, generator=g).bfloat16().cuda(),
                         req_idx=i32([b for b, _ in at]), page_table=table, max_pages_per_req=table.shape[1], batch=len(starts),
                         kv_pages=kv_pages, num_pages=total, cache_kind=mla.CACHE_FP8, status=status)
        assert int(status) == 0

    def append_block(_, table, ends):
        write(table, [n - q_len for n in ends], ends)
        seen_lens.append(list(ends))
        q = (torch.randn(len(ends), q_len, heads, 576, generator=g) * 0.5).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        probs = torch.softmax(torch.randn(len(ends), q_len - 1, vocab, generator=g), -1)
        drafts = torch.stack([torch.multinomial(p, 1, generator=g)[:, 0] for p in probs]).int()
        return q, drafts.cuda(), probs.cuda()

    base = pool.alloc((prompt + 31) // 32)
    write(table_of([base]), [0], [prompt])
    forked, src, dst, rows = pool.fork(base, prompt, 2)
    mla.copy_pages(kv_pages, kv_pages, src, dst, rows)
    at = dict(mla=mla, np=np, torch=torch, pool=pool, kv_pages=kv_pages, steps=steps, q_len=q_len, page_lists=[base, *forked],
              kv_lens=[prompt] * 3, table_of=table_of, append_block=append_block, uniforms=torch.rand(3, q_len, generator=g).cuda(),
              target_probs=lambda out: torch.softmax(torch.randn(3, q_len, vocab, generator=g), -1).cuda())
    exec(code[0], at)
    assert len(seen_lens) == steps and max(seen_lens[0]) > prompt and max(seen_lens[-1]) < 17000
    lens, weights = at["kv_lens"], at["weights"]
    # With every step's rows a request has gathered heads * q_len * (1 + 0.9 + ...) at most, less
    # what went with its evicted keys and rejected drafts.
    for b, n in enumerate(lens):
        assert 0.5 * heads * q_len < float(weights[b, :n].sum()) < heads * q_len * 10.0
    assert pool.free_pages == total - sum(len(p) for p in at["page_lists"])
