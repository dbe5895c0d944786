"""Seeded randomized sweep of the 4-bit decode: the shapes, plans and options of
the E4M3 sweep over re-encoded caches, against the oracle, the E4M3 decode of
the expanded cache and the item-list launch."""
import numpy as np
import pytest
import torch

import oracle
import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build
from synth import PAGE_SIZE
from fp4_testutil import equal_outputs, fp4_case, same_outputs
from mla_testutil import assert_parity
from test_fuzz_gpu import _case as random_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


@pytest.mark.parametrize("seed", range(500, 560))
def test_random_case(seed):
    H, q_len, B, lens, causal, opts, plan_kind, target, scale = random_case(seed)
    inp, pool = fp4_case(B, H, q_len, lens, seed=seed, extra_pages=1)
    sel = opts.get("block_idx")
    plan_lens = lens if sel is None else [PAGE_SIZE * sel.shape[1]] * B
    if plan_kind == "gb300":
        plan = mla.mla_decode_plan(plan_lens, H, q_len, sm_count=152)
    else:
        plan = mla.mla_decode_plan(plan_lens, H, q_len, target_ctas=target)

    def run(kv, items):
        out = mla.decode(inp.q.cuda(), kv.cuda(), inp.page_table.cuda(), inp.kv_lens, num_heads=H, q_len=q_len, causal=causal,
                         softmax_scale=scale, plan=plan, want_f32=True, use_items=items, **opts)
        torch.cuda.synchronize()
        return out
    got = run(pool, False)
    same_outputs(got, run(pool, True))
    out, lse, o32 = got
    ref_o, ref_l = oracle.decode_rows(inp.q, inp.kv, inp.page_table, inp.kv_lens, q_len=q_len, num_heads=H, causal=causal,
                                      softmax_scale=scale, **opts)
    fin = np.isfinite(ref_l).reshape(-1)
    assert np.array_equal(np.isfinite(lse.cpu().numpy().reshape(-1)), fin), "empty-row pattern"
    keep = torch.from_numpy(fin).cuda()
    o = out.reshape(-1, 512)
    assert (o[~keep] == 0).all()
    if fin.any():
        assert_parity(o[keep], lse.reshape(-1)[keep], ref_o.reshape(-1, 512)[fin], ref_l.reshape(-1)[fin], what=f"case {seed}")
    assert torch.equal(o32.to(torch.bfloat16), out)
    # The E4M3 cache's masked rows may hold NaNs (the tail of a page that a key
    # window ends in); with those cleared the two decodes agree.
    want = run(torch.where((inp.kv & 0x7F) == 0x7F, 0, inp.kv), False)
    lse0, lse1 = (torch.where(keep, x[1].reshape(-1), 0.0) for x in (got, want))
    equal_outputs((out, lse0, o32), (want[0], lse1, want[2]), H * q_len)
