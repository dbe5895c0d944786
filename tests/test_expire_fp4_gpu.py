"""GPU: test hooks for waits that a 4-bit decode does not make change nothing.

Role 4 (a free P^T buffer) has no wait in 16-row CTAs, and role 5 only one, at
tile 0.  The reference is taken before a hook is set, under the same plan."""
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE
from fp4_testutil import fp4_case, same_outputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


@pytest.mark.parametrize("q_len, role, tile", [(1, 4, 0), (1, 4, 3)] + [(q, 5, t) for q in (1, 2, 4, 8) for t in (1, 3)])
def test_hooks_without_a_wait_leave_the_results(q_len, role, tile):
    inp, pool = fp4_case(1, 12, q_len, [5000], seed=97)
    d = [t.cuda() for t in (inp.q, pool, inp.page_table)]

    def call():
        out = mla.decode(*d, inp.kv_lens, num_heads=12, q_len=q_len, causal=q_len > 1, softmax_scale=SOFTMAX_SCALE,
                         want_f32=True, target_ctas=2)
        torch.cuda.synchronize()
        return out
    want = call()
    mla.mla_debug_set_expire(role, tile)
    try:
        same_outputs(call(), want)
    finally:
        mla.mla_debug_set_expire(-1)
