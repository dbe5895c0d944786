"""GPU: expired waits of key weights where the epilogue warps still have steps with
new query rows before them, at whose named barriers they have to meet."""
import functools
import time

import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE
from test_key_weights_gpu import _case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


# Many requests of one or two tiles (every step of a CTA has rows of its own), row groups
# in turn, and both.
CASES = {"short": (12, 1, [130] * 500), "groups": (128, 8, [152 * 128 * 2]), "both": (100, 4, [300, 128, 40] * 90)}


@functools.lru_cache(maxsize=1)
def _inputs(kind, case):
    heads, q_len, lens = CASES[case]
    inp, pool, _, _ = _case(kind, heads, q_len, lens, 2)
    return inp.q.cuda(), pool.cuda(), inp.page_table.cuda(), torch.zeros(len(lens), q_len, heads, device="cuda")


@pytest.mark.parametrize("role,step", [(0, 0), (0, 2), (1, 0), (1, 1), (1, 3), (3, 0), (3, 1), (3, 2)])
@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("kind", ["fp8", "bf16", "fp4"])
def test_the_call_ends_and_the_next_one_is_right(kind, case, role, step):
    heads, q_len, lens = CASES[case]
    qd, kvd, pt, lse = _inputs(kind, case)
    kw = dict(num_heads=heads, q_len=q_len, causal=q_len > 1, softmax_scale=SOFTMAX_SCALE)
    ref = mla.key_weights(qd, kvd, pt, lens, lse, **kw)
    for _ in range(10):
        began = time.monotonic()
        mla.mla_debug_set_expire(role, step)
        try:
            with pytest.raises(mla.MlaError) as err:
                mla.key_weights(qd, kvd, pt, lens, lse, **kw)
            assert err.value.status == mla.MLA_ERR_TIMEOUT
        finally:
            mla.mla_debug_set_expire(-1)
        assert time.monotonic() - began < 1.0  # no wait ran to its limit of some two seconds
    assert torch.equal(mla.key_weights(qd, kvd, pt, lens, lse, **kw), ref)
