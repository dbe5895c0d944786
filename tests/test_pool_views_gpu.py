"""GPU: which cache decode() takes a pool for, however its pages are viewed."""
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build
from synth import SOFTMAX_SCALE, decode_inputs
from fp4_testutil import fp4_case, same_outputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _decode(inp, kv, **kw):
    out = mla.decode(inp.q.cuda(), kv, inp.page_table.cuda(), inp.kv_lens, num_heads=inp.num_heads, q_len=inp.q_len,
                     causal=False, softmax_scale=SOFTMAX_SCALE, want_f32=True, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("kw", [{}, dict(output_scale=0.5), dict(persistent_ctas=3),
                                dict(block_idx=torch.tensor([[0, 2], [0, -1]], dtype=torch.int32))])
def test_an_e4m3_pool_of_flat_pages(kw):
    inp = decode_inputs(2, 12, 1, [700, 33], 5, extra_pages=1)
    kv = inp.kv.cuda()
    want = _decode(inp, kv, **kw)
    for view in (kv.view(-1, 32 * 576), kv.view(torch.float8_e4m3fn), kv.view(torch.float8_e4m3fn).view(-1, 32 * 576)):
        same_outputs(_decode(inp, view, **kw), want)


def test_a_four_bit_pool_is_one_by_its_width():
    inp, pool = fp4_case(2, 12, 1, [700, 33], seed=6)
    want = _decode(inp, pool.cuda())
    assert torch.isfinite(want[2]).all()
    with pytest.raises(ValueError):
        _decode(inp, pool.cuda(), persistent_ctas=2)
