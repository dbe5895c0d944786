"""GPU: verification of drafted tokens where little lies between a kernel's start and
its exchange across CTAs, against the definition in whole numbers."""
import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build
from test_verify_gpu import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


@pytest.mark.parametrize("vocab", [1, 3, 40])
def test_many_requests_of_a_small_vocabulary(vocab):
    # Most warps have no tokens and hand over their 0 at once; more clusters than run at a time.
    g = torch.Generator().manual_seed(vocab)
    target = torch.softmax(torch.randn(3000, 1, vocab, generator=g), -1)
    u = torch.rand(3000, 1, generator=g)
    none = torch.zeros(3000, 0, dtype=torch.int32)
    ref = _check(target, None, none, u, torch.ones(3000, dtype=torch.int32))
    for _ in range(20):
        tokens, accepted, _ = mla.verify_drafts(target.cuda(), none.cuda(), u.cuda())
        assert np.array_equal(tokens.cpu().numpy(), ref[0]) and not accepted.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_single_tokens_with_draft_probabilities_of_no_rows(dtype):
    target, _, tokens, u, lens = _inputs(5, 1, 777, 4, dtype)
    _check(target, torch.zeros(5, 0, 777, dtype=dtype), tokens, u, lens)


def test_the_smallest_uniform_numbers():
    # Probabilities of a few units of 2^-50 in front: thresholds just below, at and above
    # their sums, where u has bits below 2^-64.
    units = np.array([1, 2, 4, 1 << 20, (1 << 50) - (1 << 20) - 7], np.float64) * 2.0 ** -50
    row = torch.from_numpy(units.astype(np.float32))
    assert (row.double().numpy()[:4] == units[:4]).all()
    u = [0.0, -0.0, 2.0 ** -149, 2.0 ** -126, 2.0 ** -65, 2.0 ** -64, 2.0 ** -51]
    for n in (1, 3, 7, 7 + (1 << 20)):
        at = np.float32(n * 2.0 ** -50)
        u += [at, np.nextafter(at, np.float32(0)), np.nextafter(at, np.float32(1))]
    u = torch.tensor(np.array(u, np.float32))[:, None]
    ref = _check(row.repeat(len(u), 1, 1), None, torch.zeros(len(u), 0, dtype=torch.int32), u, torch.ones(len(u), dtype=torch.int32))
    assert {0, 1, 2, 3, 4} == set(ref[0][:, 0].tolist())
