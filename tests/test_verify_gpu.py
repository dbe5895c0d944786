"""GPU: verification of drafted tokens (mla_verify_drafts).

The plain implementation walks the definition with Python integers: a probability
is a multiple of 2^-50 as the header says, sums are exact, so every output has to
be equal, whatever the sizes."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mla_build.build()
    mla.load_library()


def _fixed(row):
    """Probabilities as integers in units of 2^-50 (nearest, ties to even)."""
    x = np.nan_to_num(row.astype(np.float64), nan=0.0).clip(0.0, 1.0) * 2.0 ** 50
    return np.rint(x).astype(np.int64).astype(object)


def _plain(target, draft, tokens, u, query_lens, lens):
    batch, q_len, vocab = target.shape
    out = np.full((batch, q_len), -1, np.int32)
    accepted, new = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        n = (q_len if query_lens is None else query_lens[b]) - 1
        a = 0
        while a < n:
            x = tokens[b, a]
            if not 0 <= x < vocab:
                break
            p, q = float(target[b, a, x]), 1.0 if draft is None else float(draft[b, a, x])
            if np.isnan(p) or np.isnan(q) or not Fraction(float(u[b, a])) * Fraction(q) < Fraction(p):
                break
            out[b, a] = x
            a += 1
        w = _fixed(target[b, a])
        if a < n:
            if draft is not None:
                rest = np.maximum(w - _fixed(draft[b, a]), 0)
            else:
                rest = w.copy()
                if 0 <= tokens[b, a] < vocab:
                    rest[tokens[b, a]] = 0
            w = rest if rest.sum() > 0 else w
        c = np.cumsum(w)
        past = np.nonzero(c > Fraction(float(u[b, -1])) * int(c[-1]))[0] if c[-1] > 0 else []
        out[b, a] = past[0] if len(past) else -1
        accepted[b], new[b] = a, lens[b] - n + a
    return out, accepted, new


def _inputs(batch, q_len, vocab, seed, dtype=torch.float32, spread=3.0, near=0.4):
    g = torch.Generator().manual_seed(seed)
    z = spread * torch.randn(batch, q_len, vocab, generator=g)
    target = torch.softmax(z, -1).to(dtype)
    draft = torch.softmax(z[:, :max(q_len - 1, 1)] + near * torch.randn(batch, max(q_len - 1, 1), vocab, generator=g), -1).to(dtype)
    tokens = torch.stack([torch.multinomial(d.float(), 1, generator=g)[:, 0] for d in draft])[:, :q_len - 1].int()
    return target, draft[:, :q_len - 1], tokens, torch.rand(batch, q_len, generator=g), torch.randint(q_len, 9999, (batch,), generator=g).int()


def _check(target, draft, tokens, u, lens, query_lens=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = mla.verify_drafts(dev(target), dev(tokens), dev(u), draft_probs=dev(draft), kv_lens=dev(lens),
                            query_lens=None if query_lens is None else torch.tensor(query_lens, dtype=torch.int32).cuda())
    ref = _plain(target.float().numpy(), None if draft is None else draft.float().numpy(), tokens.numpy(), u.numpy(), query_lens, lens.numpy())
    for x, y in zip(got, ref):
        assert np.array_equal(x.cpu().numpy(), y)
    return ref


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("batch,q_len,vocab", [(1, 1, 1), (2, 2, 1), (3, 4, 7), (2, 3, 31), (1, 2, 128), (5, 8, 1000), (2, 5, 8191),
                                               (3, 2, 8192), (2, 4, 50021), (4, 8, 32000), (1, 40, 515)])
def test_matches_the_definition(batch, q_len, vocab, drafts, dtype):
    target, draft, tokens, u, lens = _inputs(batch, q_len, vocab, batch * vocab, dtype)
    _check(target, draft if drafts else None, tokens, u, lens)


def test_every_number_of_accepted_drafts():
    target, draft, tokens, u, lens = _inputs(64, 5, 300, 5, near=0.8)
    accepted = _check(target, draft, tokens, u, lens)[1]
    assert set(accepted.tolist()) == {0, 1, 2, 3, 4}


def test_ragged_query_counts():
    target, draft, tokens, u, lens = _inputs(6, 5, 777, 6)
    _check(target, draft, tokens, u, lens, [1, 2, 3, 4, 5, 1])


def test_borders():
    # Eighths: every sum and threshold is exact, and u on a border belongs to the token behind it.
    p = torch.tensor([0.125, 0.0, 0.25, 0.0, 0.5, 0.125])
    target = p.repeat(9, 1, 1)
    u = torch.tensor([[0.0], [0.124], [0.125], [0.374], [0.375], [0.874], [0.875], [0.9999999], [0.99999994]])
    got = _check(target, None, torch.zeros(9, 0, dtype=torch.int32), u, torch.ones(9, dtype=torch.int32))[0]
    assert got[:, 0].tolist() == [0, 0, 2, 2, 4, 4, 5, 5, 5]


def test_acceptance_is_strict_and_exact():
    # u q == p is a rejection; one step below is not.
    target = torch.tensor([0.25, 0.75]).repeat(2, 2, 1)
    draft = torch.tensor([0.5, 0.5]).repeat(2, 1, 1)
    u = torch.tensor([[0.5, 0.1], [np.nextafter(np.float32(0.5), np.float32(0)), 0.1]])
    got = _check(target, draft, torch.zeros(2, 1, dtype=torch.int32), u, torch.full((2,), 9, dtype=torch.int32))
    assert got[1].tolist() == [0, 1] and got[0][:, 0].tolist() == [1, 0]


def test_rejection_with_equal_probabilities_draws_from_the_target():
    # q == p, yet the draft has probability 0 in both: the residual is 0 everywhere.
    p = torch.tensor([0.0, 0.5, 0.25, 0.25])
    target, draft = p.repeat(1, 2, 1), p.repeat(1, 1, 1)
    got = _check(target, draft, torch.zeros(1, 1, dtype=torch.int32), torch.tensor([[0.0, 0.6]]), torch.full((1,), 9, dtype=torch.int32))
    assert got[0].tolist() == [[2, -1]]


def test_odd_values_count_as_nothing():
    nan, inf = float("nan"), float("inf")
    rows = torch.tensor([[nan, -1.0, 0.0, 0.25, nan], [0.0, 0.0, 0.0, 0.0, 0.0], [nan] * 5, [inf, 0.0, 2.0, 0.0, 0.0], [0.0, 1e-30, 0.0, 0.0, 0.0]])
    target = rows[:, None]
    lens = torch.ones(5, dtype=torch.int32)
    got = _check(target, None, torch.zeros(5, 0, dtype=torch.int32), torch.full((5, 1), 0.7), lens)[0]
    assert got[:, 0].tolist() == [3, -1, -1, 2, -1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows(dtype):
    target, draft, tokens, u, lens = _inputs(3, 4, 1001, 12, dtype)
    wide = torch.zeros(3, 6, 1024, dtype=dtype, device="cuda")
    wide[:, 1:5, 5:1006] = target.cuda()
    thin = torch.zeros(4, 3, 1003, dtype=dtype, device="cuda")
    thin[:3, :, :1001] = draft.cuda()
    got = mla.verify_drafts(wide[:, 1:5, 5:1006], tokens.cuda(), u.cuda(), draft_probs=thin[:3, :, :1001], kv_lens=lens.cuda())
    ref = _plain(target.float().numpy(), draft.float().numpy(), tokens.numpy(), u.numpy(), None, lens.numpy())
    for x, y in zip(got, ref):
        assert np.array_equal(x.cpu().numpy(), y)


def test_bad_requests_are_reported():
    target, draft, tokens, u, lens = _inputs(3, 4, 100, 13)
    tokens[1, 0] = 100
    ref = _plain(target.numpy(), draft.numpy(), tokens.numpy(), u.numpy(), None, lens.numpy())
    out, acc = torch.full((3, 4), -7, dtype=torch.int32).cuda(), torch.full((3,), -7, dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    args = (target.cuda(), tokens.cuda(), u.cuda(), out, acc)
    mla.mla_verify_drafts(*args, draft_probs=draft.cuda(), status=status)
    assert int(status) == mla.MLA_ERR_INVALID_ARG
    assert np.array_equal(out.cpu().numpy(), ref[0]) and np.array_equal(acc.cpu().numpy(), ref[1])
    status.zero_()
    out.fill_(-7)
    ql = torch.tensor([4, 5, 0], dtype=torch.int32).cuda()
    mla.mla_verify_drafts(*args, draft_probs=draft.cuda(), query_lens=ql, status=status)
    assert int(status) == mla.MLA_ERR_INVALID_ARG
    assert np.array_equal(out[0].cpu().numpy(), ref[0][0]) and (out[1:] == -7).all()


def test_lengths_in_place_another_stream_and_a_graph():
    target, draft, tokens, u, lens = (t.cuda() for t in _inputs(4, 4, 5000, 14))
    ref = _plain(target.cpu().numpy(), draft.cpu().numpy(), tokens.cpu().numpy(), u.cpu().numpy(), None, lens.cpu().numpy())
    out, acc = torch.empty(4, 4, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mla.mla_verify_drafts(target, tokens, u, out, acc, draft_probs=draft, kv_lens=lens, new_lens=lens)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), ref[0]) and np.array_equal(lens.cpu().numpy(), ref[2])
    u.copy_(torch.rand(4, 4, generator=torch.Generator().manual_seed(3)))
    again = _plain(target.cpu().numpy(), draft.cpu().numpy(), tokens.cpu().numpy(), u.cpu().numpy(), None, lens.cpu().numpy())
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), again[0]) and np.array_equal(lens.cpu().numpy(), again[2])
