"""CPU: structures of the verification, key-weight and shared-prefix calls against
the header, and the refusals of verification, key weights and eviction that need no
GPU.  Addresses given here are never used: every call is refused or does nothing."""
import ctypes
import os
import subprocess

import pytest
import torch

import split_kv_mla_paged_gb300 as mla
from split_kv_mla_paged_gb300 import build as mla_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = 1 << 20


@pytest.fixture(scope="module")
def lib():
    mla_build.build()
    return mla.load_library()


def test_structures_match_the_header(tmp_path):
    types = {"mla_verify_args_t": mla.VerifyArgs, "mla_key_weights_args_t": mla.KeyWeightsArgs, "mla_shared_plan_t": mla._SharedPlanInfo}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "mla_decode.h"', "int main(void) {"]
    for name, t in types.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in t._fields_]
    (tmp_path / "t.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "t.c"), "-o", str(tmp_path / "t")], check=True)
    got = iter(int(x) for x in subprocess.run([str(tmp_path / "t")], check=True, capture_output=True).stdout.split())
    for t in types.values():
        assert next(got) == ctypes.sizeof(t)
        for f, _ in t._fields_:
            assert next(got) == getattr(t, f).offset, f


def _verify(lib, **over):
    a = dict(target_probs=AT, uniforms=AT, tokens_out=AT, accepted_out=AT, draft_tokens=AT, batch=2, q_len=3, vocab=100, probs_type=0)
    a.update(over)
    return lib.mla_verify_drafts(ctypes.byref(mla.VerifyArgs(**a)), None)


@pytest.mark.parametrize("bad,status", [
    (dict(target_probs=None), 1), (dict(uniforms=None), 1), (dict(tokens_out=None), 1), (dict(accepted_out=None), 1), (dict(draft_tokens=None), 1),
    (dict(new_lens=AT), 1), (dict(batch=-1), 1), (dict(q_len=0), 1), (dict(vocab=0), 1), (dict(probs_type=2), 1), (dict(probs_type=-1), 1),
    (dict(target_row_stride=-1), 1), (dict(draft_batch_stride=-4), 1), (dict(target_probs=AT + 2), 1), (dict(draft_probs=AT + 1, probs_type=1), 1),
    (dict(vocab=(1 << 27) + 1), 2), (dict(q_len=1025), 2), (dict(batch=(1 << 24) + 1), 2), (dict(batch=0), 0)])
def test_verify_refusals(lib, bad, status):
    assert _verify(lib, **bad) == status
    assert lib.mla_verify_drafts(None, None) == mla.MLA_ERR_INVALID_ARG


def _weights(lib, **over):
    a = dict(q=AT, kv_pages=AT, num_pages=4, page_table=AT, kv_lens=AT, lse=AT, weights=AT, weights_stride=100, max_pages_per_req=4, batch=2,
             q_len=1, num_heads=12, cache_kind=0, q_scale=1.0, kv_scale=1.0, softmax_scale=0.1, decay=1.0)
    a.update(over)
    return lib.mla_key_weights(ctypes.byref(mla.KeyWeightsArgs(**a)), None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), 1), (dict(kv_pages=None), 1), (dict(page_table=None), 1), (dict(kv_lens=None), 1), (dict(lse=None), 1), (dict(weights=None), 1),
    (dict(q=AT + 8), 1), (dict(kv_pages=AT + 4), 1), (dict(batch=-1), 1), (dict(q_len=0), 1), (dict(num_heads=0), 1), (dict(num_pages=0), 1),
    (dict(max_pages_per_req=0), 1), (dict(weights_stride=-1), 1), (dict(previous=AT, previous_stride=-1), 1), (dict(cache_kind=3), 1),
    (dict(softmax_scale=float("nan")), 1), (dict(previous=AT, previous_stride=9, decay=float("inf")), 1), (dict(cache_kind=1, kv_scale=0.5), 1),
    (dict(cache_kind=1, q_scale_dev=AT), 1), (dict(num_heads=129, q_len=8), 2), (dict(batch=65536), 2), (dict(num_pages=1 << 27), 2),
    (dict(batch=0), 0), (dict(weights_stride=0), 0)])
def test_key_weights_refusals(lib, bad, status):
    assert _weights(lib, **bad) == status
    assert lib.mla_key_weights(None, None) == mla.MLA_ERR_INVALID_ARG


def _select(lib, **over):
    a = dict(weights=AT, stride=100, lens=AT, keep=AT, batch=2, first=0, last=0, kept=AT, kept_stride=10, new_lens=AT, nw=None, nws=0)
    a.update(over)
    return lib.mla_evict_select(a["weights"], a["stride"], a["lens"], a["keep"], a["batch"], a["first"], a["last"], a["kept"], a["kept_stride"],
                                a["new_lens"], a["nw"], a["nws"], None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(weights=None), 1), (dict(lens=None), 1), (dict(keep=None), 1), (dict(kept=None), 1), (dict(new_lens=None), 1), (dict(batch=-1), 1),
    (dict(first=-1), 1), (dict(last=-1), 1), (dict(stride=-1), 1), (dict(kept_stride=-1), 1), (dict(nw=AT, nws=-1), 1), (dict(batch=65536), 2),
    (dict(stride=1 << 31), 2), (dict(batch=0), 0)])
def test_evict_select_refusals(lib, bad, status):
    assert _select(lib, **bad) == status


def _move(lib, **over):
    a = dict(src=AT, sp=4, st=AT, sw=2, dst=AT, dp=4, dt=AT, dw=2, kind=0, kept=AT, ks=10, counts=AT, batch=2)
    a.update(over)
    return lib.mla_rows_move(a["src"], a["sp"], a["st"], a["sw"], a["dst"], a["dp"], a["dt"], a["dw"], a["kind"], a["kept"], a["ks"], a["counts"],
                             a["batch"], None, None)


@pytest.mark.parametrize("bad,status", [
    (dict(src=None), 1), (dict(dst=None), 1), (dict(st=None), 1), (dict(dt=None), 1), (dict(kept=None), 1), (dict(counts=None), 1),
    (dict(src=AT + 8), 1), (dict(dst=AT + 8), 1), (dict(sp=-1), 1), (dict(dw=-1), 1), (dict(ks=-1), 1), (dict(kind=3), 1), (dict(batch=-1), 1),
    (dict(batch=65536), 2), (dict(ks=1 << 31), 2), (dict(batch=0), 0), (dict(ks=0), 0)])
def test_rows_move_refusals(lib, bad, status):
    assert _move(lib, **bad) == status


class On:
    """A CPU tensor that says it is on CUDA device `index`."""
    is_cuda = True

    def __init__(self, t, index=0):
        self._t, self._index = t, index

    def get_device(self):
        return self._index

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def no_launch(monkeypatch):
    def refused(*args, **kw):
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(mla, "_call_on", refused)


def _verify_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(target_probs=torch.zeros(2, 3, 10), draft_tokens=i32(2, 2), uniforms=torch.zeros(2, 3), tokens_out=i32(2, 3), accepted_out=i32(2),
                draft_probs=torch.zeros(2, 2, 10), query_lens=i32(2), kv_lens=i32(2), new_lens=i32(2), status=i32(1))


def _weights_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=torch.zeros(2, 1, 3, 576, dtype=torch.uint8), kv_pages=torch.zeros(4, 32, 576, dtype=torch.uint8), page_table=i32(2, 2),
                kv_lens=i32(2), lse=torch.zeros(2, 1, 3), weights=torch.zeros(2, 40), previous=torch.zeros(2, 40), query_lens=i32(2),
                q_scale_dev=torch.zeros(1), status=i32(1))


def _select_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(weights=torch.zeros(2, 40), kv_lens=i32(2), keep=i32(2), kept=i32(2, 9), new_lens=i32(2), new_weights=torch.zeros(2, 9), status=i32(1))


def _move_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros(4, 32, 576, dtype=torch.uint8)
    return dict(src_pool=pool, src_table=i32(2, 2), dst_pool=pool, dst_table=i32(2, 2), kept=i32(2, 9), counts=i32(2), status=i32(1))


def _call_verify(t):
    mla.mla_verify_drafts(**t)


def _call_weights(t):
    mla.mla_key_weights(t.pop("q"), t.pop("kv_pages"), 4, t.pop("page_table"), 2, t.pop("kv_lens"), t.pop("lse"), t.pop("weights"), 2, 1, 3, False,
                        1.0, 1.0, 0.1, cache_kind=0, **t)


def _call_select(t):
    mla.mla_evict_select(**t)


def _call_move(t):
    mla.mla_rows_move(t["src_pool"], 4, t["src_table"], t["dst_pool"], 4, t["dst_table"], t["kept"], t["counts"], cache_kind=0, status=t["status"])


CALLS = [(_call_verify, _verify_tensors), (_call_weights, _weights_tensors), (_call_select, _select_tensors), (_call_move, _move_tensors)]


@pytest.mark.parametrize("call,tensors", CALLS)
def test_bindings_check_device_type_layout_and_size(call, tensors, no_launch, lib):
    with pytest.raises(AssertionError):
        call({k: On(v) for k, v in tensors().items()})
    for name, v in tensors().items():
        wrong = [On(v, 1), v]
        if not name.endswith("_pool"):  # pools of any type that are large enough (views) are taken
            wrong.append(On(v.to(torch.float64)))
        # An empty batch is a call that does nothing.
        if name != "target_probs" and not (name in ("kv_lens", "counts") and call in (_call_select, _call_move)):
            wrong.append(On(v[:0]))
        if v.dim() > 1 and v.shape[0] > 1 and name not in ("target_probs", "draft_probs"):
            wrong.append(On(v.transpose(0, -1)))
        for w in wrong:
            t = {k: On(x) for k, x in tensors().items()}
            t[name] = w
            with pytest.raises(ValueError):
                call(t)


def test_probabilities_of_other_shapes_are_refused(no_launch, lib):
    for name, v in (("target_probs", torch.zeros(2, 30)), ("target_probs", torch.zeros(2, 3, 20)[..., ::2]), ("draft_probs", torch.zeros(2, 1, 10)),
                    ("draft_probs", torch.zeros(1, 2, 10)), ("draft_probs", torch.zeros(2, 2, 11)), ("draft_probs", torch.zeros(2, 1, 10).expand(2, 2, 10)),
                    ("target_probs", torch.zeros(1, 3, 10).expand(2, 3, 10)), ("draft_probs", torch.zeros(2, 2, 10, dtype=torch.bfloat16)),
                    ("target_probs", torch.zeros(2, 3, 10, dtype=torch.float16)), ("kv_lens", None), ("new_lens", None)):
        t = {k: On(x) for k, x in _verify_tensors().items()}
        t[name] = None if v is None else On(v)
        with pytest.raises(ValueError):
            _call_verify(t)


def test_evict_refuses_bad_host_lists(lib):
    pool = mla.PagePool(8)
    pages, w = pool.alloc(2), torch.zeros(1, 64)
    data = torch.zeros(8, 32, 576, dtype=torch.uint8)
    for lists, lens, keep in (([pages], [65], 3), ([pages], [-1], 3), ([pages], [40], -1), ([pages[:1]], [40], 3), ([[8, 9]], [40], 3),
                              ([pages, pages], [40], 3), ([pages], [40], 1.5)):
        with pytest.raises(ValueError):
            mla.evict(pool, data, lists, lens, w, keep)
    assert pool.free_pages == 6
