"""CPU: the bindings take tensors, not numbers that could be addresses."""
import numpy as np
import pytest
import torch

import split_kv_mla_paged_gb300 as mla


class Library:
    """Stands in for the library: no call of these tests may get to it."""

    def __getattr__(self, name):
        def reached(*args):
            raise AssertionError(f"{name} was reached")
        return reached


@pytest.fixture(autouse=True)
def _no_library(monkeypatch):
    monkeypatch.setattr(mla, "load_library", lambda: Library())


T = torch.zeros(1)


def _decode(**over):
    a = dict(q=T, kv=T, table=T, lens=T, splits=T, chunks=T, ws=T, out=T, lse=T)
    a.update(over)
    mla.mla_decode(a["q"], a["kv"], 1, a["table"], 1, a["lens"], a["splits"], a["chunks"], 1, 1, 1, 1, 1, False, 1.0, 1.0, 1.0, a["ws"], 256,
                   a["out"], a["lse"], stream=0)


def test_tensors_get_to_the_library():
    with pytest.raises(AssertionError, match="reached"):
        _decode()


@pytest.mark.parametrize("name", ["q", "kv", "table", "lens", "splits", "chunks", "ws", "out", "lse"])
@pytest.mark.parametrize("number", [5, 1 << 20, True])
def test_numbers_are_no_addresses(name, number):
    with pytest.raises((AttributeError, TypeError, ValueError)):
        _decode(**{name: number})


def test_other_calls_refuse_numbers():
    for call in (lambda: mla.mla_decode_workspace_init(7, 256, stream=0),
                 lambda: mla.mla_merge(9, T, 1, 1, 1, T, stream=0),
                 lambda: mla.mla_kv_append(T, 1, 3, T, T, 1, 1, T, 1, 1.0, stream=0)):
        with pytest.raises((AttributeError, TypeError, ValueError)):
            call()
    assert mla._ptr(None) is None and mla._ptr(np.zeros(2)) > 0
