"""CPU: loads of kernels that are launched as programmatic dependents.

Such a kernel is alive while the one before it on the stream still writes, so that it may
not read what that one writes through the non-coherent path, which is for data that stays
read-only for the kernel's whole life.  No run shows this reliably, the source does."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "split_kv_mla_paged_gb300", "csrc")
# The loads of the split kernels choose by kShared: only the decode over shared prefixes is
# a programmatic dependent of other calls.
CHOICE = re.compile(r"if constexpr \(kShared\)\s*return ldg_stream8?_coherent\(p\);\s*else\s*return ldg_stream8?\(p\);")


def _sources():
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(f).read())
        if "ProgrammaticStreamSerialization" in text:
            yield os.path.basename(f), text


SOURCES = dict(_sources())


def test_the_programmatic_launches_are_found():
    assert sorted(SOURCES) == ["evict.cu", "key_weights.cu", "mla_decode_bf16.cu", "mla_merge.cu", "mla_split_kv.cuh", "verify.cu"]


@pytest.mark.parametrize("name", sorted(SOURCES))
def test_no_non_coherent_loads(name):
    text = CHOICE.sub("", SOURCES[name])
    assert not re.search(r"\bldg_stream8?\(|\b__ldg\(|\.nc\b|__restrict__", text)
