"""CPU: the sources by which a recorded DRAM traffic is known to be that of the
kernel that runs."""
import os
import re

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = "split_kv_mla_paged_gb300/csrc"
# The public header states the ABI; its prose is not a kernel's source.
ROOTS = {"e4m3": f"{CSRC}/mla_decode.cu", "bf16": f"{CSRC}/mla_decode_bf16.cu"}


def _reachable(path):
    found, todo = set(), [path]
    while todo:
        f = todo.pop()
        if f in found:
            continue
        found.add(f)
        with open(os.path.join(ROOT, f), encoding="utf-8") as fh:
            names = re.findall(r'^\s*#include\s+"([^"]+)"', fh.read(), re.M)
        todo += [p for p in (os.path.normpath(os.path.join(os.path.dirname(f), n)) for n in names) if p.startswith(CSRC)]
    return found


@pytest.mark.parametrize("dtype", sorted(ROOTS))
def test_every_source_of_the_kernel_is_listed(dtype):
    assert set(bench.KERNEL_SOURCES[dtype]) == _reachable(ROOTS[dtype])


def test_the_hash_follows_the_kernel(monkeypatch, tmp_path):
    before = bench.kernel_hash("e4m3")
    for f in bench.KERNEL_SOURCES["e4m3"]:
        os.makedirs(tmp_path / os.path.dirname(f), exist_ok=True)
        with open(os.path.join(ROOT, f), encoding="utf-8") as fh:
            (tmp_path / f).write_text(fh.read(), encoding="utf-8")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_hash("e4m3") == before
    kernel = tmp_path / CSRC / "mla_split_kv.cuh"
    text = kernel.read_text(encoding="utf-8")
    kernel.write_text("// a comment\n" + text, encoding="utf-8")
    assert bench.kernel_hash("e4m3") == before
    kernel.write_text(text + "static int more;\n", encoding="utf-8")
    assert bench.kernel_hash("e4m3") != before
