"""Kernels that start while the one before them on the stream ends (programmatic dependent launch) read
operands that it may still be writing.  Non-coherent loads are not ordered by the wait for it, so their
sources hold none.  Read from the sources: on a GPU the mistake shows only by chance."""
import os
import re

import pytest

from self_attention_gb300.build import CSRC

NON_COHERENT = r"__ldg\b|ld\.global(\.\w+)*\.nc\b|ld\.global\.L\w+::\w+\.nc\b|__restrict__|\b__builtin_assume_noalias\b"


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def _overlapped():
    """The sources that launch such kernels, and the headers they include."""
    names = [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "launch_overlapped(" in _code(n)]
    todo, seen = list(names), set()
    while todo:
        n = todo.pop()
        if n in seen or not os.path.exists(os.path.join(CSRC, n)):
            continue
        seen.add(n)
        todo += re.findall(r'#include "(\w+\.cuh)"', _code(n))
    return sorted(seen)


def test_overlapped_sources_are_found():
    assert {"linear.cu", "norm.cu", "sum_rows.cuh", "cluster.cuh", "act.cuh"} <= set(_overlapped())


@pytest.mark.parametrize("name", _overlapped())
def test_no_non_coherent_loads(name):
    found = [line.strip() for line in _code(name).splitlines() if re.search(NON_COHERENT, line)]
    assert not found, f"{name}: {found}"


def test_every_overlapped_kernel_waits_before_it_reads():
    """Each __global__ function of these sources signals and waits once, by every thread."""
    for name in _overlapped():
        if not name.endswith(".cu"):
            continue
        kernels = re.split(r"__global__", _code(name))[1:]
        assert kernels
        for k in kernels:
            body = k.split("\n}\n")[0]
            assert body.count("grid_dep_wait()") == 1, f"{name}: {body[:80]}"


def test_tensor_maps_that_are_not_made_are_not_touched():
    """A launch may leave some of its maps out (a backward of one product alone): they are zeros, not what the
    host's stack held, and the kernel prefetches none of them."""
    code = _code("linear.cu")
    assert not re.findall(r"\b(?:GemmMaps|GemmParams|SplitParams) \w+;", code)
    block = re.search(r"if \(warp == 2 && ptx::elect_one\(\)\) \{(.*?)\n    \}\n", code, flags=re.S).group(1)
    guards = {"maps.a2": "n_items > 0", "maps.b2": "n_items > 0"}
    for line in block.splitlines():
        for name, guard in guards.items():
            if f"&{name})" in line:
                assert guard in line, line
    assert re.search(r"if \(P != Bwd \|\| p\.q\[0\]\.n_items > 0\) \{\s*ptx::tma_prefetch_desc\(&maps\.a\);\s*"
                     r"ptx::tma_prefetch_desc\(&maps\.b\);\s*\}", block)
