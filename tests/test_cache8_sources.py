"""Kernels of the 8-bit cache may begin while the kernel ahead of them runs (cache8.cuh, launch()).  What
that one still writes may not be read before the wait, nor through the read-only path, whose data
must not change while a kernel runs.  Read from the sources, without a GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "eviction_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "cache8*.cu*")))


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _kernels(code):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__[^{;]*?(\w+)\((?:[^()]|\([^()]*\))*\)\s*\{", code):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[at], 0)
            at += 1
        yield m.group(1), code[m.end():at - 1]


def test_the_sources_are_found():
    names = [n for f in FILES for n, _ in _kernels(_code(f))]
    assert sorted(names) == ["append_kernel", "attend_few_kernel", "attend_many_join_kernel",
                             "attend_many_kernel", "compact_kernel", "fork_copy_kernel", "fork_kernel",
                             "free_kernel", "gather_kernel", "grow_kernel"]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_load_through_the_read_only_path(path):
    code = _code(path)
    assert not re.search(r"__ldg\b|\.global\.nc\b|__restrict__", code)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_every_kernel_waits_before_it_reads(path):
    for name, body in _kernels(_code(path)):
        assert body.count("before_all();") == 1, name
        ahead = body[:body.index("before_all();")]
        assert not re.search(r"\bc\.(table|seq_len|free_top|ref_count|err|status)\b\s*[\[)]|\*\s*c\.|"
                             r"atomic|\breturn\b", ahead), name
