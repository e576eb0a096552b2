"""The prompt's kernels, read from the sources without a GPU: all of them are found, and none reads what
the kernel ahead of it may still write before it waits (cache8.cuh, launch())."""
import re

from tests.test_prompt_ops import SOURCES, _code, _kernels

READS = (r"\ba\.(pos|n_tok|first|lse|w|seq_len|status|n_q)\b\s*\[|\bc\.(table|seq_len|scale|pool|status)\b\s*[\[+)]|"
         r"\bp\.part\b|lengths_of\(|length_of\(|plan_of\(|old_weight|atomic|\breturn\b")


def test_the_kernels_are_found():
    names = [n for f in SOURCES for n, _ in _kernels(_code(f))]
    assert sorted(names) == ["heaviest_kernel", "heaviest_stream_kernel", "prompt_attend_kernel", "rotary_kernel",
                             "weigh_few_kernel", "weigh_join_kernel", "weigh_many_kernel"]


def test_every_kernel_waits_before_it_reads_anything():
    for path in SOURCES:
        for name, body in _kernels(_code(path)):
            assert body.count("before_all();") == 1, name
            assert not re.search(READS, body[:body.index("before_all();")]), name
