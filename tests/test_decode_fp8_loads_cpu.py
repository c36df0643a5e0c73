"""Kernels that are launched as programmatic dependents read what the grid ahead of them may
still be writing when they start: never by the non-coherent path, and not before they wait."""
import os
import re

import pytest

from exact_attention_55_gb300 import build

CSRC = build.CSRC


def code_of(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def dependent_sources():
    """The files with such a launch or wait."""
    names = [n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))]
    return sorted(n for n in names if re.search(r"griddepcontrol\.wait|ProgrammaticStreamSerialization", code_of(n)))


def test_the_files_are_found():
    assert {"decode_fp8.cu", "decode_fp8.cuh", "decode_fp8_wide.cu"} <= set(dependent_sources())


@pytest.mark.parametrize("name", dependent_sources())
def test_no_loads_by_the_non_coherent_path(name):
    code = code_of(name)
    assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code)


@pytest.mark.parametrize("name", dependent_sources())
def test_kernels_wait_before_they_read(name):
    """A kernel that waits names none of its global inputs before."""
    bodies = [b for b in re.split(r"__global__", code_of(name))[1:] if "griddepcontrol.wait" in b]
    assert bodies
    for body in bodies:
        before = body[body.index("{"):body.index("griddepcontrol.wait")]
        assert not re.search(r"p\.(q|ks|vs|kc|vc|ws|o|lse|page_table|seq_lens)\b|tma_load|dec8_line|dec8_seq", before)
