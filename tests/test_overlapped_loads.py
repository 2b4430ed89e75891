"""Kernels that a programmatic launch starts before their predecessor ends may not read what
it writes through the read-only path: those loads are for data that nobody writes while the
kernel runs, and griddepcontrol.wait does not order them (CPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "split_kv_decode_gb300", "csrc")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def overlapped():
    """The sources with a griddep_wait: their kernels are launched ahead of time."""
    return [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "griddep_wait" in code(f)]


def test_the_overlapped_kernels_are_known():
    assert overlapped() == ["append.cu", "combine.cu", "gqa_8bit.cu", "tables.cu"]


@pytest.mark.parametrize("name", overlapped())
def test_no_read_only_loads_behind_the_wait(name):
    found = [l.strip() for l in code(name).splitlines()
             if re.search(r"__ldg\s*\(|ld\.global\.nc|LDG", l)]
    assert not found, found


def test_tma_reads_of_the_8bit_pools_are_fenced():
    # the append writes the pools by ordinary stores; copies read them through the async proxy
    text = code("gqa_8bit.cu")
    wait, fence = text.index("griddep_wait();"), text.find("fence_proxy_async_global();")
    assert wait < fence < text.index("tma_load_4d(")


def test_the_append_lets_others_start_only_after_its_own_wait():
    # a kernel two places on (a projection whose weights are fetched before its wait) may start
    # once the append says so; what ran before the append must have ended by then
    text = code("append.cu")
    text = text[text.index("append_kernel("):]
    assert text.index("griddep_wait();") < text.index("griddep_launch_dependents();")
