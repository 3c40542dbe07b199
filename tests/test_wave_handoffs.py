"""CPU test on the sources: lanes of one wave that exchange values through LDS
do so around wave_handoff() (device_common.h).  The hardware keeps a wave's LDS
operations in order, but without a fence the compiler need not: to it another
lane's store is a data race, and it may hand a lane its own earlier store."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_mssm_amd", "csrc")
FENCE = r"(?:wave_handoff|__syncthreads|tile_barrier)\(\);"


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, head):
    """The braces' content behind the first match of `head`."""
    at = re.search(head, text)
    assert at, head
    i = text.index("{", at.end())
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError(head)


def fenced(text, first, then):
    """Every text between a match of `first` and the next one of `then` holds a fence."""
    found = re.findall(f"{first}(.*?){then}", text, re.S)
    assert found, (first, then)
    return all(re.search(FENCE, part) for part in found)


def test_the_fence_binds_compiler_and_wave():
    fence = body(source("device_common.h"), r"void wave_handoff\(\)")
    assert "__ATOMIC_RELEASE" in fence and "__ATOMIC_ACQUIRE" in fence and "__builtin_amdgcn_wave_barrier" in fence


@pytest.mark.parametrize("function,first,then", [
    (r"uint64_t best_of\(", r"rank \+=", r"sorted\[lane\] = 0"),
    (r"uint64_t best_of\(", r"sorted\[lane\] = 0;", r"sorted\[rank\] ="),
    (r"uint64_t best_of\(", r"sorted\[rank\] =", r"return lane < K"),
    (r"int pick_in_passes\(", r"hits\[k\] =", r"return K"),
    (r"void beam_part_kernel\(", r"hits\[place\] =", r"pick_in_passes"),
    (r"void beam_part_kernel\(", r"best_of\(held, n", r"hits\[lane\] ="),
    (r"void beam_part_kernel\(", r"all\[total \+ lane\] =", r"all\[i \* 64"),
])
def test_beam_candidates(function, first, then):
    assert fenced(body(source("beam.hip"), function), first, then)


def test_linear_output_blocks():
    kernel = body(source("linear.hip"), r"void linear_tile_kernel\(")
    stage = body(kernel, r"auto stage =")
    assert re.search(rf"^{{\s*{FENCE}", stage), "the block before may still be read"
    assert re.search(rf"{FENCE}\s*}}$", stage), "other lanes read the block next"
    # nothing else writes or reads the blocks: stored by stage(), read by the calls behind it
    assert len(re.findall(r"out\.stage\(", kernel)) == len(re.findall(r"out\.stage\(", stage)) == 1
