"""CPU test: h_final of the gated delta rule may be h0's own buffer, also where a sequence is gone through in pieces
by workgroups that nothing orders.  Asked of the library's own rule (csrc/gdr.h, compiled alone with g++), which
launch's workgroups read h0 and which write h_final; and on the source, that the kernels go by it."""
import os
import re
import subprocess

from test_wave_handoffs import CSRC, body, source

ROOT = os.path.dirname(CSRC[:CSRC.rindex(os.sep)])
MAIN = r"""
#include <cstdio>
#include "gdr.h"
int main() {
    for (int ends = 0; ends < 2; ++ends)
        for (int first = 0; first < 2; ++first)
            for (int last = 0; last < 2; ++last)
                std::printf("%d%d%d %d %d\n", ends, first, last, mssm::gdr_reads_h0(ends, first, last), mssm::gdr_writes_h_final(ends, last));
}
"""


def rule(folder):
    """(launch for the pieces' ends, first piece, last piece) -> (reads h0, writes h_final)"""
    src, exe = os.path.join(folder, "rule.cpp"), os.path.join(folder, "rule")
    with open(src, "w") as f:
        f.write(MAIN)
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-w", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, src, "-o", exe], check=True)
    lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    return {tuple(c == "1" for c in k): (r == "1", w == "1") for k, r, w in (x.split() for x in lines if x)}


def test_no_workgroup_reads_what_another_writes_in_the_same_launch(tmp_path):
    does = rule(str(tmp_path))
    for pieces in range(1, 6):
        places = [(i == 0, i == pieces - 1) for i in range(pieces)]
        read = set()
        for ends in (True, False):
            here = [p for p in places if not (ends and p[1])]  # the pass for the ends leaves the last piece out
            readers = [i for i, p in enumerate(here) if does[(ends, *p)][0]]
            writers = [i for i, p in enumerate(here) if does[(ends, *p)][1]]
            assert all(r == w for r in readers for w in writers), (pieces, ends)
            assert writers == ([] if ends else [pieces - 1])
            read.update(readers)
        assert read == {0}  # the first piece's state comes from h0, by one launch or the other


def test_the_kernel_goes_by_it():
    kernel = body(source("gdr_fwd.hip"), r"void gdr_fwd_kernel\(FwdArgs a\)")
    assert re.findall(r"[^;{}]*\ba\.h0\b[^;{}]*;", kernel) == ["\n    const float* start = initial ? a.h0 : ENDS ? nullptr : a.starts;"]
    assert "const bool initial = !PIECES || gdr_reads_h0(ENDS, sp.first, sp.last);" in kernel
    (write,) = re.findall(r"if \(([^{}]*)\) \{[^{}]*for[^{}]*a\.h_final \+", kernel)
    assert "gdr_writes_h_final(ENDS, sp.last)" in write
    # the launch for the ends leaves what the other one takes
    assert re.search(r"if \(initial && of_v && col < K\)\s*\*reinterpret_cast<f32x4\*>\(a\.starts \+", kernel)
