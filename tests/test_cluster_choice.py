"""The cluster size of the page plan where the device cannot hold 16 CTAs (C++, no GPU)."""
import os
import subprocess

import weight_streaming_warp_gb300 as wsw

CSRC = os.path.join(os.path.dirname(wsw.__file__), "csrc")
PROGRAM = r"""
#include <cstdio>

#include "cluster_choice.h"

int main() {
    wsw::ClusterChoice choice;
    int asked = 0;
    auto answer = [&](bool yes) { return [&asked, yes] { ++asked; return yes; }; };
    const unsigned got[] = {choice.of(0, answer(false)), choice.of(0, answer(true)), choice.of(1, answer(true)),
                            choice.of(1, answer(false))};
    std::printf("%u %u %u %u asked %d\n", got[0], got[1], got[2], got[3], asked);
}
"""


def test_a_device_that_cannot_hold_sixteen_takes_eight(tmp_path):
    src = tmp_path / "choice.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-pthread", "-I", CSRC, str(src), "-o", str(tmp_path / "choice")], check=True)
    r = subprocess.run([str(tmp_path / "choice")], capture_output=True, text=True, timeout=60, check=True)
    assert r.stdout == "8 8 16 16 asked 2\n"
