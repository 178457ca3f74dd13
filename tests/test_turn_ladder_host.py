"""The rotary ladders' frequencies (csrc/turn_ladder.h, tests/turn_ladder_host.cpp) against
60-digit arithmetic, on the host."""
import os
import struct
import subprocess
from decimal import Decimal as D
from decimal import getcontext

import pytest

from paged_sparse_attention_gb300 import build

getcontext().prec = 60
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def tool(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("ladder") / "turn_ladder")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "turn_ladder_host.cpp")
    # -O3 as in the library; contraction of products into sums is a compiler's default on Arm
    subprocess.run(["g++", "-O3", "-std=c++17", "-ffp-contract=fast", "-I", build.CSRC, src, "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("theta", [1e6, 1e4, 500000.0, 2.0, 1.0000001192092896, 3e38, 10007.3])
@pytest.mark.parametrize("c", [1, 2, 3, 5, 21, 22, 32, 43, 64])
def test_frequencies(tool, theta, c):
    out = subprocess.run([tool, repr(theta), str(c)], check=True, capture_output=True, text=True).stdout.split()
    exact_theta = D(struct.unpack("f", struct.pack("f", theta))[0])
    for r in range(c):
        got = D(int(out[2 * r], 16) * 2 ** 32 + int(out[2 * r + 1], 16)) / D(2 ** 96)
        want = (-exact_theta.ln() * r / c).exp() / (2 * PI)
        assert abs(got - want) < D(2) ** -95, (theta, c, r, got - want)  # one unit for what is cut off, one before
