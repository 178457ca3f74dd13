"""The loss's workspace against what its launches write (csrc/head_plan.h, tests/head_plan_host.cpp), on the host."""
import os
import subprocess

import pytest

from paged_sparse_attention_gb300 import build


@pytest.fixture(scope="module")
def tool(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "head_plan")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "head_plan_host.cpp")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.CSRC, src, "-o", exe], check=True)
    return exe


def test_every_region_holds_what_is_written(tool):
    r = subprocess.run([tool], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
