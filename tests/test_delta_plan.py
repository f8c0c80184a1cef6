"""The plan of the gated delta rule over packed prompts, on the CPU."""
import os
import subprocess

import pytest

from hyper_connection_residual_call_gb300 import build as b

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """Compiles one of tests/native against the plan's header and runs it."""
    include = os.path.join(os.path.dirname(os.path.dirname(b.nvcc_path())), "include")

    def run(name):
        exe = str(tmp_path_factory.mktemp("plan") / name)
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", include, "-I", b.CSRC, os.path.join(HERE, "native", name + ".cpp"), "-o", exe], check=True)
        return subprocess.run([exe], capture_output=True, text=True)

    return run


def test_walks_of_a_launch_do_not_meet(plan):
    run = plan("delta_walks")
    assert run.returncode == 0, run.stdout[:2000]
