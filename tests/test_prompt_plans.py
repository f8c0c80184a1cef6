"""The plans of the operators over packed prompts, on the CPU: how the delta rule is cut into segments, how the
attention counts its blocks."""
import os
import subprocess

import pytest

from hyper_connection_residual_call_gb300 import binding as B, build as b

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def lib():
    b.build()
    return B.library()


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """Compiles one of tests/native against the plans' headers and runs it."""
    include = os.path.join(os.path.dirname(os.path.dirname(b.nvcc_path())), "include")

    def run(name):
        exe = str(tmp_path_factory.mktemp("plan") / name)
        subprocess.run(["g++", "-std=c++17", "-O1", "-I", include, "-I", b.CSRC, os.path.join(HERE, "native", name + ".cpp"), "-o", exe], check=True)
        return subprocess.run([exe], capture_output=True, text=True)

    return run


def test_walks_of_a_launch_do_not_meet(plan):
    run = plan("delta_walks")
    assert run.returncode == 0, run.stdout[:2000]


@pytest.mark.parametrize("hk,hv,d", [(1, 1, 128), (2, 4, 64), (16, 32, 128), (8, 8, 128), (5, 50, 64), (51, 51, 64)])
def test_workspace_grows_with_tokens_and_sequences(hk, hv, d):
    """What is enough for a call is enough for every one of no more tokens and sequences."""
    of = B.ts_hc_delta_prompt_workspace_bytes
    tokens = sorted({n for base in (0, 64, 1536, 2048, 8192, 39424, 65536, 300000) for n in (base, base + 1, base + 63, base + 64, base + 4000)})
    sizes = [[of(n, s, hk, hv, d) for s in (0, 1, 2, 3, 5, 8, 16, 17, 50, 51, 200, 65535)] for n in tokens]
    for row in sizes:
        assert row == sorted(row)
    for column in zip(*sizes):
        assert list(column) == sorted(column)


def test_segments_fit_the_workspace(plan):
    run = plan("delta_workspace")
    assert run.returncode == 0, run.stdout[:2000]


def test_attention_blocks_are_counted(plan):
    run = plan("attn_blocks")
    assert run.returncode == 0, run.stdout[:2000]
