"""The attention's kernels are made ready on every device that they are launched on, and a refusal is not kept."""
import os
import subprocess

from hyper_connection_residual_call_gb300 import build as b

HERE = os.path.dirname(os.path.abspath(__file__))


def test_attributes_belong_to_a_device(tmp_path):
    objects = [os.path.join(b.BUILD_DIR, name + ".o") for name in ("hc_attn", "hc_attn_tc", "hc_tc")]
    b.build()
    if not all(os.path.exists(o) for o in objects):
        b.build(force=True)
    include = os.path.join(os.path.dirname(os.path.dirname(b.nvcc_path())), "include")
    exe = str(tmp_path / "attn_devices")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", include, "-I", b.CSRC, "-I", b.INCLUDE,
                    os.path.join(HERE, "native", "attn_devices.cpp"), *objects, "-o", exe, "-lpthread"], check=True)
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[:2000]
