"""Host logic of the few-token adapter projection's look-ahead loads of X (csrc/lora_small_x.h), for
rows of every length modulo 128 and every range of steps (compiled with the host C++ compiler)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "post_weight_quantization_17_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_no_load_behind_a_row(tmp_path):
    exe = tmp_path / "lora_small_x_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "lora_small_x_check.cpp")], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr


def test_the_kernel_loads_by_the_rule():
    with open(os.path.join(CSRC, "k_lora_small.cu")) as f:
        src = f.read()
    assert "small_x_piece(p.d, s, q, s1, ragged, t4)" in src
