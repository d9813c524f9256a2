"""Host logic of the code units' barriers in the adapter projection (csrc/lora_rings.h): with copies
landing in any order, no group of warps passes its wait before its own unit has landed, and the
pipeline never stops (compiled with the host C++ compiler)."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "post_weight_quantization_17_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_code_unit_barriers(tmp_path):
    exe = tmp_path / "lora_rings_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "lora_rings_check.cpp")], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "bad=0 odd_found=1" in out.stdout


def test_the_kernel_takes_its_barriers_from_the_rule():
    with open(os.path.join(CSRC, "k_lora_tc.cu")) as f:
        src = f.read()
    assert "NB = lora_code_barriers(NC)" in src
    assert re.search(r"NC = FWD \? kLoraCodeSlotsForward : kLoraCodeSlotsBackward", src)



def test_barriers_across_the_pair_have_cluster_scope():
    with open(os.path.join(CSRC, "k_lora_tc.cu")) as f:
        src = f.read()
    waits = re.findall(r'"mbarrier\.(?:try|test)_wait[^ ]*', src)
    assert len(waits) == 2 and all(".acquire.cluster." in w for w in waits)
    arrivals = re.findall(r'"mbarrier\.arrive[^ ]*', src)
    assert len(arrivals) == 1 and ".relaxed.cluster." in arrivals[0]
    assert "fence.release.sync_restrict::shared::cta.cluster;" in src
    body = src[src.index("k_lora_tc(const"):]
    body = body[:body.index("\n}")]
    groups = re.findall(r"lt_release\(\);\s*(?:(?:lt_arrive_remote\([^;]*\);\s*)+)", body)
    assert sum(g.count("lt_arrive_remote") for g in groups) == body.count("lt_arrive_remote") == 4
