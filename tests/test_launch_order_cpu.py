"""Source check of programmatic dependent launch: a kernel lets its successor start only after it has
itself waited for its predecessor, so that what was written two kernels back is always complete."""
import glob
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "post_weight_quantization_17_b200", "csrc")


def test_kernels_wait_before_they_release():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "k_*.cu"))):
        with open(path) as f:
            src = re.sub(r"//[^\n]*", "", f.read())
        for body in re.split(r"\b__global__\b", src)[1:]:
            # the kernel's own body ends at the first closing brace in column 0
            body = body[:body.index("\n}")]
            release = body.find("pdl_release()")
            if release < 0:
                continue
            seen += 1
            assert 0 <= body.find("pdl_wait()") < release, f"{os.path.basename(path)}: {body[:120]}"
    assert seen >= 20
