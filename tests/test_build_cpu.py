"""The build refuses a compilation whose kernels could not share out their registers as they do."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _build_module():
    spec = importlib.util.spec_from_file_location(
        "_gptq_build_check", os.path.join(ROOT, "post_weight_quantization_17_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _log(name, registers):
    return (f"ptxas info    : Compiling entry function '_ZN4gptq{len(name)}{name}ILb1ELi256ELb0EEEvi' for 'sm_100a'\n"
            f"ptxas info    : Function properties for _ZN4gptq{len(name)}{name}ILb1ELi256ELb0EEEvi\n"
            f"    80 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
            f"ptxas info    : Used {registers} registers, used 0 barriers\n")


def test_register_counts_are_checked_at_build_time():
    check = _build_module().check_registers
    assert check(_log("k_lora_tc", 96) + _log("k_lora_shrink", 40)) == 1
    assert check(_log("k_lora_tc", 96) * 8) == 8
    assert check(_log("k_lora_shrink", 40)) == 0
    with pytest.raises(RuntimeError, match="88 registers"):
        check(_log("k_lora_tc", 96) + _log("k_lora_tc", 88))


def test_the_shares_fit_the_launch():
    """640 threads: 128 with 40 registers, 256 with 64 and 256 with 152, of what the launch brings."""
    import re
    with open(os.path.join(ROOT, "post_weight_quantization_17_b200", "csrc", "k_lora_tc.cu")) as f:
        src = f.read()
    shares = [int(n) for n in re.findall(r"setmaxnreg\.(?:inc|dec)\.sync\.aligned\.u32 (\d+);", src)]
    assert shares == [40, 64, 152]
    assert 128 * 40 + 256 * 64 + 256 * 152 <= 640 * _build_module().LAUNCH_REGISTERS["k_lora_tc"]
