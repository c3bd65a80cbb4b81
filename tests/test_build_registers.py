"""The build's check of kernels that share out the registers of a CTA among their warps (no GPU)."""
import glob
import os
import re

import pytest

from bit_quantized_linear_rmsnorm_b200 import _build

SRC = os.path.join(_build.CSRC, "kv4_prefill.cu")
TEXT = "constexpr int kLaunchRegs = 80, kSoftmaxRegs = 88, kOtherRegs = 64;"


def printed(*counts):
    return "".join(f"ptxas info    : Compiling entry function '_Z18kv4_prefill_kernel{i}' for 'sm_100a'\n"
                   f"ptxas info    : Function properties for _Z18kv4_prefill_kernel{i}\n"
                   f"    104 bytes stack frame, 200 bytes spill stores, 356 bytes spill loads\n"
                   f"ptxas info    : Used {c} registers, used 1 barriers\n"
                   f"ptxas info    : Compiling entry function '_Z15kv4_join_kernel{i}' for 'sm_100a'\n"
                   f"ptxas info    : Used 32 registers, used 1 barriers\n" for i, c in enumerate(counts))


def test_the_exact_count_passes():
    _build.check_registers(SRC, TEXT, printed(80, 80))


@pytest.mark.parametrize("counts", [(72, 80), (80, 72), (80, 84), ()])
def test_any_other_count_fails_the_build(counts):
    with pytest.raises(RuntimeError, match="registers"):
        _build.check_registers(SRC, TEXT, printed(*counts))


def test_the_shares_add_up_to_what_a_block_is_launched_with():
    with open(SRC) as f:
        text = f.read()
    launch, softmax, other = (int(re.search(n + r" = (\d+)", text).group(1))
                              for n in ("kLaunchRegs", "kSoftmaxRegs", "kOtherRegs"))
    threads = int(re.search(r"kPThreads = (\d+)", text).group(1))
    assert 512 * softmax + (threads - 512) * other <= threads * launch <= 65536
    assert launch % 8 == softmax % 8 == other % 8 == 0


def test_every_kernel_that_shares_registers_is_checked():
    for path in glob.glob(os.path.join(_build.CSRC, "*.cu")):
        with open(path) as f:
            if "setmaxnreg" in f.read():
                assert os.path.basename(path) in _build.EXACT_REGISTERS
