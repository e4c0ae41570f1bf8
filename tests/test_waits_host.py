"""The bounded waits of the tensor-core products' kernels, looked for in their sources: what goes wrong when one runs out for a
part of a warp cannot be shown by running it (no GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trellis_quantized_weight_gb300", "csrc")


@pytest.mark.parametrize("name,first,roles", [("gemm_q4.cu", "q4_kernel(", 6), ("gemm_tc_kernel.cu", "gemm_tc_kernel(const", 3),
                                              ("gemm_tc_kernel.cu", "gemm_tca_kernel(const", 3)])
def test_waits_of_whole_warps_are_agreed_on(name, first, roles):
    """A bounded wait may run out for some lanes of a warp only.  Before something that needs all of them (a warp barrier, a
    vote, tensor memory, an arrival for the warp) they vote on it; the warps that load tiles wait with one lane, and so do those
    that issue products, where no other lane has a part in it."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index(first):]
    kernel = kernel[:kernel.index("\n}\n")]
    parts = re.split(r"\n    \} else (?:if \(warp\b[^\n]*)?\{?", kernel[kernel.index("bool alive = true;"):])
    assert len(parts) == roles
    waits = 0
    for part in parts:
        if re.match(r"\s*if \(lane == 0\) \{", re.sub(r"^[^\n]*\{?\n", "\n", part, count=1)) or "lane == 0) {\n            uint32_t i = 0;" in part:
            continue
        open_wait = stays = False
        for line in part.split("\n"):
            if "__all_sync(0xffffffffu, alive" in line or "mbar_wait_warp(" in line:
                open_wait = stays = False
                waits += 1
            elif "alive &= " in line:               # goes on with the others, whatever came of it
                stays = True
            elif "mbar_wait(" in line and "(void)" not in line:
                open_wait = True
            elif re.search(r"__syncwarp|_sync\(|tmem_|tcgen05|mbar_arrive|mma_|fence_", line):
                assert not open_wait, line
            assert not (stays and re.search(r"if \(!alive\)|&& alive\b", line)), line
    assert waits >= 1
