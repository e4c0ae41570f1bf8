"""The bounded waits of the 4-bit products' kernel, looked for in its source: what goes wrong when one runs out for a part of
a warp cannot be shown by running it (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trellis_quantized_weight_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_of_whole_warps_are_agreed_on():
    """A bounded wait may run out for some lanes of a warp only.  Before something that needs all of them (a warp barrier, a
    vote, tensor memory, an arrival for the warp) they vote on it; the warps that load tiles wait with one lane."""
    text = source("gemm_q4.cu")
    kernel = text[text.index("q4_kernel("):text.index("q4_widen_kernel")]
    roles = re.split(r"\n    \} else if \(warp\b", kernel[kernel.index("bool alive = true;"):])
    assert len(roles) == 6
    for role in roles:
        if "lane == 0) {\n            uint32_t i = 0;" in role:
            continue
        open_wait = stays = False
        for line in role.split("\n"):
            if "__all_sync(0xffffffffu, alive" in line or "mbar_wait_warp(" in line:
                open_wait = stays = False
            elif "alive &= mbar_try(" in line:               # goes on with the others, whatever came of it
                stays = True
            elif "mbar_wait(" in line and "(void)" not in line:
                open_wait = True
            elif re.search(r"__syncwarp|_sync\(|tmem_|tcgen05|mbar_arrive|mma_|fence_", line):
                assert not open_wait, line
            assert not (stays and re.search(r"!alive|&& alive|break;\n", line)), line
