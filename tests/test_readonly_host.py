"""What the kernels may read as read-only, looked for in their sources (no GPU): a read that is too early would be rare."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trellis_quantized_weight_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# The page kernels, the norm and the 4-bit products let the next grid start beside them, so what they write is not read-only for as
# long as that grid lives, which is what ld.global.nc promises.  A caller's weights, tables and scales are.  (silu_mul reads what the
# packed products wrote, which let nothing start before they have.)
CONSTANT = {
    "kv_cache.cuh": [], "kv_pages.cu": [], "copy_groups.cu": [], "kv_attention.cuh": [], "kv_attention.cu": [],
    "kv_append.cu": ["a.rope"], "kv_attention_stream.cu": [], "kv_attention_tile.cu": [], "gemm_q4.cu": ["a.scales", "a.biases"],
    "rms_norm.cu": ["a.weight"], "lora.cu": ["p.starts", "p.which", "p.scales"], "gemm_smallm_kernel.cuh": ["rs.scales", "nrs.scales", "codes"],
}


@pytest.mark.parametrize("name", sorted(CONSTANT))
def test_only_constants_are_read_as_read_only(name):
    text = source(name)
    for m in re.finditer(r"__ldg\(", text):
        depth, end = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
        arg = text[m.end():end - 1]
        assert any(re.search(re.escape(ok) + r"\b", arg) for ok in CONSTANT[name]), arg
    if name != "gemm_smallm_kernel.cuh":            # there: the words of the packed codes
        assert "ld.global.nc" not in text
