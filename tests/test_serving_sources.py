"""The serving kernels that start before the kernel ahead of them has ended
(programmatic dependent launch) read what that one writes with plain loads:
__ldg needs data that stay as they are for the whole life of the kernel."""
import os
import re

import pytest

from quantized_attention_block_b200 import build

# written by a kernel of the same call: the selection's output, the split's partial results and the scores
WRITTEN = {"kv_cache.cu": ["kept", "new_lens", "weight", "ks", "vs"],
           "decode.cu": ["prefix", "part_m", "part_l", "part_o", "lse2", "scores", "weight"]}


@pytest.mark.parametrize("name", sorted(WRITTEN))
def test_no_non_coherent_load_of_what_the_kernel_ahead_writes(name):
    with open(os.path.join(build.CSRC, name)) as f:
        src = re.sub(r"//.*", "", f.read())
    assert "pdl_wait()" in src
    loads = re.findall(r"__ldg\(([^;]*?)\)\s*[;:]", src)
    assert loads  # page numbers, at least
    for x in loads:
        assert not re.search(r"\b(%s)\b" % "|".join(WRITTEN[name]), x), x
