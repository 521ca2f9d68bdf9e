"""The barriers that free a slot of an LDS ring, by reading the sources: a wave that passes one has the data of its own
LDS reads, wherever the compiler put their use, or the next loads into the slot could overtake them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_prefill_ffn_amd", "csrc")


def barriers(source):
    with open(os.path.join(CSRC, source)) as f:
        return re.findall(r'asm volatile\("([^"]*s_barrier[^"]*)"', f.read())


def test_the_adapters_rings():
    found = barriers("moe_lora.hip")
    assert len(found) == 6 and all("lgkmcnt(0)" in b.split("s_barrier")[0] for b in found), found


@pytest.mark.parametrize("source", ["moe_gemm16_kernels.h", "moe_mx.hip"])
def test_the_products_rings(source):
    """Two barriers a list of tiles, before any stage is read; every one inside the stages waits."""
    found = barriers(source)
    assert len(found) == 4 and [("lgkmcnt(0)" in b) for b in found] == [False, False, True, True], found
