"""What the prompts' attention stores to tensor memory and loads again, read from its source (no GPU needed).

tcgen05.st and tcgen05.ld are not ordered with one another: a load of columns that the same warp has stored needs
tcgen05.wait::st between the two.  tmem_store waits; tmem_store_nowait leaves it to what comes behind it.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hadamard_rotation_gb300", "csrc")


@pytest.fixture(scope="module")
def kernel():
    with open(os.path.join(CSRC, "hq_kv_prompt.cuh")) as f:
        source = f.read()
    at = source.index(" k_kv_prompt(")
    return re.sub(r"//[^\n]*", "", source[at:source.index("\n}\n", at)])


def test_weights_loaded_again(kernel):
    """The weights of a tile's first columns, scaled where the later ones move the reference."""
    assert kernel.count("tmem_store_nowait(") == 1  # (the weights, column by column of the loop over them)
    loops = kernel[kernel.index("for (int c0 = 0; c0 < kKeys; c0 += 64)"):kernel.index("tmem_store_nowait(")]
    again = re.findall(r"(\w+\([^;]*\);\s*)scale\(tp,", loops)
    assert loops.count("scale(tp,") == 1 and [s.strip() for s in again] == ["tmem_store_wait();"]


def test_weights_before_the_product(kernel):
    """All of a tile's weights are stored before the warp arrives for the product that reads them."""
    tail = kernel[kernel.index("tmem_store_nowait("):]
    assert tail.index("tmem_store_wait();") < tail.index("umma_fence_before();") < tail.index("bars.p_full")
