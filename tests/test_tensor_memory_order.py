"""The order in which the tensor-core kernels take and free tensor memory, read from their source (no GPU needed).

tcgen05.alloc waits, without a limit, until the SM has the columns.  CTAs of several launches share an SM, so a CTA that
holds columns must not wait for another that may still be waiting for its own:

  - the adapters' first product, of which several CTAs fit on an SM, waits for the kernel before it before it takes
    columns, and frees them before any barrier of its cluster;
  - a kernel lets the one after it start only once it holds its own columns;
  - of the products, which hold theirs across their cluster's barriers, no two CTAs fit on an SM (a static_assert).

And the arithmetic of the first product's launch: no size asks for more columns than are left beside a CTA of the
products that has 256 of the 512.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hadamard_rotation_gb300", "csrc")


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(CSRC, "hq_gemm.cuh")) as f:
        return f.read()


def body(source, name):
    """The body of a kernel: from its name to the brace in the first column that ends it."""
    at = source.index(name + "(")
    text = source[source.index("{\n", at):source.index("\n}\n", at)]
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def places(text, word):
    return [m.start() for m in re.finditer(re.escape(word), text)]


def test_first_product_of_the_adapters(source):
    k = body(source, "k_lora_shrink")
    alloc, free, wait, start, cluster = (places(k, w) for w in (
        "tcgen05.alloc", "tcgen05.dealloc", "griddepcontrol.wait", "griddepcontrol.launch_dependents", "cluster_sync()"))
    assert len(alloc) == len(free) == len(wait) == len(start) == 1 and cluster
    assert wait[0] < alloc[0] < start[0]
    assert free[0] < cluster[0]


def test_products(source):
    k = body(source, "k_fp4_gemm")
    alloc, start = places(k, "tcgen05.alloc"), places(k, "griddepcontrol.launch_dependents")
    assert len(alloc) == 2 and len(start) == 1  # (of one CTA, of a pair)
    assert max(alloc) < start[0]
    # issued by the warp that allocates, in the block that allocates
    block = k[k.index("if (warp == 2) {"):]
    block = block[:block.index("\n  }\n")]
    assert "tcgen05.alloc" in block and "griddepcontrol.launch_dependents" in block
    assert re.search(r"static_assert\(2 \* kSmemBytes > 228 \* 1024", source)


def test_columns_of_the_first_product():
    """Columns per CTA over every rank, row count and number of adapters, as launch_shrink works them out."""
    with open(os.path.join(CSRC, "hq_gemm.cu")) as f:
        text = f.read()
    assert "const int columns = p.cols + (adapters * padded > p.cols ? padded : 0);" in text
    for R in range(8, 129, 8):
        padded = (R + 15) // 16 * 16
        for adapters in range(1, 129):
            cols = min(adapters * padded, 128 // padded * padded)
            columns = cols + (padded if adapters * padded > cols else 0)
            taken = 32
            while taken < columns:
                taken *= 2
            assert taken <= 512 - 256
