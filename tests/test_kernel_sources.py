"""Orders in the kernels' sources that no run on today's register counts would show."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "trainable_block_sparse_pooled_b200", "csrc")


def kernels():
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name), encoding="utf-8").read())
        for body in text.split("__global__")[1:]:
            yield name, body


def test_dependents_start_after_the_tensor_memory_is_taken():
    """A kernel that holds tensor memory lets its dependents start only when all its blocks have theirs: a
    dependent block on the same SM could take it first, and waits for the whole grid before it gives any back."""
    both = [(n, k) for n, k in kernels() if "tmem_alloc(" in k and "pdl_trigger()" in k]
    assert both
    for name, k in both:
        taken = k.index("__syncthreads()", k.index("tmem_alloc("))
        assert k.index("pdl_trigger()") > taken, name
