"""The order of waits and fences in the microscaled 4-bit kernels, read from their source: what
they keep from happening (a warp that parts ways, a store that races with the tensor cores) does
not show in results, and is not to be made to happen on a device."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_additive_b200", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["mx4_gemv.cu", "mx4_linear.cu", "mx4_product.cu"])
def test_a_warp_waits_as_one(name):
    """Every bounded wait of a role is agreed on by the warp: whole-warp instructions follow, and
    lanes that gave up would leave the others in them for good."""
    text = source(name)
    waits = list(re.finditer(r"\bwait(?:_pair)?\(&", text))
    assert waits
    for m in waits:
        before = text[:m.start()]
        assert re.search(r"(__all_sync\(0xFFFFFFFFu, |warp_ok\(\[&\] \{ return )$", before), \
            (name, before.count("\n") + 1, text[m.start():m.start() + 60])
