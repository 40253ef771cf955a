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


def mma_role(text):
    """The role that issues MMAs, where there is one: only its elected lane does anything."""
    start = re.search(r"\} else if \(warp == (kWarpMma|1)\) \{", text)
    return text[start.start():text.index("umma_commit_cg<CG>(&acc_full[acc])")] if start else ""


@pytest.mark.parametrize("name", ["mx4_gemv.cu", "mx4_linear.cu", "mx4_product.cu"])
def test_a_warp_waits_as_one(name):
    """Every bounded wait of a role is agreed on by the warp: whole-warp instructions follow, and
    lanes that gave up would leave the others in them for good."""
    text = source(name)
    text = text.replace(mma_role(text), "")
    waits = list(re.finditer(r"\bwait(?:_pair)?\(&", text))
    assert waits
    for m in waits:
        before = text[:m.start()]
        assert re.search(r"(__all_sync\(0xFFFFFFFFu, |warp_ok\(\[&\] \{ return )$", before), \
            (name, before.count("\n") + 1, text[m.start():m.start() + 60])


@pytest.mark.parametrize("name", ["mx4_linear.cu", "mx4_product.cu"])
def test_the_warp_that_issues_agrees_once_a_tile(name):
    """There the lanes wait by themselves: no whole-warp instruction stands between the waits of a
    tile, and the warp agrees before the tile's commit."""
    role = mma_role(source(name))
    assert len(re.findall(r"\bwait(?:_pair)?\(&", role)) >= 2
    tile, agreed = role.split("for (int t = first;")[1].split("ok = __all_sync(0xFFFFFFFFu, ok);")
    assert not re.search(r"_sync\(|\.aligned|shfl|tmem_ld|tmem_st", tile.replace("tc_fence_after_sync();", ""))
    assert agreed.strip() == "if (ok && issuer)"


def between(text, start, end):
    """What follows each `start` up to the next `end`."""
    parts = [p.split(end)[0] for p in text.split(start)[1:] if end in p]
    assert parts, (start, end)
    return parts


def test_a_decoded_stage_is_overwritten_behind_a_fence():
    """The MMAs that read a stage of tensor memory are seen to be over by a wait; the stores that
    follow are ordered behind it by tcgen05.fence::after_thread_sync alone."""
    text = source("mx4_linear.cu").split("tc_fence_after_sync();\n  const uint32_t tmem")[1]  # the kernel's roles
    parts = [p for p in between(text, "wait(&done[stage]", "mbar_arrive(&ready[stage])") if "tmem_st_x32" in p]
    assert len(parts) == 1
    assert "tc_fence_after_sync();" in parts[0].split("tmem_st_x32")[0]
    assert "tmem_st_wait();" in parts[0] and "tc_fence_before_sync();" in parts[0].split("tmem_st_wait();")[1]


def test_the_pair_announces_decoded_stages_between_fences():
    """The second CTA's decoded stages are tcgen05.st results of its decoding warps, read by MMAs
    that the first CTA issues: the warp that passes the word on is a link of that chain, with the
    fence after its wait and the one before its arrival."""
    parts = between(source("mx4_linear.cu"), "warp == kWarpMma && CG > 1 && rank > 0", "mbar_arrive_leader(&ready[r.slot])")
    assert len(parts) == 1
    order = [parts[0].find(s) for s in ("wait(&ready[r.slot]", "tc_fence_after_sync();", "tc_fence_before_sync();")]
    assert -1 not in order and order == sorted(order)


@pytest.mark.parametrize("name", ["mx4_linear.cu", "mx4_product.cu"])
def test_tensor_memory_is_freed_behind_a_fence(name):
    """Other warps read it last: the barrier between is passed with both fences."""
    text = source(name)
    assert text.count("tmem_dealloc_cg") == 1
    before = text.split("tmem_dealloc_cg")[0]
    last = before.rindex("__syncthreads();")
    assert "tc_fence_after_sync();" in before[last:]
    assert "tc_fence_before_sync();" in before[before.rindex("}", 0, last):last]
