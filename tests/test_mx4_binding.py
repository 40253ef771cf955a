"""The binding of the microscaled 4-bit operators without a GPU: what a user's program may do
with an Mx4Tensor besides calling the kernels."""
import copy
import dataclasses
import os
import subprocess
import sys

import pytest
import torch

from weight_only_additive_b200 import mx4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def tensor(rows=4, K=64, fmt=1, **kw):
    d = dict(packed=torch.zeros((rows, K // 2), dtype=torch.uint8),
             scales=torch.zeros(mx4.scale_tiles(rows, K, fmt), dtype=torch.uint8), format=fmt)
    return mx4.Mx4Tensor(**{**d, **kw})


@pytest.mark.parametrize("name,value,err", [
    ("tensor_scale", torch.ones(1, device="meta"), ValueError),  # another device's memory
    ("tensor_scale", torch.ones(2), ValueError),
    ("tensor_scale", torch.ones(1, dtype=torch.float64), TypeError),
    ("packed", torch.zeros((200, 32), dtype=torch.uint8), ValueError),  # more rows than scales
    ("packed", torch.zeros((4, 64), dtype=torch.uint8), ValueError),
    ("packed", torch.zeros((4, 32), dtype=torch.uint8, device="meta"), ValueError),
    ("scales", torch.zeros((1, 1, 256), dtype=torch.uint8), ValueError),
    ("scales", torch.zeros((1, 1, 512)), TypeError),
    ("format", 2, ValueError)])
def test_an_assignment_is_checked_like_an_argument(name, value, err):
    """The kernels read the sizes that the fields imply: one changed later is checked too."""
    t = tensor()
    before = getattr(t, name)
    with pytest.raises(err):
        setattr(t, name, value)
    assert getattr(t, name) is before


def test_a_format_of_other_tiles_is_refused_by_assignment():
    t = tensor(K=256)  # 4 tiles of NVFP4 scales, 2 of MXFP4
    with pytest.raises(ValueError):
        t.format = mx4.Format.MXFP4


def test_good_assignments_copies_and_names():
    t = tensor()
    g = torch.full((1,), 0.5)
    t.tensor_scale = g
    assert t.tensor_scale is g
    t.tensor_scale = None
    p = torch.ones((7, 32), dtype=torch.uint8)
    t.packed = p
    assert t.rows == 7 and t.packed is p
    t = tensor(fmt=0, K=32)
    t.format = 1
    assert t.format is mx4.Format.NVFP4
    t.label = "up_proj"  # a program's own
    for u in (copy.copy(t), copy.deepcopy(t)):
        assert (u.rows, u.K, u.format, u.label) == (4, 32, mx4.Format.NVFP4, "up_proj")
    u = dataclasses.replace(t, tensor_scale=g)
    assert u.tensor_scale is g and u.packed is t.packed
    assert [f.name for f in dataclasses.fields(t)] == ["packed", "scales", "format", "tensor_scale"]


def test_the_module_needs_no_torch_with_cuda():
    """Of a torch built without CUDA the module can be imported, and refuses its tensors."""
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "from weight_only_additive_b200 import mx4\n"
            "try:\n"
            "    mx4.quantize(torch.zeros(3, 64), mx4.Format.MXFP4)\n"
            "except ValueError as e:\n"
            "    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-500:]
    assert "CUDA device" in r.stdout
