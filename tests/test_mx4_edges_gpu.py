"""The microscaled 4-bit kernels where a short form of their arithmetic would leave the definition:
tensor scales next to the end of fp32, special activations in every kernel, activations of any
magnitude.  Inputs are whole numbers times powers of two wherever a sum is compared, so that
every partial sum is exact in fp32 in any order and the result is the exact one rounded once;
where another rounding takes part it is counted beside the comparison.
"""
import random

import pytest
import torch

from tests import mx4_reference as ref
from tests.test_mx4_gpu import MX, NV, check_quantize, dev, gen, once, status_ok, whole  # noqa: F401
from weight_only_additive_b200 import mx4

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# quantisation with tensor scales near the bottom of fp32
# --------------------------------------------------------------------------
def low_gammas():
    r = random.Random(11)
    some = [float.fromhex(h) for h in ("0x1.573802p-120", "0x1.900d54p-120", "0x1p-120", "0x1.000002p-120",
                                       "0x1.fffffep-101", "0x1p-100", "0x1.000002p-100")]
    return some + [(1 + r.randrange(1 << 23) / (1 << 23)) * 2.0 ** e for e in (*range(-123, -114), -110, -103, -101, -100, -99)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gamma", low_gammas())
def test_quantize_with_small_tensor_scales(dev, dtype, gamma):  # noqa: F811
    """Block maxima at and next to every border between two e4m3 scales, elements at and next to
    the borders of their block's unit."""
    grid = ref.e4m3_values()
    g = torch.tensor(gamma, dtype=torch.float32).double()
    ints = torch.int32 if dtype == torch.float32 else torch.int16
    blocks = []
    for step in (-2, -1, 0, 1, 2):
        v = ((grid[1:] + grid[:-1]) / 2 * 6 * g).to(dtype).view(ints)
        for t in (v + step).clamp(min=0).view(dtype):
            b = torch.zeros(16, dtype=dtype)
            b[5], b[11] = -t, t / 2
            blocks.append(b)
    mids = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.125])
    for s in grid[1::5]:
        for step in (-1, 0, 1):
            v = (mids.double() * s * g).to(dtype).view(ints)
            v[1:] = (v[1:] + step).clamp(min=0)
            blocks.append(v.view(dtype))
    if len(blocks) % 2:
        blocks.append(torch.zeros(16, dtype=dtype))
    check_quantize(torch.stack(blocks).view(-1, 32), NV, gamma, dev)


# --------------------------------------------------------------------------
# infinities and NaN of every pattern
# --------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype,patterns", [
    (torch.float16, (0x7C00, 0xFC00, 0x7C01, 0xFC07, 0x7C04, 0x7E00, 0x7FFF, 0xFFFF)),
    (torch.bfloat16, (0x7F80, 0xFF80, 0x7F81, 0xFF81, 0x7F84, 0x7FC0, 0x7FFF, 0xFFFF))])
@pytest.mark.parametrize("batch", [1, 2, 3, 5, 8, 9, 40, 140])
def test_special_activations_in_every_kernel(dev, fmt, dtype, patterns, batch):  # noqa: F811
    """An infinite or NaN activation makes its token's outputs what the definition says, whatever
    the NaN's bits, and no other token's."""
    N, K = 70, 160
    w, W = whole(N, K, fmt, 15, dev)
    for i, bits in enumerate(patterns):
        x = torch.randint(1, 4, (batch, K), generator=gen(16, i)).to(dtype)
        at = i % batch, (37 * i + 5) % K
        x.view(torch.int16)[at] = bits - (1 << 16 if bits >> 15 else 0)
        assert not torch.isfinite(x[at])
        y = mx4.matmul(x.to(dev), w).cpu()
        want = x.double() @ W.T
        assert torch.equal(torch.isnan(y), torch.isnan(want)), hex(bits)
        inf = torch.isinf(want)
        assert torch.equal(y[inf].double(), want[inf]), hex(bits)
        fine = torch.isfinite(want)
        assert torch.equal(y[fine], once(want[fine], dtype)), hex(bits)
    status_ok()
