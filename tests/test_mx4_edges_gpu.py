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


def scaled(rows, K, fmt, seed, dev, low, gamma=None):
    """Like whole(), with block scales 2^low and 2^(low + 1)."""
    codes = torch.randint(0, 16, (rows, K), generator=gen(seed, rows, K, fmt))
    pick = torch.randint(0, 2, (rows, K // ref.BLOCK[fmt]), generator=gen(seed, rows, K, fmt, 1))
    if fmt == MX:
        bytes_ = 127 + low + pick
    else:
        bytes_ = (1 << (low + 9)) << pick if low < -6 else 56 + 8 * (low + pick)  # 2^-9, 2^-8, 2^-7: codes 1, 2, 4
    g = None if gamma is None else torch.tensor([gamma], dtype=torch.float32, device=dev)
    t = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), bytes_.to(torch.uint8).to(dev), fmt, g)
    return t, ref.values(codes, bytes_, fmt)


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


# --------------------------------------------------------------------------
# both tensor scales of a 4-bit product
# --------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,low_x,low_w,gx,gw", [
    (NV, 7, 7, 1.1e-22, 0.9e-22),      # their product is subnormal in fp32, the result is not
    (NV, 7, 7, 3e-38, 2e-6),
    (MX, 20, 40, 7e-30, 3e-25),        # it underflows to zero
    (MX, 20, 40, 3e-25, 7e-30),
    (MX, -50, -60, 3e25, 5e21),        # it overflows
    (MX, -60, -50, -5e21, 3e25),
    (MX, -50, -60, 7.0, 3e38)])
@pytest.mark.parametrize("batch,N,K", [(3, 40, 64), (70, 130, 544), (70, 131, 4128), (300, 4800, 96), (300, 9601, 32)])
def test_tensor_scales_whose_product_leaves_fp32(dev, fmt, low_x, low_w, gx, gw, batch, N, K):  # noqa: F811
    """y = sum * gx * gw + bias: the sum is exact, two products and the sum with the bias round to
    fp32 (half a step of 2^-24 each), then y to its type."""
    x, X = scaled(batch, K, fmt, 31, dev, low_x, gx)
    w, W = scaled(N, K, fmt, 32, dev, low_w, gw)
    gx, gw = x.tensor_scale.item(), w.tensor_scale.item()
    sums = X @ W.T
    want = sums * gx * gw
    assert torch.isfinite(want.float()).all() and want.abs().max() > 2.0 ** -126
    for dtype in (torch.float32, torch.bfloat16):
        y = mx4.matmul(x, w, out_dtype=dtype).cpu().double()
        bound = want.abs() * (3 * 2.0 ** -24 + torch.finfo(dtype).eps / 2 * (dtype != torch.float32)) * (1 + 2.0 ** -7)
        bound += torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
        worst = ((y - want).abs() / bound).max().item()
        assert worst <= 1, (dtype, worst)
        # a bias far above the product comes through
        b = torch.full((N,), 3.0, dtype=dtype, device=dev)
        if want.abs().max() < 2.0 ** -40:
            assert (mx4.matmul(x, w, b, out_dtype=dtype) == 3).all()
    status_ok()


@pytest.mark.parametrize("gx,gw", [(0.0, 3e38), (3e38, 0.0), (0.0, 1.0)])
def test_a_tensor_scale_of_zero(dev, gx, gw):  # noqa: F811
    x, _ = scaled(5, 64, MX, 33, dev, 3, gx)
    w, _ = scaled(40, 64, MX, 34, dev, 3, gw)
    assert (mx4.matmul(x, w, out_dtype=torch.float32) == 0).all()


# --------------------------------------------------------------------------
# activations of any magnitude
# --------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("batch", [1, 2, 8, 9, 70])
def test_large_activations_under_small_scales(dev, fmt, batch):  # noqa: F811
    """Blocks whose unscaled products with x would pass the end of fp32: their scales bring them back."""
    for N, K in ((5, 32), (130, 544), (300, 1056)):
        w, W = scaled(N, K, fmt, 35, dev, -9)
        x = (torch.randint(-3, 4, (batch, K), generator=gen(36, batch)).double() * 2.0 ** 120).to(torch.bfloat16)
        y = mx4.matmul(x.to(dev), w).cpu()
        want = x.double() @ W.T
        assert torch.isfinite(want.float()).all()
        assert torch.equal(y, once(want, torch.bfloat16)), (N, K)
    # every value the largest of its type: 32 * 6 * 2^-9 of it
    codes = torch.full((40, 32), 7)
    bytes_ = torch.full((40, 32 // ref.BLOCK[fmt]), 118 if fmt == MX else 1)
    w = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), bytes_.to(torch.uint8).to(dev), fmt)
    x = torch.full((batch, 32), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16)
    want = x.double() @ ref.values(codes, bytes_, fmt).T
    assert torch.equal(mx4.matmul(x.to(dev), w).cpu(), once(want, torch.bfloat16))
    status_ok()


@pytest.mark.parametrize("batch", [1, 2, 8, 9, 70])
def test_small_activations_under_large_scales(dev, batch):  # noqa: F811
    """Subnormal bf16 activations that MXFP4 scales bring into the ordinary range."""
    for N, K in ((5, 32), (130, 544)):
        w, W = scaled(N, K, MX, 37, dev, 100)
        x = torch.randint(-3, 4, (batch, K), generator=gen(38, batch)).double() * 2.0 ** -133
        x = x.to(torch.bfloat16)
        assert x.any() and (x.abs() < torch.finfo(torch.bfloat16).smallest_normal).all()
        assert torch.equal(mx4.matmul(x.to(dev), w).cpu(), once(x.double() @ W.T, torch.bfloat16))
    status_ok()
