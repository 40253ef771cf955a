"""The microscaled 4-bit entry points without a GPU: exported names, argument checks of
the C ABI and of the binding, and the scale layout."""
import ctypes
import os
import re

import pytest
import torch

from tests import mx4_reference as ref
from weight_only_additive_b200 import build, mx4, native
from weight_only_additive_b200.native import Status

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mx4.h")
A = 1 << 32          # fake 16-byte aligned buffers, never dereferenced: far apart
STEP = 1 << 34
D = [A + i * STEP for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return native.lib()


def test_header_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(mx4_[a-z_0-9]+)\s*\(", text))) == sorted(native.MX4_EXPORTS)
    for name in native.MX4_EXPORTS:
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr)


@pytest.mark.parametrize("rows,K,fmt,want", [
    (1, 32, 0, 512), (128, 128, 0, 512), (129, 128, 0, 1024), (128, 160, 0, 1024),
    (1, 32, 1, 512), (128, 64, 1, 512), (300, 96, 1, 3 * 2 * 512),
    (0, 32, 0, 0), (1, 0, 0, 0), (1, 48, 1, 0), (1, 32, 2, 0), (1 << 25, 32, 0, 0), (1, (1 << 20) + 32, 0, 0)])
def test_scales_bytes(lib, rows, K, fmt, want):
    assert native.mx4_scales_bytes(rows, K, fmt) == want
    if want:
        a, b, c = mx4.scale_tiles(rows, K, mx4.Format(fmt))
        assert a * b * c == want


def quantize(x=D[0], xt=0, p=D[1], s=D[2], g=None, rows=8, K=64, fmt=0):
    return native.lib().mx4_quantize(x, xt, p, s, g, rows, K, fmt, None)


def dequantize(p=D[0], s=D[1], g=None, out=D[2], t=0, rows=8, K=64, fmt=0):
    return native.lib().mx4_dequantize(p, s, g, out, t, rows, K, fmt, None)


def matmul(x=D[0], t=0, p=D[1], s=D[2], g=None, bias=None, y=D[4], N=64, K=64, batch=3, fmt=0):
    return native.lib().mx4_matmul(x, t, p, s, g, bias, y, N, K, batch, fmt, D[5], 1 << 30, None)


def product(xp=D[0], xs=D[1], xg=None, p=D[2], s=D[3], g=None, bias=None, y=D[5], t=0, N=64, K=64, batch=3, fmt=0):
    return native.lib().mx4_matmul_mx4(xp, xs, xg, p, s, g, bias, y, t, N, K, batch, fmt, None)


def grad(dy=D[0], t=0, p=D[1], s=D[2], g=None, dx=D[4], N=64, K=64, batch=3, fmt=0):
    return native.lib().mx4_input_grad(dy, t, p, s, g, dx, N, K, batch, fmt, D[5], 1 << 30, None)


INVALID, MISALIGNED = Status.INVALID_ARG, Status.MISALIGNED


@pytest.mark.parametrize("call,bad,want", [
    (f, kw, w) for f, cases in (
        (quantize, [(dict(x=None), INVALID), (dict(p=None), INVALID), (dict(s=None), INVALID),
                    (dict(x=D[0] + 8), MISALIGNED), (dict(p=D[1] + 4), MISALIGNED), (dict(s=D[2] + 8), MISALIGNED),
                    (dict(g=D[3] + 2, fmt=1), MISALIGNED), (dict(g=D[3]), INVALID), (dict(xt=3), INVALID),
                    (dict(xt=-1), INVALID), (dict(p=D[0] + 16), INVALID), (dict(s=D[0]), INVALID),
                    (dict(s=D[1] + 32), INVALID), (dict(g=D[1] + 16, fmt=1), INVALID)]),
        (dequantize, [(dict(p=None), INVALID), (dict(out=None), INVALID), (dict(s=D[1] + 4), MISALIGNED),
                      (dict(out=D[2] + 8), MISALIGNED), (dict(t=3), INVALID), (dict(out=D[0]), INVALID),
                      (dict(out=D[1] + 16), INVALID), (dict(g=D[2] + 64), INVALID)]),
        (matmul, [(dict(x=None), INVALID), (dict(y=None), INVALID), (dict(p=None), INVALID), (dict(s=None), INVALID),
                  (dict(x=D[0] + 2), MISALIGNED), (dict(y=D[4] + 8), MISALIGNED), (dict(bias=D[3] + 4), MISALIGNED),
                  (dict(g=D[3] + 1), MISALIGNED), (dict(t=2), INVALID), (dict(y=D[0] + 16), INVALID),
                  (dict(y=D[1]), INVALID), (dict(y=D[2]), INVALID), (dict(bias=D[4]), INVALID),
                  (dict(batch=0), INVALID), (dict(N=0), INVALID), (dict(batch=(1 << 24) + 1), INVALID)]),
        (product, [(dict(xp=None), INVALID), (dict(xs=None), INVALID), (dict(p=None), INVALID), (dict(y=None), INVALID),
                   (dict(xp=D[0] + 8), MISALIGNED), (dict(xs=D[1] + 8), MISALIGNED), (dict(xg=D[4] + 2), MISALIGNED),
                   (dict(y=D[5] + 4), MISALIGNED), (dict(t=3), INVALID), (dict(y=D[0]), INVALID),
                   (dict(y=D[3]), INVALID), (dict(batch=0), INVALID), (dict(N=-1), INVALID)]),
        (grad, [(dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(p=None), INVALID),
                (dict(dy=D[0] + 8), MISALIGNED), (dict(dx=D[4] + 2), MISALIGNED), (dict(t=2), INVALID),
                (dict(dx=D[0]), INVALID), (dict(dx=D[1]), INVALID), (dict(batch=0), INVALID), (dict(N=0), INVALID)]),
    ) for kw, w in cases + [(dict(K=0), INVALID), (dict(K=48), INVALID), (dict(K=-32), INVALID),
                            (dict(K=(1 << 20) + 32), INVALID), (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID)]])
def test_bad_arguments_are_refused_before_any_launch(lib, call, bad, want):
    assert call(**bad) == want


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (128, 256), (129, 160), (300, 64)])
def test_scale_layout_round_trip(fmt, rows, K):
    g = torch.Generator().manual_seed(rows * K)
    b = torch.randint(0, 127, (rows, K // ref.BLOCK[fmt]), generator=g, dtype=torch.uint8)
    t = mx4.Mx4Tensor.from_block_scales(torch.zeros((rows, K // 2), dtype=torch.uint8), b, fmt)
    assert torch.equal(t.scales, ref.tile(b))
    assert torch.equal(t.block_scales(), b)
    assert (t.rows, t.K, t.format) == (rows, K, mx4.Format(fmt))


def test_binding_refuses_wrong_tensors():
    def t(rows=4, K=64, fmt=0, **kw):
        d = dict(packed=torch.zeros((rows, K // 2), dtype=torch.uint8),
                 scales=torch.zeros(mx4.scale_tiles(rows, K, fmt), dtype=torch.uint8), format=fmt)
        return mx4.Mx4Tensor(**{**d, **kw})

    t()
    for kw, err in ((dict(packed=torch.zeros((4, 24), dtype=torch.uint8)), ValueError),
                    (dict(packed=torch.zeros((4, 0), dtype=torch.uint8)), ValueError),
                    (dict(packed=torch.zeros((0, 32), dtype=torch.uint8)), ValueError),
                    (dict(packed=torch.zeros((64, 4), dtype=torch.uint8).t()), ValueError),
                    (dict(packed=torch.zeros((4, 32), dtype=torch.int8)), TypeError),
                    (dict(scales=torch.zeros((1, 1, 256), dtype=torch.uint8)), ValueError),
                    (dict(scales=torch.zeros((1, 1, 512))), TypeError), (dict(format=2), ValueError),
                    (dict(tensor_scale=torch.ones(2)), ValueError),
                    (dict(tensor_scale=torch.ones(1, dtype=torch.float64)), TypeError)):
        with pytest.raises(err):
            t(**kw)
    with pytest.raises(ValueError):
        mx4.Mx4Tensor.from_block_scales(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 3), dtype=torch.uint8), 0)
    x = torch.zeros((3, 64), dtype=torch.float16)
    # sizes, types and devices: a CPU tensor is refused too, as nothing runs there
    for f, err in ((lambda: mx4.quantize(x, 0), ValueError),
                   (lambda: mx4.quantize(x[:, :48], 0), ValueError), (lambda: mx4.quantize(x[:0], 0), ValueError),
                   (lambda: mx4.quantize(x.double(), 0), TypeError), (lambda: mx4.quantize(x[0], 0), ValueError),
                   (lambda: mx4.quantize(x, 0, torch.ones(1)), ValueError), (lambda: mx4.quantize(x, 7), ValueError),
                   (lambda: mx4.quantize(x[:, ::2].repeat(1, 2)[:, ::2], 0), ValueError),
                   (lambda: mx4.dequantize(t()), ValueError), (lambda: mx4.dequantize(t(), torch.int8), TypeError),
                   (lambda: mx4.matmul(x, t()), ValueError), (lambda: mx4.matmul(x[:, :32], t()), ValueError),
                   (lambda: mx4.matmul(x.float(), t()), TypeError), (lambda: mx4.matmul(x[:0], t()), ValueError),
                   (lambda: mx4.matmul(x, t(), torch.zeros(4)), TypeError),
                   (lambda: mx4.matmul(x, t(), torch.zeros(5, dtype=torch.float16)), ValueError),
                   (lambda: mx4.matmul(x, t(), out_dtype=torch.float32), TypeError),
                   (lambda: mx4.matmul(t(fmt=1), t()), ValueError), (lambda: mx4.matmul(t(K=32), t()), ValueError),
                   (lambda: mx4.matmul(t(), t(), out_dtype=torch.int8), TypeError),
                   (lambda: mx4.input_grad(x, t()), ValueError), (lambda: mx4.input_grad(x[:, :4].float(), t()), TypeError),
                   (lambda: mx4.input_grad(x[:0, :4].contiguous(), t()), ValueError)):
        with pytest.raises(err):
            f()
