"""The microscaled 4-bit kernels against their definition in 64 bits.

Quantisation is compared bit for bit, dequantisation with the once-rounded exact value.
Products are compared twice: with whole-number operands, where every partial sum is
exact in fp32 in any order, so the result must be the exact one rounded once; and with
ordinary values, where a sum of n products in fp32 is off by at most n 2^-23 of the sum
of their magnitudes (each of n - 1 additions rounds or truncates to 24 bits), to which the
tensor scale, the bias and the rounding to the output's type add half a step each.
"""
import pytest
import torch

from tests import mx4_reference as ref
from weight_only_additive_b200 import layer as L
from weight_only_additive_b200 import mx4, native
from weight_only_additive_b200.native import Status

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]
MX, NV = 0, 1


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    native.lib()
    torch.cuda.set_device(0)
    return torch.device("cuda", 0)


def status_ok():
    st, detail = L.check_device_status()
    assert st == Status.OK, (st, hex(detail))


def gen(*seed):
    return torch.Generator().manual_seed(hash(seed) % (1 << 31))


def same(a, b):
    """Equal, NaN and the sign of zero counted too."""
    a, b = a.double(), b.double()
    nan = torch.isnan(a) & torch.isnan(b)
    return bool((nan | ((a == b) & (torch.signbit(a) == torch.signbit(b)))).all())


# --------------------------------------------------------------------------
# quantisation
# --------------------------------------------------------------------------
def check_quantize(x, fmt, gamma, dev):
    gamma = None if gamma is None else torch.tensor(gamma, dtype=torch.float32).item()
    codes, bytes_ = ref.quantize(x, fmt, gamma)
    g = None if gamma is None else torch.tensor([gamma], dtype=torch.float32, device=dev)
    q = mx4.quantize(x.to(dev), fmt, g)
    torch.cuda.synchronize()
    assert torch.equal(q.block_scales().cpu().long(), bytes_)
    got = ref.unpack(q.packed.cpu())
    bad = (got != codes).nonzero()
    assert not len(bad), (len(bad), bad[:4].tolist(), x[tuple(bad[0])].item())
    # the scale bytes behind a row's last block are zero
    cols = x.shape[1] // ref.BLOCK[fmt]
    up, across, _ = q.scales.shape
    flat = q.scales.view(up, across, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(up * 128, across * 4)
    assert not flat[:x.shape[0], cols:].any()
    return q


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (2, 96), (33, 128), (127, 160), (129, 416), (5, 4128), (260, 1024)])
def test_quantize_every_size(dev, fmt, dtype, rows, K):
    g = gen(fmt, rows, K)
    x = torch.randn((rows, K), generator=g, dtype=torch.float64)
    x *= 2.0 ** torch.randint(-9, 9, (rows, K // 32), generator=g).repeat_interleave(32, 1)
    x = x.to(dtype)
    check_quantize(x, fmt, None, dev)
    if fmt == NV:
        check_quantize(x, fmt, float(x.abs().max().float() / 2688), dev)


@pytest.mark.parametrize("gamma", [None, 0.7310585975646973, 3.0517578125e-05, 1.1e-38, 2.5e-45, 1e37, 3e38])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_nvfp4_at_the_borders(dev, dtype, gamma):
    """Elements at and next to every midpoint of their block's unit, block maxima at and
    next to every midpoint of the scale."""
    f = torch.float32
    g32 = torch.tensor(1.0 if gamma is None else gamma, dtype=f).double()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.125], dtype=torch.float64)
    grid = ref.e4m3_values()
    blocks = []
    for s in grid[1::7].tolist():
        for step in (-1, 0, 1):
            b = torch.cat([torch.tensor([6.0], dtype=torch.float64), mids]) * s * g32
            v = b.to(dtype).view(torch.int32 if dtype == f else torch.int16)
            v[1:] = (v[1:] + step).clamp(min=0)
            blocks.append(v.view(dtype))
    half = ((grid[1:] + grid[:-1]) / 2 * 6 * g32)
    for step in (-1, 0, 1):
        v = half.to(dtype).view(torch.int32 if dtype == f else torch.int16)
        top = (v + step).clamp(min=0).view(dtype)
        for t in top:
            b = torch.zeros(16, dtype=dtype)
            b[3], b[7] = t, -t / 2
            blocks.append(b)
    if len(blocks) % 2:
        blocks.append(torch.zeros(16, dtype=dtype))
    x = torch.stack(blocks).view(-1, 32)
    x[::2] = -x[::2]
    check_quantize(x, NV, gamma, dev)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_mxfp4_at_the_borders(dev, dtype):
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0], dtype=torch.float64)
    lo, hi = (-24, 15) if dtype == torch.float16 else (-133, 127)
    blocks = []
    for e in range(lo, hi - 2):
        for step in (-1, 0, 1):
            v = (mids * 2.0 ** e).to(dtype).view(torch.int32 if dtype == torch.float32 else torch.int16)
            v = (v + step).clamp(min=0).view(dtype)
            blocks.append(torch.cat([v, -v.flip(0)]))
    for top in (torch.finfo(dtype).max, torch.finfo(dtype).tiny, torch.finfo(dtype).smallest_normal / 2 ** 3, 0.0):
        blocks.append(torch.full((32,), top, dtype=dtype))
    check_quantize(torch.stack(blocks), MX, None, dev)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top", [5.03125, 3.0, 7.0, 1.3125, 6.5625, 10.5, 441.0])
def test_quantize_with_the_usual_tensor_scale(dev, dtype, top):
    """tensor_scale = max / 2688, rounded to fp32: quotients of few bits, so that many values
    lie on a border but for that rounding."""
    g = gen(int(top * 32))
    x = (torch.randn((64, 2048), generator=g) * top / 3).clamp(-top, top)
    x = (x * 8).round() / 8 if top < 20 else x.round()
    x[7, 9] = top
    x = x.to(dtype)
    check_quantize(x, NV, float(torch.tensor(top) / 2688), dev)
    check_quantize(x, NV, 1.0, dev)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_values(dev, fmt, dtype):
    x = torch.randn((8, 128), generator=gen(1)).to(dtype)
    x[0, 5], x[1, 40], x[2, 127] = float("inf"), float("nan"), float("-inf")
    x[3] = 0.0
    x[4, :64] = -0.0
    x[5, 3] = torch.finfo(dtype).max
    x[6] = torch.finfo(dtype).smallest_normal / 4
    q = check_quantize(x, fmt, None, dev)
    y = mx4.dequantize(q, torch.float32).cpu()
    block = ref.BLOCK[fmt]
    bad = ~torch.isfinite(x.float()).view(8, -1, block).all(-1)
    assert torch.equal(torch.isnan(y).view(8, -1, block).all(-1), bad)
    assert torch.equal(torch.isnan(y).view(8, -1, block).any(-1), bad)


@pytest.mark.parametrize("gamma", [0.0, -1.0, float("nan"), float("inf")])
def test_quantize_with_a_tensor_scale_that_is_none(dev, gamma):
    x = torch.randn((4, 64), generator=gen(2))
    check_quantize(x, NV, gamma, dev)


def test_quantize_leaves_the_bytes_behind_the_last_row(dev):
    for fmt in (MX, NV):
        x = torch.randn((37, 96), generator=gen(3)).half()
        out = mx4.Mx4Tensor(torch.full((37, 48), 0xAA, dtype=torch.uint8, device=dev),
                            torch.full(mx4.scale_tiles(37, 96, fmt), 0xAA, dtype=torch.uint8, device=dev), fmt)
        assert mx4.quantize(x.to(dev), fmt, out=out) is out
        assert torch.equal(out.scales.cpu(), ref.tile(ref.quantize(x, fmt)[1], fill=0xAA))


def test_quantize_unaligned_to_32_bytes(dev):
    """Inputs and outputs at 16-byte addresses that are not 32-byte ones."""
    for dtype in TYPES:
        n = 16 // torch.empty((), dtype=dtype).element_size()
        x = torch.randn((3 * 96 + n,), generator=gen(4)).to(dtype)
        xd = x.to(dev)[n:].view(3, 96)
        assert xd.data_ptr() % 32 == 16
        for fmt in (MX, NV):
            codes, bytes_ = ref.quantize(x[n:].view(3, 96), fmt)
            q = mx4.quantize(xd, fmt)
            assert torch.equal(q.packed.cpu(), ref.pack(codes))
            out = torch.full((3 * 96 + 2 * n,), 7.0, dtype=dtype, device=dev)
            mx4.dequantize(q, dtype, out=out[n:-n].view(3, 96))
            assert same(out[n:-n].view(3, 96).cpu(), ref.values(codes, bytes_, fmt).to(dtype))
            assert (out[:n] == 7).all() and (out[-n:] == 7).all()


# --------------------------------------------------------------------------
# dequantisation
# --------------------------------------------------------------------------
@pytest.mark.parametrize("gamma", [None, 0.375, 1.7e-3])
@pytest.mark.parametrize("fmt,top", [(MX, 253), (NV, 127)])
@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(dev, fmt, top, dtype, gamma):
    block = ref.BLOCK[fmt]
    bytes_ = torch.arange(top).view(-1, 1).repeat(1, 2)
    bytes_[:, 1] = 255 if fmt == MX else 127  # the second block is NaN
    bytes_ = bytes_.repeat(1, 32 // block)
    codes = (torch.arange(block * bytes_.shape[1]) % 16).repeat(top, 1)
    g = None if gamma is None else torch.tensor([gamma], device=dev)
    t = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), bytes_.to(torch.uint8).to(dev), fmt, g)
    got = mx4.dequantize(t, dtype).cpu()
    exact = ref.values(codes, bytes_, fmt)  # has few bits: fp32 holds it
    want = exact.float() if gamma is None else exact.float() * torch.tensor(gamma)
    assert same(got, want.to(dtype))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("rows,K", [(1, 32), (7, 160), (129, 96), (1000, 544)])
def test_dequantize_every_size(dev, fmt, rows, K):
    g = gen(fmt, rows, K)
    codes = torch.randint(0, 16, (rows, K), generator=g)
    bytes_ = torch.randint(0, 127, (rows, K // ref.BLOCK[fmt]), generator=g) + (64 if fmt == MX else 0)
    bytes_ = bytes_.clamp(max=140 if fmt == MX else 126)
    t = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), bytes_.to(torch.uint8).to(dev), fmt)
    for dtype in TYPES:
        assert same(mx4.dequantize(t, dtype).cpu(), ref.values(codes, bytes_, fmt).to(dtype))


# --------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------
def whole(rows, K, fmt, seed, dev, gamma=None):
    """A 4-bit tensor of small whole or half numbers: scales 1 and 2, so that sums of its
    products stay exact in fp32."""
    g = gen(seed, rows, K, fmt)
    codes = torch.randint(0, 16, (rows, K), generator=g)
    pick = torch.randint(0, 2, (rows, K // ref.BLOCK[fmt]), generator=g)
    bytes_ = 127 + pick if fmt == MX else 56 + 8 * pick
    gt = None if gamma is None else torch.tensor([gamma], device=dev)
    t = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), bytes_.to(torch.uint8).to(dev), fmt, gt)
    return t, ref.values(codes, bytes_, fmt, gamma)


def ordinary(rows, K, fmt, seed, dev):
    w = torch.randn((rows, K), generator=gen(seed, rows, K)) * 0.05
    gamma = None if fmt == MX else float(w.abs().max() / 2688)
    codes, bytes_ = ref.quantize(w, fmt, gamma)
    gt = None if gamma is None else torch.tensor([gamma], dtype=torch.float32, device=dev)
    t = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), bytes_.to(torch.uint8).to(dev), fmt, gt)
    return t, ref.values(codes, bytes_, fmt, None if gt is None else gt.item())


def once(exact, dtype):
    """The exact result rounded once (through fp32, which holds these results exactly)."""
    assert torch.equal(exact.float().double(), exact)
    return exact.float().to(dtype)


def close(y, exact, mags, n, dtype):
    """|y - exact| within the bound of the module's docstring."""
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    sums = n * 2.0 ** -23 * mags + 2 * 2.0 ** -24 * mags
    bound = sums + eps * (exact.abs() + sums) + tiny
    err = (y.double() - exact).abs()
    assert torch.isfinite(y).all()
    worst = (err / bound).max().item()
    assert worst <= 1, worst


BATCHES = [1, 2, 3, 7, 8, 9, 16, 17, 33, 64, 65, 127, 128, 129, 200, 257]
SHAPES = [(1, 32), (5, 64), (64, 96), (127, 128), (128, 160), (129, 256), (200, 544), (300, 1056), (96, 4128)]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("N,K", SHAPES)
def test_matmul_16bit_exact(dev, fmt, dtype, N, K):
    w, W = whole(N, K, fmt, 5, dev)
    for batch in BATCHES:
        g = gen(batch, N, K)
        x = torch.randint(-3, 4, (batch, K), generator=g).to(dtype)
        bias = torch.randint(-8, 9, (N,), generator=g).to(dtype) if batch % 2 else None
        y = mx4.matmul(x.to(dev), w, None if bias is None else bias.to(dev)).cpu()
        want = x.double() @ W.T + (0 if bias is None else bias.double())
        assert torch.equal(y, once(want, dtype)), (batch, (y.double() - want).abs().max())
    status_ok()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,K", SHAPES)
def test_matmul_4bit_exact(dev, fmt, dtype, N, K):
    w, W = whole(N, K, fmt, 6, dev, gamma=0.5)
    for batch in BATCHES:
        x, X = whole(batch, K, fmt, 7 + batch, dev, gamma=None if batch % 3 else 0.25)
        bias = torch.randint(-8, 9, (N,), generator=gen(batch, N)).to(dtype) if batch % 2 else None
        y = mx4.matmul(x, w, None if bias is None else bias.to(dev), out_dtype=dtype).cpu()
        want = X @ W.T + (0 if bias is None else bias.double())
        assert torch.equal(y, once(want, dtype)), (batch, (y.double() - want).abs().max())
    status_ok()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("N,K", SHAPES + [(4100, 64), (1032, 160)])
def test_input_grad_exact(dev, fmt, dtype, N, K):
    w, W = whole(N, K, fmt, 8, dev, gamma=0.5)
    for batch in BATCHES:
        dy = torch.randint(-2, 3, (batch, N), generator=gen(batch, N, 1)).to(dtype)
        dx = mx4.input_grad(dy.to(dev), w).cpu()
        want = dy.double() @ W
        assert torch.equal(dx, once(want, dtype)), (batch, (dx.double() - want).abs().max())
    status_ok()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("batch", [130, 256, 257, 700])
def test_products_over_many_features_exact(dev, fmt, dtype, batch):
    """Enough output tiles to fill the device, with a last one of few features."""
    w, W = whole(9500, 544, fmt, 17, dev)
    x = torch.randint(-3, 4, (batch, 544), generator=gen(batch, 3)).to(dtype)
    assert torch.equal(mx4.matmul(x.to(dev), w).cpu(), once(x.double() @ W.T, dtype))
    q, X = whole(batch, 544, fmt, 18, dev)
    assert torch.equal(mx4.matmul(q, w, out_dtype=dtype).cpu(), once(X @ W.T, dtype))
    w, W = whole(600, 9504, fmt, 19, dev)
    dy = torch.randint(-2, 3, (batch, 600), generator=gen(batch, 4)).to(dtype)
    assert torch.equal(mx4.input_grad(dy.to(dev), w).cpu(), once(dy.double() @ W, dtype))
    w, W = whole(601, 9504, fmt, 19, dev)
    dy = torch.randint(-2, 3, (batch, 601), generator=gen(batch, 4)).to(dtype)
    assert torch.equal(mx4.input_grad(dy.to(dev), w).cpu(), once(dy.double() @ W, dtype))
    status_ok()


@pytest.mark.parametrize("seed", range(48))
def test_products_of_any_size_exact(dev, seed):
    import random
    r = random.Random(seed)
    log = lambda lo, hi: int(lo * (hi / lo) ** r.random())  # noqa: E731
    fmt, dtype = r.choice((MX, NV)), r.choice(TYPES[:2])
    batch, N, K = log(1, 700), log(1, 3000), 32 * log(1, 100)
    w, W = whole(N, K, fmt, seed, dev)
    x = torch.randint(-3, 4, (batch, K), generator=gen(seed, 5)).to(dtype)
    what = (fmt, dtype, batch, N, K)
    assert torch.equal(mx4.matmul(x.to(dev), w).cpu(), once(x.double() @ W.T, dtype)), what
    q, X = whole(batch, K, fmt, seed + 1, dev)
    assert torch.equal(mx4.matmul(q, w, out_dtype=dtype).cpu(), once(X @ W.T, dtype)), what
    dy = torch.randint(-2, 3, (batch, N), generator=gen(seed, 6)).to(dtype)
    assert torch.equal(mx4.input_grad(dy.to(dev), w).cpu(), once(dy.double() @ W, dtype)), what
    status_ok()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("batch,N,K", [(1, 1024, 4096), (5, 500, 2080), (40, 384, 4096), (300, 700, 1024)])
def test_products_of_ordinary_values(dev, fmt, dtype, batch, N, K):
    w, W = ordinary(N, K, fmt, 9, dev)
    g = gen(batch, N, K, 2)
    x = torch.randn((batch, K), generator=g).to(dtype)
    bias = torch.randn((N,), generator=g).to(dtype)
    mags = x.double().abs() @ W.abs().T + bias.double().abs()
    y = mx4.matmul(x.to(dev), w, bias.to(dev)).cpu()
    close(y, x.double() @ W.T + bias.double(), mags, K, dtype)

    # quantise, multiply in 4 bits, in every output type
    gx = None if fmt == MX else (x.abs().max().float() / 2688).reshape(1)
    q = mx4.quantize(x.to(dev), fmt, None if gx is None else gx.to(dev))
    X = ref.values(*ref.quantize(x, fmt, None if gx is None else gx.item()), fmt, None if gx is None else gx.item())
    assert torch.allclose(mx4.dequantize(q, torch.float32).cpu().double(), X, rtol=2.0 ** -23, atol=0)
    for out in TYPES:
        b = bias.to(out)
        y4 = mx4.matmul(q, w, b.to(dev), out_dtype=out).cpu()
        mags4 = X.abs() @ W.abs().T + b.double().abs()
        close(y4, X @ W.T + b.double(), mags4, K, out)

    # the gradient of the 16-bit product, from the same weights
    dy = torch.randn((batch, N), generator=g).to(dtype)
    dx = mx4.input_grad(dy.to(dev), w).cpu()
    close(dx, dy.double() @ W, dy.double().abs() @ W.abs(), N, dtype)
    status_ok()


def test_input_grad_against_differences(dev):
    """dx . d = (L(x + d) - L(x - d)) / 2 for L = sum(dy * y): whole numbers, so exact."""
    w, W = whole(96, 128, NV, 10, dev)
    g = gen(11)
    x = torch.randint(-3, 4, (9, 128), generator=g).half()
    dy = torch.randint(-2, 3, (9, 96), generator=g).half()
    dx = mx4.input_grad(dy.to(dev), w).double().cpu()
    for _ in range(4):
        d = torch.randint(-1, 2, x.shape, generator=g).half()
        up = (mx4.matmul((x + d).to(dev), w).double().cpu() * dy.double()).sum()
        down = (mx4.matmul((x - d).to(dev), w).double().cpu() * dy.double()).sum()
        assert (dx * d.double()).sum() == (up - down) / 2


@pytest.mark.parametrize("batch", [1, 8, 40, 200])
@pytest.mark.parametrize("dtype", TYPES[:2])
def test_mxfp4_scales_far_apart(dev, dtype, batch):
    """Block scales that no 16-bit type holds together: 2^-60 beside 2^3."""
    N, K = 130, 128
    codes = torch.randint(0, 16, (N, K), generator=gen(12))
    bytes_ = torch.tensor([127 - 60, 127 + 3, 127 - 30, 127 - 90]).repeat(N, 1)
    bytes_[::2] = bytes_[::2].flip(1)
    W = ref.values(codes, bytes_, MX)
    w = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), bytes_.to(torch.uint8).to(dev), MX)
    x = torch.randn((batch, K), generator=gen(13)).to(dtype)
    y = mx4.matmul(x.to(dev), w, out=None).cpu()
    close(y, x.double() @ W.T, x.double().abs() @ W.abs().T, K, dtype)
    # the small blocks alone count where x is zero elsewhere
    x[:, 32:64] = 0
    if dtype == torch.bfloat16:
        w2 = bytes_.clone()
        w2[1::2, 0] = 127 - 100
        W = ref.values(codes, w2, MX)
        w = mx4.Mx4Tensor.from_block_scales(ref.pack(codes).to(dev), w2.to(torch.uint8).to(dev), MX)
    y = mx4.matmul(x.to(dev), w).cpu()
    close(y, x.double() @ W.T, x.double().abs() @ W.abs().T, K, dtype)
    dy = torch.randn((batch, N), generator=gen(14)).to(dtype)
    dx = mx4.input_grad(dy.to(dev), w).cpu()
    close(dx, dy.double() @ W, dy.double().abs() @ W.abs(), N, dtype)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("batch", [1, 9, 70, 140])
def test_nan_and_infinity_stay_in_their_rows(dev, fmt, batch):
    """A NaN block spoils its weight row's outputs alone, a NaN or infinite activation its
    token's; in the gradient a NaN block spoils its own features."""
    N, K = 140, 192
    t, W = whole(N, K, fmt, 15, dev)
    b = t.block_scales()
    b[137, 2] = 255 if fmt == MX else 127
    t = mx4.Mx4Tensor.from_block_scales(t.packed, b, fmt)
    block = ref.BLOCK[fmt]
    W = W.clone()
    W[137, 2 * block:3 * block] = torch.nan
    x = torch.randint(1, 4, (batch, K), generator=gen(16)).half()
    x[batch // 2, 50], x[batch - 1, 3] = float("inf"), float("nan")
    y = mx4.matmul(x.to(dev), t).cpu()
    want = x.double() @ W.T
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    fine = torch.isfinite(want)
    assert torch.equal(y[fine], once(want[fine], torch.float16))
    assert torch.equal(y[torch.isinf(want)].double(), want[torch.isinf(want)])
    q = mx4.quantize(x.to(dev), fmt)
    y = mx4.matmul(q, t).cpu()
    X = mx4.dequantize(q, torch.float32).cpu().double()
    want = X @ W.T
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    dx = mx4.input_grad(torch.ones((batch, N), dtype=torch.float16, device=dev), t).cpu()
    want = torch.ones((batch, N), dtype=torch.float64) @ W
    assert torch.equal(torch.isnan(dx), torch.isnan(want))
    status_ok()


# --------------------------------------------------------------------------
# as a program uses them
# --------------------------------------------------------------------------
def mlp(x, up, down, b):
    """Two layers, the second with 4-bit activations, and the first's gradient."""
    h = mx4.matmul(x, up, b)
    y = mx4.matmul(mx4.quantize(h, down.format), down, out_dtype=x.dtype)
    return h, y, mx4.input_grad(h, up)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES[:2])
@pytest.mark.parametrize("batch", [1, 13, 150])
def test_run_together_on_streams_and_in_graphs(dev, fmt, dtype, batch):
    up, _ = ordinary(512, 256, fmt, 20, dev)
    down, _ = ordinary(256, 512, fmt, 21, dev)
    b = torch.randn((512,), generator=gen(22)).to(dev, dtype)
    xs = [torch.randn((batch, 256), generator=gen(23, i)).to(dev, dtype) for i in range(3)]
    want = [mlp(x, up, down, b) for x in xs]
    torch.cuda.synchronize()
    # two streams at once, many times over
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate((s1, s2)):
            with torch.cuda.stream(s):
                got[k].append(mlp(xs[k], up, down, b))
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            assert all(torch.equal(p, q) for p, q in zip(r, want[k]))
    # two captured graphs, replayed at once on two streams with new inputs
    graphs = []
    for k in range(2):
        x = xs[k].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = mlp(x, up, down, b)
        graphs.append((g, x, r))
    torch.cuda.synchronize()
    for _ in range(3):
        for k, s in enumerate((s1, s2)):
            with torch.cuda.stream(s):
                graphs[k][1].copy_(xs[2 - k])
                graphs[k][0].replay()
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(p, q) for p, q in zip(graphs[k][2], want[2 - k]))
    # an explicit stream, and buffers of the caller's
    y = torch.empty((batch, 512), dtype=dtype, device=dev)
    s1.wait_stream(torch.cuda.current_stream())
    assert mx4.matmul(xs[0], up, b, out=y, stream=s1) is y
    s1.synchronize()
    assert torch.equal(y, want[0][0])
    status_ok()


def test_offsets_past_32_bits(dev):
    """A tensor of more than 2^32 values: the rows at its end."""
    rows, K = (1 << 17) + 3, 1 << 15
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device=dev)
    end = torch.randn((3, K), generator=gen(30)).to(torch.bfloat16)
    x[-3:] = end.to(dev)
    for fmt in (MX, NV):
        q = mx4.quantize(x, fmt)
        codes, bytes_ = ref.quantize(end, fmt)
        assert torch.equal(q.packed[-3:].cpu(), ref.pack(codes))
        tail = mx4.Mx4Tensor(q.packed[-3:], q.scales[-1:].contiguous(), fmt)
        assert torch.equal(tail.block_scales().cpu().long(), bytes_)
        y = mx4.dequantize(q, torch.bfloat16)
        assert same(y[-3:].cpu(), ref.values(codes, bytes_, fmt).to(torch.bfloat16))
        assert not y[:1000].any()
        del y
        W = ref.values(codes, bytes_, fmt)
        for batch in (2, 20):  # the kernels for a few tokens and for more
            one = torch.ones((batch, K), dtype=torch.bfloat16, device=dev)
            want, mags = torch.ones((batch, K), dtype=torch.float64) @ W.T, W.abs().sum(1).expand(batch, 3)
            close(mx4.matmul(one, q).cpu()[:, -3:], want, mags, K, torch.bfloat16)
        y = mx4.matmul(mx4.quantize(one, fmt), q, out_dtype=torch.bfloat16)
        close(y.cpu()[:, -3:], want, mags, K, torch.bfloat16)
        dy = torch.zeros((5, rows), dtype=torch.bfloat16, device=dev)
        dy[:, -3:] = 1
        close(mx4.input_grad(dy, q).cpu(), W.sum(0).expand(5, K), W.abs().sum(0).expand(5, K), 3, torch.bfloat16)
        del q
