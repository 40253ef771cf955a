"""The microscaled 4-bit definitions in 64 bits (torch, CPU), written from the formulas of
include/mx4.h for the tests alone."""
import torch

BLOCK = {0: 32, 1: 16}  # MXFP4, NVFP4
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
TABLE = torch.cat([E2M1, -E2M1])


def e4m3_values():
    """The value of every e4m3 code 0..126, ascending."""
    c = torch.arange(127)
    e, m = c >> 3, (c & 7).double()
    return torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7).double(), m / 8 * 2.0 ** -6)


def nearest(a, grid):
    """Index of the grid value nearest to each a >= 0, ties to the even index, the top kept."""
    code = torch.zeros(a.shape, dtype=torch.int64)
    for i in range(len(grid) - 1):
        mid = (grid[i] + grid[i + 1]) / 2
        code += (a > mid) | ((a == mid) & (i % 2 == 1))
    return code


def scale_values(b, fmt):
    b = b.long()
    if fmt == 0:
        return torch.where(b == 255, torch.nan, 2.0 ** (b.double() - 127))
    grid = torch.cat([e4m3_values(), torch.tensor([torch.nan], dtype=torch.float64)])
    return grid[b]


def quantize(x, fmt, gamma=None):
    """(codes [rows, K], scale bytes [rows, K / block])."""
    rows, K = x.shape
    b = x.double().view(rows, -1, BLOCK[fmt])
    a = b.abs()
    bad = ~torch.isfinite(b).all(-1)
    top = torch.where(bad, 0.0, a.amax(-1))
    if fmt == 0:
        e = torch.frexp(top)[1].long() - 1  # floor(log2)
        byte = torch.where(top > 0, (e - 2).clamp(min=-127), torch.tensor(-127)) + 127
        unit, bad_byte = 2.0 ** (byte - 127).double(), 255
    else:
        g = 1.0 if gamma is None else float(gamma)
        g_bad = not (0 <= g < float("inf"))
        if g_bad:
            bad = torch.ones_like(bad)
        # amax against each midpoint times 6 gamma: the products are exact in 64 bits
        byte = torch.zeros_like(top, dtype=torch.int64) if g_bad or g == 0 else nearest(top, e4m3_values() * (6 * g))
        unit, bad_byte = e4m3_values()[byte] * (0.0 if g_bad else g), 127
    u = unit[..., None]
    codes = torch.zeros(b.shape, dtype=torch.int64)
    for i in range(7):
        mid = (E2M1[i] + E2M1[i + 1]) / 2 * u
        codes += ((a > mid) | ((a == mid) & (i % 2 == 1))) & (u > 0)
    codes += torch.where(torch.signbit(b) & (u > 0), 8, 0)
    codes = torch.where(bad[..., None], 0, codes)
    return codes.view(rows, K), torch.where(bad, bad_byte, byte)


def pack(codes):
    c = codes.to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def unpack(packed):
    p = packed.long()
    return torch.stack((p & 15, p >> 4), -1).view(p.shape[0], -1)


def tile(bytes_, fill=0):
    """Row-major scale bytes as 512-byte tiles; rows past the last hold `fill`."""
    rows, cols = bytes_.shape
    up, across = -(-rows // 128), -(-cols // 4)
    out = torch.full((up, across, 512), fill, dtype=torch.uint8)
    for c in range(across * 4):
        for r0 in range(0, rows, 32):
            r = torch.arange(r0, min(rows, r0 + 32))
            v = bytes_[r, c].to(torch.uint8) if c < cols else torch.zeros(len(r), dtype=torch.uint8)
            out[r0 // 128, c // 4, (r % 32) * 16 + (r0 % 128) // 32 * 4 + c % 4] = v
    return out


def values(codes, bytes_, fmt, gamma=None):
    rows, K = codes.shape
    v = TABLE[codes.long()].view(rows, -1, BLOCK[fmt]) * scale_values(bytes_, fmt)[..., None]
    v = v.view(rows, K)
    return v if gamma is None else v * float(gamma)
