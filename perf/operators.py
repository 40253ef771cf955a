"""The microscaled 4-bit operators as they are measured: plain torch forms beside the framework's calls.

Formats (weights and activations are blocks along K with one scale each):
  mx  MXFP4: e2m1 values, blocks of 32, a power-of-two (e8m0) scale
  nv  NVFP4: e2m1 values, blocks of 16, an e4m3 scale, and one fp32 scale for the whole tensor

Packed rows hold two values a byte (even k in the low four bits).  Scales are held in tiles of 128 rows by
4 blocks, 512 bytes a tile: block (r, c) at byte (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4 of tile
(r // 128, c // 4).
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEVICE = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token's activations through 4 bits and back: the smallest call, latency alone
        {"name": "roundtrip 1x4096 mx f16", "op": "roundtrip", "format": "mx", "type": "f16", "rows": 1, "K": 4096},
        # a long prompt's activations, one tensor scale: bandwidth
        {"name": "roundtrip 8192x11008 nv bf16", "op": "roundtrip", "format": "nv", "type": "bf16", "rows": 8192, "K": 11008},
        # a small odd weight read back in 32 bits, K no multiple of a scale tile
        {"name": "dequantize 1100x4128 nv f32", "op": "dequantize", "format": "nv", "type": "f32", "rows": 1100, "K": 4128},
        # a 70B-shaped up projection restored to 16 bits
        {"name": "dequantize 28672x8192 mx bf16", "op": "dequantize", "format": "mx", "type": "bf16", "rows": 28672, "K": 8192},
        # token generation, one 4096 x 4096 projection: latency
        {"name": "linear b1 4096x4096 mx f16", "op": "linear", "format": "mx", "type": "f16", "batch": 1, "N": 4096, "K": 4096},
        # token generation for a few streams on a 70B-shaped layer: bandwidth of the weights
        {"name": "linear b4 28672x8192 nv bf16", "op": "linear", "format": "nv", "type": "bf16", "batch": 4, "N": 28672, "K": 8192},
        # an odd batch of streams between the two regimes
        {"name": "linear b37 11008x4096 nv f16", "op": "linear", "format": "nv", "type": "f16", "batch": 37, "N": 11008, "K": 4096},
        # a prompt through 16-bit activations
        {"name": "linear b2048 4096x11008 mx bf16", "op": "linear", "format": "mx", "type": "bf16", "batch": 2048, "N": 4096, "K": 11008},
        # a batch of streams with 4-bit activations, quantised in the call
        {"name": "linear4 b64 14336x4096 mx f16", "op": "linear4", "format": "mx", "type": "f16", "batch": 64, "N": 14336, "K": 4096},
        # a long prompt with 4-bit activations on a 70B-shaped layer: the largest product
        {"name": "linear4 b4096 28672x8192 nv bf16", "op": "linear4", "format": "nv", "type": "bf16", "batch": 4096, "N": 28672, "K": 8192},
        # fine-tuning through a frozen layer: few tokens, odd
        {"name": "grad b33 4096x11008 nv f16", "op": "grad", "format": "nv", "type": "f16", "batch": 33, "N": 4096, "K": 11008},
        # the same at a training batch, Mixtral expert shape
        {"name": "grad b1024 14336x4096 mx bf16", "op": "grad", "format": "mx", "type": "bf16", "batch": 1024, "N": 14336, "K": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("roundtrip", "dequantize", "linear", "linear", "linear4", "linear4", "grad"))
    case = {"op": op, "format": rng.choice(("mx", "nv")), "type": rng.choice(("f16", "bf16"))}
    if op in ("roundtrip", "dequantize"):
        case["type"] = rng.choice(("f16", "bf16", "f32"))
        case["rows"] = _log(rng, 1, 8192)
        case["K"] = 32 * _log(rng, 4, 344)
    else:
        # from one token to a long prompt; layers from an eighth of a projection to a 70B-shaped one
        case["batch"] = _log(rng, 1, 4096)
        case["N"] = _log(rng, 512, 14336)
        case["K"] = 32 * _log(rng, 16, 344)
    return case


def work(case):
    per = 0.5 + 1.0 / BLOCK[case["format"]]  # bytes of a value in 4 bits with its share of a scale
    size = 4 if case["type"] == "f32" else 2
    if case["op"] in ("roundtrip", "dequantize"):
        n = case["rows"] * case["K"]
        # the round trip stores the 4-bit tensor (its result) and reads it back once
        return {"bytes": n * (size + per) if case["op"] == "dequantize" else n * (2 * size + 2 * per), "flops": 2 * n}
    batch, N, K = case["batch"], case["N"], case["K"]
    return {"bytes": N * K * per + batch * (N + K) * size, "flops": 2 * batch * N * K}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _generator(seed, what):
    g = torch.Generator(device=DEVICE)
    g.manual_seed((seed * 1000003 + what * 7919 + 17) % (1 << 62))
    return g


def _activations(rows, K, dtype, seed, what):
    """Activations as a layer sees them: normal values, and a few channels far above the rest."""
    g = _generator(seed, what)
    x = torch.randn((rows, K), generator=g, device=DEVICE)
    loud = torch.rand((K,), generator=g, device=DEVICE) < 0.002
    return (x * (1 + 24 * loud)).to(dtype)


def _tensor_scale(x):
    """The largest value of the tensor at the top of the format: 6 in e2m1 times 448 in e4m3."""
    return (x.abs().amax().float() / 2688).reshape(1)


def _quantized_weights(N, K, fmt, seed, what):
    """A weight matrix as a checkpoint holds it: packed values, tiled scales, the tensor scale."""
    g = _generator(seed, what)
    w = torch.randn((N, K), generator=g, device=DEVICE)
    w *= 0.02 * (0.5 + torch.rand((N, 1), generator=g, device=DEVICE))
    gamma = _tensor_scale(w) if fmt == "nv" else None
    q, s = [], []
    for part in w.split(4096):  # a part at a time: the 64-bit steps of a whole large matrix would not fit
        a, b = _quantize(part, fmt, gamma)
        q.append(_to_codes(a))
        s.append(_scale_bytes(b, fmt))
    q, s = torch.cat(q), torch.cat(s)
    return {"packed": q[:, 0::2] | (q[:, 1::2] << 4), "scales": _tile(s), "tensor_scale": gamma}


def _to_codes(q):
    a = q.abs()
    mag = (a > 0.25).to(torch.uint8)
    for t in (0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        mag += a > t
    return mag | (torch.signbit(q).to(torch.uint8) << 3)


def _scale_bytes(s, fmt):
    if fmt == "nv":
        return s.to(torch.float8_e4m3fn).view(torch.uint8)
    return (torch.frexp(s)[1] + 126).to(torch.uint8)


def _tile(s):
    rows, cols = s.shape
    up, across = -(-rows // 128), -(-cols // 4)
    full = torch.zeros((up * 128, across * 4), dtype=torch.uint8, device=s.device)
    full[:rows, :cols] = s
    return full.view(up, 4, 32, across, 4).permute(0, 3, 2, 1, 4).reshape(up, across, 512).contiguous()


def prepare(case, seed):
    dtype, fmt, K = TYPES[case["type"]], case["format"], case["K"]
    state = {"case": dict(case), "dtype": dtype}
    if case["op"] == "roundtrip":
        state["x"] = _activations(case["rows"], K, dtype, seed, 1)
        # a calibrated scale that the program keeps for this activation
        state["x_scale"] = _tensor_scale(state["x"]) if fmt == "nv" else None
        return state
    state["w"] = _quantized_weights(case["rows"] if case["op"] == "dequantize" else case["N"], K, fmt, seed, 2)
    if case["op"] in ("linear", "linear4"):
        state["x"] = _activations(case["batch"], K, dtype, seed, 1)
        state["x_scale"] = _tensor_scale(state["x"]) if fmt == "nv" and case["op"] == "linear4" else None
        state["bias"] = torch.randn((case["N"],), generator=_generator(seed, 3), device=DEVICE).to(dtype)
    elif case["op"] == "grad":
        state["dy"] = torch.randn((case["batch"], case["N"]), generator=_generator(seed, 1), device=DEVICE).to(dtype)
    return state


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _quantize(x, fmt, gamma):
    """(values of the blocks' elements in units of their scale, scales), exact at the borders: the quotients
    are taken in 64 bits for nv; dividing by a power of two (mx) is exact in 32."""
    rows, K = x.shape
    block = BLOCK[fmt]
    if fmt == "mx":
        b = x.float().view(rows, K // block, block)
        e = torch.frexp(b.abs().amax(-1))[1] - 3  # floor(log2 amax) - 2
        e = torch.where(b.abs().amax(-1) > 0, e, -127).clamp(min=-127)
        s = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e).float()
        t = b / s[..., None]
    else:
        b = x.double().view(rows, K // block, block)
        g = gamma.double()
        v = b.abs().amax(-1) / (6 * g)
        step = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=-6).double() - 3)
        s = (torch.round(v / step) * step).clamp(max=448.0)
        t = torch.where(s[..., None] > 0, b / (g * s[..., None]), 0.0)
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    q = (torch.round(a / step) * step).clamp(max=6.0)
    q = torch.copysign(q, t)
    return q.view(rows, K).float(), s.float()


def _untile(s, rows, cols):
    up, across = s.shape[:2]
    return s.view(up, across, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(up * 128, across * 4)[:rows, :cols]


def _values(w, rows, K, fmt):
    """The 4-bit tensor's values in 32 bits, without the tensor scale."""
    p = w["packed"]
    codes = torch.stack((p & 15, p >> 4), -1).view(rows, K).int()
    e, m = (codes >> 1) & 3, (codes & 1).float()
    mag = torch.where(e > 0, (1 + 0.5 * m) * torch.exp2((e - 1).float()), 0.5 * m)
    q = torch.where(codes > 7, -mag, mag)
    b = _untile(w["scales"], rows, K // BLOCK[fmt])
    s = b.contiguous().view(torch.float8_e4m3fn).float() if fmt == "nv" else torch.exp2(b.float() - 127)
    return (q.view(rows, -1, BLOCK[fmt]) * s[..., None]).view(rows, K)


def _plain(state):
    case, dtype = state["case"], state["dtype"]
    fmt, K = case["format"], case["K"]
    if case["op"] == "roundtrip":
        q, s = _quantize(state["x"], fmt, state["x_scale"])
        y = (q.view(case["rows"], -1, BLOCK[fmt]) * s[..., None]).view(case["rows"], K)
        return (y if state["x_scale"] is None else y * state["x_scale"]).to(dtype)
    w = state["w"]
    W = _values(w, case["rows"] if case["op"] == "dequantize" else case["N"], K, fmt)
    if case["op"] == "dequantize":
        return (W if w["tensor_scale"] is None else W * w["tensor_scale"]).to(dtype)
    if case["op"] == "grad":
        y = state["dy"].float() @ W
    elif case["op"] == "linear":
        y = state["x"].float() @ W.t()
    else:
        q, s = _quantize(state["x"], fmt, state["x_scale"])
        x = (q.view(case["batch"], -1, BLOCK[fmt]) * s[..., None]).view(case["batch"], K)
        y = x @ W.t()
        if state["x_scale"] is not None:
            y = y * state["x_scale"]
    if w["tensor_scale"] is not None:
        y = y * w["tensor_scale"]
    if case["op"] != "grad":
        y = y + state["bias"].float()
    return y.to(dtype)


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------
def _framework(state):
    from weight_only_additive_b200 import mx4

    case = state["case"]
    fmt = mx4.Format.MXFP4 if case["format"] == "mx" else mx4.Format.NVFP4
    if case["op"] == "roundtrip":
        return mx4.dequantize(mx4.quantize(state["x"], fmt, state["x_scale"]), state["dtype"])
    w = mx4.Mx4Tensor(state["w"]["packed"], state["w"]["scales"], fmt, state["w"]["tensor_scale"])
    if case["op"] == "dequantize":
        return mx4.dequantize(w, state["dtype"])
    if case["op"] == "grad":
        return mx4.input_grad(state["dy"], w)
    if case["op"] == "linear":
        return mx4.matmul(state["x"], w, state["bias"])
    return mx4.matmul(mx4.quantize(state["x"], fmt, state["x_scale"]), w, state["bias"])


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(v, grid):
    """The grid's nearest value to each |v| (ties to the even index), by comparison with the midpoints."""
    a, out = v.abs(), torch.zeros_like(v)
    for i in range(1, len(grid)):
        mid = (grid[i - 1] + grid[i]) / 2
        up = a > mid if i % 2 else a >= mid
        out = torch.where(up, torch.full_like(out, grid[i]), out)
    return torch.where(torch.signbit(v), -out, out)


def _exact_rounded(x, fmt, gamma):
    """x through 4 bits and back, tensor scale left out."""
    rows, K = x.shape
    b = x.double().view(rows, -1, BLOCK[fmt])
    top = b.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        s = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2).clamp(min=-127))
        g = 1.0
    else:
        # every finite e4m3 value from 0 up: the code's index is its rank, so ties go to even codes
        grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
        g = gamma.double()
        mids = (grid[1:] + grid[:-1]) / 2
        want = (top / (6 * g)).contiguous()
        low = torch.bucketize(want, mids)               # ties stay below
        high = torch.bucketize(want, mids, right=True)  # ties go above
        s = grid[torch.where((low != high) & (low % 2 == 1), high, low)]
    unit = g * s
    q = torch.where(unit > 0, _nearest(b / torch.where(unit > 0, unit, 1.0), MAGNITUDES), 0.0)
    return (q * s).view(rows, K)


def _exact_values(w, rows, K, fmt):
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float64, device=DEVICE)
    p = w["packed"].long()
    out = torch.empty((rows, K), dtype=torch.float64, device=DEVICE)
    out[:, 0::2], out[:, 1::2] = table[p % 16], table[p // 16]
    cols = K // BLOCK[fmt]
    r = torch.arange(rows, device=DEVICE)[:, None]
    c = torch.arange(cols, device=DEVICE)[None, :]
    byte = w["scales"][r // 128, c // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4]
    s = byte.view(torch.float8_e4m3fn).double() if fmt == "nv" else torch.exp2(byte.double() - 127)
    return out * s.repeat_interleave(BLOCK[fmt], 1)


def exact(case, seed):
    state = prepare(case, seed)
    fmt, K = case["format"], case["K"]
    if case["op"] == "roundtrip":
        y = _exact_rounded(state["x"], fmt, state["x_scale"])
        return y if fmt == "mx" else y * state["x_scale"].double()
    w = state["w"]
    scale = 1.0 if w["tensor_scale"] is None else w["tensor_scale"].double()
    rows = case["rows"] if case["op"] == "dequantize" else case["N"]
    W = _exact_values(w, rows, K, fmt)
    if case["op"] == "dequantize":
        return W * scale
    if case["op"] == "grad":
        return state["dy"].double() @ W * scale
    x = state["x"].double()
    if case["op"] == "linear4":
        x = _exact_rounded(state["x"], fmt, state["x_scale"])
        scale = scale if state["x_scale"] is None else scale * state["x_scale"].double()
    return x @ W.t() * scale + state["bias"].double()
