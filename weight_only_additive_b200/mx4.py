"""Microscaled 4-bit floating point (MXFP4, NVFP4) over the C ABI of include/mx4.h:
quantisation, dequantisation, the linear layer with 4-bit weights and 16-bit or 4-bit
activations, and its input gradient.  Torch provides device memory and streams only;
the arithmetic happens in the library's kernels.
"""
from __future__ import annotations

import enum
from dataclasses import dataclass
from typing import Optional, Union

import torch

from . import native
from .layer import _check_tensor


class Format(enum.IntEnum):
    """MXFP4: blocks of 32 with a power-of-two scale (e8m0).  NVFP4: blocks of 16 with
    an e4m3 scale, and one fp32 scale per tensor."""
    MXFP4 = 0
    NVFP4 = 1

    @property
    def block(self) -> int:
        return 16 if self else 32


_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _type(dtype, name: str, wide: bool = False) -> int:
    t = _TYPES.get(dtype)
    if t is None or (t == 2 and not wide):
        raise TypeError(f"{name} must be float16{', bfloat16 or float32' if wide else ' or bfloat16'}, got {dtype}")
    return t


def scale_tiles(rows: int, K: int, format: Format):
    """Shape of the tiled scales of a rows x K tensor: [row tiles, tiles along K, 512]."""
    return (rows + 127) // 128, -(-K // (4 * Format(format).block)), 512


@dataclass(init=False)
class Mx4Tensor:
    """A rows x K tensor in 4 bits on a CUDA device (layout: include/mx4.h).

    Types and sizes are checked, the scales' bytes are not read: those behind a row's last
    block must be 0, as quantize() and from_block_scales() leave them (a NaN code there
    would reach the row's results)."""
    packed: torch.Tensor                 # [rows, K/2] uint8, even k in the low four bits
    scales: torch.Tensor                 # [row tiles, tiles along K, 512] uint8
    format: Format
    tensor_scale: Optional[torch.Tensor] = None  # one fp32 on the device

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, format: Format,
                 tensor_scale: Optional[torch.Tensor] = None):
        # the kernels read exactly the sizes that rows, K and the format imply
        if type(format) is not Format:
            format = Format(format)
        if packed.dim() != 2 or packed.shape[1] == 0 or packed.shape[1] % 16 or packed.shape[0] == 0:
            raise ValueError(f"packed must be [rows, K/2] with K a multiple of 32, got shape {tuple(packed.shape)}")
        dev = packed.device
        tiles = scale_tiles(packed.shape[0], 2 * packed.shape[1], format)
        if not (packed.dtype is scales.dtype is torch.uint8 and scales.shape == tiles and scales.device == dev
                and packed.is_contiguous() and scales.is_contiguous()):
            _check_tensor(packed, "packed", torch.uint8, dev)
            _check_tensor(scales, "scales", torch.uint8, dev, tiles)
        if tensor_scale is not None:
            _check_scale(tensor_scale, dev)
        self.__dict__.update(packed=packed, scales=scales, format=format, tensor_scale=tensor_scale)

    def __setattr__(self, name, value):
        if name in Mx4Tensor.__dataclass_fields__:  # checked like the constructor's arguments
            args = {f: self.__dict__[f] for f in Mx4Tensor.__dataclass_fields__}
            value = Mx4Tensor(**{**args, name: value}).__dict__[name]
        object.__setattr__(self, name, value)

    @classmethod
    def _of(cls, packed, scales, format, tensor_scale) -> "Mx4Tensor":
        """Of tensors made here, which need no checks."""
        t = object.__new__(cls)
        t.__dict__.update(packed=packed, scales=scales, format=format, tensor_scale=tensor_scale)
        return t

    @property
    def rows(self) -> int:
        return self.packed.shape[0]

    @property
    def K(self) -> int:
        return 2 * self.packed.shape[1]

    @property
    def device(self):
        return self.packed.device

    def block_scales(self) -> torch.Tensor:
        """The scales as a row-major [rows, K / block] uint8 tensor (a copy)."""
        up, across, _ = self.scales.shape
        s = self.scales.view(up, across, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(up * 128, across * 4)
        return s[:self.rows, :self.K // self.format.block].contiguous()

    @classmethod
    def from_block_scales(cls, packed: torch.Tensor, scales: torch.Tensor, format: Format,
                          tensor_scale: Optional[torch.Tensor] = None) -> "Mx4Tensor":
        """From row-major scales [rows, K / block] (one byte each), as checkpoints hold them."""
        format = Format(format)
        rows, K = packed.shape[0], 2 * packed.shape[1]
        if scales.element_size() != 1 or tuple(scales.shape) != (rows, K // format.block):
            raise ValueError(f"scales must be [rows, K / {format.block}] bytes, got {scales.dtype} "
                             f"{tuple(scales.shape)}")
        up, across, _ = scale_tiles(rows, K, format)
        full = torch.zeros((up * 128, across * 4), dtype=torch.uint8, device=packed.device)
        full[:rows, :scales.shape[1]] = scales.view(torch.uint8)
        tiled = full.view(up, 4, 32, across, 4).permute(0, 3, 2, 1, 4).reshape(up, across, 512).contiguous()
        return cls(packed, tiled, format, tensor_scale)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_scale(g: torch.Tensor, dev):
    _check_tensor(g, "tensor_scale", torch.float32, dev)
    if g.numel() != 1:
        raise ValueError(f"tensor_scale must hold one value, got shape {tuple(g.shape)}")


def _elsewhere(dev: torch.device, stream: Optional[torch.cuda.Stream]) -> bool:
    """Whether a call has to change the current device or stream: the library launches on the
    current device, and what a call allocates belongs to the stream that it runs on."""
    return stream is not None or dev.type != "cuda" or dev.index != torch.cuda.current_device()


def _on(dev: torch.device, stream: Optional[torch.cuda.Stream]):
    """The context that makes them current."""
    if dev.type != "cuda":
        raise ValueError(f"mx4 tensors must live on a CUDA device, got {dev}")
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)  # sets the device too


# The handle of a device's current stream (torch.cuda.current_stream builds an object, which
# takes as long as a small kernel).  A torch without CUDA has none, and no tensor that gets there.
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _matrix(t: torch.Tensor, name: str, cols: Optional[int], what: str, dev):
    if t.dim() != 2:
        raise ValueError(f"{name} must be [batch, {what}], got shape {tuple(t.shape)}")
    if cols is not None and t.shape[1] != cols:
        raise ValueError(f"{name} has {what}={t.shape[1]}, weights have {what}={cols}")
    _check_tensor(t, name, t.dtype, dev)


def quantize(x: torch.Tensor, format: Format, tensor_scale: Optional[torch.Tensor] = None,
             out: Optional[Mx4Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> Mx4Tensor:
    """x [rows, K] (fp16, bf16 or fp32, K a multiple of 32) in 4 bits.

    tensor_scale: one fp32 on the device, NVFP4 only (None: 1); a usual choice is
    max|x| / 2688, which puts the largest value at the top of the format.
    out: an Mx4Tensor of the same rows, K and format to write into (its own
    tensor_scale must be the call's).  Rounding and NaN: include/mx4.h."""
    fmt = format if type(format) is Format else Format(format)
    dev = x.device
    _matrix(x, "x", None, "K", dev)
    xt = _type(x.dtype, "x", wide=True)
    rows, K = x.shape
    if rows == 0 or K == 0 or K % 32:
        raise ValueError(f"x must have at least one row and K a multiple of 32, got shape {tuple(x.shape)}")
    if tensor_scale is not None:
        if fmt == Format.MXFP4:
            raise ValueError("MXFP4 is quantised without a tensor scale")
        _check_scale(tensor_scale, dev)
    if out is not None and ((out.rows, out.K, out.format, out.device) != (rows, K, fmt, dev) or
                            _ptr(out.tensor_scale) != _ptr(tensor_scale)):
        raise ValueError("out must have x's rows and K, its device, the format and the tensor scale of the call")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return quantize(x, fmt, tensor_scale, out)
    if out is None:
        up, across, _ = scale_tiles(rows, K, fmt)
        out = Mx4Tensor._of(torch.empty(rows, K // 2, dtype=torch.uint8, device=dev),
                            torch.empty(up, across, 512, dtype=torch.uint8, device=dev), fmt, tensor_scale)
    native.mx4_quantize(x.data_ptr(), xt, out.packed.data_ptr(), out.scales.data_ptr(), _ptr(tensor_scale), rows, K,
                        fmt, _current(dev.index))
    return out


def dequantize(t: Mx4Tensor, dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The tensor's values [rows, K] in fp16, bf16 or fp32: computed in fp32, rounded once."""
    code = _type(dtype, "dtype", wide=True)
    packed = t.packed
    dev = packed.device
    rows, half = packed.shape
    if out is not None:
        _check_tensor(out, "out", dtype, dev, (rows, 2 * half))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return dequantize(t, dtype, out)
    if out is None:
        out = torch.empty(rows, 2 * half, dtype=dtype, device=dev)
    native.mx4_dequantize(packed.data_ptr(), t.scales.data_ptr(), _ptr(t.tensor_scale), out.data_ptr(), code, rows,
                          2 * half, t.format, _current(dev.index))
    return out


def matmul(x: Union[torch.Tensor, Mx4Tensor], w: Mx4Tensor, bias: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y = x . W^T + bias [batch, N] for 4-bit weights w [N, K].

    x: a [batch, K] fp16 or bf16 tensor (weights taken exactly; y in x's type), or an
    Mx4Tensor of w's format, whose product runs on the block-scaled tensor-core path (y
    in out_dtype: fp16, bf16 or fp32; out's or bias's type if None, else fp16, which ends at
    65504: a 4-bit tensor does not know the type that it was quantised from, so name it).
    bias: [N] in y's type."""
    four = isinstance(x, Mx4Tensor)
    packed = w.packed
    dev = packed.device
    N, half = packed.shape
    K = 2 * half
    if four:
        if x.device != dev:
            raise ValueError(f"x must be on {dev}, got {x.device}")
        if x.K != K:
            raise ValueError(f"x has K={x.K}, weights have K={K}")
        if x.format != w.format:
            raise ValueError(f"x is {x.format.name}, weights are {w.format.name}")
        batch = x.rows
        if out_dtype is None:
            out_dtype = out.dtype if out is not None else bias.dtype if bias is not None else torch.float16
        code = _type(out_dtype, "out_dtype", wide=True)
    else:
        _matrix(x, "x", K, "K", dev)
        code = _type(x.dtype, "x")
        batch = x.shape[0]
        if batch == 0:
            raise ValueError("x must have at least one row")
        if out_dtype is not None and out_dtype != x.dtype:
            raise TypeError(f"y has x's type, {x.dtype}, for 16-bit x; got out_dtype={out_dtype}")
        out_dtype = x.dtype
    if bias is not None:
        _check_tensor(bias, "bias", out_dtype, dev, (N,))
    if out is not None:
        _check_tensor(out, "out", out_dtype, dev, (batch, N))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return matmul(x, w, bias, out, out_dtype)
    if out is None:
        out = torch.empty(batch, N, dtype=out_dtype, device=dev)
    if four:
        native.mx4_matmul_mx4(x.packed.data_ptr(), x.scales.data_ptr(), _ptr(x.tensor_scale), packed.data_ptr(),
                              w.scales.data_ptr(), _ptr(w.tensor_scale), _ptr(bias), out.data_ptr(), code, N, K, batch,
                              w.format, _current(dev.index))
    else:
        ws, need = None, 0
        if code == 0 and not w.format:  # fp16 x with MXFP4 weights alone can need one
            need = native.mx4_matmul_workspace_size(code, N, K, batch, w.format)
            ws = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
        native.mx4_matmul(x.data_ptr(), code, packed.data_ptr(), w.scales.data_ptr(), _ptr(w.tensor_scale), _ptr(bias),
                          out.data_ptr(), N, K, batch, w.format, _ptr(ws), need, _current(dev.index))
    return out


def input_grad(dy: torch.Tensor, w: Mx4Tensor, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """dx = dy . W [batch, K] for dy [batch, N] fp16 or bf16: the gradient of matmul() with
    respect to 16-bit x (the weights are fixed, and taken exactly)."""
    packed = w.packed
    dev = packed.device
    N, half = packed.shape
    _matrix(dy, "dy", N, "N", dev)
    code = _type(dy.dtype, "dy")
    batch = dy.shape[0]
    if batch == 0:
        raise ValueError("dy must have at least one row")
    if out is not None:
        _check_tensor(out, "out", dy.dtype, dev, (batch, 2 * half))
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return input_grad(dy, w, out)
    if out is None:
        out = torch.empty(batch, 2 * half, dtype=dy.dtype, device=dev)
    need = native.mx4_input_grad_workspace_size(code, N, 2 * half, batch, w.format)
    ws = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    native.mx4_input_grad(dy.data_ptr(), code, packed.data_ptr(), w.scales.data_ptr(), _ptr(w.tensor_scale),
                          out.data_ptr(), N, 2 * half, batch, w.format, _ptr(ws), need, _current(dev.index))
    return out
