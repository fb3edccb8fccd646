"""Projections in 8 bits: what a decoder layer computes around its attention and
its MoE FFN.  ``rms_norm8`` adds the residual, norms, and gives the rows in 8
bits (or bf16, as the router takes them); ``quantize8`` gives rows in 8 bits (the
attention's output; SiLU(gate) * up of a dense FFN); ``Linear8`` multiplies such
rows by a weight in 8 bits.  Each call is one C entry point (``moe_rms_norm8``,
``moe_quantize8``, ``moe_quantize8_weight``, ``moe_linear8``; the format, layouts
and refusals are documented in ``include/moe_ffn.h``).  PyTorch provides the
memory and the streams.

A matrix in 8 bits is a pair of uint8 tensors: e4m3 codes [R, K] and exponent
bytes of the scales, [R, ceil(K / 128)] for rows and [ceil(R / 128), ceil(K /
128)] for weights (``codes.view(torch.float8_e4m3fn)`` and
``scales.view(torch.float8_e8m0fnu)`` are their values).
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B
from .kv_cache import _call, _current, _device


# The calls are a few microseconds of kernels at decode sizes, and the host has to
# keep ahead of them: the checks are a few comparisons a tensor.  They are made of every
# tensor of every call, of results given back and of weights too, since any tensor may
# have been changed in place (set_, resize_, .data) since the last one.


class Block8(NamedTuple):
    """A matrix in 8 bits: codes, scales."""
    codes: torch.Tensor
    scales: torch.Tensor


class Norm8(NamedTuple):
    """What ``rms_norm8`` gives: codes, scales, h, y; None for what was not asked for."""
    codes: torch.Tensor | None
    scales: torch.Tensor | None
    h: torch.Tensor | None
    y: torch.Tensor | None


_BF16, _U8, _INT_MAX = torch.bfloat16, torch.uint8, 2 ** 31 - 1


def _empty8(rows, K, high, device):
    # Rows of codes lie a multiple of 128 bytes apart, so that the product's copies of 128 bytes a row read whole
    # lines (8192 x 4096 x 2000 50 us, with rows of 2000 bytes 68).
    blocks = -(-K // 128)
    codes = (torch.empty((rows, K), dtype=_U8, device=device) if K % 128 == 0 else
             torch.empty_strided((rows, K), (128 * blocks, 1), dtype=_U8, device=device))
    return codes, torch.empty((-(-rows // high), blocks), dtype=_U8, device=device)


def rows8(codes: torch.Tensor, scales: torch.Tensor) -> Block8:
    """Codes and scales from elsewhere (uint8 [R, K]; uint8 [.., ceil(K / 128)]),
    each copied where its rows do not lie as the results here do: codes a multiple
    of 128 bytes apart (of 16 is enough for the calls), scales contiguous in a row."""
    R, K = codes.shape
    if (codes.stride(1) != 1 and K > 1) or (codes.stride(0) % 128 and R > 1) or codes.data_ptr() % 128:
        codes = torch.empty(R, -(-K // 128) * 128, dtype=codes.dtype, device=codes.device)[:, :K].copy_(codes)
    if scales.stride(1) != 1 and scales.shape[1] > 1:
        scales = scales.contiguous()
    return Block8(codes, scales)


def _rows(name, t, dtype, dev, shape):
    """The stride of t's rows.  Raises ValueError unless t has that type, device and shape, its rows contiguous."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        apart, step = t.stride()
        if step == 1 or shape[1] == 1:
            return apart
    raise ValueError(f"{name}: want {dtype} {tuple(shape)} with contiguous rows on device {dev}, got {t.dtype} "
                     f"{tuple(t.shape)} of strides {tuple(t.stride())} on {t.device}")


def _input(name, x):
    """Shape, device and stride of the rows of x.  Raises ValueError unless x is a bf16 matrix with contiguous rows on a
    CUDA device, of sizes that the C calls take."""
    shape, dev, strides = x.shape, x.get_device(), x.stride()
    if x.dtype is not _BF16 or len(shape) != 2 or dev < 0 or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}: want 2-d {_BF16} with contiguous rows on a CUDA device, got {x.dim()}-d {x.dtype} of "
                         f"strides {tuple(strides)} on {x.device}")
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:
        raise ValueError(f"{name}: want sizes of 31 bits, got {tuple(shape)}")
    return shape, dev, strides[0]


def _made(stream, device, make):
    """What a call on `stream` (torch's, or a handle) allocates."""
    if stream is None:
        return make()
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream):
        return make()


def rms_norm8(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, residual: torch.Tensor | None = None,
              outputs: str = "codes", into: Norm8 | None = None, stream=None) -> Norm8:
    """h = x + residual (bf16), y = RMS norm of h's rows times weight.  x and
    residual bf16 [T, H], rows any multiple of 8 elements apart; weight bf16 [H]
    (None: ones).  outputs: "codes" (y in 8 bits), "y" (in bf16) or "both".
    `into` takes the results of an earlier call of the same sizes, or a Norm8 of
    other tensors; its h may be x or residual themselves.  Without a residual, h is
    None (it would be x)."""
    shape, dev, stride = _input("x", x)
    if _device() != dev:   # (the library works on the current device)
        with torch.cuda.device(dev):
            return rms_norm8(x, weight, eps, residual, outputs, into, stream)
    T, H = shape
    if residual is None:
        r, r_stride = None, 0
    else:
        r_stride = _rows("residual", residual, _BF16, dev, shape)
        r = residual.data_ptr()
    if weight is not None and (weight.dtype is not _BF16 or weight.shape != shape[1:] or weight.get_device() != dev or
                               not weight.is_contiguous()):
        raise ValueError(f"weight: want contiguous {_BF16} ({H},) on {x.device}, got {weight.dtype} {tuple(weight.shape)} on {weight.device}")
    if outputs not in ("codes", "y", "both"):
        raise ValueError(f"outputs: want 'codes', 'y' or 'both', got {outputs!r}")
    if into is None:
        def make():
            row = lambda: torch.empty(shape, dtype=_BF16, device=x.device)  # noqa: E731
            q = _empty8(T, H, 1, x.device) if outputs != "y" else (None, None)
            return Norm8(*q, None if residual is None else row(), None if outputs == "codes" else row())
        into = _made(stream, x.device, make)
    elif not isinstance(into, Norm8):
        into = Norm8(*into)
    codes, scales, h, y = into
    no8 = outputs == "y"
    if (codes is None) != no8 or (scales is None) != no8 or (y is None) != (outputs == "codes") or (h is None) != (r is None):
        raise ValueError(f"into: not the results of a call with outputs={outputs!r} and {'no' if r is None else 'a'} residual")
    ld = 0 if no8 else _rows("into.codes", codes, _U8, dev, shape)
    lds = 0 if no8 else _rows("into.scales", scales, _U8, dev, (T, -(-H // 128)))
    h_stride = 0 if h is None else _rows("into.h", h, _BF16, dev, shape)
    y_stride = 0 if y is None else _rows("into.y", y, _BF16, dev, shape)
    _call("moe_rms_norm8", B.lib().moe_rms_norm8(
        x.data_ptr(), stride, r, r_stride, None if weight is None else weight.data_ptr(), eps, T, H,
        None if h is None else h.data_ptr(), h_stride, None if y is None else y.data_ptr(), y_stride,
        None if codes is None else codes.data_ptr(), ld, None if scales is None else scales.data_ptr(), lds,
        _current(dev) if stream is None else B.handle(stream)))
    return into


def quantize8(x: torch.Tensor, silu_mul: bool = False, into: Block8 | None = None, stream=None) -> Block8:
    """The rows of x (bf16 [T, K], any multiple of 8 elements apart) in 8 bits;
    silu_mul: of SiLU(x[:, :K]) * x[:, K:], x bf16 [T, 2K].  `into` takes the
    results of an earlier call of the same sizes, or a Block8 of other tensors."""
    (T, K), dev, stride = _input("x", x)
    if _device() != dev:
        with torch.cuda.device(dev):
            return quantize8(x, silu_mul, into, stream)
    if silu_mul:
        if K % 2:
            raise ValueError(f"x: want an even number of columns (gate, up), got {K}")
        K //= 2
    if into is None:
        into = Block8(*_made(stream, x.device, lambda: _empty8(T, K, 1, x.device)))
    elif not isinstance(into, Block8):
        into = Block8(*into)
    codes, scales = into
    ld = _rows("into.codes", codes, _U8, dev, (T, K))
    lds = _rows("into.scales", scales, _U8, dev, (T, -(-K // 128)))
    _call("moe_quantize8", B.lib().moe_quantize8(
        x.data_ptr(), stride, T, K, 1 if silu_mul else 0, codes.data_ptr(), ld, scales.data_ptr(), lds,
        _current(dev) if stream is None else B.handle(stream)))
    return into


def quantize8_weight(w: torch.Tensor, stream=None) -> Block8:
    """A weight bf16 [N, K] (rows any multiple of 8 elements apart) in 8 bits, with
    a scale per block of 128 x 128."""
    (N, K), dev, stride = _input("w", w)
    if _device() != dev:
        with torch.cuda.device(dev):
            return quantize8_weight(w, stream)
    device = w.device
    codes, scales = _empty8(N, K, 128, device) if stream is None else _made(stream, device, lambda: _empty8(N, K, 128, device))
    _call("moe_quantize8_weight", B.lib().moe_quantize8_weight(
        w.data_ptr(), stride, N, K, codes.data_ptr(), codes.stride(0), scales.data_ptr(), scales.stride(0),
        _current(dev) if stream is None else B.handle(stream)))
    return Block8(codes, scales)


class Linear8:
    """A weight in 8 bits: codes uint8 [N, K], scales uint8 [ceil(N / 128), ceil(K /
    128)] (kept, not copied, where their rows lie as ``rows8`` leaves them)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() != 2 or not codes.is_cuda:
            raise ValueError(f"codes: want 2-d on a CUDA device, got {codes.dim()}-d on {codes.device}")
        self.N, self.K = codes.shape
        self.device, self._dev = codes.device, codes.get_device()
        self._of = of = (-(-self.N // 128), -(-self.K // 128))
        if codes.dtype is not _U8:
            raise ValueError(f"codes: want {_U8}, got {codes.dtype}")
        if scales.dtype is not _U8 or scales.shape != of or scales.device != codes.device:
            raise ValueError(f"scales: want {_U8} {of} on {codes.device}, got {scales.dtype} {tuple(scales.shape)} on {scales.device}")
        if self.N > _INT_MAX or self.K > _INT_MAX:
            raise ValueError(f"codes: want sizes of 31 bits, got {tuple(codes.shape)}")
        self._codes, self._scales = rows8(codes, scales)

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)

    def __reduce__(self):
        return type(self), (self._codes, self._scales)

    @classmethod
    def from_weight(cls, w: torch.Tensor) -> "Linear8":
        """From a weight bf16 [N, K]."""
        return cls(*quantize8_weight(w))

    def forward(self, codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """out bf16 [T, N] = A W^T of A in 8 bits (codes uint8 [T, K], scales uint8
        [T, ceil(K / 128)], as ``rms_norm8`` and ``quantize8`` give them)."""
        T, K, N, dev = codes.shape[0], self.K, self.N, self._dev
        if T > _INT_MAX:
            raise ValueError(f"codes: want sizes of 31 bits, got {tuple(codes.shape)}")
        ld, lds = _rows("codes", codes, _U8, dev, (T, K)), _rows("scales", scales, _U8, dev, (T, self._of[1]))
        w, ws = self._codes, self._scales
        ldw, lws = _rows("weight's codes", w, _U8, dev, (N, K)), _rows("weight's scales", ws, _U8, dev, self._of)
        if _device() != dev:
            with torch.cuda.device(dev):
                return self.forward(codes, scales, out, stream)
        if out is None:
            out, out_stride = _made(stream, self.device, lambda: torch.empty((T, N), dtype=_BF16, device=self.device)), N
        else:
            out_stride = _rows("out", out, _BF16, dev, (T, N))
        if N == 0:   # (a weight of no rows: the C call wants one)
            return out
        _call("moe_linear8", B.lib().moe_linear8(
            codes.data_ptr(), ld, scales.data_ptr(), lds, w.data_ptr(), ldw, ws.data_ptr(), lws, T, N, K,
            out.data_ptr(), out_stride, _current(dev) if stream is None else B.handle(stream)))
        return out

    __call__ = forward
