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


class Block8(NamedTuple):
    """A matrix in 8 bits."""
    codes: torch.Tensor
    scales: torch.Tensor


class Norm8(NamedTuple):
    """What ``rms_norm8`` gives; None for what was not asked for."""
    codes: torch.Tensor | None
    scales: torch.Tensor | None
    h: torch.Tensor | None
    y: torch.Tensor | None


def _empty8(rows, K, high, device) -> Block8:
    # (rows of scales lie a multiple of 4 bytes apart: the product reads four at a time)
    blocks = -(-K // 128)
    scales = torch.empty(-(-rows // high), -(-blocks // 4) * 4, dtype=torch.uint8, device=device)
    return Block8(torch.empty(rows, K, dtype=torch.uint8, device=device), scales[:, :blocks])


def rows8(codes: torch.Tensor, scales: torch.Tensor) -> Block8:
    """Codes and scales from elsewhere (uint8 [R, K]; uint8 [.., ceil(K / 128)]),
    each copied where its rows do not lie as the calls here take them."""
    if codes.stride(1) != 1 or codes.stride(0) % 16 or codes.data_ptr() % 16:
        codes = codes.contiguous() if codes.shape[1] % 16 == 0 and not codes.is_contiguous() else codes.clone()
    if scales.stride(1) != 1 or scales.stride(0) % 4 or scales.data_ptr() % 4:
        padded = torch.empty(scales.shape[0], -(-scales.shape[1] // 4) * 4, dtype=scales.dtype, device=scales.device)
        scales = padded[:, :scales.shape[1]].copy_(scales)
    return Block8(codes, scales)


def _want_rows(name, t, dtype, dev, shape):
    """Raises ValueError unless t has that type, device and shape, its rows contiguous."""
    if t.dtype is not dtype or t.dim() != 2 or t.get_device() != dev or t.shape != shape or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name}: want {dtype} {tuple(shape)} with contiguous rows on device {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} of strides {tuple(t.stride())} on {t.device}")


def _stride(t) -> int:
    # (a single row's stride says nothing: the C call wants one that holds the row)
    n = t.shape[1]
    return t.stride(0) if t.shape[0] > 1 else -(-n // 16) * 16


def _made(stream, device, make):
    """What a call on `stream` (torch's, or a handle) allocates."""
    if stream is None:
        return make()
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream):
        return make()


def _is_bf16_rows(name, x):
    if x.dtype is not torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name}: want 2-d torch.bfloat16 on a CUDA device, got {x.dim()}-d {x.dtype} on {x.device}")


def rms_norm8(x: torch.Tensor, weight: torch.Tensor | None = None, eps: float = 1e-6, residual: torch.Tensor | None = None,
              outputs: str = "codes", into: Norm8 | None = None, stream=None) -> Norm8:
    """h = x + residual (bf16), y = RMS norm of h's rows times weight.  x and
    residual bf16 [T, H], rows any multiple of 8 elements apart; weight bf16 [H]
    (None: ones).  outputs: "codes" (y in 8 bits), "y" (in bf16) or "both".
    `into` takes the results of an earlier call of the same sizes; its h may be
    x or residual themselves.  Without a residual, h is None (it would be x)."""
    _is_bf16_rows("x", x)
    if outputs not in ("codes", "y", "both"):
        raise ValueError(f"outputs: want 'codes', 'y' or 'both', got {outputs!r}")
    dev, shape = x.get_device(), x.shape
    T, H = shape
    bf16 = torch.bfloat16
    if _device() != dev:   # (the library works on the current device)
        with torch.cuda.device(dev):
            return rms_norm8(x, weight, eps, residual, outputs, into, stream)
    if into is None:
        def make():
            q = _empty8(T, H, 1, x.device) if outputs != "y" else (None, None)
            return Norm8(*q, None if residual is None else torch.empty(shape, dtype=bf16, device=x.device),
                         None if outputs == "codes" else torch.empty(shape, dtype=bf16, device=x.device))
        into = _made(stream, x.device, make)
    codes, scales, h, y = into
    _want_rows("x", x, bf16, dev, shape)
    if (codes is None) != (outputs == "y") or (y is None) != (outputs == "codes") or (h is None) != (residual is None):
        raise ValueError(f"into: not the results of a call with outputs={outputs!r} and {'no' if residual is None else 'a'} residual")
    args = [None, 0, None, 0, None, 0, None, 0]
    if residual is not None:
        _want_rows("residual", residual, bf16, dev, shape)
        _want_rows("into.h", h, bf16, dev, shape)
        args[0], args[1] = h.data_ptr(), _stride(h)
    if weight is not None and (weight.dtype is not bf16 or weight.shape != (H,) or weight.get_device() != dev or not weight.is_contiguous()):
        raise ValueError(f"weight: want contiguous {bf16} ({H},) on {x.device}, got {weight.dtype} {tuple(weight.shape)} on {weight.device}")
    if y is not None:
        _want_rows("into.y", y, bf16, dev, shape)
        args[2], args[3] = y.data_ptr(), _stride(y)
    if codes is not None:
        _want_rows("into.codes", codes, torch.uint8, dev, shape)
        _want_rows("into.scales", scales, torch.uint8, dev, (T, -(-H // 128)))
        args[4:] = codes.data_ptr(), _stride(codes), scales.data_ptr(), _stride(scales)
    _call("moe_rms_norm8", B.lib().moe_rms_norm8(
        x.data_ptr(), _stride(x), None if residual is None else residual.data_ptr(), 0 if residual is None else _stride(residual),
        None if weight is None else weight.data_ptr(), eps, T, H, *args, _current(dev) if stream is None else B.handle(stream)))
    return into


def quantize8(x: torch.Tensor, silu_mul: bool = False, into: Block8 | None = None, stream=None) -> Block8:
    """The rows of x (bf16 [T, K], any multiple of 8 elements apart) in 8 bits;
    silu_mul: of SiLU(x[:, :K]) * x[:, K:], x bf16 [T, 2K].  `into` takes the
    results of an earlier call of the same sizes."""
    _is_bf16_rows("x", x)
    T, K = x.shape
    dev = x.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return quantize8(x, silu_mul, into, stream)
    if silu_mul:
        if K % 2:
            raise ValueError(f"x: want an even number of columns (gate, up), got {K}")
        K //= 2
    if into is None:
        into = _made(stream, x.device, lambda: _empty8(T, K, 1, x.device))
    codes, scales = into
    _want_rows("x", x, torch.bfloat16, dev, x.shape)
    _want_rows("into.codes", codes, torch.uint8, dev, (T, K))
    _want_rows("into.scales", scales, torch.uint8, dev, (T, -(-K // 128)))
    _call("moe_quantize8", B.lib().moe_quantize8(
        x.data_ptr(), _stride(x), T, K, 1 if silu_mul else 0, codes.data_ptr(), _stride(codes), scales.data_ptr(),
        _stride(scales), _current(dev) if stream is None else B.handle(stream)))
    return into


def quantize8_weight(w: torch.Tensor, stream=None) -> Block8:
    """A weight bf16 [N, K] (rows any multiple of 8 elements apart) in 8 bits, with
    a scale per block of 128 x 128."""
    _is_bf16_rows("w", w)
    N, K = w.shape
    dev = w.get_device()
    if _device() != dev:
        with torch.cuda.device(dev):
            return quantize8_weight(w, stream)
    codes, scales = made = _made(stream, w.device, lambda: _empty8(N, K, 128, w.device))
    _want_rows("w", w, torch.bfloat16, dev, w.shape)
    _call("moe_quantize8_weight", B.lib().moe_quantize8_weight(
        w.data_ptr(), _stride(w), N, K, codes.data_ptr(), _stride(codes), scales.data_ptr(), _stride(scales),
        _current(dev) if stream is None else B.handle(stream)))
    return made


class Linear8:
    """A weight in 8 bits: codes uint8 [N, K], scales uint8 [ceil(N / 128), ceil(K /
    128)] (kept, not copied, where their rows lie as ``rows8`` leaves them)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() != 2 or not codes.is_cuda:
            raise ValueError(f"codes: want 2-d on a CUDA device, got {codes.dim()}-d on {codes.device}")
        self.N, self.K = codes.shape
        self.device, self._dev = codes.device, codes.get_device()
        self._blocks = -(-self.K // 128)
        if codes.dtype is not torch.uint8:
            raise ValueError(f"codes: want torch.uint8, got {codes.dtype}")
        if scales.dtype is not torch.uint8 or scales.shape != (-(-self.N // 128), self._blocks) or scales.device != codes.device:
            raise ValueError(f"scales: want torch.uint8 {(-(-self.N // 128), self._blocks)} on {codes.device}, got "
                             f"{scales.dtype} {tuple(scales.shape)} on {scales.device}")
        self.codes, self.scales = rows8(codes, scales)
        self._w = (self.codes.data_ptr(), _stride(self.codes), self.scales.data_ptr(), _stride(self.scales))

    @classmethod
    def from_weight(cls, w: torch.Tensor) -> "Linear8":
        """From a weight bf16 [N, K]."""
        return cls(*quantize8_weight(w))

    def forward(self, codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """out bf16 [T, N] = A W^T of A in 8 bits (codes uint8 [T, K], scales uint8
        [T, ceil(K / 128)], as ``rms_norm8`` and ``quantize8`` give them)."""
        T, dev = codes.shape[0], self._dev
        _want_rows("codes", codes, torch.uint8, dev, (T, self.K))
        _want_rows("scales", scales, torch.uint8, dev, (T, self._blocks))
        if _device() != dev:
            with torch.cuda.device(dev):
                return self.forward(codes, scales, out, stream)
        if out is None:
            out = _made(stream, self.device, lambda: torch.empty(T, self.N, dtype=torch.bfloat16, device=self.device))
        _want_rows("out", out, torch.bfloat16, dev, (T, self.N))
        _call("moe_linear8", B.lib().moe_linear8(
            codes.data_ptr(), _stride(codes), scales.data_ptr(), _stride(scales), *self._w, T, self.N, self.K,
            out.data_ptr(), out.stride(0) if T > 1 else self.N, _current(dev) if stream is None else B.handle(stream)))
        return out

    __call__ = forward
