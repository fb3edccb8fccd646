"""SiLU(gate) * up in 8 bits, on the GPU, as near float64 over the whole range of gates as fp32 allows.

Derived, in units of 2^-24 of the value: the exponential of half the gate is off by 4 (2 ulp) and once more by 1 where the
rest of its argument is put in, whose second order is 1.5 (a rest of 174 * 3.6e-6 ln 2), and comes in twice: 13; 1 + h^2
rounds (1), its reciprocal is off by 2 (1 ulp), and four products round (4): 20 in all.  A code's value is then half a step of the
exact value's own binade away from it at most (2^-4 of the power of two under it; 2^-10 of the scale under the normal
range), and ERR of it."""
import numpy as np
import pytest
import torch

import test_linear8 as tl
from moe_ffn_layer_gb300 import linear8 as L8
from test_linear8 import lib  # noqa: F401  (builds the library, and looks at the device's status at the end)

pytestmark = pytest.mark.gpu

ERR = 20 * 2.0 ** -24


@pytest.mark.parametrize("low,high", [(-170, -120), (-120, -87), (-87, -40), (-40, -8), (-8, 8), (8, 100)])
def test_gates_of_any_size(low, high):
    """Ups that bring the products near one another and, as far as bf16 goes, near 1, so that every code counts: 1 M of
    them, of which some thousand lie within 2^-17 of a border between codes."""
    g = torch.Generator("cuda").manual_seed(200 + low)
    T, K = 512, 2048
    base = torch.linspace(low + 2, high - 2, T, device="cuda")[:, None]
    gate = (base + 4 * torch.rand(T, K, generator=g, device="cuda") - 2).bfloat16()
    up = (0.5 + 0.5 * torch.rand(T, K, generator=g, device="cuda")) * (1 - 2 * torch.randint(0, 2, (T, K), generator=g, device="cuda"))
    up *= torch.exp2((-1.4427 * base).clamp(0, 126).floor())
    x = torch.cat([gate, up.bfloat16()], 1)
    codes, scales = L8.quantize8(x, silu_mul=True)
    y, scales = tl.lo.silu_mul(tl.np64(x)), tl.np8(scales)
    s = tl.lo.quantize(y)[1]
    off = scales != s
    if off.any():   # the block's largest lies within ERR of the border
        top = np.abs(y).reshape(T, -1, 128).max(2)[off]
        assert (np.abs(top / (448 * 2.0 ** (np.minimum(scales, s)[off].astype(float) - 127)) - 1) <= ERR).all()
    unit = tl.lo.spread(scales, 1, T, K)
    half = 2.0 ** (np.maximum(np.floor(np.log2(np.abs(y) / unit)), -6) - 4) * unit
    assert (np.abs(tl.lo.VALUES[tl.np8(codes)] * unit - y) <= half + ERR * np.abs(y)).all()


def test_ends():
    """Infinite, huge, tiny and NaN gates and ups."""
    inf, nan = float("inf"), float("nan")
    cases = [(inf, 1.0, nan), (inf, 0.0, nan), (-inf, 1.0, nan), (-inf, 0.0, nan), (nan, 1.0, nan), (1.0, nan, nan), (1.0, inf, nan),
             (-3e38, 3e38, 0.0), (-200.0, 3e38, 0.0), (3e38, 2.0 ** -126, 3e38 * 2.0 ** -126), (0.0, 3e38, 0.0), (-0.0, 3e38, 0.0),
             (2.0 ** -133, 2.0 ** 127, 2.0 ** -7), (-2.0 ** -130, 2.0 ** 127, -2.0 ** -4), (3e38, 3e38, nan)]
    gate, up = (torch.zeros(len(cases), 128) for _ in range(2))
    for i, (a, b, _) in enumerate(cases):
        gate[i, 5], up[i, 5] = a, b
    codes, scales = L8.quantize8(torch.cat([gate, up], 1).bfloat16().cuda(), silu_mul=True)
    got = tl.lo.values(tl.np8(codes), tl.np8(scales))[:, 5]
    for (a, b, want), v in zip(cases, got):
        a, b = (float(torch.tensor(t).bfloat16()) for t in (a, b))
        want = a * b if want == 3e38 * 2.0 ** -126 else want
        assert (v != v) if want != want else abs(v - want) <= (2.0 ** -4 + ERR) * abs(want), (a, b, want, v)
