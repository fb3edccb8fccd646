"""Norm and quantisation at the sizes that choose each form of their kernels, on the GPU: vectors a thread (1, 2, 4, 8), blocks
a thread (1, 4), ends inside a CTA's share, and nothing written beside the results."""
import numpy as np
import pytest
import torch

import test_linear8 as tl
from moe_ffn_layer_gb300 import linear8 as L8
from test_linear8 import lib  # noqa: F401  (builds the library, and looks at the device's status at the end)

pytestmark = pytest.mark.gpu


def guarded(T, K, dtype, more=8, fill=9):
    """A [T, K] matrix in a larger tensor, and a check that what is beside it is as it was."""
    base = torch.full((T + 2, K + more), fill, dtype=dtype, device="cuda")

    def check():
        assert (base[T:] == fill).all() and (base[:, K:] == fill).all()
    return base[:T, :K], check


def vectors(T, H):
    """rms_norm8_launch's rule, restated."""
    vecs, n = 1, H // 8
    while vecs < 8 and n > (512 if T <= 256 else 256) * vecs:
        vecs *= 2
    return vecs


# (vectors a thread, T, H)
NORMS = [(1, 256, 4096), (1, 300, 2048), (2, 256, 8192), (2, 257, 4096), (2, 3, 4112), (4, 300, 5136), (4, 257, 8192), (4, 3, 12304),
         (4, 256, 16384), (4, 1, 8208), (8, 300, 8208), (8, 257, 16384), (8, 3, 16400), (8, 300, 16400), (8, 260, 65536), (8, 1, 65520)]


@pytest.mark.parametrize("vecs,T,H", NORMS)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(vecs, T, H, residual):
    assert vectors(T, H) == vecs
    x, r = tl.rows(T, H, 24, T + H), tl.rows(T, H, 8, T + H + 1) if residual else None
    w = (1 + 0.2 * torch.randn(H, device="cuda")).bfloat16()
    codes, codes_kept = guarded(T, H, torch.uint8, 16)
    scales, scales_kept = guarded(T, -(-H // 128), torch.uint8, 3)
    y, y_kept = guarded(T, H, torch.bfloat16)
    h, h_kept = guarded(T, H, torch.bfloat16)
    into = L8.Norm8(codes, scales, h if residual else None, y)
    L8.rms_norm8(x, w, 1e-5, r, "both", into)
    stored = x if r is None else (x.float() + r.float()).bfloat16()
    if residual:
        assert torch.equal(h.contiguous().view(torch.int16), stored.view(torch.int16))
    want = tl.lo.rms_norm(tl.np64(stored), tl.np64(w), 1e-5)
    assert (np.abs(tl.np64(y) - want) <= (2.0 ** -8 + tl.ERR) * np.abs(want)).all()
    tl.assert_near_codes(codes, scales, want)
    for check in (codes_kept, scales_kept, y_kept, h_kept):
        check()


# 65536 blocks of 128 from which on a thread has four: under it, at it, over it with 25 blocks, one and 63 in the last CTA (of 64)
ROWS = [(7281, 1040, 0), (8192, 1024, 8), (8209, 1040, 24), (65537, 128, 0), (65599, 112, 16)]


@pytest.mark.parametrize("T,K,gap", ROWS)
@pytest.mark.parametrize("silu", [False, True])
def test_quantize(T, K, gap, silu):
    x = tl.rows(T, 2 * K if silu else K, gap, T + K)
    if silu:
        x.clamp_(-100, 100)   # as test_silu_mul, whose bound this is
    codes, codes_kept = guarded(T, K, torch.uint8, 16)
    scales, scales_kept = guarded(T, -(-K // 128), torch.uint8, 3)
    L8.quantize8(x, silu, L8.Block8(codes, scales))
    if silu:
        tl.assert_near_codes(codes, scales, tl.lo.silu_mul(tl.np64(x)), err=64 * 2.0 ** -23)
    else:
        want, s = tl.lo.quantize(tl.np64(x))
        assert np.array_equal(tl.np8(scales), s) and np.array_equal(tl.np8(codes), want)
    codes_kept()
    scales_kept()


def test_last_blocks_are_uneven():
    blocks = [T * -(-K // 128) for T, K, _ in ROWS]
    assert [b >= 1 << 16 for b in blocks] == [False, True, True, True, True]
    assert [b % 64 for b in blocks[1:]] == [0, 25, 1, 63]
