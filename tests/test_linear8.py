"""The 8-bit projections on the GPU against float64.

Tolerances, derived.  Quantising bf16 values is exact but for the one rounding,
which the oracle makes as well: codes and scales are equal.  Where the value is
computed in fp32 (the norm, SiLU * up), with a relative error of at most ERR, a
code may fall to the other side of a rounding border: |value - exact| is then at
most half a step of e4m3 (2^-4 of the value, or 2^-10 of the scale under the
normal range) more than ERR of it; a scale may differ only where the block's
largest lies within ERR of the border.  ERR: a sum of H squares in fp32 in at
most 64 + 32 + 5 steps a thread and its tree (each 2^-24, under the square root
half of it), the division, root and products: (0.5 * 101 + 6) * 2^-24 < 2^-18.
The product's sums are in fp32: K / 32 additions of partial sums and 32 products
to each, a step at most 2^-22 of the sum of magnitudes (a truncating adder that
keeps 22 bits beside the largest), then bf16's half step 2^-8 of the result.
"""
import copy
import pickle

import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from moe_ffn_layer_gb300 import linear8 as L8
from oracle import linear8_oracle as lo

pytestmark = pytest.mark.gpu

ERR = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield B.lib()
    assert B.moe_last_device_error(torch.cuda.current_stream()) == 0


def np64(t):
    return t.double().cpu().numpy()


def np8(t):
    return t.cpu().numpy()


def rows(T, K, gap=0, seed=0):
    """bf16 rows `gap` elements apart, some channels and rows much larger, a block of zeros."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(T, K + gap, generator=g, device="cuda")
    x *= 1 + 31 * (torch.rand(K + gap, generator=g, device="cuda") < 0.02)
    x *= torch.exp2(torch.randint(-20, 20, (T, 1), generator=g, device="cuda").float())
    x[T // 2, :128] = 0
    return x.bfloat16()[:, :K]


def assert_near_codes(codes, scales, y, err=ERR):
    """codes and scales stand for y [R, K] within half a step and err."""
    want, s = lo.quantize(y)
    codes, scales = np8(codes), np8(scales)
    off = scales != s
    if off.any():   # the block's largest lies at the border
        i, j = np.nonzero(off)
        top = np.array([np.abs(y[r, 128 * b:128 * b + 128]).max() for r, b in zip(i, j)])
        border = 448 * 2.0 ** (np.minimum(scales, s)[off].astype(float) - 127)
        assert (np.abs(top / border - 1) <= err).all()
    unit = lo.spread(scales, 1, *y.shape)
    got = lo.VALUES[codes] * unit
    assert np.array_equal(np.isnan(got), ~np.isfinite(y))
    fine = np.isfinite(y)
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * unit) + err * np.abs(y)
    assert (np.abs(got - y)[fine] <= tol[fine]).all()
    # the codes differ only where a rounding may fall either way: a border is at most 2^-4 of a value away
    # from the next, so that 2 err / 2^-4 of the values lie within err of one (twice that, and a few, allowed)
    same = fine & ~off.repeat(128, 1)[:, :y.shape[1]]
    assert np.sum((codes != want)[same]) <= 4 + 64 * err * same.sum()


# ---------------------------------------------------------------- quantising
@pytest.mark.parametrize("T,K,gap", [(1, 16, 0), (1, 128, 8), (3, 144, 0), (7, 2048, 128), (257, 272, 24), (1021, 768, 0),
                                     (64, 8208, 16), (5, 112, 0)])
def test_quantize_rows_equal(T, K, gap):
    x = rows(T, K, gap, T + K)
    codes, scales = L8.quantize8(x)
    want, s = lo.quantize(np64(x))
    assert np.array_equal(np8(scales), s) and np.array_equal(np8(codes), want)


@pytest.mark.parametrize("N,K,gap", [(1, 16, 0), (128, 128, 0), (129, 144, 8), (300, 2064, 0), (1000, 768, 40)])
def test_quantize_weight_equal(N, K, gap):
    w = rows(N, K, gap, N + K)
    codes, scales = L8.quantize8_weight(w)
    want, s = lo.quantize(np64(w), 128)
    assert np.array_equal(np8(scales), s) and np.array_equal(np8(codes), want)


def special_rows():
    """Rows of one block each at the ends of bf16 and at the scales' borders."""
    out = [torch.zeros(128)]
    for e in (-133, -126, -118, -117, -30, 0, 100, 118, 119):
        for top in (1.75, 1.7578125, 1.7421875):
            r = torch.linspace(-1, 1, 128) * 2.0 ** e
            r[17] = top * 2.0 ** e
            out.append(r)
    for bad in (float("inf"), -float("inf"), float("nan")):
        r = torch.linspace(-3, 3, 128)
        r[5] = bad
        out.append(r)
        out.append(torch.full((128,), bad))
    r = torch.full((128,), -0.0)
    out.append(r)
    return torch.stack(out).bfloat16().cuda()


def test_quantize_special_values():
    x = special_rows()
    codes, scales = L8.quantize8(x)
    want, s = lo.quantize(np64(x))
    assert np.array_equal(np8(scales), s) and np.array_equal(np8(codes), want)
    one = x.reshape(1, -1)
    codes1, scales1 = L8.quantize8(one)   # and as the blocks of one row
    assert torch.equal(codes1.view(-1), codes.view(-1)) and torch.equal(scales1.view(-1), scales.view(-1))
    codes, scales = L8.quantize8_weight(x)   # one block for all
    want, s = lo.quantize(np64(x), 128)
    assert np.array_equal(np8(scales), s) and np.array_equal(np8(codes), want)


@pytest.mark.parametrize("T,K,gap", [(1, 16, 0), (333, 768, 0), (9, 1040, 8), (130, 2048, 64)])
def test_silu_mul(T, K, gap):
    """exp and the quotient by the fast instructions: 2 + |gate| 2^-1 ulp and 2 ulp; gates here stay under 100."""
    x = rows(T, 2 * K, gap, T + K).float().clamp(-100, 100).bfloat16()
    codes, scales = L8.quantize8(x, silu_mul=True)
    assert_near_codes(codes, scales, lo.silu_mul(np64(x)), err=64 * 2.0 ** -23)


def test_silu_mul_far_gates():
    """Gates whose exponential overflows give 0; an infinite gate or up gives what the formula gives."""
    inf = float("inf")
    gate = torch.tensor([-1e4, -90.0, 90.0, 1e4, inf, float("nan"), 3.0, 0.0] + [1.0] * 120)
    up = torch.tensor([2.0, 2.0, 2.0, 2.0, 1.0, 1.0, inf, 5.0] + [1.0] * 120)
    codes, scales = L8.quantize8(torch.cat([gate, up]).bfloat16().cuda()[None], silu_mul=True)
    got = lo.values(np8(codes), np8(scales))[0]
    assert got[0] == 0 and got[1] == 0 and got[7] == 0
    assert np.isnan(got[4:7]).all() and abs(got[3] / 2e4 - 1) < 2.0 ** -4 + 2.0 ** -8


def test_silu_mul_small_products():
    """Gates whose sigmoid is under the fp32 range, alone in their blocks and with ups that bring the product back into it:
    exp twice of half the gate, 2 + 1.17 |gate| / 2 ulp each, and six for the quotient and products."""
    g = torch.Generator("cuda").manual_seed(5)
    gate = -60 - 60 * torch.rand(40, 640, generator=g, device="cuda")
    up = torch.randn(40, 640, generator=g, device="cuda") * torch.exp2(torch.arange(40, device="cuda") * 3.0)[:, None]
    x = torch.cat([gate, up], 1).bfloat16()
    codes, scales = L8.quantize8(x, silu_mul=True)
    assert int(codes.count_nonzero()) > 12000
    assert_near_codes(codes, scales, lo.silu_mul(np64(x)), err=160 * 2.0 ** -23)


# ---------------------------------------------------------------- the norm
@pytest.mark.parametrize("T,H,gap,residual,weight,outputs", [
    (1, 16, 0, True, True, "both"), (1, 2048, 0, True, True, "codes"), (3, 128, 8, False, False, "both"),
    (7, 2064, 24, True, True, "both"), (300, 768, 0, True, False, "y"), (5, 4096, 128, False, True, "codes"),
    (1030, 256, 0, True, True, "both"), (2, 8192, 0, True, True, "both"), (3, 16400, 0, True, True, "both"),
    (2, 65536, 0, True, True, "codes"), (65, 112, 16, True, True, "both")])
def test_norm(T, H, gap, residual, weight, outputs):
    x = rows(T, H, gap, T + H)
    r = rows(T, H, gap // 8 * 16, T + H + 1) if residual else None
    w = (1 + 0.2 * torch.randn(H, device="cuda")).bfloat16() if weight else None
    n = L8.rms_norm8(x, w, 1e-5, r, outputs)
    h = x if r is None else (x.float() + r.float()).bfloat16()
    assert n.h is None if r is None else torch.equal(n.h.view(torch.int16), h.view(torch.int16))
    y = lo.rms_norm(np64(h), None if w is None else np64(w), 1e-5)
    assert (n.y is None) == (outputs == "codes") and (n.codes is None) == (outputs == "y")
    if n.y is not None:
        assert (np.abs(np64(n.y) - y) <= (2.0 ** -8 + ERR) * np.abs(y)).all()
    if n.codes is not None:
        assert_near_codes(n.codes, n.scales, y)


def test_norm_in_place_and_rows_behind():
    """h over the residual itself and over x; rows and columns beyond stay as they were."""
    H = 272
    x, r = rows(9, H, 16, 1), rows(9, H, 16, 2)
    want = L8.rms_norm8(x, None, 1e-6, r, "both")
    for over in ("x", "residual"):
        base = {"x": torch.full((12, H + 16), 7.0, device="cuda").bfloat16(), "residual": torch.full((12, H + 16), 7.0, device="cuda").bfloat16()}
        a, b = base["x"][:9, :H].copy_(x), base["residual"][:9, :H].copy_(r)
        codes = torch.full((12, 288), 9, dtype=torch.uint8, device="cuda")
        scales = torch.full((12, 8), 9, dtype=torch.uint8, device="cuda")
        y = torch.full((12, 280), 7.0, device="cuda").bfloat16()
        into = L8.Norm8(codes[:9, :H], scales[:9, :3], a if over == "x" else b, y[:9, :H])
        got = L8.rms_norm8(a, None, 1e-6, b, "both", into)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        for t, n in ((codes, H), (scales, 3)):
            assert (t[9:] == 9).all() and (t[:, n:] == 9).all()
        assert (y[9:] == 7).all() and (y[:, H:] == 7).all()
        assert (base[over][9:] == 7).all() and (base[over][:, H:] == 7).all()


def test_norm_special_rows():
    x = torch.zeros(4, 256, device="cuda")
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 2.0 ** 100   # the sum of squares passes fp32
    n = L8.rms_norm8(x.bfloat16(), None, 1e-6, None, "both")
    v = lo.values(np8(n.codes), np8(n.scales))
    y = np64(n.y)
    for got in (v, y):
        assert (got[0] == 0).all() and np.isnan(got[1]).all() and (got[3] == 0).all()
        assert np.isnan(got[2, 5]) and (np.delete(got[2], 5) == 0).all()


# ---------------------------------------------------------------- the product
def random8(R, K, high, seed, span=12):
    """All 254 codes that are numbers, scales of some powers of two."""
    g = torch.Generator("cuda").manual_seed(seed)
    codes = torch.randint(0, 254, (R, K), generator=g, device="cuda")
    codes += codes >= 127
    scales = torch.randint(127 - span, 127 + span, (-(-R // high), -(-K // 128)), generator=g, device="cuda")
    return L8.rows8(codes.to(torch.uint8), scales.to(torch.uint8))


def assert_linear(out, a, w, rows_of=None):
    A, W = lo.values(np8(a.codes), np8(a.scales)), lo.values(np8(w.codes), np8(w.scales), 128)
    ref, size = lo.linear(A if rows_of is None else A[rows_of], W)
    got = np64(out)
    assert got.shape == ref.shape and (np.isnan(got) == np.isnan(ref)).all()
    fine = ~np.isnan(ref)
    steps = W.shape[1] / 32 + 32
    tol = 2.0 ** -8 * np.abs(ref) + steps * 2.0 ** -22 * size
    assert (np.abs(got - ref)[fine] <= tol[fine]).all()


SIZES = [(1, 1, 16), (1, 128, 128), (1, 4096, 2048), (2, 40, 144), (7, 129, 272), (8, 256, 4096), (15, 2500, 2000),
         (16, 384, 640), (17, 128, 1024), (31, 513, 80), (33, 130, 528), (63, 2048, 768), (64, 1000, 128), (65, 64, 2064),
         (127, 300, 256), (128, 256, 512), (129, 257, 1040), (200, 2500, 2000), (255, 77, 64), (256, 512, 2048),
         (257, 1030, 384), (400, 255, 1536), (511, 8, 128), (513, 2049, 192), (1000, 640, 896), (1500, 3000, 1168),
         (2049, 1025, 336), (4100, 264, 160),
         (1, 300, 4112), (5, 129, 8208), (16, 130, 4128), (9, 7400, 272), (3, 20000, 80), (16, 257, 2064), (12, 16, 4096)]


@pytest.mark.parametrize("T,N,K", SIZES)
def test_linear(T, N, K):
    a, w = random8(T, K, 1, T + N), random8(N, K, 128, K + N)
    out = L8.Linear8(*w)(*a)
    assert_linear(out, a, w)


@pytest.mark.parametrize("T,N,K", [(1, 520, 1040), (5, 520, 1040), (5, 520, 4112), (16, 520, 1040), (16, 7400, 1040), (30, 520, 1040),
                                   (40, 520, 1040), (64, 520, 4112), (100, 2000, 1040), (128, 520, 1040), (300, 8200, 1040),
                                   (1024, 520, 1040), (1024, 5200, 528), (2100, 4520, 272)])
def test_linear_exact(T, N, K):
    """Small whole numbers, whose sums fp32 holds: every bit, on every path."""
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").float()
    m = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    e = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    sa = torch.randint(126, 129, (T, -(-K // 128)), generator=g, device="cuda", dtype=torch.uint8)
    sw = torch.randint(126, 129, (-(-N // 128), -(-K // 128)), generator=g, device="cuda", dtype=torch.uint8)
    a, w = L8.rows8(e(x), sa), L8.rows8(e(m), sw)
    out = L8.Linear8(*w)(*a)
    ref = lo.linear(lo.values(np8(a.codes), np8(a.scales)), lo.values(np8(w.codes), np8(w.scales), 128))[0]
    assert torch.equal(out.cpu().view(torch.int16), torch.from_numpy(ref).float().bfloat16().view(torch.int16))


@pytest.mark.parametrize("T,N,K,pad_s", [(3, 200, 272, 2), (2, 200, 4112, 3), (20, 200, 272, 5), (20, 200, 512, 8), (70, 136, 400, 2),
                                         (70, 136, 512, 3), (600, 300, 272, 4), (1100, 4300, 272, 1), (1100, 4300, 512, 2),
                                         (1100, 4300, 1024, 8)])
def test_linear_strides_and_rows_behind(T, N, K, pad_s):
    """Operands and outputs that lie in larger tensors; what is beyond them stays as it was."""
    big = torch.randint(0, 120, (T + 3, K + 48), dtype=torch.uint8, device="cuda")
    nb = -(-K // 128)
    apart, at_s = nb + pad_s, pad_s // 2
    bs = torch.randint(120, 130, (T + 3, apart), dtype=torch.uint8, device="cuda")
    bs[:, :at_s] = bs[:, at_s + nb:] = 255   # NaN beside what is used
    wide = torch.randint(0, 120, (N, -(-K // 128) * 128 + 128), dtype=torch.uint8, device="cuda")
    ws = torch.randint(120, 130, (-(-N // 128), apart), dtype=torch.uint8, device="cuda")
    ws[:, nb:] = 255
    a, w = L8.Block8(big[:T, 16:16 + K], bs[:T, at_s:at_s + nb]), L8.Block8(wide[:, :K], ws[:, :nb])
    lin = L8.Linear8(*w)
    assert lin.codes.data_ptr() == wide.data_ptr()   # not copied
    for pad, at in ((8, 0), (7, 0), (8, 1), (0, 0)):   # 16-byte rows, odd rows, an odd start, its own rows
        out = torch.full((T + 2, N + pad), 7.0, device="cuda").bfloat16()
        view = out[:T, at:at + N]
        assert lin(*a, out=view) is view
        assert_linear(view, a, w)
        assert (out[T:] == 7).all() and (out[:, :at] == 7).all() and (out[:, at + N:] == 7).all()
    near = torch.empty(N, K + 16, dtype=torch.uint8, device="cuda")[:, :K].copy_(w.codes)   # weights' rows that begin anywhere
    got = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    B.moe_linear8(a.codes, a.codes.stride(0), a.scales, a.scales.stride(0), near, K + 16, w.scales, apart, T, N, K, got, N,
                  torch.cuda.current_stream())
    assert torch.equal(got.view(torch.int16), view.view(torch.int16))


@pytest.mark.parametrize("T,K", [(2, 528), (2, 4112), (14, 528), (40, 528), (200, 528), (700, 528), (6000, 528)])
def test_linear_nan(T, K):
    """A NaN code or scale reaches its row or column, and nothing else."""
    N = 300
    a, w = random8(T, K, 1, 1, 4), random8(N, K, 128, 2, 4)
    a.codes[1, K - 1], a.scales[T - 1, 2] = 127, 255
    w.codes[5, 0], w.scales[2, 3] = 255, 255
    out = np64(L8.Linear8(*w)(*a))
    want = np.zeros((T, N), bool)
    want[1] = want[T - 1] = True
    want[:, 5] = want[:, 256:] = True
    assert (np.isnan(out) == want).all()


@pytest.mark.parametrize("T,K", [(3, 256), (3, 4112), (50, 256), (300, 256), (6000, 256)])
def test_linear_far_scales(T, K):
    """Scales at both ends of their range, whose product is of ordinary size."""
    N = 140
    a, w = random8(T, K, 1, 3, 1), random8(N, K, 128, 4, 1)
    for la, lw in ((1, 240), (247, 10)):
        a.scales.fill_(la)
        w.scales.fill_(lw)
        assert_linear(L8.Linear8(*w)(*a), a, w)


@pytest.mark.parametrize("T,N,K", [(1, 4096, 2048), (4, 600, 8192), (60, 640, 4096), (500, 1000, 1024), (1500, 4000, 512)])
def test_same_bits_again(T, N, K):
    a, w = random8(T, K, 1, 5), random8(N, K, 128, 6)
    lin = L8.Linear8(*w)
    first = lin(*a)
    for _ in range(5):
        assert torch.equal(lin(*a).view(torch.int16), first.view(torch.int16))


# ---------------------------------------------------------------- streams, graphs, a run of them
def chain(x, r, weight, lin1, lin2, stream=None):
    """norm -> gate_up -> SiLU * up -> down, the dense FFN of a layer."""
    n = L8.rms_norm8(x, weight, 1e-6, r, stream=stream)
    gu = lin1(n.codes, n.scales, stream=stream)
    q = L8.quantize8(gu, silu_mul=True, stream=stream)
    return n, gu, q, lin2(*q, stream=stream)


@pytest.mark.parametrize("T,H,I", [(1, 256, 384), (37, 512, 272), (600, 256, 640)])
def test_dense_ffn(T, H, I):
    x, r = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda").bfloat16()
    weight = torch.rand(H, device="cuda").bfloat16()
    w1 = L8.quantize8_weight((torch.randn(2 * I, H, device="cuda") * H ** -0.5).bfloat16())
    w2 = L8.quantize8_weight((torch.randn(H, I, device="cuda") * I ** -0.5).bfloat16())
    lin1, lin2 = L8.Linear8(*w1), L8.Linear8(*w2)
    n, gu, q, out = chain(x, r, weight, lin1, lin2)
    assert_near_codes(n.codes, n.scales, lo.rms_norm(np64((x.float() + r.float()).bfloat16()), np64(weight), 1e-6))
    assert_linear(gu, L8.Block8(n.codes, n.scales), w1)
    assert_near_codes(*q, lo.silu_mul(np64(gu)), err=64 * 2.0 ** -23)
    assert_linear(out, q, w2)
    # against the unquantised layer: each of the four quantised operands is off by 2^-4 of a value at most,
    # about 2^-5.3 in the root mean square, independently: 5 % of the output
    h = np64(x) + np64(r)
    full = lo.silu_mul(lo.rms_norm(h, np64(weight), 1e-6) @ lo.values(np8(w1.codes), np8(w1.scales), 128).T) \
        @ lo.values(np8(w2.codes), np8(w2.scales), 128).T
    assert np.linalg.norm(np64(out) - full) <= 0.1 * np.linalg.norm(full)

    # on another stream, by object and by handle
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = chain(x, r, weight, lin1, lin2, s)[3]
        side.synchronize()
        assert torch.equal(got, out)

    # captured, then replayed over new inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = chain(x, r, weight, lin1, lin2)[3]
    x.copy_(torch.randn(T, H, device="cuda").bfloat16())
    fresh = chain(x, r, weight, lin1, lin2)[3]
    for _ in range(3):
        captured.zero_()
        graph.replay()
        assert torch.equal(captured, fresh)


def test_wrappers_refuse():
    x = torch.zeros(4, 256, device="cuda").bfloat16()
    q = L8.quantize8(x)
    lin = L8.Linear8(*L8.quantize8_weight(torch.zeros(40, 256, device="cuda").bfloat16()))
    for bad in (lambda: L8.quantize8(x.float()), lambda: L8.quantize8(x[0]), lambda: L8.quantize8(x.t()),
                lambda: L8.quantize8(x[:, :255], silu_mul=True), lambda: L8.quantize8(x, into=L8.quantize8(x[:, :128])),
                lambda: L8.rms_norm8(x, outputs="h"), lambda: L8.rms_norm8(x, torch.ones(256, device="cuda")),
                lambda: L8.rms_norm8(x, residual=x[:3]), lambda: L8.rms_norm8(x, residual=x.cpu()),
                lambda: L8.rms_norm8(x, into=L8.rms_norm8(x, outputs="y")),
                lambda: L8.rms_norm8(x, residual=x, into=L8.rms_norm8(x)), lambda: L8.rms_norm8(x[:2], into=L8.rms_norm8(x)),
                lambda: L8.rms_norm8(x, into=L8.Norm8(q.codes, q.scales[:2], None, None)),
                lambda: L8.quantize8(x[:3], into=q), lambda: L8.quantize8(x, into=L8.Block8(q.codes, q.scales.float())),
                lambda: lin(x, q.scales), lambda: lin(q.codes[:, :128], q.scales), lambda: lin(q.codes, q.scales[:2]),
                lambda: lin(*q, out=torch.empty(4, 39, device="cuda").bfloat16()), lambda: lin(*q, out=torch.empty(4, 40, device="cuda")),
                lambda: L8.Linear8(q.codes, q.scales), lambda: L8.Linear8(x, q.scales)):
        with pytest.raises(ValueError):
            bad()
    many = x[:1, :16].expand(2 ** 32 + 1, 16)   # (a 32-bit count of its rows is one)
    for bad in (lambda: L8.quantize8(many), lambda: L8.rms_norm8(many), lambda: L8.quantize8_weight(many),
                lambda: lin(q.codes[:1].expand(2 ** 32 + 1, 256), q.scales[:1].expand(2 ** 32 + 1, 2), out=x),
                lambda: L8.Linear8(q.codes[:1].expand(2 ** 32 + 1, 256), q.scales[:1].expand(2 ** 25 + 1, 2))):
        with pytest.raises(ValueError, match="31 bits"):
            bad()
    with pytest.raises(AttributeError):
        lin.codes = q.codes
    host = torch.empty(4, 40, dtype=torch.bfloat16)
    for bad in (lambda: L8.quantize8(x[:, :40]), lambda: L8.quantize8(x[:, 4:20]),
                lambda: B.moe_linear8(q.codes, 256, q.scales, 4, lin.codes, 256, lin.scales, 4, 4, 40, 256, host, 40, None)):
        with pytest.raises(B.MoEError) as e:
            bad()
        assert e.value.code == -2
    assert L8.quantize8(x[:0]).codes.shape == (0, 256) and lin(*L8.quantize8(x[:0])).shape == (0, 40)
    assert L8.rms_norm8(x[:0], residual=x[:0], outputs="both").y.shape == (0, 256)


@pytest.mark.parametrize("again", [copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))])
def test_copies_are_matrices_of_their_own(again):
    """A copy of results, or of a weight, has its own memory: written and read there, the original as it was."""
    x, y = rows(5, 256, 0, 1), rows(5, 256, 0, 2)
    lin = L8.Linear8(*L8.quantize8_weight(rows(40, 256, 0, 3)))
    for make in (lambda x, into=None: L8.quantize8(x, into=into), lambda x, into=None: L8.rms_norm8(x, None, 1e-6, x, "both", into)):
        q = make(x)
        kept, other = [t.clone() for t in q], again(q)
        assert type(other) is type(q) and all(torch.equal(t, u) for t, u in zip(q, other))
        make(y, other)
        assert all(torch.equal(t, u) for t, u in zip(q, kept)) and all(torch.equal(t, u) for t, u in zip(other, make(y)))
    q, twin = L8.quantize8(x), again(lin)
    want = lin(*q)
    assert torch.equal(twin(*q), want)
    lin.codes.zero_()
    assert torch.equal(twin(*q), want) and not lin(*q).any()


@pytest.mark.parametrize("T,N,K", [(3, 128, 4112), (3, 300, 8192), (3, 7400, 272), (20, 300, 2048), (40, 520, 1024), (300, 2048, 512),
                                   (1100, 512, 640), (1200, 4100, 640)])
def test_expired_waits_write_nothing(T, N, K):
    """With the wait limit at 0 a wait that is not complete at its first test expires: the product records it,
    lets its copies and MMAs in flight end, and writes nothing; the next call is clean."""
    a, w = random8(T, K, 1, 8), random8(N, K, 128, 9)
    lin = L8.Linear8(*w)
    fresh = lin(*a)
    out = torch.full_like(fresh, 5.0)
    s = torch.cuda.current_stream()
    assert B.moe_last_device_error(s) == 0
    try:
        B.moe_debug_set_wait_limit_ns(0)
        lin(*a, out=out)
    finally:
        B.moe_debug_set_wait_limit_ns(2_000_000_000)
    assert B.moe_last_device_error(s) == -5
    assert (out == 5.0).all()
    assert torch.equal(lin(*a).view(torch.int16), fresh.view(torch.int16))
    assert B.moe_last_device_error(s) == 0


def test_first_call_inside_a_capture():
    """In a process that has made no call before."""
    code = """
import torch
from moe_ffn_layer_gb300 import linear8 as L8
x = torch.ones(600, 256, device="cuda").bfloat16()
w = L8.Block8(torch.full((4000, 256), 56, dtype=torch.uint8, device="cuda"), torch.full((32, 4), 127, dtype=torch.uint8, device="cuda")[:, :2])
lin, outs = L8.Linear8(*w), []
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for T in (1, 12, 20, 60, 128, 600):
        n = L8.rms_norm8(x[:T], None, 0.0, x[:T])
        outs.append(lin(n.codes, n.scales))
graph.replay()
torch.cuda.synchronize()
assert all((o == 256).all() for o in outs), [o.float().mean() for o in outs]
print("fine")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_calls_on_two_streams_at_once():
    """Nothing is shared between calls: two streams' results are those of one after the other."""
    work = []
    for i, (T, N, K) in enumerate([(3, 4096, 2048), (50, 3000, 2048), (400, 1000, 1024), (1500, 4000, 512)]):
        a, w = random8(T, K, 1, i), random8(N, K, 128, 9 + i)
        work.append((L8.Linear8(*w), a))
    want = [lin(*a) for lin, a in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for s, out, order in zip(streams, got, (work, work[::-1])):
            with torch.cuda.stream(s):
                out.append([lin(*a) for lin, a in order])
    torch.cuda.synchronize()
    for outs in got[0]:
        assert all(torch.equal(o.view(torch.int16), x.view(torch.int16)) for o, x in zip(outs, want))
    for outs in got[1]:
        assert all(torch.equal(o.view(torch.int16), x.view(torch.int16)) for o, x in zip(outs[::-1], want))


def test_offsets_past_32_bits():
    """Rows whose bytes and elements lie past 2^32: quantised, normed and multiplied as the same rows by themselves."""
    T, K = 1100000, 4096
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").zero_()
    at = torch.tensor([0, 1, 524288, 1048575, 1048576, T - 2, T - 1], device="cuda")
    few = rows(len(at), K, 0, 11)
    x[at] = few
    q, want = L8.quantize8(x), L8.quantize8(few)
    assert torch.equal(q.codes[at], want.codes) and torch.equal(q.scales[at], want.scales)
    assert int(q.codes.count_nonzero()) == int(want.codes.count_nonzero())
    n, some = L8.rms_norm8(x, None, 1e-6, x, "both"), L8.rms_norm8(few, None, 1e-6, few, "both")
    for t, u in zip(n, some):
        assert torch.equal(t[at].view(torch.uint8), u.view(torch.uint8))
    del n, x
    w = random8(40, K, 128, 3, 4)
    lin = L8.Linear8(*w)
    out, rest = lin(*q)[at], lin(*want)   # (by other kernels: the same up to the order of their sums)
    assert (out.float() - rest.float()).abs().max() <= 2.0 ** -7 * rest.float().abs().max()
    big = L8.Block8(q.codes[:1048600], q.scales[:1048600])   # as weights: 4 GB of rows
    ones = torch.full((8208, 32), 127, dtype=torch.uint8, device="cuda")[:-(-1048600 // 128)]
    a = random8(3, K, 1, 4, 4)
    y = L8.Linear8(big.codes, ones)(*a)
    ref, size = lo.linear(lo.values(np8(a.codes), np8(a.scales)), lo.VALUES[np8(big.codes[at[:5]])])
    assert (np.abs(np64(y[:, at[:5]]) - ref) <= 2.0 ** -8 * np.abs(ref) + 160 * 2.0 ** -22 * size).all()
