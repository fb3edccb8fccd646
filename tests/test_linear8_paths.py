"""Every kernel of the 8-bit product, by the rules that choose (restated here): sizes that reach each, held to those rules
without a GPU; and on it, exact bits, random codes, strides, NaN, scales at their ends and the same bits again at each."""
import pytest
import torch

import test_linear8 as tl
from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from moe_ffn_layer_gb300 import linear8 as L8

# the kernel, and sizes that reach it on 148 to 160 SMs
SIZES = [
    ("few<2, 2>", 12, 304, 2032), ("few<2, 2>", 9, 2049, 640),
    ("few<2, 1>", 1, 4096, 2048), ("few<2, 1>", 7, 333, 1040),
    ("few<1, 1>", 8, 6144, 2064), ("few<1, 1>", 3, 520, 272), ("few<1, 1>", 2, 7000, 1168), ("few<1, 1>", 5, 129, 4096),
    ("narrow<16>", 1, 8192, 4112), ("narrow<16>", 16, 7400, 1040), ("narrow<16>", 13, 130, 8208), ("narrow<16>", 2, 20000, 144),
    ("narrow<32>", 17, 128, 1024), ("narrow<32>", 31, 2049, 528), ("narrow<32>", 32, 20000, 400),
    ("narrow<64>", 33, 130, 528), ("narrow<64>", 64, 6144, 4096), ("narrow<64>", 777, 2500, 2000), ("narrow<64>", 130, 4000, 3216),
    ("narrow<128>", 256, 6144, 4096), ("narrow<128>", 200, 6100, 3216), ("narrow<128>", 384, 4999, 3216), ("narrow<128>", 100, 12790, 3344),
    ("wide<1>", 1024, 4032, 2048), ("wide<1>", 2100, 4519, 272), ("wide<1>", 300, 8201, 1040), ("wide<1>", 513, 5000, 4112),
    ("wide<2>", 1500, 9000, 1168), ("wide<2>", 1100, 4297, 656), ("wide<2>", 2049, 2504, 4112),
]
NAMES = ["few<1, 1>", "few<2, 1>", "few<2, 2>", "narrow<16>", "narrow<32>", "narrow<64>", "narrow<128>", "wide<1>", "wide<2>"]
IDS = [f"{name}-{T}-{N}-{K}" for name, T, N, K in SIZES]


def kernel_of(T, N, K, sms):
    """linear8_few_takes, linear8_few_launch, linear8_launch, linear8_wide_launch."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    ctas = up(N, 16)
    if T <= 8 and K <= 4096 and ctas <= 3 * sms or 8 < T <= 16 and K <= 2048 and ctas <= 2 * sms:
        return "few<2, 2>" if T > 8 else "few<2, 1>" if 1024 < K <= 2048 and ctas <= 2 * sms else "few<1, 1>"
    for high in (16, 32, 64):
        if T <= high:
            return f"narrow<{high}>"
    if up(N, 128) * up(T, 64) <= (2 if K <= 24 * 128 else 1) * sms:
        return "narrow<64>"
    if up(N, 128) * up(T, 128) <= sms:
        return "narrow<128>"
    one, two = (up(up(N, 224) * up(T, high), sms // 2) for high in (256, 512))
    return "wide<1>" if 4 * one < 7 * two else "wide<2>"


def test_sizes_reach_every_kernel():
    for sms in (148, 152, 160):
        for name, *size in SIZES:
            assert kernel_of(*size, sms) == name, (size, sms)
    assert {name for name, *_ in SIZES} == set(NAMES)
    for name in NAMES:   # with rows that are whole vectors of 16 bytes, and rows that are not
        assert {N % 8 == 0 for of, _, N, _ in SIZES if of == name} == {True, False}


def gpu(test):
    return pytest.mark.gpu(pytest.mark.parametrize("name,T,N,K", SIZES, ids=IDS)(test))


@pytest.fixture
def clean():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert B.moe_last_device_error(torch.cuda.current_stream()) == 0


def random_pair(T, N, K, span=12):
    return tl.random8(T, K, 1, T + N, span), tl.random8(N, K, 128, K + N, span)


@gpu
def test_on_this_gpu(clean, name, T, N, K):
    assert kernel_of(T, N, K, torch.cuda.get_device_properties(0).multi_processor_count) == name


@gpu
def test_exact(clean, name, T, N, K):
    """Small whole numbers, whose sums fp32 holds (|a w| <= 16, scales' products 1/4 to 4, K <= 8208: multiples of 1/4 under 2^20):
    every bit.  One output column or token off, or a scale of another block or row, would show."""
    g = torch.Generator("cuda").manual_seed(T + N)
    small = lambda r: torch.randint(-4, 5, (r, K), generator=g, device="cuda").float()  # noqa: E731
    power = lambda r: torch.randint(126, 129, (r, -(-K // 128)), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    a, w = (L8.rows8(small(r).to(torch.float8_e4m3fn).view(torch.uint8), power(s)) for r, s in ((T, T), (N, -(-N // 128))))
    ref = tl.lo.linear(tl.lo.values(tl.np8(a.codes), tl.np8(a.scales)), tl.lo.values(tl.np8(w.codes), tl.np8(w.scales), 128))[0]
    ref = torch.from_numpy(ref).float().bfloat16().view(torch.int16)
    lin = L8.Linear8(*w)
    for pad, at in ((0, 0), (9, 1)):
        out = torch.empty(T, N + pad, dtype=torch.bfloat16, device="cuda")[:, at:at + N]
        assert torch.equal(lin(*a, out=out).cpu().view(torch.int16), ref)


@gpu
def test_random(clean, name, T, N, K):
    """All codes, and the same bits again, into rows of any place, from scales of any place, with what is beside untouched."""
    a, w = random_pair(T, N, K)
    lin = L8.Linear8(*w)
    first = lin(*a)
    tl.assert_linear(first, a, w)
    nb = a.scales.shape[1]
    beside = torch.full((T, nb + 5), 255, dtype=torch.uint8, device="cuda")   # NaN
    beside[:, 2:2 + nb] = a.scales
    wide = torch.full((w.scales.shape[0], nb + 3), 255, dtype=torch.uint8, device="cuda")
    wide[:, 1:1 + nb] = w.scales
    other = L8.Linear8(w.codes, wide[:, 1:1 + nb])
    for pad, at in ((0, 0), (8 - N % 8, 0), (16, 8), (7, 3)):
        out = torch.full((T + 2, N + pad), 7.0, device="cuda").bfloat16()
        view = out[:T, at:at + N]
        other(a.codes, beside[:, 2:2 + nb], out=view)
        assert torch.equal(view.view(torch.int16), first.view(torch.int16))
        assert (out[T:] == 7).all() and (out[:, :at] == 7).all() and (out[:, at + N:] == 7).all()


@gpu
def test_nan(clean, name, T, N, K):
    """NaN codes and scales reach their rows and columns, the last ones among them, and nothing else."""
    a, w = random_pair(T, N, K, 4)
    last = (K - 1) // 128
    a.codes[T - 1, K - 1] = 127
    a.scales[T // 2, last] = 255
    w.codes[N - 1, K - 1], w.codes[N // 2, 0] = 255, 127
    w.scales[0, last] = 255
    want = torch.zeros(T, N, dtype=torch.bool)
    want[[T // 2, T - 1]] = True
    want[:, [N // 2, N - 1]] = True
    want[:, :128] = True
    assert torch.equal(L8.Linear8(*w)(*a).isnan().cpu(), want)


@gpu
def test_far_scales(clean, name, T, N, K):
    a, w = random_pair(T, N, K, 1)
    lin = L8.Linear8(*w)
    for la, lw in ((1, 240), (247, 10)):
        a.scales.fill_(la)
        lin.scales.fill_(lw)
        tl.assert_linear(lin(*a), a, w)


@pytest.mark.gpu
@pytest.mark.parametrize("name,T,N,K", [s for s in SIZES if s[0].startswith(("narrow", "wide")) and s[3] >= 1024])
def test_expired_waits_write_nothing(clean, name, T, N, K):
    """With the wait limit at 0 a wait that is not complete at its first test expires: status -5, nothing written, and the
    next call is clean."""
    a, w = random_pair(T, N, K)
    lin, s = L8.Linear8(*w), torch.cuda.current_stream()
    fresh = lin(*a)
    out = torch.full_like(fresh, 5.0)
    assert B.moe_last_device_error(s) == 0
    try:
        B.moe_debug_set_wait_limit_ns(0)
        lin(*a, out=out)
    finally:
        B.moe_debug_set_wait_limit_ns(2_000_000_000)
    assert B.moe_last_device_error(s) == -5
    assert (out == 5.0).all()
    assert torch.equal(lin(*a).view(torch.int16), fresh.view(torch.int16))
