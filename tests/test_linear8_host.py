"""The 8-bit projections without a GPU: the oracle's pins, and what the C calls and their wrappers refuse."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from moe_ffn_layer_gb300 import linear8 as L8
from oracle import linear8_oracle as lo

INVALID, UNSUPPORTED = -1, -2
P = 1 << 20   # an aligned address that no refused call reads


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.lib()


def test_oracle_codes_are_torchs():
    x = torch.cat([torch.randn(4096) * 2.0 ** e for e in range(-12, 8)]).clamp(-448, 448)
    assert np.array_equal(lo.encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    c = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(lo.VALUES, c.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


def test_oracle_scales_are_the_least():
    for e in range(-117, 119):
        top = 448 * 2.0 ** e
        for amax, want in ((top, e), (np.nextafter(top, np.inf), e + 1), (np.nextafter(top, 0), e)):
            assert lo.scale_byte(np.float64(amax)) == max(want, -126) + 127
    assert lo.scale_byte(np.float64(0)) == 1 and lo.scale_byte(np.float64(2.0 ** -133)) == 1


def test_oracle_blocks_of_a_weight():
    """A weight that is a power of two per block comes back whole, ends included."""
    e = np.arange(6).reshape(2, 3) * 7 - 20
    w = (2.0 ** e).repeat(128, 0).repeat(128, 1)[:200, :272]
    codes, s = lo.quantize(w, 128)
    assert s.shape == (2, 3) and np.array_equal(lo.values(codes, s, 128), w)


NORM = dict(x=P, x_stride=256, residual=P, r_stride=256, weight=P, eps=1e-6, T=4, H=256, h=P, h_stride=256, y=None,
            y_stride=0, codes=P, ld=256, scales=P, lds=4, stream=None)
ROWS = dict(x=P, x_stride=256, T=4, K=256, act=0, codes=P, ld=256, scales=P, lds=4, stream=None)
WEIGHT = dict(w=P, w_stride=256, N=4, K=256, codes=P, ld=256, scales=P, lds=4, stream=None)
LINEAR = dict(a=P, lda=256, a_scales=P, las=4, w=P, ldw=256, w_scales=P, lws=4, T=4, N=40, K=256, out=P, out_stride=40,
              stream=None)


@pytest.mark.parametrize("name,base,change,want", [
    # null and inconsistent arguments
    ("moe_rms_norm8", NORM, dict(x=None), INVALID),
    ("moe_rms_norm8", NORM, dict(h=None), INVALID),
    ("moe_rms_norm8", NORM, dict(residual=None), INVALID),
    ("moe_rms_norm8", NORM, dict(codes=None), INVALID),
    ("moe_rms_norm8", NORM, dict(codes=None, scales=None), INVALID),   # no output
    ("moe_rms_norm8", NORM, dict(T=-1), INVALID),
    ("moe_rms_norm8", NORM, dict(H=0), INVALID),
    ("moe_rms_norm8", NORM, dict(eps=-1e-6), INVALID),
    ("moe_rms_norm8", NORM, dict(eps=float("nan")), INVALID),
    ("moe_rms_norm8", NORM, dict(eps=float("inf")), INVALID),
    ("moe_rms_norm8", NORM, dict(x_stride=248), INVALID),
    ("moe_rms_norm8", NORM, dict(r_stride=248), INVALID),
    ("moe_rms_norm8", NORM, dict(h_stride=0), INVALID),
    ("moe_rms_norm8", NORM, dict(y=P, y_stride=8), INVALID),
    ("moe_rms_norm8", NORM, dict(ld=240), INVALID),
    ("moe_rms_norm8", NORM, dict(lds=1), INVALID),
    ("moe_quantize8", ROWS, dict(x=None), INVALID),
    ("moe_quantize8", ROWS, dict(act=2), INVALID),
    ("moe_quantize8", ROWS, dict(act=1), INVALID),                     # rows of 2 K lie too near
    ("moe_quantize8", ROWS, dict(scales=None), INVALID),
    ("moe_quantize8", ROWS, dict(K=-16), INVALID),
    ("moe_quantize8_weight", WEIGHT, dict(w=None), INVALID),
    ("moe_quantize8_weight", WEIGHT, dict(N=-1), INVALID),
    ("moe_quantize8_weight", WEIGHT, dict(N=400, lds=1), INVALID),
    ("moe_linear8", LINEAR, dict(a=None), INVALID),
    ("moe_linear8", LINEAR, dict(w_scales=None), INVALID),
    ("moe_linear8", LINEAR, dict(out=None), INVALID),
    ("moe_linear8", LINEAR, dict(out_stride=39), INVALID),
    ("moe_linear8", LINEAR, dict(N=0), INVALID),
    ("moe_linear8", LINEAR, dict(T=-1), INVALID),
    ("moe_linear8", LINEAR, dict(lda=240), INVALID),
    ("moe_linear8", LINEAR, dict(las=1), INVALID),
    # sizes, strides and alignments that the kernels do not take
    ("moe_rms_norm8", NORM, dict(H=248), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(H=65552, x_stride=65552, r_stride=65552, h_stride=65552, ld=65552, lds=516), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(x=P + 2), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(residual=P + 8), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(h=P + 8), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(weight=P + 2), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(x_stride=260), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(y=P, y_stride=257), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(codes=P + 8), UNSUPPORTED),
    ("moe_rms_norm8", NORM, dict(ld=264), UNSUPPORTED),
    ("moe_quantize8", ROWS, dict(K=40, x_stride=256), UNSUPPORTED),
    ("moe_quantize8", ROWS, dict(x=P + 4), UNSUPPORTED),
    ("moe_quantize8", ROWS, dict(T=2 ** 31 - 1), UNSUPPORTED),         # more blocks than are counted
    ("moe_quantize8_weight", WEIGHT, dict(N=65535 * 128 + 1), UNSUPPORTED),
    ("moe_quantize8_weight", WEIGHT, dict(K=8), UNSUPPORTED),
    ("moe_quantize8_weight", WEIGHT, dict(K=2 ** 31 - 16, w_stride=2 ** 31, ld=2 ** 31, lds=2 ** 24), UNSUPPORTED),
    ("moe_quantize8", ROWS, dict(K=2 ** 30, x_stride=2 ** 31, ld=2 ** 30, lds=2 ** 23), UNSUPPORTED),
    ("moe_linear8", LINEAR, dict(K=136), UNSUPPORTED),
    ("moe_linear8", LINEAR, dict(a=P + 8), UNSUPPORTED),
    ("moe_linear8", LINEAR, dict(ldw=264), UNSUPPORTED),
    ("moe_linear8", LINEAR, dict(out=P + 1), UNSUPPORTED),
    ("moe_linear8", LINEAR, dict(T=2 ** 31 - 1), UNSUPPORTED),
    ("moe_linear8", LINEAR, dict(N=2 ** 31 - 1, out_stride=2 ** 31), UNSUPPORTED),
    ("moe_linear8", LINEAR, dict(), UNSUPPORTED),                      # memory that is no device's
])
def test_refused(name, base, change, want):
    with pytest.raises(B.MoEError) as e:
        getattr(B, name)(**{**base, **change})
    assert e.value.code == want
    assert B.moe_last_launch_count() == 0


@pytest.mark.parametrize("name,base,rows", [("moe_rms_norm8", NORM, "T"), ("moe_quantize8", ROWS, "T"),
                                            ("moe_quantize8_weight", WEIGHT, "N"), ("moe_linear8", LINEAR, "T")])
def test_no_rows_launch_nothing(name, base, rows):
    assert getattr(B, name)(**{**base, rows: 0}) == 0
    assert B.moe_last_launch_count() == 0


def test_wrappers_refuse_what_is_on_no_gpu():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    for call in (lambda: L8.rms_norm8(x), lambda: L8.quantize8(x), lambda: L8.quantize8_weight(x),
                 lambda: L8.Linear8(torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rows8_lays_out_what_lies_otherwise():
    def apart(n, K, step):   # codes whose rows begin at multiples of `step`, from 128 bytes on
        base = torch.zeros(n * step + 256, dtype=torch.uint8)
        return base[-base.data_ptr() % 128:].as_strided((n, K), (step, 1))

    values = torch.arange(3 * 144).to(torch.uint8).view(3, 144)
    scales = torch.arange(6, dtype=torch.uint8).view(3, 2)
    codes = apart(3, 144, 256).copy_(values)
    c, s = L8.rows8(codes, scales)
    assert c.data_ptr() == codes.data_ptr() and s.data_ptr() == scales.data_ptr()   # as they are
    s = L8.rows8(codes, torch.zeros(2, 3, dtype=torch.uint8).t().copy_(scales))[1]
    assert s.is_contiguous() and torch.equal(s, scales)
    wide = torch.zeros(144, 3, dtype=torch.uint8).t().copy_(values)
    for other in (values, wide, apart(3, 144, 160).copy_(values)):   # rows 144 bytes, columns, 160 bytes apart
        c, _ = L8.rows8(other, scales)
        assert c.stride() == (256, 1) and c.data_ptr() != other.data_ptr() and torch.equal(c, values)
    one = apart(1, 144, 16)   # a single row has no stride
    assert L8.rows8(one, scales[:1])[0].data_ptr() == one.data_ptr()
