"""Output rows of the pairs' tiles of 256 tokens that do not leave by tensor copies, on the GPU: the second epilogue
group's 96 of a tile's 224 columns begin at another alignment than the first's 128, and N ends inside either."""
import pytest
import torch

import test_linear8 as tl
from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import linear8 as L8
from test_linear8 import lib  # noqa: F401  (builds the library, and looks at the device's status at the end)

pytestmark = pytest.mark.gpu

# tiles of 256 tokens on 148 to 160 SMs; N ends 39 columns into a tile, in the first group's part; 137, in the second's;
# 224, at its end; 1; and 161
SIZES = [(2100, 4519, 272), (300, 8201, 1040), (300, 8288, 1040), (700, 4033, 144), (515, 4865, 128)]


def takes_256(T, N, K, sms):
    """The rule for products of more than 64 tokens (linear8_launch, linear8_wide_launch), restated."""
    wide, n, pairs = -(-N // 128), -(-N // 224), sms // 2
    narrow = wide * -(-T // 64) <= (2 if K <= 24 * 128 else 1) * sms or wide * -(-T // 128) <= sms
    waves = lambda high: -(-n * -(-T // high) // pairs)  # noqa: E731
    return T > 64 and not narrow and 4 * waves(256) < 7 * waves(512)


@pytest.mark.parametrize("T,N,K", SIZES)
def test_tiles_of_256_tokens(T, N, K):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert takes_256(T, N, K, sms)


@pytest.mark.parametrize("T,N,K", SIZES)
def test_rows_anywhere(T, N, K):
    """Rows some elements apart that begin anywhere; the same bits as rows by themselves, and nothing beside them."""
    a, w = tl.random8(T, K, 1, T), tl.random8(N, K, 128, N)
    lin = L8.Linear8(*w)
    own = lin(*a)
    tl.assert_linear(own, a, w)
    for pad, at in ((8, 0), (7, 0), (-N % 8, 0), (8, 1), (9, 3), (13, 5), (24, 7), (3, 2)):
        out = torch.full((T + 2, N + pad), 7.0, device="cuda").bfloat16()
        lin(*a, out=out[:T, at:at + N])
        assert torch.equal(out[:T, at:at + N].view(torch.int16), own.view(torch.int16))
        assert (out[T:] == 7).all() and (out[:, :at] == 7).all() and (out[:, at + N:] == 7).all()


@pytest.mark.parametrize("T,N,K", SIZES)
def test_exact(T, N, K):
    """Small whole numbers: every bit."""
    g = torch.Generator("cuda").manual_seed(T)
    small = lambda r: torch.randint(-4, 5, (r, K), generator=g, device="cuda").float()  # noqa: E731
    power = lambda r: torch.randint(126, 129, (r, -(-K // 128)), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    a, w = (L8.rows8(small(r).to(torch.float8_e4m3fn).view(torch.uint8), power(s)) for r, s in ((T, T), (N, -(-N // 128))))
    out = torch.empty(T, N + 5, dtype=torch.bfloat16, device="cuda")[:, 3:N + 3]
    L8.Linear8(*w)(*a, out=out)
    ref = tl.lo.linear(tl.lo.values(tl.np8(a.codes), tl.np8(a.scales)), tl.lo.values(tl.np8(w.codes), tl.np8(w.scales), 128))[0]
    assert torch.equal(out.cpu().view(torch.int16), torch.from_numpy(ref).float().bfloat16().view(torch.int16))


@pytest.mark.parametrize("T,N,K", [(2100, 4520, 640), (2100, 4519, 640), (300, 8201, 1040)])
def test_expired_waits_write_nothing(T, N, K):
    a, w = tl.random8(T, K, 1, 8), tl.random8(N, K, 128, 9)
    assert takes_256(T, N, K, torch.cuda.get_device_properties(0).multi_processor_count)
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
    assert B.moe_last_device_error(s) == 0
