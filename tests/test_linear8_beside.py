"""What lies beside a product's output rows stays as it was, on the GPU: every width modulo 16, rows a multiple of 8
elements apart that begin at 16-byte boundaries."""
import pytest
import torch

import test_linear8 as tl
from moe_ffn_layer_gb300 import linear8 as L8
from test_linear8 import lib  # noqa: F401  (builds the library, and looks at the device's status at the end)

pytestmark = pytest.mark.gpu


# by tiles of 512 and 256 tokens, and of 128 weight rows with few tokens
@pytest.mark.parametrize("T,N,K", [(1100, 4288, 272), (300, 8192, 272), (200, 600, 272), (40, 600, 272), (20, 600, 272), (12, 600, 4112),
                                   (3, 600, 272)])
@pytest.mark.parametrize("more", range(16))
def test_columns_behind(T, N, K, more):
    N += more
    a, w = tl.random8(T, K, 1, T), tl.random8(N, K, 128, N)
    apart = -(-N // 8) * 8 + 8
    out = torch.full((T + 1, apart), 7.0, device="cuda").bfloat16()
    L8.Linear8(*w)(*a, out=out[:T, :N])
    assert (out[T:] == 7).all() and (out[:, N:] == 7).all()
    some = torch.cat([torch.arange(0, T, 7, device="cuda"), torch.tensor([T - 1], device="cuda")])
    tl.assert_linear(out[some][:, :N], L8.Block8(a.codes[some], a.scales[some]), w)
    # and the vector behind the last row's end, where memory that is the caller's may end
    flat = torch.full((T * apart + 16,), 7.0, device="cuda").bfloat16()
    L8.Linear8(*w)(*a, out=flat.as_strided((T, N), (apart, 1)))
    assert (flat[(T - 1) * apart + N:] == 7).all()
