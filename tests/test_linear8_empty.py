"""Matrices of no rows in 8 bits, on the GPU: no tokens, no weight rows, neither; the checks of the other arguments stay."""
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import linear8 as L8
from test_linear8 import lib  # noqa: F401  (builds the library, and looks at the device's status at the end)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N", [(0, 40), (0, 0), (1, 0), (5, 0), (700, 0)])
def test_no_rows(T, N):
    a = L8.quantize8(torch.ones(T, 272, device="cuda").bfloat16())
    w = L8.quantize8_weight(torch.ones(N, 272, device="cuda").bfloat16())
    assert a.codes.shape == (T, 272) and a.scales.shape == (T, 3) and w.codes.shape == (N, 272) and w.scales.shape == (-(-N // 128), 3)
    lin = L8.Linear8(*w)
    out = torch.empty(T, N, device="cuda").bfloat16()
    assert lin(*a).shape == (T, N) and lin(*a, out=out) is out
    assert lin(*a, stream=torch.cuda.Stream()).shape == (T, N)
    assert B.moe_last_launch_count() == 0
    assert L8.Linear8.from_weight(torch.ones(N, 272, device="cuda").bfloat16())(*a).shape == (T, N)
    for bad in (lambda: lin(a.codes[:, :256], a.scales), lambda: lin(a.codes, a.scales[:, :2]), lambda: lin(*a, out=out.float()),
                lambda: lin(*a, out=torch.empty(T + 1, N, device="cuda").bfloat16())):
        with pytest.raises(ValueError):
            bad()
