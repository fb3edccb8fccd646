"""Results and weights of the 8-bit projections that were changed in place between calls, without a GPU: the C entry
points are recorded, not called, and tensors say that they are on device 0.  A call may only be made with the rows
that its tensors have now."""
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import linear8 as L8


class OnDevice0(torch.Tensor):
    """A CPU tensor that says so."""
    is_cuda = True

    def get_device(self):
        return 0


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16).as_subclass(OnDevice0)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).as_subclass(OnDevice0)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def calls(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(B, "_lib", rec)
    monkeypatch.setattr(L8, "_current", lambda device: 0)
    monkeypatch.setattr(L8, "_device", lambda: 0)
    return rec.calls


# each leaves another tensor where a [5, 256] (or its scales) was
CHANGES = {
    "set_": lambda t: t.set_(t[:2].clone()),
    "data": lambda t: setattr(t, "data", torch.zeros(2, t.shape[1], dtype=t.dtype)),
    "resize_": lambda t: t.resize_(2, t.shape[1]),
    "columns": lambda t: t.set_(torch.zeros(t.shape[::-1], dtype=t.dtype).t()),
    "type": lambda t: setattr(t, "data", torch.zeros(t.shape, dtype=torch.int32)),
}


@pytest.mark.parametrize("change", CHANGES.values(), ids=CHANGES)
@pytest.mark.parametrize("name", ["codes", "scales"])
def test_quantize_into_changed_results(calls, name, change):
    x, into = bf16(5, 256), L8.Block8(u8(5, 256), u8(5, 2))
    assert L8.quantize8(x, into=into) is into and L8.quantize8(x, into=into) is into
    change(getattr(into, name))
    with pytest.raises(ValueError, match=name):
        L8.quantize8(x, into=into)
    assert len(calls) == 2


@pytest.mark.parametrize("change", CHANGES.values(), ids=CHANGES)
@pytest.mark.parametrize("name", ["codes", "scales", "h", "y"])
def test_norm_into_changed_results(calls, name, change):
    x, into = bf16(5, 256), L8.Norm8(u8(5, 256), u8(5, 2), bf16(5, 256), bf16(5, 256))
    for _ in range(2):
        assert L8.rms_norm8(x, residual=x, outputs="both", into=into) is into
    change(getattr(into, name))
    with pytest.raises(ValueError, match=name):
        L8.rms_norm8(x, residual=x, outputs="both", into=into)
    assert len(calls) == 2


@pytest.mark.parametrize("change", CHANGES.values(), ids=CHANGES)
@pytest.mark.parametrize("name", ["codes", "scales"])
def test_changed_weights(calls, name, change):
    w = L8.Block8(u8(300, 256), u8(3, 2))
    lin = L8.Linear8(*w)
    lin._codes, lin._scales = w   # (the layout of host memory may have had them copied)
    a, out = L8.Block8(u8(5, 256), u8(5, 2)), bf16(5, 300)
    lin(*a, out=out)
    change(getattr(w, name))
    with pytest.raises(ValueError, match=name):
        lin(*a, out=out)
    assert len(calls) == 1


def test_rows_that_moved_apart(calls):
    """Of the same sizes but other strides: the call is made with those."""
    x, into = bf16(5, 256), L8.Block8(u8(5, 256), u8(5, 2))
    lin, out = L8.Linear8(u8(5, 256), u8(1, 2)), bf16(5, 5)
    for apart in (256, 384):
        into.codes.set_(torch.zeros(5, apart, dtype=torch.uint8)[:, :256])
        into.scales.set_(torch.zeros(5, apart // 64, dtype=torch.uint8)[:, :2])
        lin.codes.set_(torch.zeros(5, apart, dtype=torch.uint8)[:, :256])
        L8.quantize8(x, into=into)
        n = L8.rms_norm8(x, into=L8.Norm8(*into, None, None))
        L8.rms_norm8(x, into=n)
        lin(*into, out=out)
        quantize, norm, again, linear = (args for _, args in calls[-4:])
        assert quantize[6] == norm[13] == again[13] == linear[1] == apart
        assert quantize[8] == norm[15] == again[15] == linear[3] == apart // 64
        assert linear[5] == apart
    into.codes.untyped_storage().resize_(0)   # memory that was given back has no address, which the C calls refuse
    L8.quantize8(x, into=into)
    assert calls[-1][1][5] == 0


def test_no_scales_beside_codes(calls):
    x = bf16(5, 256)
    for into in (L8.Norm8(u8(5, 256), None, None, None), L8.Norm8(None, u8(5, 2), None, None)):
        with pytest.raises(ValueError, match="into"):
            L8.rms_norm8(x, into=into)
        with pytest.raises(ValueError, match="into"):
            L8.rms_norm8(x, outputs="y", into=into._replace(y=bf16(5, 256)))
    assert not calls
