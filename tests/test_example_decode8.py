"""The decoder layer of examples/decode_with_cache.py with its projections in 8 bits."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from moe_ffn_layer_gb300 import build as build_mod
    build_mod.build()
    import decode_with_cache
    return decode_with_cache


def step(example, layer, x, lens, new):
    to = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = to([[5, 9, 2], [7, 1, 0]])
    cu = [0, new[0], sum(new)]
    return layer(x, table, to(lens), to(cu), max(new), max(lens))


def test_near_the_bf16_layer(example):
    """A prompt and a step.  Rows and weights in 8 bits are each off by at most 2^-4 of a value, evenly spread within
    a step so by 2^-4 / sqrt(3) = 0.036 in the root mean square, and a product of them by sqrt(2) of that, 0.051.  The
    attention's input and its output projection add such an error each, and so does the cache's rounding of K and V that
    fall on other codes; the FFN's input carries them on, and a token whose last two experts lie near may take the
    other.  The residual stream itself, of the same size, has no error: three such errors, 0.15, bound the sum."""
    from moe_ffn_layer_gb300 import binding as B
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(103, 512, generator=g, device="cuda").bfloat16()
    y = {}
    for kind in (example.DecoderLayer, example.DecoderLayer8):
        layer = example.make_layer(kind=kind)
        first = step(example, layer, x, [70, 33], [70, 33])
        y[kind] = (first, step(example, layer, x[[3, 80]], [71, 34], [1, 1]))
    assert B.moe_last_device_error(torch.cuda.current_stream()) == 0
    for a, b in zip(y[example.DecoderLayer], y[example.DecoderLayer8]):
        assert torch.isfinite(b).all()
        assert (a.float() - b.float()).norm() <= 0.15 * a.float().norm()


def test_serves(example):
    from moe_ffn_layer_gb300 import binding as B
    y, lens, evictions = example.serve(example.make_layer(kind=example.DecoderLayer8), [60, 20], 40, limit=96, budget=64)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and evictions > 0 and B.moe_last_device_error(torch.cuda.current_stream()) == 0
