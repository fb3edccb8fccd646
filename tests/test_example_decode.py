"""The decoder layer of examples/decode_with_cache.py: against a float64 layer
over the same quantised cache, and through evictions."""
import os
import sys

import numpy as np
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


def test_prompt_and_step_against_float64(example):
    """The projections round to bf16 (2^-9 each), the attention and the FFN are
    held to 2^-8 and 1e-2 by their own tests; a K or V that rounds to the
    neighbouring code moves its term by 2^-4: 2e-2 of the output bounds the sum."""
    from moe_ffn_layer_gb300 import binding as B
    from moe_ffn_layer_gb300 import synth
    from oracle import kv_oracle as ko
    from oracle import moe_oracle as om
    layer = example.make_layer()
    H, Hq, Hkv, D, P = 512, 8, 2, 64, 32
    lens, table = [70, 33], np.array([[5, 9, 2], [7, 1, 0]], np.int32)
    x = torch.randn(sum(lens), H, device="cuda").bfloat16()
    to = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    cu = [0, 70, 103]
    y1 = layer(x, to(table), to(lens), to(cu), 70, 70)
    x2 = y1[[69, 102]].clone()
    y2 = layer(x2, to(table), to([71, 34]), to([0, 1, 2]), 1, 71)
    assert B.moe_last_device_error(torch.cuda.current_stream()) == 0

    pool = dict(k=np.zeros((64, Hkv, P, D), np.uint8), v=np.zeros((64, Hkv, P, D), np.uint8),
                ks=np.zeros((64, Hkv), np.float32), vs=np.zeros((64, Hkv), np.float32))
    inp = synth.make_inputs(synth.Workload("example", 8, H, 8, 2, 256, 256, sigma_router=0.1), 0)
    bf = lambda a: torch.from_numpy(a).bfloat16().double().numpy()  # noqa: E731
    w_qkv, w_o = (t.double().cpu().numpy() for t in (layer.w_qkv, layer.w_o))

    def norm(x):
        return bf(x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6))

    def reference(x, lens, cu):
        qkv = bf(norm(x) @ w_qkv.T).reshape(-1, Hq + 2 * Hkv, D)
        ko.append(pool, table, lens, cu, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:])
        att = bf(ko.attention(pool, table, lens, cu, qkv[:, :Hq], D ** -0.5)[0])
        x = bf(x + bf(att.reshape(len(x), -1) @ w_o.T))
        bits = torch.from_numpy(norm(x)).bfloat16().view(torch.int16).numpy().view(np.uint16)
        return x + om.forward(dict(inp, x=bits), 2)["out"]

    for got, ref in ((y1, reference(x.double().cpu().numpy(), lens, cu)),
                     (y2, reference(x2.double().cpu().numpy(), [71, 34], [0, 1, 2]))):
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - ref) <= 2e-2 * np.linalg.norm(ref)


def test_serving_through_evictions(example):
    from moe_ffn_layer_gb300 import binding as B
    runs = []
    for _ in range(2):
        y, lens, evictions = example.serve(example.make_layer(), [60, 21, 96], 90, limit=100, budget=48, recent=8)
        assert B.moe_last_device_error(torch.cuda.current_stream()) == 0
        assert evictions == 2 and all(48 < L <= 100 for L in lens) and bool(y.isfinite().all())
        runs.append((y, lens))
    assert torch.equal(runs[0][0], runs[1][0]) and runs[0][1] == runs[1][1]
