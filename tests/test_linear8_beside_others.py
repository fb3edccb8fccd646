"""The 8-bit projections while the MoE layer and the cache's attention run on other streams, on the GPU.  Kernels of all
three hold tensor memory while they wait for the launch before them; a CTA that waits for tensor memory waits for one
that ends by itself, and results are those of one stream."""
import pytest
import torch

import test_linear8 as tl
from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import linear8 as L8
from moe_ffn_layer_gb300 import synth
from moe_ffn_layer_gb300.kv_cache import KVCache8
from moe_ffn_layer_gb300.layer import MoEFFN, bf16_tensor
from test_linear8 import lib  # noqa: F401  (builds the library, and looks at the device's status at the end)

pytestmark = pytest.mark.gpu

# every kernel of the product, one after another, and the norm and quantisation between them
PRODUCTS = [(1, 4096, 2048), (8, 6144, 4096), (12, 304, 2032), (16, 7400, 1040), (20, 4096, 2048), (64, 6144, 4096), (256, 6144, 4096),
            (777, 2500, 2000), (1024, 4032, 2048), (1500, 9000, 1168)]


def projections():
    parts = []
    for i, (T, N, K) in enumerate(PRODUCTS):
        a, w = tl.random8(T, K, 1, i), tl.random8(N, K, 128, 20 + i)
        x = torch.randn(T, K, device="cuda").bfloat16()
        parts.append((L8.Linear8(*w), a, x))

    def run():
        out = []
        for lin, a, x in parts:
            out.append(lin(*a))
            n = L8.rms_norm8(x, None, 1e-6, x)
            out.append(lin(n.codes, n.scales))
            out.append(lin(*L8.quantize8(x)))
        return out
    return run


def experts(T):
    w = synth.Workload("beside", T, 1024, 16, 4, 512, 512, sigma_router=0.1)
    inp = synth.make_inputs(w, T)
    layer, x = MoEFFN.from_inputs(inp, w.k, "cuda:0"), bf16_tensor(inp["x"], "cuda:0")
    lin = L8.Linear8.from_weight(torch.randn(1024, 1024, device="cuda").bfloat16())

    def run():   # (norm, layer, projection: one stream's launches among each other)
        y = layer(L8.rms_norm8(x, outputs="y").y)
        return [y, lin(*L8.quantize8(y))]
    return run


def attention():
    Hkv, Hq, D, page = 2, 8, 128, 64
    cache = KVCache8(40, Hkv, D, page, "cuda")
    to = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    new = [700, 333]
    kv = torch.randn(2, sum(new), Hkv, D, device="cuda").bfloat16()
    q, one = torch.randn(sum(new), Hq, D, device="cuda").bfloat16(), torch.randn(2, Hq, D, device="cuda").bfloat16()
    table, lens, cu, ends = to([list(range(11)), list(range(11, 22))]), to(new), to([0, 700, 1033]), to([0, 1, 2])

    def run():
        cache.append(kv[0], kv[1], table, lens, cu)
        a = cache.attend(q, table, lens, cu, 700, 700)
        return [a, cache.attend(one, table, lens, ends, 1, 700)]
    return run


@pytest.mark.parametrize("other", ["decode", "batch", "prompt", "attention", "all"])
def test_beside(other):
    runs = [projections()]
    if other in ("decode", "all"):
        runs += [experts(1), experts(8)]
    if other in ("batch", "all"):
        runs += [experts(64)]
    if other in ("prompt", "all"):
        runs += [experts(2048)]
    if other in ("attention", "all"):
        runs += [attention()]
    want = [run() for run in runs]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        got = [[] for _ in runs]
        for _ in range(6):
            for s, run, out in zip(streams, runs, got):
                with torch.cuda.stream(s):
                    out.append(run())
        torch.cuda.synchronize()
        for s in streams:
            assert B.moe_last_device_error(s) == 0
        for outs, first in zip(got, want):
            for out in outs:
                assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(out, first))


def test_beside_in_graphs():
    """The same as graphs that are replayed at once."""
    runs = [projections(), experts(8), experts(2048), attention()]
    want = [run() for run in runs]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for run in runs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run())
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert B.moe_last_device_error(torch.cuda.current_stream()) == 0
    for out, first in zip(outs, want):
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(out, first))
