"""Calls of the 8-bit projections that the documentation allows, on the GPU: outputs past 2^32 elements, results in larger
tensors through the C call, the same memory as both operands, streams by handle, copies and fills before a captured call,
threads."""
import threading

import numpy as np
import pytest
import torch

import test_linear8 as tl
from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import linear8 as L8
from test_linear8 import lib  # noqa: F401  (builds the library, and looks at the device's status at the end)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [4104, 4103])
def test_outputs_past_32_bits(N):
    """By tensor copies and by vectors; whole numbers, whose sums are exact."""
    T, K = 1050000, 64
    few = torch.randint(-4, 5, (16, K), device="cuda").bfloat16()
    x = few[torch.arange(T, device="cuda") % 16]
    w = torch.randint(-4, 5, (N, K), device="cuda").bfloat16()
    a, lin = L8.quantize8(x), L8.Linear8.from_weight(w)
    del x
    out = lin(*a)
    want = (few.float() @ w.float().t()).bfloat16()
    assert torch.equal(lin(*L8.quantize8(few)), want)
    for t in range(0, T, 1 << 16):   # all of it, a part at a time
        part = out[t:t + (1 << 16)]
        assert (part.view(-1, 16, N) == want).all()


@pytest.mark.parametrize("N,K", [(300, 272), (128, 128), (1, 400)])
def test_weight_into_larger_tensors(N, K):
    w = tl.rows(N, K, 8, N)
    codes = torch.full((N + 3, K + 32), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-N // 128) + 2, -(-K // 128) + 3), 9, dtype=torch.uint8, device="cuda")
    B.moe_quantize8_weight(w, w.stride(0), N, K, codes, K + 32, scales, scales.stride(0), torch.cuda.current_stream())
    want, s = tl.lo.quantize(tl.np64(w), 128)
    assert np.array_equal(tl.np8(codes[:N, :K]), want) and np.array_equal(tl.np8(scales[:s.shape[0], :s.shape[1]]), s)
    assert (codes[N:] == 9).all() and (codes[:, K:] == 9).all()
    assert (scales[s.shape[0]:] == 9).all() and (scales[:, s.shape[1]:] == 9).all()


@pytest.mark.parametrize("T", [8, 16, 30, 60, 128, 2304])
def test_the_same_memory_twice(T):
    """Rows times themselves: one codes tensor as both operands; x as its own residual."""
    q = tl.random8(T, 528, 1, 7, 1)
    w = L8.Block8(q.codes, torch.full((-(-T // 128), 5), 127, dtype=torch.uint8, device="cuda"))
    tl.assert_linear(L8.Linear8(*w)(*q), q, w)
    x = tl.rows(T, 528, 8, 3)
    n = L8.rms_norm8(x, x[0, :528].contiguous(), 1e-6, x, "both")
    assert torch.equal(n.h.view(torch.int16), (2 * x.float()).bfloat16().view(torch.int16))


def test_rows_at_one_place():
    """Inputs may be one row again and again only where there is one row; results never may."""
    x = torch.ones(1, 256, device="cuda").bfloat16()
    assert torch.equal(L8.quantize8(x.expand(1, 256)).codes, L8.quantize8(x).codes)
    lin = L8.Linear8(*L8.quantize8_weight(x))
    for bad in (lambda: L8.quantize8(x.expand(5, 256)), lambda: L8.rms_norm8(x.expand(5, 256)), lambda: L8.quantize8_weight(x.expand(5, 256)),
                lambda: lin(*L8.quantize8(x.repeat(2, 1)), out=torch.empty(1, 1, device="cuda").bfloat16().expand(2, 1))):
        with pytest.raises(B.MoEError) as e:
            bad()
        assert e.value.code == -1


def test_the_default_stream_by_handle():
    x = tl.rows(5, 256, 0, 1)
    lin = L8.Linear8(*L8.quantize8_weight(tl.rows(40, 256, 0, 3)))
    q, n = L8.quantize8(x, stream=0), L8.rms_norm8(x, stream=0)
    y = lin(*q, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(q.codes, L8.quantize8(x).codes) and torch.equal(n.codes, L8.rms_norm8(x).codes)
    assert torch.equal(y, lin(*q))


@pytest.mark.parametrize("T", [1, 20, 70, 600])
def test_captured_behind_copies_and_fills(T):
    """Nodes that are no kernels stand before the captured calls, which are to wait for them all the same."""
    K, N = 4096, 4032
    src, x = tl.rows(T, K, 0, 1), torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    a = L8.quantize8(src)
    codes, out = torch.empty_like(a.codes), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    lin = L8.Linear8.from_weight(tl.rows(N, K, 0, 2))
    want_q, want = L8.quantize8(src), lin(*a)
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(src)
        q = L8.quantize8(x)
        codes.copy_(a.codes)
        out.zero_()
        lin(codes, a.scales, out=out)
        side.wait_stream(torch.cuda.current_stream())   # a fork, and two calls that join before a third
        with torch.cuda.stream(side):
            n = L8.rms_norm8(x, None, 1e-6, x)
            done.record()
        again = lin(*q)
        done.wait()
        last = lin(n.codes, n.scales)
    for t in (x, codes, out):
        t.zero_()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q.codes, want_q.codes) and torch.equal(out, want) and torch.equal(again, want)
        fresh = L8.rms_norm8(src, None, 1e-6, src)
        assert torch.equal(last, lin(fresh.codes, fresh.scales))
        for t in (x, codes, out):
            t.zero_()


def test_threads():
    """Calls of several threads at once, each on a stream of its own, the sizes' first calls among them."""
    sizes = [(1, 520, 1040), (20, 521, 1040), (40, 522, 1040), (200, 6100, 3216), (300, 8200, 1040), (1100, 4300, 272)]
    work = []
    for i, (T, N, K) in enumerate(sizes):
        a, w = tl.random8(T, K, 1, i), tl.random8(N, K, 128, 9 + i)
        work.append((L8.Linear8(*w), a))
    torch.cuda.synchronize()
    got, wrong = [None] * 6, []

    def call(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()) as _:
                got[i] = [[lin(*a) for lin, a in work[i:] + work[:i]] for _ in range(10)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=call, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    want = [lin(*a) for lin, a in work]
    for i in range(6):
        for outs in got[i]:
            assert all(torch.equal(o.view(torch.int16), w.view(torch.int16)) for o, w in zip(outs, want[i:] + want[:i]))
