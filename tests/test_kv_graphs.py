"""Attention calls in CUDA graphs: what is called, captured or replayed besides
does not reach a graph's workspace.  The calls are of units cut between CTAs, whose
parts and counters lie there."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from test_kv_cache import i32, make_pool, make_table, status, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return B.lib()


class Calls:
    """Calls of n queries over one sequence of L tokens, with weights."""

    def __init__(self, L=9000, Hkv=2, g=4, D=128, P=64, seed=70):
        rng = np.random.default_rng(seed)
        table, pages = make_table(rng, [L], P)
        self.cache = upload(make_pool(rng, pages, Hkv, P, D))
        self.q = torch.from_numpy(rng.standard_normal((300, Hkv * g, D))).bfloat16().cuda()
        self.table, self.L = i32(table), L
        self.lens, self.cu = i32([L]), {n: i32([0, n]) for n in (1, 3, 300)}
        self.w = torch.zeros(1, Hkv, L, device="cuda")

    def __call__(self, n, out, w=None, stream=None):
        return self.cache.attend(self.q[:n], self.table, self.lens, self.cu[n], n, self.L, weights=w, out=out, stream=stream)

    def out(self, n):
        return torch.full_like(self.q[:n], 7.0)

    def graph(self, n, w=None, stream=None, pool=None):
        out, g = self.out(n), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream, pool=pool):
            self(n, out, w)
        return g, out


def new_stream():
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    return side


@pytest.mark.parametrize("n", [1, 3, 300])
def test_replay_after_a_larger_call_on_the_same_stream(n):
    c, side = Calls(), new_stream()
    with torch.cuda.stream(side):
        want = c(n, c.out(n)).clone()
    torch.cuda.synchronize()
    graph, out = c.graph(n, stream=side)
    with torch.cuda.stream(side):
        c(300, c.out(300), c.w)                                                   # needs a larger workspace
        others = [torch.full((m << 20,), 0xAB, dtype=torch.uint8, device="cuda") for m in (1, 2, 5, 6, 20, 30, 60)]
    torch.cuda.synchronize()
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((t == 0xAB).all()) for t in others) and status() == 0


@pytest.mark.parametrize("shared_pool", [False, True])
def test_graphs_of_a_stream_without_a_warm_up_in_any_order(shared_pool):
    c, want = Calls(), {}
    for n in (1, 3, 300):
        want[n] = c(n, c.out(n))
    fresh, side = Calls(), new_stream()
    pool = torch.cuda.graph_pool_handle() if shared_pool else None
    graphs = {n: fresh.graph(n, stream=side, pool=pool) for n in (3, 300, 1)}
    with torch.cuda.stream(side):
        eager = fresh(3, fresh.out(3)).clone()      # before any replay
    torch.cuda.synchronize()
    assert torch.equal(eager, want[3])
    for n in (1, 300, 3, 300, 1):
        graph, out = graphs[n]
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n]), n
    assert status() == 0


def test_graphs_of_one_stream_replayed_on_two():
    c, side = Calls(), new_stream()
    with torch.cuda.stream(side):
        want = {n: c(n, c.out(n)).clone() for n in (1, 3)}
    torch.cuda.synchronize()
    graphs = {n: c.graph(n, stream=side) for n in (1, 3)}
    streams = {n: new_stream() for n in graphs}
    wrong = {n: torch.zeros((), dtype=torch.long, device="cuda") for n in graphs}
    torch.cuda.synchronize()
    for _ in range(50):
        for n, (graph, out) in graphs.items():
            with torch.cuda.stream(streams[n]):
                out.fill_(7)
                graph.replay()
                wrong[n] += (out != want[n]).sum()
    torch.cuda.synchronize()
    assert not any(int(x) for x in wrong.values()) and status() == 0


def test_several_calls_and_streams_of_one_capture():
    """Two calls in a row and one on a forked stream, with weights: one graph, replayed twice."""
    c = Calls()
    w, w2 = torch.zeros_like(c.w), torch.zeros_like(c.w)
    want = {n: c(n, c.out(n)).clone() for n in (1, 3)}
    once = torch.zeros_like(c.w)
    c(1, c.out(1), once)
    main, fork = new_stream(), torch.cuda.Stream()
    outs = [c.out(1), c.out(3), c.out(1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        fork.wait_stream(main)
        c(1, outs[0], w)
        c(3, outs[1])
        c(1, outs[2], w2, stream=fork)
        main.wait_stream(fork)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1]) and torch.equal(outs[1], want[3]) and torch.equal(outs[2], want[1])
    assert torch.equal(w, once + once) and torch.equal(w2, w) and status() == 0


def test_stream_given_by_handle():
    c, side = Calls(), new_stream()
    want, w = c(3, c.out(3)), torch.rand_like(c.w)
    dst, to = i32([[0, 1]]), upload(make_pool(np.random.default_rng(1), 2, 2, 64, 128))
    torch.cuda.synchronize()
    got = c.cache.attend(c.q[:3], c.table, c.lens, c.cu[3], 3, c.L, stream=side.cuda_stream)
    lens, _, kept = c.cache.evict(w, c.table, c.lens, c.L, 100, 4, 16, dst, dst=to, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and int(lens) == 100 and bool((kept >= 0).all()) and status() == 0
