"""The 8-bit product's bounded waits beside a long launch before it, on the GPU."""
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from moe_ffn_layer_gb300 import linear8 as L8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield B.lib()
    assert B.moe_last_device_error(torch.cuda.current_stream()) == 0


def random8(R, K, high, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    codes = torch.randint(0, 120, (R, K), generator=g, device="cuda", dtype=torch.uint8)
    return L8.rows8(codes, torch.full((-(-R // high), -(-K // 128)), 120, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T,N,K", [(3, 300, 2048), (12, 300, 8192), (40, 520, 1024), (256, 6144, 4096), (600, 4000, 640), (1200, 4100, 640)])
def test_limit_counts_no_earlier_launch(T, N, K):
    """A product whose limit is a quarter of the time that the launch before it runs on for, and far above its own: the
    launch before, one tile of a long K on eight SMs, lets it set itself up on the others from the start."""
    a, w = random8(T, K, 1, 1), random8(N, K, 128, 2)
    lin = L8.Linear8(*w)
    fresh = lin(*a)
    far = 1 << 24
    b, long = random8(20, far, 1, 3), L8.Linear8(*random8(1, far, 128, 4))
    before = long(*b)
    s = torch.cuda.current_stream()
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ends[0].record()
    long(*b, out=before)
    ends[1].record()
    assert B.moe_last_device_error(s) == 0
    ns = int(ends[0].elapsed_time(ends[1]) * 1e6)
    assert ns > 1_000_000   # (a limit of 250 us; the products take 30 at most)
    got = torch.empty_like(fresh)
    try:
        long(*b, out=before)
        B.moe_debug_set_wait_limit_ns(ns // 4)
        lin(*a, out=got)
    finally:
        B.moe_debug_set_wait_limit_ns(2_000_000_000)
    assert B.moe_last_device_error(s) == 0
    assert torch.equal(got.view(torch.int16), fresh.view(torch.int16))
