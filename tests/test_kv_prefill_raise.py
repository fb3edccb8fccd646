"""Attention of many query rows where the running maximum rises inside a step:
scores that jump at the second 32 tokens of a step of 64, also right after a
rise at its first 32, so that weights and outputs of the same step are scaled
down a second time.  Bounds are test_kv_cache.py's."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from test_kv_cache import check_attention, make_pool, make_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return B.lib()


# what the score gains, in powers of two, at the first and at the second half of each step in turn
JUMPS = {
    "second half": [(0, 11)],
    "both halves": [(10.5, 11)],
    "in turn": [(0, 12), (0, 0), (13, 10), (11, 0), (0.5, 30)],
    "down and up": [(-9, 12), (-20, 35), (6, 10)],
}


@pytest.mark.parametrize("kind", JUMPS)
@pytest.mark.parametrize("L,n,Hkv,g,D", [(700, 700, 1, 2, 128), (650, 300, 2, 3, 64), (1500, 100, 1, 8, 128),
                                         (1400, 640, 1, 2, 64)])
def test_scores_that_jump_inside_a_step(kind, L, n, Hkv, g, D):
    rng = np.random.default_rng(L + g)
    P, scale = 16, 1.0 / 64
    table, pages = make_table(rng, [L], P)
    pool = make_pool(rng, pages, Hkv, P, D)
    # a page's keys are its level in every channel, 1/8 of it up or down at random; queries are near one
    pool["k"][:] = rng.integers(0x37, 0x3A, pool["k"].shape, dtype=np.uint8)
    level = 0.0
    for i in range(-(-L // P)):
        if i % 2 == 0:
            level += JUMPS[kind][i // 4 % len(JUMPS[kind])][i // 2 % 2]
        pool["ks"][table[0, i]] = abs(level) * np.log(2) / (scale * D)
        if level < 0:
            pool["k"][table[0, i]] |= 0x80
    q = 1 + 0.05 * rng.standard_normal((n, Hkv * g, D))
    w = rng.random((1, Hkv, L)).astype(np.float32) if kind == "in turn" else None
    check_attention(pool, table, [L], [n], q, g, w, scale=scale)
