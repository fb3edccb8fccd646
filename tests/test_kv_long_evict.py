"""Eviction from long sequences, on either side of the length up to which the
selection keeps the weights in shared memory.  Everything equals the oracle's
exactly."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import build as build_mod
from test_kv_cache import check_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("lens", [[24577], [49152], [49153], [60001, 300, 1, 0, 50000]])
@pytest.mark.parametrize("budget,sink,recent", [(3001, 16, 200), (20000, 0, 0)])
def test_evict(lens, budget, sink, recent):
    check_evict(np.random.default_rng(sum(lens) + budget), lens, 2, 64, 64, budget, sink, recent)


@pytest.mark.parametrize("L", [30000, 52000])
@pytest.mark.parametrize("kind", ["equal", "few", "odd"])
def test_evict_equal_and_odd_weights(kind, L):
    rng = np.random.default_rng(31)
    w = np.ones((1, 2, L), np.float32)
    if kind == "few":
        w = rng.integers(0, 3, (1, 2, L)).astype(np.float32)
    if kind == "odd":
        w = rng.standard_normal((1, 2, L)).astype(np.float32)
        w[0, :, ::7], w[0, :, 5::11], w[0, :, 3::13] = np.nan, np.inf, -np.inf
    check_evict(rng, [L], 2, 64, 64, 9000, 3, 40, w)
