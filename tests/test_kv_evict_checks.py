"""Device-side checks of the eviction's sequences."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import build as build_mod
from oracle import kv_oracle as ko
from test_kv_cache import B_CHECK, i32, make_pool, status, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def test_evict_skips_a_sequence_longer_than_its_pages():
    """A length within max_len and beyond the table's width keeps nothing, as the other calls skip it."""
    rng = np.random.default_rng(65)
    lens, P, D, Hkv, budget = [100, 40, 64], 32, 64, 2, 30
    table = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    pool, dst = make_pool(rng, 6, Hkv, P, D), make_pool(rng, 3, Hkv, P, D)
    w = rng.random((3, Hkv, 100)).astype(np.float32)
    dst_table = np.array([[2], [0], [1]], np.int32)
    cache, to = upload(pool), upload(dst)
    lens_out, wk, kept = cache.evict(torch.from_numpy(w).cuda(), i32(table), i32(lens), 100, budget, 2, 5,
                                     i32(dst_table), dst=to)
    assert status() == B_CHECK and status() == 0
    want = ko.evict(pool, table, np.array([0, 40, 64]), w, budget, 2, 5, dst, dst_table)
    for x, y in zip((lens_out, wk, kept), want):
        assert np.array_equal(x.cpu().numpy(), y)
    for n, t in (("k", to.k), ("v", to.v), ("ks", to.k_scale), ("vs", to.v_scale)):
        assert np.array_equal(t.cpu().numpy(), dst[n]), n
