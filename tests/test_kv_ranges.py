"""Attention over the cache at the ends of its ranges."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from oracle import kv_oracle as ko
from test_kv_cache import B_CHECK, bf16_round, i32, make_pool, make_table, status, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return B.lib()


@pytest.mark.parametrize("n,L", [(200, 1500), (640, 900)])
def test_subnormal_v_scales(n, L):
    """A page's V scale below 2^-126: the values are as small, not zero."""
    rng = np.random.default_rng(62)
    table, pages = make_table(rng, [L], 32)
    pool = make_pool(rng, pages, 2, 32, 128)
    pool["vs"] = np.ldexp(rng.uniform(1, 2, pool["vs"].shape), -129).astype(np.float32)
    pool["vs"][table[0, 1]] = 0
    assert 0 < pool["vs"].max() < 2.0 ** -126
    q = bf16_round(rng.standard_normal((n, 8, 128)))
    ref, _, mass, _ = ko.attention(pool, table, [L], np.array([0, n]), q, 128 ** -0.5)
    out = upload(pool).attend(torch.from_numpy(q).bfloat16().cuda(), i32(table), i32([L]), i32([0, n]), n, L)
    # the scale's own 21 bits and the sums' are below bf16's 8; 2^-132 is what subnormal bf16 results round by
    e = np.abs(out.double().cpu().numpy() - ref) - 2.0 ** -8 * np.abs(ref) - 2.0 ** -10 * mass - 2.0 ** -132
    assert e.max() <= 0 and status() == 0


def test_rows_times_tokens_past_32_bits():
    """128 heads on one kv head over 25 million tokens (a few pages, many times over), one page missing:
    the tokens beside it gain what their like gain elsewhere."""
    Hkv, g, D, P, n_pages = 1, 128, 64, 16, 1_570_000
    L = n_pages * P - 3
    rng = np.random.default_rng(63)
    pool = make_pool(rng, 4, Hkv, P, D, scales=(-10, -8))
    cache = upload(pool)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").remainder(3)[None].contiguous()
    table[0, 0] = table[0, 4] = 3
    table[0, 1] = -1
    q = torch.from_numpy(rng.standard_normal((1, g, D))).bfloat16().cuda()
    w = torch.zeros(1, 1, L, device="cuda")
    out = cache.attend(q, table, i32([L]), i32([0, 1]), 1, L, weights=w)
    assert status() == B_CHECK and status() == 0
    assert not w[0, 0, P:2 * P].any()
    assert bool((w[0, 0, :P] > 0).all()) and torch.equal(w[0, 0, :P], w[0, 0, 4 * P:5 * P])
    assert bool(out.isfinite().all())
