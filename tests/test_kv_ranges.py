"""The cache's calls at the ends of their ranges: scales, sizes, numbers of sequences."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from oracle import kv_oracle as ko
from test_kv_cache import (B_CHECK, bf16_round, check_append, check_attention, check_evict, i32, make_pool, make_table, status,
                           upload)

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


@pytest.mark.parametrize("B_,kind", [(33, "ones"), (65, "mixed"), (129, "mixed"), (300, "ones"), (300, "mixed"),
                                     (260, "chunks"), (513, "last")])
@pytest.mark.parametrize("weights", [False, True])
def test_many_sequences(B_, kind, weights):
    """More than one round of either kernel's search for a sequence (32 and 128 of them)."""
    rng = np.random.default_rng(B_)
    lens = rng.integers(1, 60, B_).tolist()
    new = [1] * B_
    if kind == "chunks":
        lens = rng.integers(40, 90, B_).tolist()
        new = [int(rng.integers(20, L + 1)) for L in lens]
    elif kind != "ones":
        at = [B_ - 1] if kind == "last" else [0, 31, 32, B_ // 2, B_ - 2, *([127, 128] if B_ > 128 else [])]
        for b in at:
            lens[b] = int(rng.integers(300, 700))
            new[b] = int(rng.integers(70, 300))
        for b in (5, 30, B_ - 3):
            new[b] = 0
    table, pages = make_table(rng, lens, 16)
    pool = make_pool(rng, pages, 1, 16, 64)
    q = rng.standard_normal((sum(new), 4, 64))
    w = rng.random((B_, 1, max(lens))).astype(np.float32) if weights else None
    check_attention(pool, table, lens, new, q, 4, w)


@pytest.mark.parametrize("B_", [32, 33, 200, 1025, 1100])
@pytest.mark.parametrize("P,D", [(16, 64), (32, 128)])
def test_append_to_many_sequences(B_, P, D):
    """One, two and three rounds of the search for a page's sequence."""
    rng = np.random.default_rng(B_ + P)
    lens = rng.integers(1, 50, B_)
    new = np.minimum(lens, np.where(rng.random(B_) < 0.2, 0, rng.integers(1, 40, B_)))
    check_append(rng, lens.tolist(), new.tolist(), 1, P, D, 2.0)


@pytest.mark.parametrize("lens,new,Hkv,g,D", [([700], [1], 2, 4, 128), ([700, 30], [3, 2], 2, 8, 64),
                                              ([1300, 200], [200, 3], 2, 8, 128), ([900], [900], 2, 4, 64)])
def test_negative_scale(lens, new, Hkv, g, D):
    """-c times q . K is c times (-q) . K, to the bit."""
    rng = np.random.default_rng(61)
    table, pages = make_table(rng, lens, 32)
    cache = upload(make_pool(rng, pages, Hkv, 32, D))
    cu = [0, *np.cumsum(new).tolist()]
    q = torch.from_numpy(rng.standard_normal((cu[-1], Hkv * g, D))).bfloat16().cuda()

    def run(q, scale):
        w, lse = torch.zeros(len(lens), Hkv, max(lens), device="cuda"), torch.empty(cu[-1], Hkv * g, device="cuda")
        out = cache.attend(q, i32(table), i32(lens), i32(cu), max(new), max(lens), scale=scale, weights=w, lse=lse)
        assert status() == 0
        return out, lse, w

    assert all(torch.equal(a, b) for a, b in zip(run(q, -0.11), run(-q, 0.11)))
    out, lse, w = run(q, 0.0)   # every visible token alike
    assert bool((lse[-1] - np.log(lens[-1])).abs().max() < 1e-5) and bool(w.isfinite().all())


@pytest.mark.parametrize("L", [30000, 50001])
@pytest.mark.parametrize("Hkv,P,D", [(1, 16, 128), (3, 128, 128), (2, 32, 64)])
def test_long_evictions_of_other_layouts(L, Hkv, P, D):
    check_evict(np.random.default_rng(L + P), [L, 700], Hkv, P, D, 5001, 16, 100)
