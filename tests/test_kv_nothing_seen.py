"""Query rows that are left with nothing to see: every page of theirs missing, or
more queries than tokens, whatever the row itself holds."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from test_kv_cache import B_CHECK, i32, make_pool, make_table, status, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return B.lib()


@pytest.mark.parametrize("n", [1, 2, 40, 129])
@pytest.mark.parametrize("D", [64, 128])
def test_a_sequence_whose_pages_are_all_missing(n, D):
    """Out 0, lse -inf and no weight gained; the sequences beside it as without it."""
    rng = np.random.default_rng(40 + n)
    lens, P, Hkv, g = [300, 290, 310], 32, 2, 4
    table, pages = make_table(rng, lens, P)
    cache = upload(make_pool(rng, pages, Hkv, P, D))
    q = torch.from_numpy(rng.standard_normal((3 * n, Hkv * g, D))).bfloat16().cuda()
    w0 = torch.from_numpy(rng.random((3, Hkv, 310)).astype(np.float32)).cuda()
    args = (i32(lens), i32([0, n, 2 * n, 3 * n]), n, 310)
    want_w, want_lse = w0.clone(), torch.empty(3 * n, Hkv * g, device="cuda")
    want = cache.attend(q, i32(table), *args, weights=want_w, lse=want_lse)
    assert status() == 0
    broken = table.copy()
    broken[1] = [-1, pages] * (table.shape[1] // 2) + [-5] * (table.shape[1] % 2)
    w, lse = w0.clone(), torch.empty(3 * n, Hkv * g, device="cuda")
    out = cache.attend(q, i32(broken), *args, weights=w, lse=lse)
    assert status() == B_CHECK and status() == 0
    assert not out[n:2 * n].any() and bool(lse[n:2 * n].isneginf().all()) and torch.equal(w[1], w0[1])
    for b in (0, 2):
        assert torch.equal(out[b * n:b * n + n], want[b * n:b * n + n]) and torch.equal(w[b], want_w[b])
        assert torch.equal(lse[b * n:b * n + n], want_lse[b * n:b * n + n])


@pytest.mark.parametrize("n", [1, 4, 70, 200])
def test_a_prompt_whose_first_pages_are_missing(n):
    """Its first queries see nothing, the later ones what is left."""
    rng = np.random.default_rng(50 + n)
    P, Hkv, g, D = 16, 2, 2, 64
    table, pages = make_table(rng, [n], P)
    cache = upload(make_pool(rng, pages, Hkv, P, D))
    q = torch.from_numpy(rng.standard_normal((n, Hkv * g, D))).bfloat16().cuda()
    broken = table.copy()
    gone = min(3, table.shape[1])
    broken[0, :gone] = -1
    w0 = torch.from_numpy(rng.random((1, Hkv, n)).astype(np.float32)).cuda()
    w, lse = w0.clone(), torch.empty(n, Hkv * g, device="cuda")
    out = cache.attend(q, i32(broken), i32([n]), i32([0, n]), n, n, weights=w, lse=lse)
    assert status() == B_CHECK
    blind = min(gone * P, n)
    assert not out[:blind].any() and bool(lse[:blind].isneginf().all())
    assert bool(lse[blind:].isfinite().all()) and bool(out.isfinite().all())
    assert torch.equal(w[..., :blind], w0[..., :blind])
    gained = (w - w0).double().sum(-1).cpu()
    assert torch.allclose(gained, torch.full_like(gained, g * (n - blind)), rtol=1e-4, atol=1e-6)


# lens, new, kv heads, heads of each, head size
@pytest.mark.parametrize("lens,new,Hkv,g,D", [([3], [5], 2, 2, 128), ([3, 40], [9, 1], 1, 4, 64),
                                              ([100, 3000], [200, 300], 2, 8, 128), ([70, 900], [100, 640], 2, 4, 64),
                                              ([40, 8000], [90, 33], 1, 4, 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_row_that_sees_nothing_may_hold_anything(lens, new, Hkv, g, D, value):
    """As rows that a program never filled do: they give 0 and -inf like any other that sees nothing."""
    rng = np.random.default_rng(sum(lens))
    table, pages = make_table(rng, lens, 16)
    cache = upload(make_pool(rng, pages, Hkv, 16, D))
    cu = np.concatenate([[0], np.cumsum(new)])
    q = torch.from_numpy(rng.standard_normal((cu[-1], Hkv * g, D))).bfloat16().cuda()

    def run(q):
        w, lse = torch.zeros(len(lens), Hkv, max(lens), device="cuda"), torch.empty(cu[-1], Hkv * g, device="cuda")
        out = cache.attend(q, i32(table), i32(lens), i32(cu), max(new), max(lens), weights=w, lse=lse)
        assert status() == 0
        return out, lse, w

    want = run(q)
    bad = q.clone()
    blind = new[0] - lens[0]                        # the first queries of sequence 0
    bad[:blind, :, D // 2] = value
    bad[blind - 1, 0] = value
    got = run(bad)
    assert not got[0][:blind].any() and bool(got[1][:blind].isneginf().all())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
