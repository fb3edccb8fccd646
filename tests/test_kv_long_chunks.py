"""Attention of many query rows over long sequences: the key axis cut into
parts, and both ways of computing the same rows.  Bounds are
test_kv_cache.py's: joining parts adds a few fp32 roundings (2^-24 each) to sums
whose allowance is 2^-10 of their magnitudes, and scales by powers of two."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from oracle import kv_oracle as ko
from test_kv_cache import bf16_round, check_attention, i32, make_pool, make_table, spoil_tails, status, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return B.lib()


# lens, new, kv heads, heads of each, head size, page
SHAPES = [
    ([5000], [300], 1, 4, 128, 64),                        # few rows' tiles: many parts
    ([1025], [257], 2, 8, 128, 16),
    ([3000, 40, 0, 1999], [200, 40, 3, 1], 2, 8, 128, 64),  # sequences of no, one and several parts' steps
    ([2500], [2500], 1, 1, 64, 32),                        # causal: the first rows see nothing of later parts
    ([4097, 1100], [33, 1024], 1, 16, 64, 128),
    ([1600, 1500], [1200, 1500], 2, 4, 128, 64),
    ([200] * 7, [150, 200, 1, 0, 129, 64, 200], 3, 7, 128, 32),   # enough rows to fill the GPU uncut
    ([130] * 24, [40] * 24, 4, 4, 64, 16),
    ([2, 1300], [600, 600], 2, 4, 128, 64),                # more queries than tokens
    # single tokens, sequences that ask for nothing and chunks together
    ([900, 1, 3000, 0, 64, 2100] + [33] * 30, [1, 1, 300, 1, 0, 16] + [1] * 30, 2, 4, 128, 64),
    ([2000] + [70 + i for i in range(40)], [65] + [1 + i % 3 for i in range(40)], 1, 16, 64, 16),
    ([500, 3000, 20], [17, 16, 1], 4, 4, 128, 32),         # 68 rows beside 64
    ([1100, 5, 1500, 1500], [200, 5, 1, 1400], 2, 2, 64, 64),
]


@pytest.mark.parametrize("lens,new,Hkv,g,D,P", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_attention(lens, new, Hkv, g, D, P, weights):
    rng = np.random.default_rng(sum(lens) + 5 * g + D)
    table, pages = make_table(rng, lens, P)
    pool = make_pool(rng, pages, Hkv, P, D)
    spoil_tails(pool, table, lens)
    q = rng.standard_normal((sum(new), Hkv * g, D))
    w = rng.random((len(lens), Hkv, max(lens) + 3)).astype(np.float32) if weights else None
    check_attention(pool, table, lens, new, q, g, w)


@pytest.mark.parametrize("n,L", [(100, 1500), (300, 900), (700, 2000)])
def test_sizes_of_values(n, L):
    """Page scales 2^20 apart and zero ones in either pool, rows from 1e-30 to 1e4,
    and the whole weight of a row in one part."""
    rng = np.random.default_rng(21)
    table, pages = make_table(rng, [L], 32)
    pool = make_pool(rng, pages, 2, 32, 128, scales=(-14, 6))
    pool["ks"] = np.minimum(pool["ks"], 2.0 ** -4).astype(np.float32)
    for m in ("ks", "vs"):
        pool[m][rng.random(pool[m].shape) < 0.15] = 0.0
    q = rng.standard_normal((n, 8, 128)) * np.exp2(rng.uniform(-100, 6, (n, 8, 1)))
    check_attention(pool, table, [L], [n], q, 4)


@pytest.mark.parametrize("n,L", [(100, 1500), (300, 900), (700, 2000)])
def test_nan_row_stays_its_own(n, L):
    rng = np.random.default_rng(22)
    table, pages = make_table(rng, [L], 64)
    cache = upload(make_pool(rng, pages, 2, 64, 128))
    q = torch.from_numpy(rng.standard_normal((n, 8, 128))).bfloat16().cuda()
    args = (i32(table), i32([L]), i32([0, n]), n, L)
    want = cache.attend(q, *args)
    bad = q.clone()
    bad[n // 2, 3, 5], bad[n - 1, 6, 0] = float("nan"), float("inf")
    got = cache.attend(bad, *args)
    assert status() == 0
    hit = torch.zeros(n, 8, dtype=torch.bool, device="cuda")
    hit[n // 2, 3] = hit[n - 1, 6] = True
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("n,L", [(100, 1500), (300, 900), (700, 2000)])
def test_page_that_is_not_there_is_masked(n, L):
    """Missing pages, one part's every page among them."""
    rng = np.random.default_rng(23)
    P = 32
    table, pages = make_table(rng, [L], P)
    pool = make_pool(rng, pages, 1, P, 64)
    cache = upload(pool)
    q = torch.randn(n, 4, 64, device="cuda").bfloat16()
    broken = table.copy()
    broken[0, 2], broken[0, 5], broken[0, 8:32] = pages, -1, -1
    gone = {2, 5, *range(8, 32)}
    out = cache.attend(q, i32(broken), i32([L]), i32([0, n]), n, L)
    assert status() == -6 and status() == 0
    keep = np.array([t for t in range(L) if t // P not in gone])
    k, v = (ko.rows(pool, m, table[0], L, 0)[keep] for m in "kv")
    s = q.double().cpu().numpy() @ k.T / 8
    got = out.double().cpu().numpy()
    for i in range(n):
        x = s[i][:, keep <= L - n + i]
        p = np.exp(x - x.max(-1, keepdims=True))
        ref = (p / p.sum(-1, keepdims=True)) @ v[keep <= L - n + i]
        np.testing.assert_allclose(got[i], ref, rtol=2 ** -8, atol=2 ** -9 * np.abs(v).max())


def test_graph_replay_and_later_calls_of_other_sizes():
    """The parts' workspace holds nothing that a later call reads."""
    rng = np.random.default_rng(24)
    L = 4000
    table, pages = make_table(rng, [L], 64)
    cache = upload(make_pool(rng, pages, 2, 64, 128))
    q = torch.from_numpy(rng.standard_normal((300, 16, 128))).bfloat16().cuda()
    calls = [(300, L), (1, L), (64, 1500), (300, 200), (300, L)]
    run = lambda n, m: cache.attend(q[:n], i32(table), i32([m]), i32([0, n]), n, m)
    first = [run(*c) for c in calls]
    assert all(torch.equal(a, run(*c)) for a, c in zip(first, calls)) and torch.equal(first[0], first[4])
    tbl, lens, cu = i32(table), i32([L]), i32([0, 300])
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.attend(q, tbl, lens, cu, 300, L, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cache.attend(q, tbl, lens, cu, 300, L, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and status() == 0


def test_strided_rows_and_other_stream():
    rng = np.random.default_rng(25)
    lens, n = [1333, 1290], 140
    table, pages = make_table(rng, lens, 64)
    cache = upload(make_pool(rng, pages, 2, 64, 128))
    qkv = torch.randn(2 * n, 12, 128, device="cuda").bfloat16()
    args = (i32(table), i32(lens), i32([0, n, 2 * n]), n, max(lens))
    want = cache.attend(qkv[:, :8].contiguous(), *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cache.attend(qkv[:, :8], *args)
    side.synchronize()
    assert torch.equal(got, want) and status() == 0


@pytest.mark.parametrize("n,L", [(300, 300), (300, 1100)])
def test_offsets_past_32_bits(n, L):
    Hkv, P, D, pages = 8, 128, 128, 36000
    from moe_ffn_layer_gb300.kv_cache import KVCache8
    cache = KVCache8(pages, Hkv, D, P)
    assert cache.k.numel() > 2 ** 32
    rng = np.random.default_rng(26)
    small = make_pool(rng, 9, Hkv, P, D)
    ids = np.array([35999, 20000, 35000, 34001, 33, 30000, 29000, 35998, 28000])[:-(-L // P)]
    at = torch.from_numpy(ids).cuda()
    for m, t in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scale), ("vs", cache.v_scale)):
        t[at] = torch.from_numpy(small[m][:len(ids)]).cuda()
    q = bf16_round(rng.standard_normal((n, Hkv, D)))
    ref, _, mass, size = ko.attention(small, [list(range(len(ids)))], [L], np.array([0, n]), q, D ** -0.5)
    out = cache.attend(torch.from_numpy(q).bfloat16().cuda(), i32(ids[None]), i32([L]), i32([0, n]), n, L)
    ds = (D / 16) * 2.0 ** -22 * size + 2.0 ** -21 * size
    e = np.abs(out.double().cpu().numpy() - ref) - 2.0 ** -8 * np.abs(ref) - (2.0 ** -10 + 2 * ds.max()) * mass
    assert e.max() <= 0 and status() == 0


@pytest.mark.parametrize("bad", [0, 2, 34])
def test_sequences_of_a_mixed_batch_that_fail_their_checks_are_skipped(bad):
    rng = np.random.default_rng(27)
    lens, new = [1500, 40, 1200] + [50] * 32, [200, 1, 130] + [1] * 32
    table, pages = make_table(rng, lens, 16)
    cache = upload(make_pool(rng, pages, 2, 16, 128))
    cu = np.concatenate([[0], np.cumsum(new)])
    q = torch.from_numpy(rng.standard_normal((cu[-1], 8, 128))).bfloat16().cuda()
    run = lambda ls, **kw: cache.attend(q, i32(table), i32(ls), i32(cu), 200, 1500, **kw)
    want = run(lens)
    assert status() == 0
    out = torch.full_like(want, 3.0)
    run([-1 if b == bad else L for b, L in enumerate(lens)], out=out)
    assert status() == -6 and status() == 0
    rows = torch.arange(cu[-1], device="cuda")
    gone = (rows >= int(cu[bad])) & (rows < int(cu[bad + 1]))
    assert bool((out[gone] == 3).all())
    # (the cut of the key axis goes by the units there are, so the sums' order may differ)
    torch.testing.assert_close(out[~gone].float(), want[~gone].float(), rtol=2.0 ** -7, atol=2.0 ** -9)
