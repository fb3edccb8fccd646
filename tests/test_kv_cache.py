"""The 8-bit paged KV cache on the GPU against its float64 oracle.

Tolerances, from the arithmetic the header states.  A score is one fp32 sum of
D exact products, added in D / 16 steps whose rounding (or truncation) is at
most 2^-22 of the sum of magnitudes `size`: |ds| <= (D / 16) 2^-22 size, plus a
few fp32 roundings of s itself.  lse moves by at most max |ds| plus its own
roundings; a softmax weight by twice that, relatively.  The weights enter the
second product with f16's 11 bits: each by 2^-11 of itself at most, so out moves
by 2^-11 of `mass` = sum p |V| plus twice ds of it, and then rounds to bf16 (2^-8
of itself covers the nearest rounding and its neighbour)."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import binding as B
from moe_ffn_layer_gb300 import build as build_mod
from moe_ffn_layer_gb300.kv_cache import KVCache8
from oracle import kv_oracle as ko

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return B.lib()


def status():
    return B.moe_last_device_error(torch.cuda.current_stream())


def bf16_round(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().double().numpy()


def make_pool(rng, pages, Hkv, P, D, scales=(-10, -4)):
    """Random valid codes and scales, as numpy (the oracle's form)."""
    def codes():
        c = rng.integers(0, 127, (pages, Hkv, P, D), dtype=np.uint8)
        return c | (rng.integers(0, 2, c.shape, dtype=np.uint8) << 7)

    def scale():
        return np.exp2(rng.uniform(*scales, (pages, Hkv))).astype(np.float32)

    return dict(k=codes(), v=codes(), ks=scale(), vs=scale())


def upload(pool):
    return KVCache8.from_tensors(*(torch.from_numpy(pool[n].copy()).cuda() for n in ("k", "v", "ks", "vs")))


def make_table(rng, lens, P, spare=1):
    """A shuffled page for every page of tokens; entries beyond a length hold an id that is not there."""
    need = [-(-L // P) for L in lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max([1, *need])), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(need) + spare


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def spoil_tails(pool, table, lens):
    """Slots beyond a sequence's end hold NaN codes."""
    P = pool["k"].shape[2]
    for b, L in enumerate(lens):
        if L % P:
            for n in "kv":
                pool[n][table[b, L // P], :, L % P:] = 0x7F


def check_attention(pool, table, lens, new, q, g, weights=None, scale=None, cache=None, **kw):
    T, Hq, D = q.shape
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    scale = D ** -0.5 if scale is None else scale
    q64 = bf16_round(q)
    w64 = None if weights is None else weights.astype(np.float64)
    out64, lse64, mass, size = ko.attention(pool, table, lens, cu, q64, scale, w64)
    cache = upload(pool) if cache is None else cache
    w = None if weights is None else torch.from_numpy(weights).cuda()
    lse = torch.full((T, Hq), 7.0, device="cuda")
    qt = torch.from_numpy(q64).to(torch.bfloat16).cuda()
    args = (i32(table), i32(lens), i32(cu), max([0, *new]), max([0, *lens]))
    out = cache.attend(qt, *args, scale=scale, lse=lse, weights=w, **kw)
    assert status() == 0
    ds = (D / 16) * 2.0 ** -22 * size + 2.0 ** -21 * size
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(lse64)
    assert np.array_equal(np.isneginf(got_lse), empty) and not got[empty].any()
    e = np.abs(got - out64) - 2.0 ** -8 * np.abs(out64) - (2.0 ** -10 + 2 * ds.max(initial=0)) * mass
    assert e.max(initial=0) <= 1e-30, e.max()
    e = np.abs(got_lse - lse64)[~empty] - ds[~empty] - 2.0 ** -21 * (1 + np.abs(lse64[~empty]))
    assert e.max(initial=0) <= 0, e.max()
    if weights is not None:
        gain = w64 - weights
        e = np.abs(w.double().cpu().numpy() - w64) - (2 * ds.max(initial=0) + 2.0 ** -18) * gain - 2.0 ** -23 * np.abs(w64)
        assert e.max() <= 0, e.max()
        # the same bits again
        again = torch.from_numpy(weights).cuda()
        assert torch.equal(cache.attend(qt, *args, scale=scale, weights=again, **kw), out) and torch.equal(again, w)
    assert torch.equal(cache.attend(qt, *args, scale=scale, **kw), out)
    return out


# lens, new, kv heads, heads of each, head size, page
SHAPES = [
    ([1], [1], 1, 1, 128, 64),
    ([64], [1], 2, 8, 128, 64),
    ([65, 63, 128, 1], [1, 1, 1, 1], 2, 4, 128, 64),
    ([31, 32, 33, 17, 16, 15], [1] * 6, 3, 3, 64, 16),
    ([700, 0, 301], [1, 0, 1], 1, 16, 128, 32),          # a sequence that is not in the call
    ([0, 40], [1, 1], 2, 2, 64, 128),                    # an empty one that asks
    ([3, 130], [5, 130], 2, 3, 128, 64),                 # more queries than tokens
    ([5000], [1], 2, 8, 128, 64),                        # cut along its length
    ([4097, 2, 1025], [1, 1, 1], 1, 7, 64, 32),
    ([900, 300], [4, 3], 2, 8, 128, 64),                 # drafted tokens
    ([513, 77, 260], [140, 77, 1], 2, 4, 128, 64),       # prompts beside a decode step
    ([400], [400], 1, 1, 64, 64),
    ([259, 1300], [257, 150], 1, 5, 128, 16),
    ([700], [33], 2, 16, 64, 128),
    ([2100, 150], [1, 129], 4, 2, 64, 64),
]


@pytest.mark.parametrize("lens,new,Hkv,g,D,P", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_attention(lens, new, Hkv, g, D, P, weights):
    rng = np.random.default_rng(sum(lens) + 3 * g + D)
    table, pages = make_table(rng, lens, P)
    pool = make_pool(rng, pages, Hkv, P, D)
    spoil_tails(pool, table, lens)
    q = rng.standard_normal((sum(new), Hkv * g, D))
    w = rng.random((len(lens), Hkv, max(lens) + 3)).astype(np.float32) if weights else None
    check_attention(pool, table, lens, new, q, g, w)


@pytest.mark.parametrize("n", [1, 130])
def test_attention_sizes_of_values(n):
    """Page scales 2^20 apart in either pool, zero ones among them, and query
    rows from 1e-30 to 1e4 with elements far below their row's largest."""
    rng = np.random.default_rng(11)
    lens, new = [450], [n]
    table, pages = make_table(rng, lens, 32)
    pool = make_pool(rng, pages, 2, 32, 128, scales=(-14, 6))
    pool["ks"] = np.minimum(pool["ks"], 2.0 ** -4).astype(np.float32)
    pool["vs"][table[0, 2]] = 0
    pool["ks"][table[0, 3]] = 0
    q = rng.standard_normal((n, 8, 128)) * np.exp2(rng.integers(-12, 1, (n, 8, 128)))
    q[:, 0] *= 1e-30
    q[:, 1] *= 20
    q[:, 2] = 0
    check_attention(pool, table, lens, new, q, 4, scale=0.05)


def test_attention_long_tail_of_small_weights():
    """One token far above 3000 others of e^-13 each: their sum still counts."""
    L, D = 3001, 128
    rng = np.random.default_rng(5)
    table, pages = make_table(rng, [L], 64)
    pool = make_pool(rng, pages, 1, 64, D)
    pool["ks"][:] = pool["vs"][:] = 1
    pool["k"][:] = 0
    pool["k"][table[0, 7], 0, 3] = 0x38            # 1.0
    q = np.full((1, 1, D), 13.0 / (D * D ** -0.5))
    pool["v"][:] = 0x38
    pool["v"][table[0, 7], 0, 3] = 0
    out = check_attention(pool, table, [L], [1], q, 1)
    assert float(out.float().mean()) == pytest.approx(3000 * np.exp(-13) / (1 + 3000 * np.exp(-13)), rel=1e-2)


@pytest.mark.parametrize("n", [1, 150])
def test_attention_nan_row_stays_its_own(n):
    rng = np.random.default_rng(6)
    table, pages = make_table(rng, [500], 64)
    pool = make_pool(rng, pages, 2, 64, 128)
    q = rng.standard_normal((n, 8, 128))
    cache = upload(pool)
    args = (i32(table), i32([500]), i32([0, n]), n, 500)
    qt = torch.from_numpy(q).bfloat16().cuda()
    clean = cache.attend(qt, *args)
    bad = qt.clone()
    bad[0, 3, 17] = float("nan")
    bad[n - 1, 5, 0] = float("inf")
    lse = torch.empty(n, 8, device="cuda")
    out = cache.attend(bad, *args, lse=lse)
    rows = torch.zeros(n, 8, dtype=torch.bool, device="cuda")
    rows[0, 3] = rows[n - 1, 5] = True
    assert out[rows].isnan().all() and lse[rows].isnan().all()
    assert torch.equal(out[~rows], clean[~rows]) and status() == 0


@pytest.mark.parametrize("n", [1, 140])
def test_attention_strided_rows_other_stream_and_given_out(n):
    rng = np.random.default_rng(7)
    lens = [333, 290]
    table, pages = make_table(rng, lens, 64)
    pool = make_pool(rng, pages, 2, 64, 128)
    cache = upload(pool)
    qkv = torch.randn(2 * n, 12, 128, device="cuda").bfloat16()   # heads of q, k and v of one projection
    args = (i32(table), i32(lens), i32([0, n, 2 * n]), n, max(lens))
    want = cache.attend(qkv[:, :8].contiguous(), *args)
    out = torch.full((2 * n + 3, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.attend(qkv[:, :8], *args, out=out[:2 * n], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out[:2 * n], want) and bool((out[2 * n:] == 5).all()) and status() == 0


@pytest.mark.parametrize("n", [1, 129])
def test_attention_page_that_is_not_there_is_masked(n):
    rng = np.random.default_rng(8)
    L, P = 300, 32
    table, pages = make_table(rng, [L], P)
    pool = make_pool(rng, pages, 1, P, 64)
    q = torch.randn(n, 4, 64, device="cuda").bfloat16()
    cache = upload(pool)
    broken = table.copy()
    broken[0, 2], broken[0, 5] = pages, -1
    w = torch.zeros(1, 1, L, device="cuda")
    out = cache.attend(q, i32(broken), i32([L]), i32([0, n]), n, L, weights=w)
    assert status() == B_CHECK and status() == 0
    keep = np.array([t for t in range(L) if t // P not in (2, 5)])
    k, v = (ko.rows(pool, m, table[0], L, 0)[keep] for m in "kv")
    s = q.double().cpu().numpy() @ k.T / 8
    for i in range(n):
        x = s[i][:, keep <= L - n + i]
        p = np.exp(x - x.max(-1, keepdims=True))
        ref = (p / p.sum(-1, keepdims=True)) @ v[keep <= L - n + i]
        np.testing.assert_allclose(out[i].double().cpu().numpy(), ref, rtol=2 ** -8, atol=2 ** -9 * np.abs(v).max())
    gone = torch.tensor([t // P in (2, 5) for t in range(L)], device="cuda")
    assert bool((w[0, 0, gone] == 0).all()) and bool((w[0, 0, ~gone][:64] > 0).all())


B_CHECK = -6


def test_sequences_that_fail_their_checks_are_skipped():
    rng = np.random.default_rng(9)
    lens = [40, 50, 60]
    table, pages = make_table(rng, lens, 16)
    cache = upload(make_pool(rng, pages, 1, 16, 64))
    q = torch.randn(3, 2, 64, device="cuda").bfloat16()
    want = cache.attend(q, i32(table), i32(lens), i32([0, 1, 2, 3]), 1, 60)
    for lens_bad, cu in (([40, 61, 60], [0, 1, 2, 3]), ([40, -1, 60], [0, 1, 2, 3])):
        out = torch.full_like(want, 3.0)
        cache.attend(q, i32(table), i32(lens_bad), i32(cu), 1, 60, out=out)
        assert status() == B_CHECK
        assert torch.equal(out[[0, 2]], want[[0, 2]]) and bool((out[1] == 3).all())
    out = torch.full_like(want, 3.0)
    cache.attend(q, i32(table), i32(lens), i32([0, 2, 1, 4]), 1, 60, out=out)   # too many, negative, beyond the rows
    assert status() == B_CHECK and bool((out == 3).all())
    before = cache.k.clone()
    cache.append(torch.ones(3, 1, 64, device="cuda").bfloat16(), torch.ones(3, 1, 64, device="cuda").bfloat16(),
                 i32(table), i32([2, 999, 60]), i32([0, 3, 3, 3]))               # more new tokens than the length
    assert status() == B_CHECK and torch.equal(cache.k, before)


def test_offsets_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes into the pools."""
    Hkv, P, D, pages = 8, 128, 128, 36000
    cache = KVCache8(pages, Hkv, D, P)
    assert cache.k.numel() > 2 ** 32
    rng = np.random.default_rng(10)
    L = 300
    ids = np.array([[35999, 20000, 35000]], np.int32)
    k, v = (rng.standard_normal((L, Hkv, D)) for _ in "kv")
    small = dict(k=np.zeros((3, Hkv, P, D), np.uint8), v=np.zeros((3, Hkv, P, D), np.uint8),
                 ks=np.zeros((3, Hkv), np.float32), vs=np.zeros((3, Hkv), np.float32))
    ko.append(small, [[0, 1, 2]], [L], [0, L], bf16_round(k), bf16_round(v))
    cache.append(torch.from_numpy(k).bfloat16().cuda(), torch.from_numpy(v).bfloat16().cuda(), i32(ids), i32([L]),
                 i32([0, L]))
    for n, t in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scale), ("vs", cache.v_scale)):
        assert np.array_equal(t[torch.from_numpy(ids[0].astype(np.int64)).cuda()].cpu().numpy(), small[n])
    q = rng.standard_normal((140, Hkv, D))
    cu = np.array([0, 140])
    ref, _, mass, _ = ko.attention(small, [[0, 1, 2]], [L], cu, bf16_round(q), D ** -0.5)
    for n in (1, 140):
        out = cache.attend(torch.from_numpy(q[-n:]).bfloat16().cuda(), i32(ids), i32([L]), i32([0, n]), n, L)
        e = np.abs(out.double().cpu().numpy() - ref[-n:]) - 2 ** -8 * np.abs(ref[-n:]) - 2 ** -9 * mass[-n:]
        assert e.max() <= 0
    w = torch.rand(1, Hkv, L, device="cuda")
    _, _, kept = cache.evict(w, i32(ids), i32([L]), L, 100, 0, 0, i32([[34000]]))
    at = kept[0, 5].long().cpu().numpy()
    want = ko.rows(small, "v", [0, 1, 2], L, 5)[at]
    got = ko.VALUE[cache.v[34000, 5, :100].cpu().numpy()] * float(cache.v_scale[34000, 5])
    assert np.abs(got - want).max() <= 2.0 ** -10 * float(cache.v_scale[34000, 5]) and status() == 0


# ---------------------------------------------------------------- append

def check_append(rng, lens, new, Hkv, P, D, spread=0.0, scales=None, stride=None):
    table, pages = make_table(rng, lens, P)
    pool = make_pool(rng, pages, Hkv, P, D)
    for n in ("ks", "vs"):
        pool[n] = np.exp2(np.round(np.log2(pool[n]))).astype(np.float32) if scales is None else np.full_like(pool[n], scales)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = sum(new)
    kv = rng.standard_normal((2, T, Hkv, D)) * np.exp2(rng.uniform(-spread, spread, (2, T, Hkv, 1)))
    k, v = bf16_round(kv[0]), bf16_round(kv[1])
    cache = upload(pool)
    both = torch.from_numpy(np.stack([k, v], 1)).bfloat16().cuda()          # [T, 2, Hkv, D]
    kt, vt = (both[:, 0], both[:, 1]) if stride else (both[:, 0].contiguous(), both[:, 1].contiguous())
    cache.append(kt, vt, i32(table), i32(lens), i32(cu))
    assert status() == 0
    ko.append(pool, table, lens, cu, k, v)
    for n, t in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scale), ("vs", cache.v_scale)):
        assert np.array_equal(t.cpu().numpy(), pool[n]), n


@pytest.mark.parametrize("lens,new", [([1], [1]), ([64, 65, 128, 200], [1, 1, 1, 1]), ([64, 5, 300], [64, 0, 150]),
                                      ([500, 1, 16], [499, 1, 3]), ([129] * 7, [1, 2, 3, 0, 65, 128, 129])])
@pytest.mark.parametrize("Hkv,P,D", [(2, 64, 128), (1, 16, 64), (3, 128, 128), (2, 32, 64)])
@pytest.mark.parametrize("spread", [0.0, 9.0])
def test_append(lens, new, Hkv, P, D, spread):
    check_append(np.random.default_rng(sum(lens) + P), lens, new, Hkv, P, D, spread, stride=spread > 0)


@pytest.mark.parametrize("scales", [0.013, 0.0, 2.0 ** -126, 3.0e30])
def test_append_onto_foreign_scales(scales):
    check_append(np.random.default_rng(1), [70, 33], [3, 20], 2, 64, 128, 3.0, scales=np.float32(scales))


def test_append_step_by_step_equals_the_oracle_step_by_step():
    """Tokens of growing size, one at a time: the page's scale grows with them."""
    rng = np.random.default_rng(2)
    P, D, table = 16, 64, np.array([[2, 0, 1]], np.int32)
    pool = dict(k=np.zeros((3, 1, P, D), np.uint8), v=np.zeros((3, 1, P, D), np.uint8),
                ks=np.zeros((3, 1), np.float32), vs=np.zeros((3, 1), np.float32))
    cache = upload(pool)
    for L in range(1, 41):
        kv = bf16_round(rng.standard_normal((2, 1, 1, D)) * 2.0 ** (L % 16 - 8))
        ko.append(pool, table, [L], [0, 1], kv[0], kv[1])
        kt, vt = (torch.from_numpy(x).bfloat16().cuda() for x in kv)
        cache.append(kt, vt, i32(table), i32([L]), i32([0, 1]))
    for n, t in (("k", cache.k), ("v", cache.v), ("ks", cache.k_scale), ("vs", cache.v_scale)):
        assert np.array_equal(t.cpu().numpy(), pool[n]), n
    assert status() == 0


def test_append_of_values_that_are_not_finite():
    table = np.array([[0]], np.int32)
    pool = dict(k=np.zeros((1, 1, 64, 64), np.uint8), v=np.zeros((1, 1, 64, 64), np.uint8),
                ks=np.zeros((1, 1), np.float32), vs=np.zeros((1, 1), np.float32))
    cache = upload(pool)
    k = np.random.default_rng(3).standard_normal((3, 1, 64))
    k[0, 0, 5], k[1, 0, 6], k[2, 0, 7] = np.nan, np.inf, -np.inf
    v = np.full((3, 1, 64), np.nan)
    k = bf16_round(k)
    cache.append(torch.from_numpy(k).bfloat16().cuda(), torch.from_numpy(v).bfloat16().cuda(), i32(table), i32([3]),
                 i32([0, 3]))
    assert status() == B_CHECK
    with np.errstate(invalid="ignore"):
        ko.append(pool, table, [3], [0, 3], k, v)
    assert np.array_equal(cache.k.cpu().numpy(), pool["k"]) and np.array_equal(cache.k_scale.cpu().numpy(), pool["ks"])
    assert not cache.v.any() and float(cache.v_scale) == 2.0 ** -126
    assert cache.k[0, 0, :3, 5:8].cpu().numpy()[[0, 1, 2], [0, 1, 2]].tolist() == [0, 0x7E, 0xFE]


# ---------------------------------------------------------------- evict

def check_evict(rng, lens, Hkv, P, D, budget, sink, recent, w=None, scales=(-10, -4)):
    table, pages = make_table(rng, lens, P)
    pool = make_pool(rng, pages, Hkv, P, D, scales)
    if w is None:
        w = rng.random((len(lens), Hkv, max(lens) + 5)).astype(np.float32) ** 6
    keep = [min(L, budget) for L in lens]
    dst_table, dst_pages = make_table(rng, keep, P)
    dst = make_pool(rng, dst_pages, Hkv, P, D)
    cache, dst_cache = upload(pool), upload(dst)
    got = cache.evict(torch.from_numpy(w).cuda(), i32(table), i32(lens), max(lens), budget, sink, recent,
                      i32(dst_table), dst=dst_cache)
    assert status() == 0
    want = ko.evict(pool, table, np.array(lens), w, budget, sink, recent, dst, dst_table)
    for x, y in zip(got, want):
        assert np.array_equal(x.cpu().numpy(), y, equal_nan=True)
    for n, t in (("k", dst_cache.k), ("v", dst_cache.v), ("ks", dst_cache.k_scale), ("vs", dst_cache.v_scale)):
        assert np.array_equal(t.cpu().numpy(), dst[n]), n


@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([100], 40, 4, 10), ([100, 40, 41, 39, 1, 0], 40, 0, 0), ([300, 77], 64, 64, 0), ([300, 77], 64, 0, 64),
    ([300, 77], 65, 33, 31), ([5000, 1, 2500], 1111, 16, 128), ([9], 1, 0, 0), ([2100], 2099, 3, 5)])
@pytest.mark.parametrize("Hkv,P,D", [(2, 64, 128), (1, 16, 64), (2, 128, 64)])
def test_evict(lens, budget, sink, recent, Hkv, P, D):
    check_evict(np.random.default_rng(sum(lens) + budget), lens, Hkv, P, D, budget, sink, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "odd"])
def test_evict_equal_and_odd_weights(kind):
    rng = np.random.default_rng(4)
    L = 2500
    w = np.ones((1, 2, L), np.float32)
    if kind == "few":
        w = rng.integers(0, 3, (1, 2, L)).astype(np.float32)
    if kind == "signs":
        w = rng.choice(np.array([0.0, -0.0, -1.0, 1e-45, -1e-45], np.float32), (1, 2, L))
    if kind == "odd":
        w = rng.standard_normal((1, 2, L)).astype(np.float32)
        w[0, :, ::7], w[0, :, 5::11], w[0, :, 3::13] = np.nan, np.inf, -np.inf
    check_evict(rng, [L], 2, 64, 64, 1000, 3, 40, w)


def test_evict_scales_far_apart():
    check_evict(np.random.default_rng(12), [900], 2, 32, 128, 400, 0, 16, scales=(-30, 10))


def test_evict_then_attend_sees_the_kept_tokens_alone():
    """Within one cache: into its free pages, then a decode step over them."""
    rng = np.random.default_rng(13)
    L, P, D, K = 500, 64, 128, 200
    table, _ = make_table(rng, [L], P, spare=4)
    free = np.array([sorted(set(range(12)) - set(table[0].tolist()))], np.int32)
    pool = make_pool(rng, 12, 2, P, D)
    pool["ks"][:] = pool["vs"][:] = 2.0 ** -8
    cache = upload(pool)
    w = torch.rand(1, 2, L, device="cuda")
    lens, kw, kept = cache.evict(w, i32(table), i32([L]), L, K, 4, 32, i32(free))
    q = torch.randn(1, 8, D, device="cuda").bfloat16()
    out = cache.attend(q, i32(free), lens, i32([0, 1]), 1, K)
    for h in range(8):
        at = kept[0, h // 4].long().cpu().numpy()
        k, v = (ko.rows(pool, m, table[0], L, h // 4)[at] for m in "kv")
        s = k @ q[0, h].double().cpu().numpy() * D ** -0.5
        p = np.exp(s - s.max())
        np.testing.assert_allclose(out[0, h].double().cpu().numpy(), (p / p.sum()) @ v, rtol=2 ** -8,
                                   atol=2 ** -9 * np.abs(v).max())
    assert torch.equal(kw, w.gather(2, kept.long())) and status() == 0


def test_calls_replay_in_a_graph():
    rng = np.random.default_rng(14)
    lens = [300, 1000]
    table, pages = make_table(rng, lens, 64)
    cache = upload(make_pool(rng, pages, 2, 64, 128))
    q = torch.randn(2, 8, 128, device="cuda").bfloat16()
    args = (i32(table), i32(lens), i32([0, 1, 2]), 1, 1000)
    out, w = torch.empty_like(q), torch.zeros(2, 2, 1000, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = cache.attend(q, *args, weights=w).clone()
    torch.cuda.current_stream().wait_stream(side)
    once = w.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cache.attend(q, *args, out=out, weights=w)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.allclose(w, 3 * once, rtol=1e-6) and status() == 0
