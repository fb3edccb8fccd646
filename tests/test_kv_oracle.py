"""Pins of the KV cache oracle: its e4m3 against torch's, its scale rule, its
attention against torch's float64 softmax, its eviction against hand-made cases."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko


def test_codes_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    real = ~np.isnan(t)
    assert np.array_equal(ko.VALUE[real], t[real]) and (~real).sum() == 2
    assert np.array_equal(np.abs(ko.VALUE[~real]), [480, 480])
    x = np.random.default_rng(0).standard_normal(4096) * np.exp2(np.random.default_rng(1).uniform(-12, 8, 4096))
    x = np.clip(np.concatenate([x, ko.VALUE[real], (ko.VALUE[:126] + ko.VALUE[1:127]) / 2]), -448, 448)
    x32 = x.astype(np.float32)
    want = torch.from_numpy(x32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ko.nearest_code(x32.astype(np.float64)), want)
    assert np.array_equal(ko.VALUE[ko.nearest_code(np.array([1e9, -1e9, np.inf]))], [448, -448, 448])


@pytest.mark.parametrize("amax,s", [(0, 2.0 ** -126), (448, 1), (448.0001, 2), (1, 2.0 ** -8), (1.75, 2.0 ** -8),
                                    (1.76, 2.0 ** -7), (3e38, 2.0 ** 120), (1e-44, 2.0 ** -126)])
def test_least_scale(amax, s):
    assert ko.least_scale(amax) == s


def _pool(rng, pages, Hkv, P, D):
    codes = lambda: rng.integers(0, 127, (pages, Hkv, P, D)).astype(np.uint8) | (rng.integers(0, 2, (pages, Hkv, P, D)) << 7).astype(np.uint8)
    scale = lambda: np.exp2(rng.integers(-9, -5, (pages, Hkv))).astype(np.float32)
    return dict(k=codes(), v=codes(), ks=scale(), vs=scale())


def test_attention_matches_torch():
    rng = np.random.default_rng(3)
    Hkv, g, P, D, lens, cu = 2, 3, 16, 64, [37, 5], [0, 4, 7]
    pool = _pool(rng, 5, Hkv, P, D)
    table = [[4, 1, 0], [3, 0, 0]]
    q = rng.standard_normal((7, Hkv * g, D))
    w = np.zeros((2, Hkv, 40))
    out, lse, mass, size = ko.attention(pool, table, lens, cu, q, 0.1, w)
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for h in range(Hkv * g):
            k, v = (torch.from_numpy(ko.rows(pool, m, table[b], L, h // g)) for m in "kv")
            s = 0.1 * torch.from_numpy(q[cu[b]:cu[b + 1], h]) @ k.T
            s = s.masked_fill(torch.arange(L)[None] > torch.arange(L - n, L)[:, None], -torch.inf)
            np.testing.assert_allclose(out[cu[b]:cu[b + 1], h], torch.softmax(s, 1) @ v, rtol=1e-12, atol=1e-12)
            np.testing.assert_allclose(lse[cu[b]:cu[b + 1], h], torch.logsumexp(s, 1), rtol=1e-12)
        # every row spreads a weight of one over what it sees
        np.testing.assert_allclose(w[b].sum(-1), n * g, rtol=1e-12)
        assert not w[b, :, L:].any()


def test_attention_rows_that_see_nothing():
    pool = _pool(np.random.default_rng(0), 1, 1, 16, 64)
    out, lse, _, _ = ko.attention(pool, [[0], [0]], [0, 1], [0, 2, 5], np.ones((5, 1, 64)), 1.0)
    assert not out[:4].any() and np.all(lse[:4] == -np.inf) and np.isfinite(lse[4])
    np.testing.assert_allclose(out[4, 0], ko.rows(pool, "v", [0], 1, 0)[0])


def test_append_keeps_older_tokens_and_grows_the_scale():
    pool = dict(k=np.zeros((2, 1, 16, 64), np.uint8), v=np.zeros((2, 1, 16, 64), np.uint8),
                ks=np.zeros((2, 1), np.float32), vs=np.zeros((2, 1), np.float32))
    one = np.full((3, 1, 64), 1.75)
    ko.append(pool, [[1]], [3], [0, 3], one, one)
    assert pool["ks"][1, 0] == 2.0 ** -8
    ko.append(pool, [[1]], [4], [0, 1], one[:1] * 8, one[:1])
    assert pool["ks"][1, 0] == 2.0 ** -5 and pool["vs"][1, 0] == 2.0 ** -8
    np.testing.assert_array_equal(ko.rows(pool, "k", [1], 4, 0)[:, 0], [1.75, 1.75, 1.75, 14])


def test_evict_by_hand():
    pool = _pool(np.random.default_rng(1), 2, 1, 16, 64)
    dst = _pool(np.random.default_rng(2), 1, 1, 16, 64)
    w = np.array([[[0, 5, 1, 5, np.nan, 5, 9, 9, 0]]], np.float32)
    lens, kw, kept = ko.evict(pool, [[0]], [9], w, 5, 1, 1, dst, [[0]])
    assert lens[0] == 5
    # the first and the last; then the NaN and the two of 9 come before the 5s
    assert kept[0, 0].tolist() == [0, 4, 6, 7, 8]
    np.testing.assert_array_equal(dst["k"][0, 0, :5], pool["k"][0, 0, [0, 4, 6, 7, 8]])
    w[0, 0, 4] = 0
    assert ko.evict(pool, [[0]], [9], w, 5, 1, 1, dst, [[0]])[2][0, 0].tolist() == [0, 1, 6, 7, 8]


def test_cache_refuses_tensors_of_the_wrong_kind():
    """On the host, before any call of the library."""
    from moe_ffn_layer_gb300.kv_cache import KVCache8
    cache = KVCache8(4, 2, 64, 16, device="cpu")
    table, lens, cu = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for bad in ((k.float(), k, table, lens, cu), (k[:, :1], k, table, lens, cu), (k, k, table.long(), lens, cu),
                (k, k, table, lens, cu[:1]), (k, k, table, torch.ones(2, dtype=torch.int32), cu)):
        with pytest.raises(ValueError):
            cache.append(*bad)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for bad in ((q.half(), table, lens, cu), (q[..., :32], table, lens, cu), (q, table, lens.long(), cu)):
        with pytest.raises(ValueError):
            cache.attend(*bad, 1, 16)
    with pytest.raises(ValueError):
        KVCache8.from_tensors(cache.k, cache.v[:2], cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError):
        KVCache8.from_tensors(cache.k.transpose(1, 2), cache.v, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError):
        cache.evict(torch.zeros(1, 3, 16), table, lens, 16, 4, 0, 0, table)


def test_calls_refuse_bad_arguments_before_a_launch():
    from moe_ffn_layer_gb300 import binding as B
    from moe_ffn_layer_gb300 import build as build_mod
    build_mod.build()
    fake = 1 << 20   # never dereferenced
    good = B.moe_kv_dims(2, 128, 64)
    pool, seqs = B.moe_kv_pool(fake, fake, fake, fake, 8), B.moe_kv_seqs(fake, fake, 1, 4, 256)

    def code(fn, *args):
        with pytest.raises(B.MoEError) as e:
            fn(*args)
        return e.value.code

    def attn(d=good, p=pool, s=seqs, q=fake, stride=512, Hq=4, cu=fake, T=1, n=1, out=fake, lse=None, w=None, ws_=0,
             ws=fake, nb=1 << 30):
        return (d, p, s, q, stride, Hq, cu, T, n, 1.0, out, lse, w, ws_, ws, nb, None)

    dims = B.moe_kv_dims
    assert code(B.moe_kv_attention, *attn(d=dims(0, 128, 64))) == -1
    for d in (dims(2, 96, 64), dims(2, 128, 48), dims(2, 128, 256), dims(40000, 64, 64)):
        assert code(B.moe_kv_attention, *attn(d=d, Hq=40000 if d.Hkv > 2 else 4, stride=1 << 23)) == -2
    assert code(B.moe_kv_attention, *attn(Hq=5)) == -1
    assert code(B.moe_kv_attention, *attn(stride=511)) == -1 and code(B.moe_kv_attention, *attn(stride=516)) == -2
    assert code(B.moe_kv_attention, *attn(q=None)) == -1 and code(B.moe_kv_attention, *attn(q=fake + 8)) == -2
    assert code(B.moe_kv_attention, *attn(p=B.moe_kv_pool(fake, None, fake, fake, 8))) == -1
    assert code(B.moe_kv_attention, *attn(p=B.moe_kv_pool(fake, fake + 4, fake, fake, 8))) == -2
    assert code(B.moe_kv_attention, *attn(s=B.moe_kv_seqs(fake, fake, 70000, 4, 256))) == -2
    assert code(B.moe_kv_attention, *attn(w=fake, ws_=255)) == -1 and code(B.moe_kv_attention, *attn(nb=0)) == -3
    assert code(B.moe_kv_attention, *attn(ws=fake + 128)) == -2
    assert B.moe_kv_attention(*attn(T=0, q=None)) == 0 and B.moe_kv_attention(*attn(s=B.moe_kv_seqs(None, None, 0, 0, 0))) == 0
    assert 0 < B.moe_kv_attention_workspace_bytes(good, 4, 1, 1, 1, 256, 0) < B.moe_kv_attention_workspace_bytes(good, 4, 1, 1, 1, 256, 1)
    assert B.moe_kv_attention_workspace_bytes(good, 5, 1, 1, 1, 256, 0) == 0

    def app(d=good, p=pool, s=seqs, k=fake, v=fake, stride=256, cu=fake, T=1):
        return (d, p, s, k, v, stride, cu, T, None)

    assert code(B.moe_kv_append, *app(stride=255)) == -1 and code(B.moe_kv_append, *app(stride=260)) == -2
    assert code(B.moe_kv_append, *app(v=None)) == -1 and code(B.moe_kv_append, *app(k=fake + 2)) == -2
    assert code(B.moe_kv_append, *app(T=-1)) == -1 and code(B.moe_kv_append, *app(cu=None)) == -1
    assert B.moe_kv_append(*app(T=0, k=None)) == 0

    def ev(d=good, s=seqs, w=fake, stride=256, budget=64, sink=4, recent=8, dst=pool, table=fake, width=1, lens=fake,
           kept=fake):
        return (d, pool, s, w, stride, budget, sink, recent, dst, table, width, lens, fake, kept, None)

    assert code(B.moe_kv_evict, *ev(budget=0)) == -1 and code(B.moe_kv_evict, *ev(sink=60)) == -1
    assert code(B.moe_kv_evict, *ev(sink=-1)) == -1 and code(B.moe_kv_evict, *ev(width=0)) == -1
    assert code(B.moe_kv_evict, *ev(stride=255)) == -1 and code(B.moe_kv_evict, *ev(kept=None)) == -1
    assert code(B.moe_kv_evict, *ev(lens=fake + 2)) == -2 and code(B.moe_kv_evict, *ev(d=dims(2, 80, 64))) == -2
