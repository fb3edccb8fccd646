"""The softmax weights' sixteen bits: pages whose values cancel, so that what is left
of a weight's rounding is not hidden by that of the result.

A weight times its page's V scale enters the product as two bf16 terms, the upper
one cut off after 8 bits and the lower one rounded to 8: 2^-16 of it at most is
lost.  Exponents and scales round to fp32 (2^-18 in all), and a score's error ds
moves a weight by twice as much; so out moves by (2^-15 + 2 ds) of the mass sum p |V|
at most, and then rounds to bf16."""
import numpy as np
import pytest
import torch

from moe_ffn_layer_gb300 import build as build_mod
from oracle import kv_oracle as ko
from test_kv_cache import i32, make_pool, make_table, status, upload

SCALE = 0.125


def cancelling(n, L, Hkv, g, D=128, P=16):
    """Even pages: K 0, V +1 times a; odd ones: a score s, V -1.25 times 0.8 a e^-s; s and a by kv head.  (The weights
    times V's scale are a and 0.8 a times the same: other bits of them are lost.)"""
    rng = np.random.default_rng(64)
    table, pages = make_table(rng, [L], P)
    pool = make_pool(rng, pages, Hkv, P, D)
    s, a = rng.uniform(-3, 3, Hkv), rng.uniform(1, 2, Hkv)
    even, odd = table[0, ::2], table[0, 1::2]
    pool["k"][:] = 0
    pool["k"][odd, :, :, 5] = np.where(s < 0, 0xB8, 0x38).astype(np.uint8)[None, :, None]
    pool["v"][even], pool["v"][odd] = 0x38, 0xBA
    pool["ks"][odd] = np.abs(s) / SCALE
    s = pool["ks"][odd[0]].astype(np.float64) * np.sign(s) * SCALE      # as held
    pool["vs"][even], pool["vs"][odd] = a, 0.8 * a * np.exp(-s)
    return np.ones((n, Hkv * g, D)), pool, table


def bound_of(q, pool, table, L):
    """(the exact result, how far from it a result may lie)"""
    ref, _, mass, size = ko.attention(pool, table, [L], np.array([0, len(q)]), q, SCALE)
    ds = 8 * 2.0 ** -22 * size + 2.0 ** -21 * size
    return ref, 2.0 ** -8 * np.abs(ref) + (2.0 ** -15 + 2 * ds.max()) * mass


CASES = [(1, 700, 16, 4), (3, 900, 16, 4), (40, 700, 16, 4), (300, 3000, 4, 4)]   # queries, tokens, kv heads, heads of each


@pytest.mark.gpu
@pytest.mark.parametrize("n,L,Hkv,g", CASES)
def test_weights_keep_sixteen_bits(n, L, Hkv, g):
    build_mod.build()
    q, pool, table = cancelling(n, L, Hkv, g)
    ref, bound = bound_of(q, pool, table, L)
    out = upload(pool).attend(torch.from_numpy(q).bfloat16().cuda(), i32(table), i32([L]), i32([0, n]), n, L, scale=SCALE)
    assert (np.abs(out.double().cpu().numpy() - ref) - bound).max() <= 0 and status() == 0


@pytest.mark.parametrize("bits", [8, 11])
def test_the_bound_sees_weights_of_fewer_bits(bits):
    """The definition with weights rounded to one term of so many bits, on the CPU."""
    n, L, Hkv, g = CASES[0]
    q, pool, table = cancelling(n, L, Hkv, g)
    ref, bound = bound_of(q, pool, table, L)
    over = 0
    for h in range(Hkv):
        k, v = ko.rows(pool, "k", table[0], L, h), ko.rows(pool, "v", table[0], L, h)
        s = SCALE * (k @ q[0, h * g])
        code = np.where(v[:, 0] > 0, 1.0, -1.25)
        m, e = np.frexp(np.exp(s - s.max()) * v[:, 0] / code)           # weights times V's scale
        out = (np.ldexp(np.round(m * 2 ** bits) / 2 ** bits, e) * code).sum() / np.exp(s - s.max()).sum()
        over += abs(out - ref[0, h * g, 0]) > bound[0, h * g, 0]
    assert over > Hkv // 2
