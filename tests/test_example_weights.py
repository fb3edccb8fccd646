"""What the decoder layers of examples/decode_with_cache.py keep of their weights, without a GPU."""
import os
import sys
import types
import weakref

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_8_bit_layer_keeps_no_bf16_weight(monkeypatch):
    import decode_with_cache as example
    monkeypatch.setattr(example, "Linear8", types.SimpleNamespace(from_weight=lambda w: ("in 8 bits", tuple(w.shape))))
    w_qkv, w_o = torch.zeros(48, 32, dtype=torch.bfloat16), torch.zeros(32, 32, dtype=torch.bfloat16)
    given = [weakref.ref(w_qkv), weakref.ref(w_o)]
    layer = example.DecoderLayer8(w_qkv, w_o, "ffn", "cache", 4)
    del w_qkv, w_o
    assert [w() for w in given] == [None, None]
    assert (layer.qkv, layer.o) == (("in 8 bits", (48, 32)), ("in 8 bits", (32, 32)))
    assert (layer.ffn, layer.cache, layer.heads) == ("ffn", "cache", 4)
