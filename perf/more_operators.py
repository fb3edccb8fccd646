"""Measured cases of the 8-bit projections' operators: norm, quantise, multiply.

Rows in 8 bits: e4m3 codes ``[T, K]`` with one power of two per 128 values of a
row, held as its exponent byte (value ``2 ** (byte - 127)``), ``[T, ceil(K /
128)]``.  Weights ``[N, K]`` have one per block of 128 x 128.  A scale is the least
power of two s with ``max |x| <= 448 s``, 2^-126 at least; codes are rounded to
nearest even.

Where ``own`` is false, ``run`` is elementary torch in fp32; where it is true it
calls ``moe_ffn_layer_gb300.linear8``.
"""
import math

import torch

own = False

# Sizes are those of hidden sizes 2048 and 4096 (with the layer's 768, 1024, 2048
# and 4096 wide intermediates, 32 query heads and 8 kv heads of 128) at its
# decode, batched decode and prefill batches (1 to 256 tokens, 8192 and 16384).


def listed():
    return [
        # the norm before a projection, one token of one chat: launch latency counts
        dict(name="norm 1", op="norm", T=1, H=2048, res=True, out="codes", gap=0),
        # the norm before the MoE FFN of a batched decode step: bf16 rows, which its router takes
        dict(name="norm 256 bf16", op="norm", T=256, H=2048, res=True, out="y", gap=0),
        # a prompt's norm before its projections: memory speed
        dict(name="norm 8k", op="norm", T=8192, H=4096, res=True, out="codes", gap=0),
        # an embedding's first norm, a hidden size that ends inside a block, rows some way apart
        dict(name="norm odd", op="norm", T=1021, H=2064, res=False, out="both", gap=24),
        # SiLU(gate) * up of a dense FFN at batched decode, to 8 bits for its down projection
        dict(name="silu 333", op="silu", T=333, K=768, gap=0),
        # the attention's output of a large prefill, to 8 bits for the output projection
        dict(name="quantize 16k", op="rows", T=16384, K=4096, gap=0),
        # a gate_up weight at load
        dict(name="quantize weight", op="weight", N=8192, K=4096),
        # a projection of one token: latency and the weights' stream
        dict(name="linear 1", op="linear", T=1, N=4096, K=2048),
        # q, k and v of a batched decode step: the weights' stream
        dict(name="linear 64", op="linear", T=64, N=6144, K=4096),
        # a ragged chunk, sizes that end inside every tile
        dict(name="linear odd", op="linear", T=777, N=2500, K=2000),
        # q, k and v of a prompt
        dict(name="linear 8k", op="linear", T=8192, N=4096, K=2048),
        # gate_up of a large prefill: the tensor cores' rate
        dict(name="linear 16k", op="linear", T=16384, N=8192, K=4096),
    ]


def draw(rng):
    def logint(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["norm", "norm", "rows", "silu", "weight", "linear", "linear", "linear"])
    K = 16 * logint(4, 512) if rng.random() < 0.5 else 128 * logint(1, 64)
    if kind in ("norm", "rows", "silu"):
        T = logint(1, min(16384, (1 << 26) // K))
        gap = rng.choice([0, 0, 8, 24, 128])
        if kind == "norm":
            return dict(op="norm", T=T, H=K, res=rng.random() < 0.7, out=rng.choice(["codes", "codes", "y", "both"]), gap=gap)
        return dict(op=kind, T=T, K=K, gap=gap)
    N = rng.choice([128 * logint(1, 64), 16 * logint(4, 512), logint(64, 8192)])
    if kind == "weight":
        return dict(op="weight", N=N, K=K)
    return dict(op="linear", T=logint(1, min(16384, (1 << 39) // (N * K))), N=N, K=K)


def _scale_bytes(amax):
    """Exponent bytes of the least powers of two s with amax <= 448 s (2^-126 at least)."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    return torch.where(amax > 0, e + 127, 1).to(torch.uint8)


def _power(s):
    return torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.int() - 127)


def _blocks(x, rows):
    """x [R, K] cut in blocks of `rows` x 128, padded with zeros: [R', rows, K', 128]."""
    R, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128, 0, -R % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def _to8(x, rows=1):
    """Codes and exponent bytes of x in blocks of `rows` x 128."""
    b = _blocks(x, rows)
    s = _scale_bytes(b.abs().amax((1, 3)))
    c = (b / _power(s)[:, None, :, None]).to(torch.float8_e4m3fn)
    return c.view(c.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]].contiguous(), s


def _from8(c, s, rows=1):
    """The values that codes and exponent bytes stand for."""
    s = _power(s).repeat_interleave(rows, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :c.shape[1]]
    return c.view(torch.float8_e4m3fn).float() * s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    def rows(T, K):
        # activations: unit size, a few channels much larger, rows of different size; they lie `gap` values apart
        x = randn(T, K + case.get("gap", 0))
        x *= 1 + 15 * (torch.rand(x.shape[1], generator=g, device="cuda") < 0.01).bfloat16()
        x *= torch.rand(T, 1, generator=g, device="cuda").bfloat16() + 0.25
        return x[:, :K]

    op, st = case["op"], dict(case=case)
    if op == "norm":
        st["x"] = rows(case["T"], case["H"])
        st["w"] = (1 + 0.1 * randn(case["H"]).float()).bfloat16()
        st["r"] = 4 * randn(case["T"], case["H"]) if case["res"] else None
    elif op == "silu":
        st["x"] = rows(case["T"], 2 * case["K"])
    elif op == "rows":
        st["x"] = rows(case["T"], case["K"])
    elif op == "weight":
        st["x"] = 0.02 * randn(case["N"], case["K"])
    else:
        st["a"], st["as"] = _to8(rows(case["T"], case["K"]).float())
        st["b"], st["bs"] = _to8(0.02 * randn(case["N"], case["K"]).float(), 128)
        if own:
            from moe_ffn_layer_gb300 import linear8
            st["a"], st["as"] = linear8.rows8(st["a"].view(torch.uint8), st["as"])
            st["linear"] = linear8.Linear8(st["b"].view(torch.uint8), st["bs"])
            st["out"] = torch.empty(case["T"], case["N"], dtype=torch.bfloat16, device="cuda")
    if own and op != "linear":
        from moe_ffn_layer_gb300 import linear8
        st["linear8"] = linear8
    return st


def _as_values(codes, scales):
    return dict(codes=codes.view(torch.float8_e4m3fn), scales=scales.view(torch.float8_e8m0fnu))


def run(st):
    return {"norm": _norm, "silu": _rows, "rows": _rows, "weight": _weight, "linear": _linear}[st["case"]["op"]](st)


def _norm(st):
    out = st["case"]["out"]
    if own:
        st["into"] = n = st["linear8"].rms_norm8(st["x"], st["w"], 1e-6, residual=st["r"], outputs=out, into=st.get("into"))
        h, y, codes, scales = n.h, n.y, n.codes, n.scales
    else:
        h = st["x"]
        if st["r"] is not None:
            h = (h.float() + st["r"].float()).bfloat16()
        y = h.float()
        y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6) * st["w"].float()
        codes, scales = _to8(y) if out != "y" else (None, None)
        h, y = h if st["r"] is not None else None, y.bfloat16() if out != "codes" else None
    return dict(h=h, y=y, **(_as_values(codes, scales) if out != "y" else {}))


def _rows(st):
    silu = st["case"]["op"] == "silu"
    if own:
        st["into"] = st["linear8"].quantize8(st["x"], silu_mul=silu, into=st.get("into"))
        return _as_values(*st["into"])
    x = st["x"].float()
    if silu:
        gate, up = x.chunk(2, 1)
        x = gate / (1 + torch.exp(-gate)) * up
    return _as_values(*_to8(x))


def _weight(st):
    if own:
        return _as_values(*st["linear8"].quantize8_weight(st["x"]))
    return _as_values(*_to8(st["x"].float(), 128))


def _linear(st):
    if own:
        return st["linear"](st["a"], st["as"], out=st["out"])
    return (_from8(st["a"], st["as"]) @ _from8(st["b"], st["bs"], 128).t()).bfloat16()


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        moved = 2 + 4 * case["res"] + 2 * (case["out"] != "codes") + (case["out"] != "y")
        return dict(bytes=T * H * moved + 2 * H + (T * -(-H // 128) if case["out"] != "y" else 0), flops=6 * T * H)
    if op == "weight":
        return dict(bytes=3 * case["N"] * case["K"] + -(-case["N"] // 128) * -(-case["K"] // 128), flops=2 * case["N"] * case["K"])
    T, K = case["T"], case["K"]
    if op != "linear":
        return dict(bytes=T * K * (5 if op == "silu" else 3) + T * -(-K // 128), flops=T * K * (6 if op == "silu" else 2))
    N = case["N"]
    return dict(bytes=T * K + N * K + (T + -(-N // 128)) * -(-K // 128) + 2 * T * N, flops=2 * T * N * K)


def exact(case, seed):
    """The definitions in float64."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = dict(dtype=torch.float64, device="cuda")
    # the value of each e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits
    table8 = [((c & 7) * 2.0 ** -9 if not c & 0x78 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) * (-1) ** (c >> 7)
              for c in range(256)]
    value = torch.tensor(table8, **f64)
    grid = value[:127].contiguous()
    powers = torch.tensor([2.0 ** e for e in range(-126, 128)], **f64)

    def nearest(x):   # to the nearest e4m3 value, ties to the even code
        a = x.abs().clamp(max=448).contiguous()
        hi = torch.searchsorted(grid, a).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up, down = grid[hi] - a, a - grid[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        return torch.copysign(grid[code], x)

    def spread(s, high, R, K):   # one value a block to one an element
        i, j = torch.arange(R, device="cuda") // high, torch.arange(K, device="cuda") // 128
        return s[i][:, j]

    def eight(x, high=1):
        R, K = x.shape
        codes, scales = torch.empty_like(x), torch.empty(-(-R // high), -(-K // 128), **f64)
        for j in range(scales.shape[1]):
            col = x[:, 128 * j:128 * j + 128]
            top = col.abs().amax(1)
            if high > 1:
                top = torch.stack([t.max() for t in top.split(high)])
            s = scales[:, j] = powers[torch.searchsorted(powers, top / 448)]
            codes[:, 128 * j:128 * j + 128] = nearest(col / s.repeat_interleave(high)[:R, None])
        return dict(codes=codes, scales=scales)

    if op == "norm":
        x, w, H = st["x"].double(), st["w"].double(), case["H"]
        h = x if st["r"] is None else (x + st["r"].double()).float().bfloat16().double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / H + 1e-6) * w
        return dict(h=None if st["r"] is None else h, y=y if case["out"] != "codes" else None,
                    **(eight(y) if case["out"] != "y" else {}))
    if op == "weight":
        return eight(st["x"].double(), 128)
    if op == "silu":
        gate, up = st["x"].double().split(case["K"], 1)
        return eight(gate * torch.sigmoid(gate) * up)
    if op == "rows":
        return eight(st["x"].double())
    T, N, K = case["T"], case["N"], case["K"]
    two = torch.tensor([2.0 ** (e - 127) for e in range(256)], **f64)
    a = value[st["a"].view(torch.uint8).long()] * spread(two[st["as"].long()], 1, T, K)
    b = value[st["b"].view(torch.uint8).long()] * spread(two[st["bs"].long()], 128, N, K)
    return a @ b.t()
