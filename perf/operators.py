"""The microscaled operators: what is measured, and their plain forms.

A microscaled block is 32 consecutive values of a row that share one power of
two.  MXFP4 holds the values on the 4-bit grid {0, 0.5, 1, 1.5, 2, 3, 4, 6} with
a sign, MXINT8 as whole numbers of sixty-fourths, -127/64 .. 127/64; the shared
power is the smallest one under which no value of the block is cut off.

  quantize  rows of activations or weights to MXFP4 and the values read back
  linear    y = act(q(x) q(W)^T): rows quantised as they come, weights once
  states    recurrent states of slots saved as MXINT8 or MXFP4 entries of a
            cache, and loaded from it into other slots

`own` false: torch operations on the values themselves.  `own` true: the calls
of recurrent_decode_gb300.  Weights are quantised in `prepare`, where a program
loads them, so what `prepare` keeps of them goes by `own`: the values they stand
for, or the library's matrix.  A cache is likewise made where a program starts.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's normed rows at the 2.9B width, 64 slots
        dict(name="quant_step", op="quantize", rows=64, cols=2560, pad=0, dtype="fp16"),
        # fp32 rows cut out of a wider buffer, no size a multiple of anything
        dict(name="quant_ragged", op="quantize", rows=1001, cols=1999, pad=6, dtype="fp32"),
        # the hidden rows of sixteen prefill chunks at the 7.2B width
        dict(name="quant_prefill", op="quantize", rows=4096, cols=16384, pad=0, dtype="bf16"),
        # the 2.9B head for a single sequence: logits in fp32
        dict(name="head_one", op="linear", rows=1, cols=2560, outs=65536, dtype="fp16", out="fp32", act="none"),
        # the 2.9B channel-mix key for a decode batch
        dict(name="key_batch", op="linear", rows=64, cols=2560, outs=10240, dtype="fp16", out="fp16", act="relu2"),
        # the 7.2B channel-mix value for a full decode batch: few rows of output, a long sum
        dict(name="value_batch", op="linear", rows=256, cols=16384, outs=4096, dtype="fp16", out="fp32", act="none", hidden=True),
        # a LoRA-like odd product
        dict(name="linear_odd", op="linear", rows=37, cols=1000, outs=1337, dtype="bf16", out="bf16", act="none"),
        # a long prefill through the 7.2B channel-mix key
        dict(name="key_prefill", op="linear", rows=4096, cols=4096, outs=16384, dtype="fp16", out="fp16", act="relu2"),
        # one sequence of the 0.1B shape set aside and resumed
        dict(name="state_one", op="states", layers=12, heads=12, save=1, load=1, format="mxint8"),
        # sixteen sequences of the 2.9B shape set aside and resumed
        dict(name="state_batch", op="states", layers=32, heads=40, save=16, load=16, format="mxint8"),
        # one 7.2B prefix shared by 48 requests
        dict(name="state_fork", op="states", layers=32, heads=64, save=1, load=48, format="mxint8"),
        # an odd shape in four bits
        dict(name="state_four_bits", op="states", layers=5, heads=3, save=7, load=21, format="mxfp4"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "states"])
    if op == "quantize":
        while True:
            rows, cols = _log(rng, 1, 65536), _log(rng, 20, 16384)
            if rng.random() < 0.5:
                cols = max(32, cols // 32 * 32)
            if rows * cols <= 4096 * 16384:
                return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 1, 8, 96]),
                            dtype=rng.choice(["fp16", "bf16", "fp32"]) if rows * cols <= 1 << 25 else "bf16")
    if op == "linear":
        while True:
            rows, cols, outs = _log(rng, 1, 4096), _log(rng, 40, 16384), _log(rng, 40, 65536)
            if rng.random() < 0.5:
                cols, outs = max(64, cols // 64 * 64), max(64, outs // 64 * 64)
            if rows * cols * outs <= 1 << 38 and cols * outs <= 1 << 28 and rows * outs <= 1 << 26:
                return dict(op=op, rows=rows, cols=cols, outs=outs, dtype=rng.choice(["fp16", "bf16", "fp32"]),
                            out=rng.choice(["fp16", "bf16", "fp32"]), act=rng.choice(["none", "relu2"]),
                            hidden=rng.random() < 0.3)
    while True:
        layers, heads, save, load = rng.randint(1, 32), rng.randint(1, 64), _log(rng, 1, 32), _log(rng, 1, 64)
        if layers * heads * (save + load) <= 32 * 64 * 40:
            return dict(op=op, layers=layers, heads=heads, save=save, load=load, format=rng.choice(["mxint8", "mxfp4"]))


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed * 1000003 + 17)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "states":
        # Decayed sums of outer products: heads of different scales, values of a
        # row (one value channel, 64 key channels) of similar size; one slot fresh.
        L, H, n = case["layers"], case["heads"], case["save"] + case["load"]
        wkv = normal(L, n, H, 64, 64)
        wkv.mul_(torch.exp(normal(L, n, H, 1, 1))).mul_(torch.exp(0.5 * normal(L, n, H, 64, 1)))
        order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        if case["save"] > 2:
            wkv[:, order[0].long()] = 0
        s["states"] = (wkv, normal(L, n, H * 64), normal(L, n, H * 64))
        s["src"], s["dst"] = order[:case["save"]].contiguous(), order[case["save"]:].contiguous()
        s["kept"] = torch.arange(case["save"], dtype=torch.int32, device="cuda").flip(0).contiguous()
        s["taken"] = s["kept"][torch.arange(case["load"], device="cuda") % case["save"]].contiguous()
        if own:
            import recurrent_decode_gb300 as rd
            s["cache"] = rd.StateCache(L, H, case["save"], case["format"])
        return s
    # Normed rows with a few large channels; past a squared ReLU half of them are zero.
    R, K = case["rows"], case["cols"]
    x = normal(R, K + case.get("pad", 0)) * torch.exp(0.6 * normal(K + case.get("pad", 0)))
    if case.get("hidden"):
        x = torch.relu(x).square()
    s["x"] = x.to(TYPES[case["dtype"]])[:, :K]
    if case["op"] == "linear":
        w = s["weights"] = (0.02 * normal(case["outs"], K)).half()
        if own:
            import recurrent_decode_gb300 as rd
            s["w"] = rd.mx4_quantize(w)
        else:
            s["w"] = _mxfp4(w)
    return s


def work(case):
    if case["op"] == "states":
        one = case["layers"] * case["heads"] * 4096  # values of one state
        shift = 2 * case["layers"] * case["heads"] * 64 * 4
        entry = one * (8 if case["format"] == "mxint8" else 4) // 8 + one // BLOCK + shift
        n = case["save"] + case["load"]
        return {"bytes": (4 * one + shift) * n + 2 * entry * case["save"], "flops": 2 * one * n}
    R, K, size = case["rows"], case["cols"], 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "quantize":
        return {"bytes": 2 * R * K * size, "flops": 4 * R * K}
    N, blocks = case["outs"], -(-K // BLOCK)
    return {"bytes": R * K * size + N * (K / 2 + blocks) + R * N * (4 if case["out"] == "fp32" else 2),
            "flops": 2 * R * K * N}


# ------------------------------------------------------------------ one pass
def run(s):
    if s["op"] == "quantize":
        return _own_quantize(s) if own else _mxfp4(s["x"]).to(s["x"].dtype)
    if s["op"] == "linear":
        return _own_linear(s) if own else _plain_linear(s)
    return _own_states(s) if own else _plain_states(s)


def _own_quantize(s):
    import recurrent_decode_gb300 as rd
    return rd.mx4_quantize(s["x"]).dequantize(s["x"].dtype)


def _own_linear(s):
    import recurrent_decode_gb300 as rd
    return rd.mx4_linear(s["x"], s["w"], out_dtype=TYPES[s["out"]], activation=s["act"])


def _own_states(s):
    s["cache"].save(s["states"], s["src"], s["kept"])
    s["cache"].load(s["states"], s["taken"], s["dst"])
    return s["states"]


def _blocks(x):
    """x [..., K] in fp32 as blocks [..., ceil(K / 32), 32], the last one filled with zeros."""
    x = x.float()
    short = -x.shape[-1] % BLOCK
    if short:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], short)], -1)
    return x.reshape(*x.shape[:-1], -1, BLOCK)


def _power(top, past, less, lowest, highest):
    """(2^e, 2^-e) with e the exponent of `top` less `less`, one more where its fraction passes `past`."""
    bits = top.view(torch.int32)
    e = (bits >> 23) - less + ((bits & 0x7FFFFF) > past).int()
    e = e.clamp(lowest, highest)
    up = torch.where(e > 0, e << 23, 1 << 22).int().view(torch.float32)
    down = torch.where(e < 254, (254 - e) << 23, 1 << 22).int().view(torch.float32)
    return up, down


def _mxfp4(x):
    """The values that x stands for in MXFP4, in fp32."""
    b = _blocks(x)
    top = b.abs().amax(-1, keepdim=True)
    up, down = _power(top, 0x400000, 2, 0, 254)  # 6 = 1.5 * 2^2
    v = b * down
    size = v.abs()
    step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    q = torch.round(v / step) * step * up
    q = torch.where(torch.isfinite(top), q, torch.nan)
    return q.reshape(*x.shape[:-1], -1)[..., :x.shape[-1]]


def _mxint8(x):
    """The values that x stands for in MXINT8, in fp32."""
    b = _blocks(x)
    top = b.abs().amax(-1, keepdim=True)
    up, down = _power(top, 0x7E0000, 0, 1, 254)  # 127/64 = 1.984375
    q = torch.round(b * down * 64).clamp(-127, 127) / 64 * up
    q = torch.where(torch.isfinite(top), q, torch.nan)
    return q.reshape(*x.shape[:-1], -1)[..., :x.shape[-1]]


def _plain_linear(s):
    y = torch.matmul(_mxfp4(s["x"]), s["w"].t())
    if s["act"] == "relu2":
        y = torch.relu(y).square()
    return y.to(TYPES[s["out"]])


def _plain_states(s):
    wkv, att, ffn = s["states"]
    src, dst = s["src"].long(), s["dst"].long()
    held = torch.zeros_like(src)
    held[s["kept"].long()] = src  # the slot behind each entry
    held = held[s["taken"].long()]
    q = (_mxint8 if s["format"] == "mxint8" else _mxfp4)(wkv[:, src])
    at = torch.zeros_like(s["kept"], dtype=torch.int64)
    at[s["kept"].long()] = torch.arange(len(src), device=src.device)
    wkv[:, dst] = q[:, at[s["taken"].long()]]
    att[:, dst], ffn[:, dst] = att[:, held], ffn[:, held]
    return wkv, att, ffn


# ------------------------------------------------------------------ 64 bits
def _nearest(x, name):
    """MXFP4 or MXINT8 values of x [R, K] by the definition, in float64."""
    R, K = x.shape
    b = torch.zeros(R, -(-K // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    b[:, :K] = x
    b = b.view(R, -1, BLOCK)
    limit, lowest, highest = (6.0, -127, 127) if name == "mxfp4" else (127.0, -132, 121)
    top = b.abs().max(-1, keepdim=True).values
    bad = ~torch.isfinite(top)
    m, e = torch.frexp(torch.where(bad, 0.0, top) / limit)  # top / limit = m 2^e with 1/2 <= m < 1, or 0
    e = torch.where(m == 0, lowest, e - (m == 0.5).int()).clamp(lowest, highest)
    one = ((e.long() + 1023) << 52).view(torch.float64)
    v = torch.where(bad, 0.0, b) / one
    if name == "mxfp4":
        a = v.abs()
        q = 0.5 * ((a > 0.25).double() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5) + 2 * (a > 5.0)
        q = q * v.sign()
    else:
        q = v.round().clamp(-127, 127)
    return torch.where(bad, math.nan, q * one).view(R, -1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "states":
        wkv, att, ffn = (t.double() for t in s["states"])
        entry = dict(zip(s["kept"].tolist(), s["src"].tolist()))
        for t, d in zip(s["taken"].tolist(), s["dst"].tolist()):
            a = wkv[:, entry[t]]
            wkv[:, d] = _nearest(a.reshape(-1, 64), case["format"]).view_as(a)
            att[:, d], ffn[:, d] = att[:, entry[t]], ffn[:, entry[t]]
        return wkv, att, ffn
    x = _nearest(s["x"].double(), "mxfp4")
    if case["op"] == "quantize":
        return x
    y = x @ _nearest(s["weights"].double(), "mxfp4").t()
    return y.clamp(min=0) ** 2 if case["act"] == "relu2" else y
