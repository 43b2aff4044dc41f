"""Microscaled formats beside the decode path: many requests that share a prompt
prefix start from one packed state, and the channel mix and head of the same model
run on 4-bit weights.

    python examples/microscaled.py [--shape 0.1b] [--slots 8] [--prefix 512]

1. The shared prefix is prefilled once and its state kept as MXINT8 and as MXFP4
   (PackedPrefixStateCache); every slot is loaded from the entry and decodes one token.
   Printed: bytes of a slot's state and of an entry, and how far the logits are from those
   of an unpacked state.
2. Rows as the layer's LayerNorm gives them go through the first layer's channel mix
   (key, squared ReLU, value) and the head with MXFP4 weights (mx4_quantize once,
   mx4_linear per step).  Printed: bytes of the weights in fp16 and MXFP4, and how far
   the results are from those of the fp16 weights.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import recurrent_decode_gb300 as rd  # noqa: E402
import synth  # noqa: E402
from recurrent_decode_gb300.prefix_cache import PackedPrefixStateCache  # noqa: E402


def off(got, want):
    """Relative distance of two results."""
    got, want = got.double(), want.double()
    return float((got - want).norm() / want.norm())


def shared_prefix(ctx, dims, slots, prefix):
    dev = torch.device("cuda")
    tokens = synth.prompt_tokens(dims.vocab, 1, prefix + 1)[0]
    all_slots = torch.arange(slots, dtype=torch.int32, device=dev)
    next_token = torch.full((slots,), int(tokens[-1]), dtype=torch.int32, device=dev)

    def decode():
        logits = torch.empty(slots, dims.vocab, device=dev)
        ctx.decode_step(all_slots, next_token, logits)
        ctx.synchronize()
        return logits

    out = {}
    for format in ("mxint8", "mxfp4"):
        cache = PackedPrefixStateCache(ctx, 4, format)
        ctx.slot_reset(slots)  # the last slot of the pool prefills
        cache.prefill(slots, tokens[:-1], 0, lambda a: torch.from_numpy(a.copy()).to(dev))
        for s in range(slots):
            ctx.slot_copy(slots, s)
        exact = decode()
        for s in range(slots):
            assert cache.restore(tokens[:-1], s) == prefix
        packed = decode()
        out[format] = off(packed, exact)
        print(f"{format}: {cache.states.entry_bytes:,} bytes an entry, {ctx.state_bytes():,} a slot; "
              f"logits of {slots} requests off by {out[format]:.2e}")
    return out


def four_bit_weights(weights, dims, rows):
    names = {"key": "blocks.0.ffn.key", "value": "blocks.0.ffn.value", "head": "head"}
    w = {k: torch.from_numpy(np.ascontiguousarray(weights[n])).cuda() for k, n in names.items()}
    q = {k: rd.mx4_quantize(t) for k, t in w.items()}
    x = torch.nn.functional.layer_norm(torch.randn(rows, dims.d_model, device="cuda"), (dims.d_model,)).half()

    h = rd.mx4_linear(x, q["key"], activation="relu2")
    y = rd.mx4_linear(h, q["value"], out_dtype=torch.float32)
    logits = rd.mx4_linear(x, q["head"], out_dtype=torch.float32)
    rd.mx4_check()

    mix = torch.relu(x.float() @ w["key"].float().t()).square() @ w["value"].float().t()
    out = {"channel mix": off(y, mix), "head": off(logits, x.float() @ w["head"].float().t())}
    for k, t in w.items():
        print(f"{k}: {t.numel() * 2:,} bytes in fp16, {q[k].data.numel():,} in MXFP4")
    print(", ".join(f"{k} off by {v:.2e}" for k, v in out.items()))
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--shape", default="0.1b")
    ap.add_argument("--slots", type=int, default=8)
    ap.add_argument("--prefix", type=int, default=512)
    a = ap.parse_args(argv)
    dims = synth.Dims(a.shape)
    weights = synth.make_weights(a.shape)
    ctx = rd.Rwkv7(dims, a.slots + 1)
    ctx.set_weights(weights)
    result = {**shared_prefix(ctx, dims, a.slots, a.prefix), **four_bit_weights(weights, dims, a.slots)}
    ctx.close()
    return result


if __name__ == "__main__":
    main()
