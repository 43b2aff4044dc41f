"""Beam search beside the sampler: the most probable continuations of a few prompts, and
the same choice of tokens from a head in 4 bits.

    python examples/beam_search.py [--shape 0.1b] [--prompts 4] [--width 4] [--tokens 16]

1. Every prompt is prefilled once, its state forked to `width` slots, and beam_search keeps
   the best beams for a number of steps.  Printed: the best beam's summed log-probability and the
   greedy continuation's.
2. Random rows, normed as the final LayerNorm's are, go through the head in fp16 and in 4 bits with a
   scale for 64 columns (q4_quantize once, q4_linear a step), and beam_select picks from both.  (The decode
   step computes its head itself, in fp16; the search above does not use this one.)
   Printed: bytes of both heads, how far the logits are, how many picks agree.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import recurrent_decode_gb300 as rd  # noqa: E402
import synth  # noqa: E402


def greedy_score(ctx, prompt, n_out):
    """Summed log-probability of the greedy continuation."""
    dev = torch.device("cuda")
    slot = torch.zeros(1, dtype=torch.int32, device=dev)
    ctx.slot_reset(0)
    if len(prompt) > 1:
        ctx.prefill_seq(0, torch.from_numpy(prompt[:-1].copy()).to(dev))
    token = torch.tensor([int(prompt[-1])], dtype=torch.int32, device=dev)
    logits, total = torch.empty(1, ctx.dims.vocab, device=dev), 0.0
    for _ in range(n_out):
        ctx.decode_step(slot, token, logits)
        ctx.synchronize()
        p = torch.log_softmax(logits[0].double(), 0)
        token = p.argmax().int().view(1)
        total += float(p[token.long()])
    return total


def search(ctx, prompts, width, n_out):
    greedy = [greedy_score(ctx, p, n_out) for p in prompts]
    found = rd.beam_search(ctx, prompts, width, n_out)
    for i, (beams, g) in enumerate(zip(found, greedy)):
        print(f"prompt {i}: best of {width} beams {beams[0][0]:.3f}, greedy {g:.3f}, tokens {beams[0][1][:8].tolist()} ...")
    return found, greedy


def four_bit_head(weights, dims, requests, width):
    head = torch.from_numpy(np.ascontiguousarray(weights["head"])).cuda()
    q = rd.q4_quantize(head, group=64)
    x = torch.nn.functional.layer_norm(torch.randn(requests * width, dims.d_model, device="cuda"), (dims.d_model,)).half()
    exact = x.float() @ head.float().t()
    logits = rd.q4_linear(x, q, out_dtype=torch.float32)
    rd.q4_check()
    scores = torch.zeros(requests, width, device="cuda")
    want, got = rd.beam_select(exact, scores), rd.beam_select(logits, scores)
    off = float((logits - exact).double().norm() / exact.double().norm())
    same = float(((want.tokens == got.tokens) & (want.parents == got.parents)).float().mean())
    print(f"head: {head.numel() * 2:,} bytes in fp16, {q.data.numel():,} in 4 bits; logits off by {off:.2e}, "
          f"{100 * same:.0f} % of the picks alike")
    return off, same


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--shape", default="0.1b")
    ap.add_argument("--prompts", type=int, default=4)
    ap.add_argument("--width", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--prompt-length", type=int, default=24)
    a = ap.parse_args(argv)
    dims, weights = synth.Dims(a.shape), synth.make_weights(a.shape)
    ctx = rd.Rwkv7(dims, a.prompts * a.width)
    ctx.set_weights(weights)
    prompts = list(synth.prompt_tokens(dims.vocab, a.prompts, a.prompt_length))
    found, greedy = search(ctx, prompts, a.width, a.tokens)
    off, same = four_bit_head(weights, dims, a.prompts, a.width)
    ctx.close()
    return found, greedy, off, same


if __name__ == "__main__":
    main()
