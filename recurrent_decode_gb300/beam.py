"""Beam search over state slots (include/rwkv7.h): the selection of a request's best
continuations, the slots' states brought in line with it, and the loop of both around
the decode step.

Calls without a context run on the current stream of the device their tensors are on,
allocate outputs from torch's allocator on that stream, do not synchronise, and may be
captured into a graph.
"""
from __future__ import annotations

from functools import lru_cache
from typing import NamedTuple

import numpy as np
import torch

from . import EINVAL, RWKV7Error
from . import load_library as _library
from . import mx
from .mx import _call, _rows

MAX_WIDTH, MAX_K, MAX_SLOTS = 128, 128, 1024  # RWKV7_BEAM_MAX_*


_TICKETS, _ROOM = 4096, 2 << 20  # requests whose tickets are kept, and bytes of room


def _space(n: int, size: int, index: int):
    """(tensors that own it, address of `size` bytes of room, address of n tickets): words of
    zeros, which a selection leaves as zeros.  Kept for the next call of the same host thread
    on the same stream, as mx._room keeps its bytes; a graph, a stream that torch does not own
    and a large selection get memory of the call's own."""
    if n <= _TICKETS and size <= _ROOM and not mx._capturing(index):
        key = "beam", index, mx._raw_stream(index)
        kept = mx._kept.__dict__
        w = kept.get(key)
        if w is not None:
            return w
        stream = mx._stream_data(index)[0]
        if not stream or stream & 1:
            t = torch.zeros(4 * _TICKETS + _ROOM, dtype=torch.uint8, device=f"cuda:{index}")
            w = kept[key] = t, t.data_ptr() + 4 * _TICKETS, t.data_ptr()
            return w
    room = torch.empty(size, dtype=torch.uint8, device=f"cuda:{index}")
    tickets = torch.zeros(n, dtype=torch.int32, device=f"cuda:{index}")
    return (room, tickets), room.data_ptr(), tickets.data_ptr()


@lru_cache(256)
def _room_bytes(n: int, width: int, vocab: int, k: int) -> int:
    return _library().rwkv7_beam_room_bytes(n, width, vocab, k)


class BeamStep(NamedTuple):
    """What a selection found, [requests, k], best first; where a request has fewer
    candidates the rest is token -1, parent -1, score -inf, length 0, not ended."""
    tokens: torch.Tensor          # int32
    parents: torch.Tensor         # int32, a beam of the request
    scores: torch.Tensor          # float32, summed log-probabilities
    ended: torch.Tensor | None    # bool, with end_token
    lengths: torch.Tensor | None  # int32, with lengths


def _plain(t, dtype, shape, index, what):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != index:
        raise TypeError(f"{what} must be a contiguous {dtype} tensor on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{what} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def beam_select(logits, scores, k: int | None = None, *, ended=None, end_token: int | None = None, lengths=None,
                length_penalty: float = 0.0) -> BeamStep:
    """The k best continuations of each request by one token (rwkv7_beam_select).

    scores [requests, width] float32: the beams' summed log-probabilities, -inf for a
    beam that is not there; logits [requests * width, vocab] (float32, float16, bfloat16,
    any row stride): theirs.  k: how many, default width.  Candidate (beam, token) is ranked
    by (score + log-softmax of the beam's logits at token) / length**length_penalty, ties to
    the lowest beam, then token; NaN and infinite logits are no candidates.
    end_token: the token that ends a beam; ended [requests, width] bool: beams that have
    ended go on as themselves, with end_token and the score they have.  lengths [requests,
    width] int32: the beams' tokens so far, needed with a length_penalty (0 .. 16)."""
    rows, vocab, ld, code = _rows(logits, "logits")
    index = logits.get_device()
    if not isinstance(scores, torch.Tensor) or scores.dim() != 2:
        raise ValueError("scores must be a tensor [requests, width]")
    shape = n, width = scores.shape
    _plain(scores, torch.float32, shape, index, "scores")
    if rows != n * width:
        raise ValueError(f"{rows} rows of logits for {n} x {width} beams")
    if rows > mx._MAX_DIM or vocab > mx._MAX_DIM:
        raise RWKV7Error(EINVAL, f"{rows} beams of a vocabulary of {vocab}: at most 2^24 of both")
    if k is None:
        k = width
    if not 1 <= k <= MAX_K:
        raise RWKV7Error(EINVAL, f"k={k} is outside 1 .. {MAX_K}")
    if ended is not None:
        _plain(ended, torch.bool, shape, index, "ended")
        if end_token is None:
            raise ValueError("ended beams need an end_token")
    if end_token is not None and not 0 <= end_token < vocab:
        raise ValueError(f"end_token={end_token} is outside the vocabulary of {vocab}")
    if lengths is not None:
        _plain(lengths, torch.int32, shape, index, "lengths")
    elif length_penalty:
        raise ValueError("a length penalty needs the beams' lengths")
    # (no bytes for what the call refuses, saying why)
    own, room, zeros = _space(n, _room_bytes(n, width, vocab, k), index)
    # (An output each: views of one allocation take longer to make than allocations.)
    if k == width:
        sums = torch.empty_like(scores)
        tokens = torch.empty_like(scores if lengths is None else lengths, dtype=torch.int32)
        parents = torch.empty_like(tokens)
        after = None if lengths is None else torch.empty_like(tokens)
    else:
        size, device = (n, k), logits.device
        sums = torch.empty(size, dtype=torch.float32, device=device)
        tokens = torch.empty(size, dtype=torch.int32, device=device)
        parents = torch.empty_like(tokens)
        after = None if lengths is None else torch.empty_like(tokens)
    over = None if end_token is None else torch.empty_like(tokens, dtype=torch.bool)
    _call(_library().rwkv7_beam_select, index, logits.data_ptr(), code, ld, n, width, vocab, scores.data_ptr(),
          None if ended is None else ended.data_ptr(), -1 if end_token is None else end_token,
          None if lengths is None else lengths.data_ptr(), length_penalty, k, tokens.data_ptr(), parents.data_ptr(),
          sums.data_ptr(), None if after is None else after.data_ptr(), None if over is None else over.data_ptr(),
          room, zeros)
    return BeamStep(tokens, parents, sums, over, after)


def _beams(slots, parents, dev: torch.device):
    for what, t in (("slots", slots), ("parents", parents)):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_contiguous() \
                or t.get_device() != dev.index:
            raise TypeError(f"{what} must be a contiguous int32 tensor on {dev}")
    if slots.dim() != 2 or slots.shape != parents.shape:
        raise ValueError(f"slots and parents must be [requests, width] alike, got {tuple(slots.shape)} and "
                         f"{tuple(parents.shape)}")
    n, width = slots.shape
    if not 1 <= width <= MAX_WIDTH or n * width > MAX_SLOTS:
        raise ValueError(f"{n} requests of {width} beams: 1 to {MAX_WIDTH} beams a request and {MAX_SLOTS} in a call")
    return n, width


def _slots_out(slots):
    return torch.empty_like(slots)


def states_reorder(states, slots, parents):
    """Bring slots' states in line with a selection (rwkv7_states_reorder): beam j of a
    request goes on from the state of its beam parents[j] (-1: from any).  slots, parents:
    int32 [requests, width]; states: (wkv [L, n_slots, H, 64, 64], shift_att, shift_ffn
    [L, n_slots, 64 H]), changed in place.  Returns the beams' new slots: a parent's first
    child keeps its slot, the others take those of beams without children and a copy.
    A request with an index out of range, or a slot met twice in the call, is left as it
    was and its new slots are -1."""
    wkv, att, ffn = states
    if not isinstance(wkv, torch.Tensor) or not wkv.is_cuda:
        raise TypeError("wkv must be a CUDA tensor")
    dev = wkv.device
    for what, t in (("wkv", wkv), ("shift_att", att), ("shift_ffn", ffn)):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or not t.is_contiguous() or t.device != dev:
            raise TypeError(f"{what} must be a contiguous float32 tensor on {dev}")
    if wkv.dim() != 5 or wkv.shape[3:] != (64, 64):
        raise ValueError(f"wkv must be [L, slots, H, 64, 64], got {tuple(wkv.shape)}")
    L, n_slots, H = wkv.shape[:3]
    if att.shape != (L, n_slots, 64 * H) or ffn.shape != att.shape:
        raise ValueError(f"the token shifts must be [{L}, {n_slots}, {64 * H}]")
    n, width = _beams(slots, parents, dev)
    out = _slots_out(slots)
    _call(_library().rwkv7_states_reorder, dev.index, wkv.data_ptr(), att.data_ptr(), ffn.data_ptr(), L, H, n_slots,
          slots.data_ptr(), parents.data_ptr(), n, width, out.data_ptr())
    return out


def beam_search(ctx, prompts, width: int, n_out: int, *, end_token: int | None = None, length_penalty: float = 0.0,
                slots=None):
    """The `width` best continuations of each prompt by up to n_out tokens, best first:
    for each prompt a list of (score, tokens), tokens a numpy array that ends with end_token
    where the beam ended.  prompts: int32 arrays of at least one token.  A prompt's body is
    prefilled once into one slot; its beams' states are forked from there and moved with
    rwkv7_slots_reorder.  slots: the slots to use, width for each prompt (default: the
    context's first); what they held is lost, and they hold the last beams' states afterwards.

    Every step is decode_step, beam_select and slots_reorder on the context's stream; the
    host waits once, at the end."""
    n = len(prompts)
    if n < 1 or not 1 <= width <= MAX_WIDTH or n * width > MAX_SLOTS:
        raise ValueError(f"{n} prompts of {width} beams: at least one, 1 to {MAX_WIDTH} beams and {MAX_SLOTS} in all")
    V = ctx.dims.vocab
    if width > V:
        raise ValueError(f"{width} beams of a vocabulary of {V}")
    if n_out < 1:
        raise ValueError("n_out must be at least 1")
    prompts = [np.ascontiguousarray(p, np.int32) for p in prompts]
    if any(p.ndim != 1 or len(p) < 1 for p in prompts):
        raise ValueError("a prompt is a row of at least one token")
    slots = list(range(n * width)) if slots is None else [int(s) for s in slots]
    if len(slots) != n * width or len(set(slots)) != len(slots) or not all(0 <= s < ctx.n_slots for s in slots):
        raise ValueError(f"beam search of {n} prompts and {width} beams takes {n * width} different slots of the "
                         f"context's {ctx.n_slots}")
    dev = ctx.stream.device
    with torch.cuda.device(dev), torch.cuda.stream(ctx.stream):
        to_dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731
        at = to_dev(np.array(slots).reshape(n, width))
        for p, s in zip(prompts, slots[::width]):
            ctx.slot_reset(s)
            if len(p) > 1:
                ctx.prefill_seq(s, to_dev(p[:-1]))
        # The first token: a prompt is one beam, whose best continuations become the beams.
        logits = torch.empty(n * width, V, device=dev)
        ctx.decode_step(at[:, 0].contiguous(), to_dev([p[-1] for p in prompts]), logits[:n])
        lengths = torch.zeros(n, 1, dtype=torch.int32, device=dev)
        step = beam_select(logits[:n], torch.zeros(n, 1, device=dev), width, end_token=end_token, lengths=lengths,
                           length_penalty=length_penalty)
        steps = [step]
        at = ctx.slots_reorder(at, step.parents)
        for _ in range(n_out - 1):
            ctx.decode_step(at.view(-1), step.tokens.view(-1), logits)
            step = beam_select(logits, step.scores, ended=step.ended, end_token=end_token, lengths=step.lengths,
                               length_penalty=length_penalty)
            steps.append(step)
            at = ctx.slots_reorder(at, step.parents)
        tokens = torch.stack([s.tokens for s in steps]).cpu().numpy()
        parents = torch.stack([s.parents for s in steps]).cpu().numpy()
        scores, lengths = step.scores.cpu().numpy(), step.lengths.cpu().numpy()
    ctx.synchronize()
    found = []
    for r in range(n):
        beams = []
        for b in range(width):
            line, j = [], b
            for t in range(n_out - 1, -1, -1):
                line.append(tokens[t, r, j])
                j = parents[t, r, j]
            beams.append((float(scores[r, b]), np.array(line[::-1][:lengths[r, b]], np.int32)))
        found.append(beams)
    return found
