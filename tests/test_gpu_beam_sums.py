"""Norms of rows whose chunks lie far apart: one value, or a few, well above a long flat rest, in
which each term weighs next to nothing and all of them together do.

Tolerance.  A row's norm is log sum exp(x - top).  With the weights w of the terms, an error of e in
the terms' logarithms is one of sum w e in the norm.  A term x of a chunk with the largest value c is
exp(x - c) exp(c - top): off by at most 2^-22 (two steps of the hardware's 2^x), 8e-8 (a polynomial), and
by |x - c| and |c - top| times 2^-24 for a rounded difference, 2^-24 for a rounded product and 1.3e-8
for its constant: at most 3.2e-7 + 1.33e-7 |x - top|.  The mean of |x - top| under the weights is
largest for n equal terms below one, where it is the u with 1 + u + log u = log n: 8.9 for 160,000
terms, 10.5 for 2^20.  3.2e-7 + 1.33e-7 * 10.5 < 2e-6 = NORM; each chunk's share is cut to 2^-40
besides, 8e-9 for 2^13 of them.  A score is off by that and half a step of fp32."""
import numpy as np
import pytest
import torch

import recurrent_decode_gb300 as rd
from _beam_reference import ranks, select

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
NORM = 2e-6


def check(x, scores, k):
    """Scores of the k best of one request; tokens and parents, whose ranks must lie further apart than NORM."""
    step = rd.beam_select(x, scores.cuda(), k)
    want = select(x.double().cpu().numpy(), scores.numpy(), k)
    assert step.tokens.tolist() == want[0].tolist() and step.parents.tolist() == want[1].tolist()
    off = np.abs(step.scores.double().cpu().numpy() - want[2])
    assert (off <= NORM + 2.0 ** -24 * np.abs(want[2])).all(), float(off.max())


# Rows a call are few (chunks of 2048 values) or enough for chunks of 8192.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,V", [(1, 65536), (20, 65536), (1, 159744), (8, 159744), (1, 30011), (40, 30011)])
@pytest.mark.parametrize("below", [12.0, 15.0, 17.85, 20.8, 21.49, 22.0])
def test_one_value_over_a_flat_rest(below, rows, V, dtype):
    x = torch.full((rows, V), -below, dtype=TYPES[dtype], device="cuda")
    for r in range(rows):
        x[r, 977 * r % V] = 0.0
    step = rd.beam_select(x, torch.zeros(rows, 1, device="cuda"), 2)
    rest = float(x[0, 1])
    norm = np.log1p((V - 1) * np.exp(rest))
    want = np.array([[-norm, rest - norm]])
    assert step.tokens.tolist() == [[977 * r % V, int(977 * r % V == 0)] for r in range(rows)]
    off = np.abs(step.scores.double().cpu().numpy() - want)
    assert (off <= NORM + 2.0 ** -24 * np.abs(want)).all(), float(off.max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 20])
def test_one_value_over_a_normal_rest(rows, dtype):
    g = torch.Generator()
    g.manual_seed(rows)
    x = (0.3 * torch.randn(rows, 65536, generator=g) - 15.0).to(TYPES[dtype])
    x[:, 40000] = 0.0
    x = x.cuda()
    step = rd.beam_select(x, torch.zeros(rows, 1, device="cuda"), 1)
    score = ranks(x.double().cpu().numpy(), np.zeros((rows, 1)))[0][:, 0, 40000]
    assert step.tokens.tolist() == [[40000]] * rows
    off = np.abs(step.scores.double().cpu().numpy()[:, 0] - score)
    assert (off <= NORM + 2.0 ** -24 * np.abs(score)).all(), float(off.max())


def test_values_far_apart_in_every_chunk():
    """Chunk tops on a ladder down from the row's, each over its own flat rest."""
    V = 131072
    x = torch.empty(1, V)
    for c in range(V // 2048):
        x[0, 2048 * c:2048 * (c + 1)] = -10.0 - 0.25 * c
        x[0, 2048 * c + 5 * c] = -0.5 * c
    check(x.cuda(), torch.tensor([[-1.0]]), 10)


@pytest.mark.parametrize("ahead", [1e-5, -1e-5])
def test_the_rest_decides_between_beams(ahead):
    """A beam's best is ahead of a certain one's, or behind it, by less than its rest weighs."""
    V = 65536
    x = torch.full((2, V), -17.85)
    x[0, 5] = 0.0
    x[1] = -float("inf")
    x[1, 9] = 3.0
    norm = float(np.log1p((V - 1) * np.exp(float(x[0, 0].double()))))
    scores = torch.tensor([[0.0, -norm - ahead]], dtype=torch.float32)
    assert abs(float(scores[0, 1].double()) + norm + ahead) < 1e-9
    check(x.cuda(), scores, 2)


def test_a_large_vocabulary():
    V = 1 << 20
    x = torch.full((1, V), -16.0, device="cuda")
    x[0, V - 1] = 0.0
    check(x, torch.tensor([[0.0]]), 3)
