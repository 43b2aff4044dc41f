"""Equal beams: rows that are alike value for value, at any stride and any place between 16-byte
boundaries, have the same candidates with the same ranks, so that the order is that of the beams."""
import pytest
import torch

import recurrent_decode_gb300 as rd

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def rows(V, seed, scale=2.5):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(1, V, generator=g) * scale


# Vocabularies of one chunk and several, whole and not; few rows (chunks of 2048) and many (8192).
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,W,V", [(1, 8, 1), (1, 8, 11), (2, 8, 2041), (1, 5, 2048), (3, 4, 2049), (1, 8, 30011),
                                   (40, 8, 8191), (40, 8, 8193), (10, 8, 30011), (2, 16, 65537)])
def test_equal_beams_go_by_place(G, W, V, dtype):
    for pad in (0, 1, 3, 6):
        x = torch.zeros(G * W, V + pad, dtype=TYPES[dtype], device="cuda")[:, :V]
        one = rows(V, V + pad).to(TYPES[dtype])
        x.copy_(one)
        step = rd.beam_select(x, torch.full((G, W), -3.0, device="cuda"), W + 2)
        order = torch.sort(one[0].double(), descending=True, stable=True)[1].tolist()
        # by value, then beam, then token
        want = [(b, v) for _, b, v in sorted((-float(one[0, v]), b, v) for v in order[:W + 2] for b in range(W))][:W + 2]
        want += [(-1, -1)] * (W + 2 - len(want))
        for g in range(G):
            assert list(zip(step.parents[g].tolist(), step.tokens[g].tolist())) == want
        assert bool((step.scores[:, :W] == step.scores[0, 0]).all())


def on_grid(x):
    """The same rows, all on 16-byte boundaries."""
    n, V = x.shape
    return torch.zeros(n, V + 7 & ~7, dtype=x.dtype, device="cuda")[:, :V].copy_(x)


def everywhere(x, pads):
    """The same rows at every offset and some strides, among values that would be chosen."""
    n, V = x.shape
    for off in range(16 // x.element_size()):
        for pad in pads:
            room = torch.full((n * (V + pad) + off + 8,), 90.0, dtype=x.dtype, device="cuda")
            yield torch.as_strided(room, (n, V), (V + pad, 1), off).copy_(x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V", [(3, 5000), (24, 30011), (3, 8200)])
def test_strides_change_nothing(n, V, dtype):
    """Bit for bit the same step wherever the rows lie."""
    x = torch.cat([rows(V, s) for s in range(n)]).to(TYPES[dtype]).cuda()
    scores = torch.linspace(-1, 0, n, device="cuda").view(1, n)
    want = rd.beam_select(on_grid(x), scores, 20)
    for y in everywhere(x, (0, 1, 2)):
        assert all(torch.equal(a, b) for a, b in zip(rd.beam_select(y, scores, 20)[:3], want[:3]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [2, 160])
def test_ends_of_rows(n, dtype):
    """The best value first or last of a row, in vectors and chunks of all lengths."""
    for V in (*range(1, 19), 255, 257, 2047, 2048, 2049, 2050, 8191, 8192, 8193, 8197):
        x = torch.cat([rows(V, 1)] * n).to(TYPES[dtype])
        x[0::2, 0], x[1::2, V - 1] = 20.0, 20.0
        scores = torch.zeros(n, 1, device="cuda")
        want = rd.beam_select(on_grid(x.cuda()), scores, 3)
        assert want.tokens[:, 0].tolist() == [0, V - 1] * (n // 2)
        for y in everywhere(x.cuda(), (0, 1)):
            assert all(torch.equal(a, b) for a, b in zip(rd.beam_select(y, scores, 3)[:3], want[:3]))
