"""The microscaled operators against the plain 64-bit implementations of
_mx_reference.py: MXFP4 quantisation and its inverse, the product, and slot states
saved to and loaded from a cache.

Tolerances.  Codes and powers of two are exact, so quantised values must equal the
reference's.  A product's terms are exact in fp32 and their sum has at most K
additions, each off by at most 2^-23 of the running sum's bound S = sum |x w|
(a step of fp32, where an adder cuts instead of rounding): |sum error| <= K 2^-23 S.
relu(t)^2 turns an error d into at most 2 |t| d + d^2, and the result is rounded
once more, by half a step of its type."""
import numpy as np
import pytest
import torch

import recurrent_decode_gb300 as rd
import synth
from _harness import gpu_ctx
from _mx_reference import nearest

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def same(got, want):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def cpu(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ MXFP4 rows
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 32, 0), (3, 31, 0), (2, 33, 7), (1, 256, 0), (5, 257, 1),
                                           (128, 64, 0), (129, 40, 8), (7, 1000, 24), (131, 300, 3)])
def test_quantized_values(rows, cols, pad, dtype):
    x = (torch.randn(rows, cols + pad, generator=cpu(rows * cols)) * 3).to(TYPES[dtype])
    want = nearest(x[:, :cols].double().numpy(), "mxfp4")
    x = x.cuda()[:, :cols]
    m = rd.mx4_quantize(x)
    assert m.shape == (rows, cols)
    same(m.dequantize(), want)
    same(m.dequantize(TYPES[dtype]), want)  # few bits: exact in every type


@pytest.mark.parametrize("offset", [1, 2, 3, 5, 8])
def test_rows_at_any_address(offset):
    """Views that start and step off the 16-byte grid, for reading and writing."""
    base = torch.randn(40 * 77 + offset, generator=cpu(offset)).half().cuda()
    x = torch.as_strided(base, (40, 70), (77, 1), offset)
    m = rd.mx4_quantize(x)
    want = nearest(x.double().cpu().numpy(), "mxfp4")
    same(m.dequantize(), want)
    room = torch.full((40 * 77 + offset,), 9.0, device="cuda", dtype=torch.float16)
    out = torch.as_strided(room, (40, 70), (77, 1), offset)
    assert m.dequantize(out=out) is out
    same(out, want)
    room[offset:].view(40, 77)[:, :70] = 9.0
    assert bool((room == 9.0).all())  # nothing else was written


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(4000, 1280), (2500, 1300), (10001, 256), (3000, 1024)])
def test_many_rows_as_few(rows, cols, dtype):
    """Matrices large enough for several lines a warp, whole and ragged, against the
    reference on some rows and against the same rows quantised a few at a time."""
    x = (torch.randn(rows, cols, generator=cpu(rows)) * 5).to(TYPES[dtype])
    x[7, 9] = float("nan")
    y = rd.mx4_quantize(x.cuda()).dequantize(TYPES[dtype])
    some = [0, 1, 2, 3, 7, 8, 127, 128, 129, rows // 2, rows - 2, rows - 1]
    same(y[some], nearest(x[some].double().numpy(), "mxfp4"))
    parts = [rd.mx4_quantize(x[a:a + 800].cuda()).dequantize(TYPES[dtype]) for a in range(0, rows, 800)]
    assert torch.equal(torch.nan_to_num(y, 77.0), torch.nan_to_num(torch.cat(parts), 77.0))


def test_ties_and_signs():
    v = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    row = torch.tensor(v + [-t for t in v] + [0.0, -0.0] + [0.2499, 0.2501, 4.999, 5.001] + [0.0] * 10)
    x = torch.stack([row * 2.0 ** e for e in (-20, 0, 7, 100)]).cuda()
    want = nearest(x.double().cpu().numpy(), "mxfp4")
    same(rd.mx4_quantize(x).dequantize(), want)
    assert want[1, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]


@pytest.mark.parametrize("top", [1e-45, 1e-40, 1.1754942e-38, 1.1754944e-38, 4.7e-38, 7e-38, 7.1e-38, 1e-3,
                                 6.0, 6.0000005, 1e30, 2e38])
def test_range_of_powers(top):
    x = torch.randn(8, 64, generator=cpu(3)).clamp(-1, 1).double() * top
    x = x.float()
    x[:, 3] = top
    x[2] = 0
    want = nearest(x.double().numpy(), "mxfp4")
    same(rd.mx4_quantize(x.cuda()).dequantize(), want)


def test_no_number_in_a_block():
    x = torch.randn(4, 96, generator=cpu(4))
    x[0, 0], x[1, 40], x[2, 95] = float("nan"), float("inf"), float("-inf")
    m = rd.mx4_quantize(x.cuda())
    for dt in TYPES.values():
        bad = torch.isnan(m.dequantize(dt)).cpu()
        assert bad[0, :32].all() and bad[1, 32:64].all() and bad[2, 64:].all() and int(bad.sum()) == 96


def test_last_block_is_filled_with_zeros():
    """A short last block takes its power from its own values, not from what lies behind the row."""
    x = torch.full((3, 64), 1e6, device="cuda")
    x[:, :40] = 1.0
    same(rd.mx4_quantize(x[:, :40]).dequantize(), np.ones((3, 40)))


def test_no_rows():
    m = rd.mx4_quantize(torch.empty(0, 100, device="cuda"))
    assert m.dequantize().shape == (0, 100)
    w = rd.mx4_quantize(torch.ones(5, 100, device="cuda"))
    assert rd.mx4_linear(torch.empty(0, 100, device="cuda"), w).shape == (0, 5)


def test_fp16_range_is_kept_by_rounding():
    x = torch.tensor([[1e6, -1e-9] + [1.0] * 30], device="cuda")
    y = rd.mx4_quantize(x).dequantize(torch.float16)
    assert torch.isinf(y[0, 0]) and y[0, 1] == 0


# ------------------------------------------------------------------ the product
def product(xv, wv, act, dtype):
    """(result, how far a kernel's may be off) in 64 bits, of values xv [B, K], wv [N, K]."""
    t = xv @ wv.T
    d = xv.shape[1] * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T)
    if act == "relu2":
        d = 2 * np.abs(t) * d + d * d
        t = np.maximum(t, 0) ** 2
    return t, d + torch.finfo(dtype).eps / 2 * (np.abs(t) + d) + torch.finfo(dtype).tiny


def check_product(B, N, K, xt, yt, act, seed=0, x=None, strided=False):
    g = cpu(seed + B * 7 + N * 3 + K)
    if x is None:
        x = torch.randn(B, K, generator=g) * torch.exp(torch.randn(K, generator=g))
    w = torch.randn(N, K, generator=g) * 0.05
    x = x.to(TYPES[xt]).cuda()
    wq = rd.mx4_quantize(w.cuda())
    xv = rd.mx4_quantize(x).dequantize().double().cpu().numpy()
    wv = wq.dequantize().double().cpu().numpy()
    want, off = product(xv, wv, act, TYPES[yt])
    if strided:
        room = torch.full((B, N + 5), 3.0, dtype=TYPES[yt], device="cuda")
        y = rd.mx4_linear(x, wq, out=room[:, 2:N + 2], activation=act)
        assert bool((room[:, :2] == 3).all()) and bool((room[:, N + 2:] == 3).all())
    else:
        y = rd.mx4_linear(x, wq, out_dtype=TYPES[yt], activation=act)
    rd.mx4_check()
    assert y.dtype == TYPES[yt] and y.shape == (B, N)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= off).all(), f"worst {np.max(err / off):.3f} of the bound"
    return y


@pytest.mark.parametrize("B", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300])
def test_product_rows(B):
    check_product(B, 130, 320, "fp16", "fp32", None)


@pytest.mark.parametrize("K", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 511, 513, 1000, 2560, 5000])
def test_product_lengths(K):
    check_product(5, 70, K, "fp32", "fp32", None)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1337])
def test_product_outputs(N):
    check_product(3, N, 96, "bf16", "fp32", None)
    check_product(130, N, 288, "bf16", "fp16", "relu2")


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("yt", TYPES)
@pytest.mark.parametrize("act", [None, "relu2"])
def test_product_types(xt, yt, act):
    check_product(19, 200, 352, xt, yt, act)
    check_product(140, 200, 352, xt, yt, act, strided=True)


@pytest.mark.parametrize("B,N,K", [(1, 4096, 8192), (64, 256, 16384), (256, 640, 4096), (600, 2048, 1024), (1, 65536, 64)])
def test_product_shapes_of_a_model(B, N, K):
    check_product(B, N, K, "fp16", "fp32", None)
    check_product(B, N, K, "fp16", "bf16", "relu2")


@pytest.mark.parametrize("B,N,K", [(65, 100, 300), (80, 300, 2100), (191, 129, 600), (200, 4096, 260), (320, 200, 2048),
                                   (500, 128, 5000), (1000, 130, 520), (700, 20000, 64), (257, 19456, 256)])
def test_product_tiles_of_every_width(B, N, K):
    """Few and many tiles, tokens that end inside one, alone and over a cluster."""
    check_product(B, N, K, "bf16", "fp32", None)
    check_product(B, N, K, "fp32", "fp16", "relu2", strided=True)


@pytest.mark.parametrize("B", [3, 130])
def test_product_of_whole_numbers_is_exact(B):
    """Values on the grid with equal powers: every sum is a whole number of quarters
    below 2^24, which fp32 holds exactly in any order."""
    g = cpu(B)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    x = grid[torch.randint(0, 8, (B, 1024), generator=g)] * torch.sign(torch.randn(B, 1024, generator=g))
    w = grid[torch.randint(0, 8, (300, 1024), generator=g)] * torch.sign(torch.randn(300, 1024, generator=g))
    x[:, ::32], w[:, ::32] = 6.0, -6.0
    y = rd.mx4_linear(x.cuda(), rd.mx4_quantize(w.cuda()))
    assert torch.equal(y.cpu().double(), x.double() @ w.double().t())


def test_product_uses_each_blocks_own_powers():
    """Powers from 2^-40 to 2^40 over rows, columns and blocks, products of like size."""
    g = cpu(8)
    e = torch.randint(-40, 41, (1, 24), generator=g).repeat_interleave(32, 1).double()
    x = (torch.randn(70, 768, generator=g).double() * 2.0 ** e).float()
    w = (torch.randn(150, 768, generator=g).double() * 2.0 ** -e).float()
    wq, xq = rd.mx4_quantize(w.cuda()), rd.mx4_quantize(x.cuda())
    want, off = product(xq.dequantize().double().cpu().numpy(), wq.dequantize().double().cpu().numpy(), None, torch.float32)
    y = rd.mx4_linear(x.cuda(), wq)
    assert (np.abs(y.double().cpu().numpy() - want) <= off).all()
    assert torch.equal(rd.mx4_linear(xq, wq), y)  # quantised before or on the way: the same


@pytest.mark.parametrize("B", [4, 150])
def test_product_keeps_no_number_to_its_row_and_column(B):
    x = torch.randn(B, 300, generator=cpu(5))
    w = torch.randn(140, 300, generator=cpu(6))
    x[1, 290], w[133, 2] = float("inf"), float("nan")
    for act in (None, "relu2"):
        y = rd.mx4_linear(x.cuda(), rd.mx4_quantize(w.cuda()), activation=act)
        bad = torch.isnan(y).cpu()
        assert bad[1].all() and bad[:, 133].all() and int(bad.sum()) == B + 140 - 1


def test_zero_rows_give_zero():
    x = torch.zeros(9, 200, device="cuda")
    w = rd.mx4_quantize(torch.randn(64, 200, generator=cpu(11)).cuda())
    assert bool((rd.mx4_linear(x, w) == 0).all())
    w = rd.mx4_quantize(torch.zeros(64, 200, device="cuda"))
    assert bool((rd.mx4_linear(torch.ones(9, 200, device="cuda"), w) == 0).all())


def test_product_repeats_bit_for_bit():
    g = cpu(9)
    x = torch.randn(40, 4000, generator=g).cuda()
    w = rd.mx4_quantize(torch.randn(256, 4000, generator=g).cuda())
    a = rd.mx4_linear(x, w)
    for _ in range(5):
        assert torch.equal(rd.mx4_linear(x, w), a)


def test_product_on_its_own_stream_and_in_a_graph():
    g = cpu(10)
    x = torch.randn(12, 640, generator=g).half().cuda()
    w = rd.mx4_quantize(torch.randn(700, 640, generator=g).cuda())
    want = rd.mx4_linear(x, w)
    rd.mx4_check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = rd.mx4_linear(x, w)
    s.synchronize()
    assert torch.equal(got, want)
    other = torch.randn(12, 640, generator=g).half().cuda()
    fresh = rd.mx4_linear(other, w)
    held, out = x.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rd.mx4_linear(held, w, out=out)
    held.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fresh)


def test_products_of_two_threads():
    """Two host threads on one stream and on streams of their own: each keeps its own
    rows on the way through the product."""
    import threading
    w = rd.mx4_quantize(torch.randn(300, 900, generator=cpu(12)).cuda())
    xs = [torch.randn(40, 900, generator=cpu(20 + i)).cuda() for i in range(2)]
    want = [rd.mx4_linear(x, w) for x in xs]
    torch.cuda.synchronize()
    for streams in ([torch.cuda.current_stream()] * 2, [torch.cuda.Stream(), torch.cuda.Stream()]):
        wrong = []

        def work(i):
            with torch.cuda.stream(streams[i]):
                for _ in range(200):
                    y = rd.mx4_linear(xs[i], w)
                streams[i].synchronize()
                if not torch.equal(y, want[i]):
                    wrong.append(i)
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not wrong


def test_a_wait_that_gave_up_is_reported_once():
    """The word that the kernel sets when a wait runs out, set here by the host."""
    from recurrent_decode_gb300 import mx
    x = torch.ones(2, 64, device="cuda")
    w = rd.mx4_quantize(x)
    rd.mx4_linear(x, w)
    mx._err_word(torch.cuda.current_device()).fill_(8)
    with pytest.raises(rd.RWKV7Error) as e:
        rd.mx4_check()
    assert e.value.code == rd.ETIMEOUT
    rd.mx4_check()


def test_rows_and_states_on_a_stream_and_in_a_graph():
    x = torch.randn(9, 500, generator=cpu(13)).cuda()
    st = tuple(t.cuda() for t in pool(1, 3, 2, 14))
    cache = rd.StateCache(1, 2, 1, "mxint8")
    m, out = rd.mx4_empty(9, 500, x.device), torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rd.mx4_quantize(x, out=m).dequantize(out=out)
        cache.save(st, ints(0), ints(0))
        cache.load(st, ints(0), ints(1))
    s.synchronize()
    same(out, nearest(x.double().cpu().numpy(), "mxfp4"))
    want = nearest(st[0][:, 0].double().cpu().numpy(), "mxint8")
    same(st[0][:, 1], want)
    a, b, c = ints(0), ints(1), ints(2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rd.mx4_quantize(x, out=m).dequantize(out=out)
        cache.save(st, b, a)
        cache.load(st, a, c)
    x.mul_(-3)
    st[0][:, 1].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    cache.check()
    same(out, nearest(x.double().cpu().numpy(), "mxfp4"))
    same(st[0][:, 2], 2 * want)


def test_binding_refusals():
    w = rd.mx4_quantize(torch.ones(8, 64, device="cuda"))
    x = torch.ones(2, 64, device="cuda")
    for bad, what in ((x.double(), TypeError), (x.int(), TypeError), (x[0], ValueError), (x.t(), ValueError),
                      (x.cpu(), TypeError), (x[:, :1].expand(2, 64), ValueError)):
        with pytest.raises(what):
            rd.mx4_quantize(bad)
        with pytest.raises(what):
            rd.mx4_linear(bad, w)
    with pytest.raises(ValueError, match="columns"):
        rd.mx4_linear(torch.ones(2, 65, device="cuda"), w)
    with pytest.raises(ValueError, match="activation"):
        rd.mx4_linear(x, w, activation="gelu")
    with pytest.raises(ValueError):
        rd.mx4_linear(x, w, out=torch.empty(2, 9, device="cuda"))
    with pytest.raises(ValueError):
        rd.mx4_linear(x, w, out=torch.empty(1, 8, device="cuda").expand(2, 8))
    with pytest.raises(TypeError):
        rd.mx4_linear(x, w, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        rd.mx4_quantize(x, out=w)
    with pytest.raises(ValueError, match="bytes"):
        rd.MX4Matrix(w.data[:-16], 8, 64)
    with pytest.raises(TypeError):
        rd.MX4Matrix(w.data.cpu(), 8, 64)
    with pytest.raises(TypeError):
        rd.StateCache(1, 1, 1, device="cpu")


# ------------------------------------------------------------------ states
def pool(L, n, H, seed):
    g = cpu(seed)
    return (torch.randn(L, n, H, 64, 64, generator=g) * torch.exp(2 * torch.randn(L, n, H, 1, 1, generator=g)),
            torch.randn(L, n, 64 * H, generator=g), torch.randn(L, n, 64 * H, generator=g))


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", ["mxint8", "mxfp4"])
@pytest.mark.parametrize("L,n,H", [(1, 3, 1), (2, 5, 3)])
def test_states_move_through_the_cache(fmt, L, n, H):
    host = pool(L, n, H, n)
    host[0][0, 1] = 0
    host[0][0, 0, 0, 5, 7] = float("nan")
    host[0][-1, 0, -1, 9, 40] = float("-inf")
    host[0][0, 0, 0, 6, :32] *= 1e-40
    host[0][0, 0, 0, 7, 32:] = torch.finfo(torch.float32).max  # 4 * 2^126 in MXFP4: infinity in fp32
    st = tuple(t.cuda() for t in host)
    cache = rd.StateCache(L, H, 4, fmt)
    cache.data.fill_(0xAB)
    cache.save(st, ints(0, 1), ints(3, 1))
    cache.check()
    for a, b in zip(st, host):
        assert torch.equal(torch.nan_to_num(a.cpu()), torch.nan_to_num(b))  # saving changes no state
    rows = cache.data.view(4, -1)
    assert bool((rows[0] == 0xAB).all()) and bool((rows[2] == 0xAB).all())  # nor another entry
    cache.load(st, ints(3, 1), ints(n - 1, 0))
    cache.check()
    for to, src in ((n - 1, 0), (0, 1)):
        with np.errstate(over="ignore"):
            same(st[0][:, to], nearest(host[0][:, src].double().numpy(), fmt).astype(np.float32).astype(np.float64))
        assert torch.equal(st[1][:, to].cpu(), host[1][:, src]) and torch.equal(st[2][:, to].cpu(), host[2][:, src])
    for k in range(1, n - 1):  # the slots between keep theirs
        assert all(torch.equal(a[:, k].cpu(), b[:, k]) for a, b in zip(st, host))


@pytest.mark.parametrize("fmt", ["mxint8", "mxfp4"])
def test_state_error_is_half_a_step_of_its_block(fmt):
    """MXINT8: half of 2^e/64 with max > 127/128 2^e, within max/126.  MXFP4: half of
    at most 2 * 2^e with max > 3 * 2^e: within max/3."""
    st = tuple(t.cuda() for t in pool(2, 2, 2, 77))
    before = st[0][:, 0].clone()
    cache = rd.StateCache(2, 2, 1, fmt)
    cache.save(st, ints(0), ints(0))
    cache.load(st, ints(0), ints(1))
    d = (st[0][:, 1] - before).view(-1, 32).abs().amax(1)
    top = before.view(-1, 32).abs().amax(1)
    assert bool((d <= top / (126 if fmt == "mxint8" else 3)).all())


@pytest.mark.parametrize("fmt", ["mxint8", "mxfp4"])
def test_one_entry_for_many_slots_and_none(fmt):
    st = tuple(t.cuda() for t in pool(2, 12, 2, 5))
    cache = rd.StateCache(2, 2, 2, fmt)
    cache.save(st, ints(4), ints(1))
    before = tuple(t.clone() for t in st)
    cache.load(st, ints(), ints())
    assert all(torch.equal(a, b) for a, b in zip(st, before))
    cache.load(st, ints(*[1] * 11), ints(*[k for k in range(12) if k != 4]))
    cache.check()
    assert all(torch.equal(st[0][:, k], st[0][:, 0]) for k in range(12) if k != 4)
    assert torch.equal(st[0][:, 4], before[0][:, 4])
    again = tuple(t.clone() for t in st)  # a state read back stands for itself
    cache.save(st, ints(0), ints(0))
    cache.load(st, ints(0), ints(4))
    assert torch.equal(st[0][:, 4], again[0][:, 0])


def test_bad_and_repeated_indices_are_left_out_and_reported():
    host = pool(1, 6, 1, 6)
    st = tuple(t.cuda() for t in host)
    cache = rd.StateCache(1, 1, 3)
    cache.data.zero_()
    cache.save(st, ints(0, 6, -1, 2), ints(0, 1, 1, 3))  # only the first pair is good
    with pytest.raises(rd.RWKV7Error) as e:
        cache.check()
    assert e.value.code == rd.EINVAL and "0x1" in str(e.value)
    cache.check()  # reported once
    assert bool((cache.data.view(3, -1)[1:] == 0).all())
    cache.save(st, ints(1, 2, 3), ints(1, 2, 1))  # entry 1 twice: slot 1 stays
    with pytest.raises(rd.RWKV7Error, match="0x4"):
        cache.check()
    cache.load(st, ints(1, 2, 0), ints(5, 4, 5))
    with pytest.raises(rd.RWKV7Error, match="0x4"):
        cache.check()
    same(st[0][:, 5], nearest(host[0][:, 1].double().numpy(), "mxint8"))
    same(st[0][:, 4], nearest(host[0][:, 2].double().numpy(), "mxint8"))


def test_many_pairs_in_one_call():
    st = tuple(t.cuda() for t in pool(1, 1024, 1, 8))
    before = st[0].clone()
    cache = rd.StateCache(1, 1, 1024, "mxint8")
    perm = torch.randperm(1024, generator=cpu(1)).to(torch.int32).cuda()
    all_ = torch.arange(1024, dtype=torch.int32, device="cuda")
    cache.save(st, all_, perm)
    cache.load(st, perm, all_)
    cache.check()
    once = st[0].clone()
    assert float((once - before).abs().max()) > 0
    cache.save(st, all_, perm)
    cache.load(st, perm, all_)
    assert torch.equal(st[0], once)
    with pytest.raises(rd.RWKV7Error, match="pairs"):
        cache.save(st, torch.zeros(1025, dtype=torch.int32, device="cuda"), torch.zeros(1025, dtype=torch.int32, device="cuda"))


def test_state_binding_refusals():
    st = tuple(t.cuda() for t in pool(2, 3, 2, 9))
    cache = rd.StateCache(2, 2, 2)
    with pytest.raises(TypeError):
        cache.save((st[0].half(), st[1], st[2]), ints(0), ints(0))
    with pytest.raises(TypeError):
        cache.save((st[0].transpose(3, 4), st[1], st[2]), ints(0), ints(0))
    with pytest.raises(ValueError):
        cache.save((st[0][:1], st[1], st[2]), ints(0), ints(0))
    with pytest.raises(ValueError):
        cache.save((st[0], st[1][:, :2].contiguous(), st[2]), ints(0), ints(0))
    with pytest.raises(ValueError):
        cache.save(st, ints(0, 1), ints(0))
    with pytest.raises(TypeError):
        cache.load(st, ints(0).long(), ints(0))


@pytest.mark.parametrize("fmt", ["mxint8", "mxfp4"])
def test_slots_of_a_context(fmt):
    """A slot of the library's pool through the cache: its state is the quantised
    one, and its occurrence counts and draws restart as with slot_copy."""
    ctx, _, dims = gpu_ctx("tiny", 4)
    prompts = synth.prompt_tokens(dims.vocab, 2, 9)
    for s in range(2):
        ctx.prefill_seq(s, torch.from_numpy(prompts[s].copy()).cuda())
    before = [ctx.get_state(s) for s in range(2)]
    cache = rd.StateCache(dims.n_layer, dims.n_head, 3, fmt)
    ctx.slots_save(cache, ints(0, 1), ints(2, 0))
    for k in (2, 3):  # draws that the load has to make undone
        ctx.set_sampling(k, temperature=1.0, top_p=0.9, seed=5)
    logits = torch.randn(2, dims.vocab, generator=cpu(3)).cuda()
    first, second = ints(0, 0), ints(0, 0)
    ctx.sample_batch(ints(2, 3), logits, first)
    ctx.slots_load(cache, ints(2, 0), ints(3, 2))
    ctx.sample_batch(ints(2, 3), logits, second)
    ctx.synchronize()
    assert torch.equal(first, second)
    for to, src in ((3, 0), (2, 1)):
        got = ctx.get_state(to)
        assert np.array_equal(got[0].astype(np.float64), nearest(before[src][0], fmt))
        assert np.array_equal(got[1], before[src][1]) and np.array_equal(got[2], before[src][2])
    ctx.slots_save(cache, ints(4), ints(0))
    with pytest.raises(rd.RWKV7Error) as e:
        ctx.synchronize()
    assert e.value.code == rd.EINVAL
    ctx.synchronize()
    with pytest.raises(ValueError):
        ctx.slots_save(rd.StateCache(dims.n_layer + 1, dims.n_head, 3, fmt), ints(0), ints(0))
    with pytest.raises(rd.RWKV7Error):
        rd.Rwkv7._check(ctx, ctx.lib.rwkv7_slots_save(ctx.h, None, None, 1, cache.data.data_ptr(), 3, 1))
    ctx.close()


@pytest.mark.parametrize("fmt", ["mxint8", "mxfp4"])
def test_packed_prefix_cache(fmt):
    """The prefix cache over packed entries: the longest stored prefix comes back as its
    quantised state, the least recently used entry goes first."""
    from recurrent_decode_gb300.prefix_cache import PackedPrefixStateCache
    ctx, _, dims = gpu_ctx("tiny", 3)
    cache = PackedPrefixStateCache(ctx, 2, fmt, block=8)
    dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    body = synth.prompt_tokens(dims.vocab, 1, 12)[0]
    assert cache.restore(body, 1) == 0
    assert cache.prefill(0, body, 0, dev) == 12  # stored at 8 and at 12
    at12 = ctx.get_state(0)
    assert len(cache) == 2 and cache.restore(body, 1) == 12
    got = ctx.get_state(1)
    assert np.array_equal(got[0].astype(np.float64), nearest(at12[0], fmt))
    assert np.array_equal(got[1], at12[1]) and np.array_equal(got[2], at12[2])
    other = np.concatenate([body[:9], body[:1]])
    assert cache.restore(other, 2) == 8
    cache.store(other, 2)  # evicts the entry after 12 tokens
    assert cache.evictions == 1 and cache.restore(body, 1) == 8
    ctx.synchronize()
    ctx.close()


def test_slots_of_a_context_on_its_own_stream():
    dims = synth.Dims("tiny")
    s = torch.cuda.Stream()
    ctx = rd.Rwkv7(dims, 2, stream=s)
    state = [torch.randn(*a.shape, generator=cpu(30 + i)).numpy() for i, a in enumerate(ctx.get_state(0))]
    cache = rd.StateCache(dims.n_layer, dims.n_head, 1, "mxint8")
    zero, one = ints(0), ints(1)
    torch.cuda.synchronize()
    for _ in range(20):
        ctx.set_state(0, *state)
        ctx.slot_reset(1)
        ctx.slots_save(cache, zero, zero)
        ctx.slots_load(cache, zero, one)
        got = ctx.get_state(1)
        assert np.array_equal(got[0].astype(np.float64), nearest(state[0], "mxint8")) and np.array_equal(got[1], state[1])
        state[0] *= 2
    ctx.synchronize()
    ctx.close()


def test_example_runs():
    """The example on the tiny shape.  Rounding to MXFP4 is off by at most a fifth of a
    value past the block's smallest steps and by a third of the block's largest in all;
    independent errors of that size in both operands stay below 0.35 of a random sum, and
    two products in a row below 0.6.  The states are 1/126 and a third of a block's
    largest off, and the logits take them through one token."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import microscaled
    r = microscaled.main(["--shape", "tiny", "--slots", "3", "--prefix", "40"])
    assert 0 < r["mxint8"] < 0.01 and r["mxint8"] < r["mxfp4"] < 0.35
    assert 0 < r["head"] < 0.35 and 0 < r["channel mix"] < 0.6


@pytest.mark.parametrize("B,N,K", [(1, 300, 1), (1, 70, 5000), (2, 2560, 2560), (3, 129, 4100), (5, 200, 3333), (7, 96, 2048),
                                   (9, 1000, 700), (16, 640, 1024), (16, 640, 1100), (16, 20000, 1024), (16, 20000, 1300),
                                   (4, 20000, 4096), (4, 20000, 4200)])
def test_product_of_few_rows_quantised_on_the_way(B, N, K):
    """Up to sixteen rows go through the product's own quantisation or through the
    kernel before it, as their length has it: to the same bits."""
    g = cpu(B + N + K)
    w = rd.mx4_quantize((torch.randn(N, K, generator=g) * 0.05).cuda())
    for dt in TYPES.values():
        wide = (torch.randn(B, K + 3, generator=g) * torch.exp(torch.randn(K + 3, generator=g))).to(dt).cuda()
        for x in (wide[:, :K].contiguous(), wide[:, 3:]):  # on the 16-byte grid (where K is) and off it
            y = rd.mx4_linear(x, w, out_dtype=torch.float32)
            rd.mx4_check()
            assert torch.equal(y, rd.mx4_linear(rd.mx4_quantize(x), w))
    check_product(B, N, K, "bf16", "fp32", None)
    check_product(B, N, K, "fp32", "fp16", "relu2", strided=True)


def test_few_rows_keep_no_number_to_their_block():
    x = torch.randn(3, 300, generator=cpu(5))
    x[1, 290], x[2, 0] = float("inf"), float("nan")
    y = rd.mx4_linear(x.half().cuda(), rd.mx4_quantize(torch.randn(140, 300, generator=cpu(6)).cuda()))
    assert bool(torch.isnan(y[1:]).all()) and bool(torch.isfinite(y[0]).all())


# ------------------------------------------------------------------ far places
def test_matrix_past_32_bits():
    """Rows past 2^32 elements, codes past 2^32 bytes: the last rows of 70,000 x 131,072
    come back as those of a small matrix do."""
    R, K = 70000, 131072
    x = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    x[:64] = 1.0
    x[-130:] = torch.randn(130, K, generator=cpu(1)).cuda()
    m = rd.mx4_quantize(x)
    assert m.data.numel() > 1 << 32
    small = rd.mx4_quantize(x[-130:])
    want = small.dequantize(torch.bfloat16)
    tail = x[-130:].clone()
    del x
    y = m.dequantize(torch.bfloat16)
    assert torch.equal(y[-130:], want) and bool((y[:64] == 1).all())
    del y
    got = rd.mx4_linear(tail[:3, :], m, out_dtype=torch.float32)[:, -130:]
    rd.mx4_check()
    v = small.dequantize().double().cpu().numpy()
    want, off = product(v[:3], v, None, torch.float32)
    assert (np.abs(got.double().cpu().numpy() - want) <= off).all()


@pytest.mark.parametrize("fmt", ["mxint8", "mxfp4"])
def test_entries_and_slots_past_32_bits(fmt):
    """A pool and a cache of more than 2^32 bytes: the last slots and entries."""
    L, H, n = 4, 64, 1100  # 4.6 GB of states a layer
    cache = rd.StateCache(L, H, (1 << 32) // rd.StateCache(L, H, 1, fmt).entry_bytes + 2, fmt)
    st = (torch.zeros(L, n, H, 64, 64, device="cuda"), torch.zeros(L, n, 64 * H, device="cuda"), torch.zeros(L, n, 64 * H, device="cuda"))
    st[0][:, n - 1] = torch.randn(L, H, 64, 64, generator=cpu(2)).cuda()
    st[1][:, n - 1], st[2][:, n - 1] = 3.0, 4.0
    last = cache.n_entries - 1
    cache.save(st, ints(n - 1), ints(last))
    cache.load(st, ints(last, last), ints(0, n - 2))
    cache.check()
    want = nearest(st[0][-1, n - 1, -1].double().cpu().numpy(), fmt)
    same(st[0][-1, n - 2, -1], want)
    same(st[0][-1, 0, -1], want)
    assert bool((st[1][:, n - 2] == 3).all()) and bool((st[2][:, 0] == 4).all()) and bool((st[0][:, 1:n - 2] == 0).all())
