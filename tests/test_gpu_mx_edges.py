"""The microscaled operators where a call goes wrong beside its values: repeated and
bad indices, entries that nothing was saved to, tensors and graphs on other streams,
results over their inputs, powers at the ends of their range."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import recurrent_decode_gb300 as rd
import synth
from _mx_reference import nearest
from test_gpu_mx import cpu, ints, pool, product, same

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ indices
@pytest.mark.parametrize("first", [3, -1])
def test_a_pair_left_out_repeats_nothing(first):
    """A pair with a bad index writes nothing, so the next one with its target is the
    first: entry 0 gets slot 2's state, slot 1 entry 0's."""
    host = pool(2, 3, 2, 31)
    st = tuple(t.cuda() for t in host)
    cache = rd.StateCache(2, 2, 2)
    cache.data.fill_(0xAB)
    cache.save(st, ints(first, 2, first, 0), ints(0, 0, 1, 1))
    with pytest.raises(rd.RWKV7Error, match="0x1"):
        cache.check()
    want = [nearest(host[0][:, s].double().numpy(), "mxint8") for s in (2, 0)]
    cache.load(st, ints(5, 0, -2, 1), ints(1, 1, 0, 0))
    with pytest.raises(rd.RWKV7Error, match="0x1"):
        cache.check()
    same(st[0][:, 1], want[0])
    same(st[0][:, 0], want[1])
    assert torch.equal(st[1][:, 1].cpu(), host[1][:, 2]) and torch.equal(st[2][:, 0].cpu(), host[2][:, 0])


def test_of_good_bad_and_good_the_first_good_is_carried_out():
    host = pool(1, 4, 1, 32)
    st = tuple(t.cuda() for t in host)
    cache = rd.StateCache(1, 1, 2)
    cache.save(st, ints(1, 4, 2), ints(0, 0, 0))
    with pytest.raises(rd.RWKV7Error, match="0x5"):
        cache.check()
    cache.save(st, ints(2), ints(1))
    cache.load(st, ints(0, 2, 1), ints(3, 3, 3))
    with pytest.raises(rd.RWKV7Error, match="0x5"):
        cache.check()
    same(st[0][:, 3], nearest(host[0][:, 1].double().numpy(), "mxint8"))


@pytest.mark.parametrize("fmt", ["mxint8", "mxfp4"])
def test_an_entry_never_saved_is_a_fresh_state(fmt):
    size = rd.StateCache(2, 2, 3, fmt).data.numel()
    torch.full((size,), 0x5B, dtype=torch.uint8, device="cuda")  # what the allocator may hand out next
    cache = rd.StateCache(2, 2, 3, fmt)
    st = tuple(t.cuda() for t in pool(2, 3, 2, 33))
    kept = tuple(t[:, 1].clone() for t in st)
    cache.load(st, ints(0, 2), ints(2, 0))
    cache.check()
    for t, k in zip(st, kept):
        assert bool((t[:, 0] == 0).all()) and bool((t[:, 2] == 0).all()) and torch.equal(t[:, 1], k)


# ------------------------------------------------------------------ streams
@pytest.fixture
def own_stream():
    """A context of four slots on a stream of its own, each with its own state."""
    dims = synth.Dims("tiny")
    ctx = rd.Rwkv7(dims, 4, stream=torch.cuda.Stream())
    states = [[torch.randn(*a.shape, generator=cpu(40 + s)).numpy() for a in ctx.get_state(0)] for s in range(4)]
    for s in range(4):
        ctx.set_state(s, *states[s])
    torch.cuda.synchronize()
    yield ctx, dims, states
    ctx.synchronize()
    ctx.close()


def filled(v):
    """An index that a kernel of the current stream writes (no copy, which would wait)."""
    return torch.full((1,), v, dtype=torch.int32, device="cuda")


SOME_MS = 100_000_000  # clock ticks: 50 ms


def test_indices_of_a_busy_stream_are_read_after_they_are_written(own_stream):
    ctx, dims, states = own_stream
    cache = rd.StateCache(dims.n_layer, dims.n_head, 2)
    torch.cuda._sleep(SOME_MS)
    ctx.slots_save(cache, filled(2), filled(1))
    torch.cuda._sleep(SOME_MS)
    ctx.slots_load(cache, filled(1), filled(3))
    ctx.synchronize()
    got = ctx.get_state(3)
    same(torch.from_numpy(got[0]), nearest(states[2][0], "mxint8"))
    assert (got[1] == states[2][1]).all()


def test_indices_and_cache_may_be_dropped_at_once(own_stream):
    """Their memory is not handed out again while the context's stream has yet to read it."""
    ctx, dims, states = own_stream
    cache = rd.StateCache(dims.n_layer, dims.n_head, 2)
    size = cache.data.numel()
    with torch.cuda.stream(ctx.stream):
        torch.cuda._sleep(SOME_MS)
    ctx.slots_save(cache, filled(2), filled(1))
    others = [filled(0) for _ in range(8)]  # valid ones, in the memory of those if it were free
    ctx.slots_load(cache, filled(1), filled(3))
    others += [filled(0) for _ in range(8)]
    del cache
    others.append(torch.full((size,), 0x33, dtype=torch.uint8, device="cuda"))
    ctx.synchronize()
    got = ctx.get_state(3)
    same(torch.from_numpy(got[0]), nearest(states[2][0], "mxint8"))
    assert (got[2] == states[2][2]).all()
    assert (ctx.get_state(0)[0] == states[0][0]).all()


# ------------------------------------------------------------------ graphs
def fresh_process(code):
    """What a new process prints that runs `code` after the imports."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", "import torch\nimport recurrent_decode_gb300 as rd\n" + code],
                       cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.split()


def test_first_product_of_a_process_is_captured():
    assert fresh_process("""
x, out = torch.ones(12, 640, device="cuda"), torch.empty(12, 70, device="cuda")
w = rd.mx4_quantize(torch.ones(70, 640, device="cuda"))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    rd.mx4_linear(x, w, out=out)
out.zero_()
g.replay()
rd.mx4_check()
print(bool((out == 640).all()))
""") == ["True"]


def test_a_first_matrix_in_a_capture_refuses_the_product_and_leaves_the_capture():
    assert fresh_process("""
x, v, out = torch.ones(12, 640, device="cuda"), torch.ones(70, 640, device="cuda"), torch.empty(70, 640, device="cuda")
rd.load_library()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    w = rd.mx4_quantize(v)
    try:
        rd.mx4_linear(x, w)
    except rd.RWKV7Error as e:
        print(e.code == rd.ESTATE)
    w.dequantize(out=out)
g.replay()
print(bool((out == 1).all()), bool((rd.mx4_linear(x, rd.mx4_quantize(v)) == 640).all()))
rd.mx4_check()
""") == ["True", "True", "True"]


def test_a_cache_made_in_inference_mode_is_checked_outside():
    with torch.inference_mode():
        cache = rd.StateCache(1, 1, 1)
        cache.save(tuple(t.cuda() for t in pool(1, 1, 1, 34)), ints(0), ints(1))
    with pytest.raises(rd.RWKV7Error):
        cache.check()
    cache.check()


# ------------------------------------------------------------------ results over their inputs
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("B,K", [(1, 700), (3, 2560), (16, 640), (16, 2560), (17, 640), (130, 640)])
def test_a_product_over_its_own_rows(B, K, dtype):
    """out = x, out shifted against x in one buffer, and rows of a different step: as
    into memory of its own, whether few rows or many."""
    w = rd.mx4_quantize((torch.randn(K, K, generator=cpu(K)) * 0.05).cuda())
    x = torch.randn(B, K, generator=cpu(B)).to(dtype).cuda()
    want = rd.mx4_linear(x, w, activation="relu2")
    for shift, step in ((0, K), (8, K), (5, K), (3, K + 9)):
        flat = torch.zeros(B * (K + 9) + 64, dtype=dtype, device="cuda")
        rows, out = torch.as_strided(flat, (B, K), (K, 1), 0), torch.as_strided(flat, (B, K), (step, 1), shift)
        rows.copy_(x)
        assert torch.equal(rd.mx4_linear(rows, w, out=out, activation="relu2"), want)
    rd.mx4_check()


@pytest.mark.parametrize("B", [1, 4, 16, 40])
def test_a_product_beside_its_rows_in_one_buffer(B):
    w = rd.mx4_quantize(torch.randn(96, 300, generator=cpu(1)).cuda())
    both = torch.randn(B, 500, generator=cpu(B)).cuda()
    x = both[:, 7:307].clone()
    want = rd.mx4_linear(x, w)
    assert torch.equal(rd.mx4_linear(both[:, 7:307], w, out=both[:, 307:403]), want)
    assert torch.equal(both[:, 7:307], x)


def test_a_product_may_write_between_and_around_its_matrices():
    """Rows of y 32 KB apart with the matrices between them; over them it is refused."""
    flat = torch.zeros(6 << 15, dtype=torch.uint8, device="cuda")
    at = lambda k: flat[(k << 15) + 64:][:17408]  # noqa: E731
    x, v = torch.randn(5, 64, generator=cpu(2)).cuda(), torch.randn(32, 64, generator=cpu(3)).cuda()
    w, xq = rd.MX4Matrix(at(1), 32, 64), rd.MX4Matrix(at(3), 5, 64)
    rd.mx4_quantize(v, out=w), rd.mx4_quantize(x, out=xq)
    want = rd.mx4_linear(x, rd.mx4_quantize(v), out_dtype=torch.float16)
    out = torch.as_strided(flat.view(torch.float16), (5, 32), (1 << 14, 1), 0)
    assert torch.equal(rd.mx4_linear(xq, w, out=out), want)
    assert torch.equal(rd.mx4_linear(x, w, out=out), want)
    for shift in (1, 32, 8000):
        bad = torch.as_strided(flat.view(torch.float16), (5, 32), (1 << 14, 1), shift)
        for rows in (x, xq):
            with pytest.raises(rd.RWKV7Error, match="overlaps"):
                rd.mx4_linear(rows, w, out=bad)
    assert torch.equal(rd.mx4_linear(xq, xq), rd.mx4_linear(x, rd.mx4_quantize(x)))  # one matrix on both sides


def test_rows_may_lie_around_their_matrix():
    """Rows 32 KB apart with their matrix between them."""
    flat = torch.zeros(3 << 15, dtype=torch.uint8, device="cuda")
    x = torch.as_strided(flat.view(torch.float32), (3, 40), (1 << 13, 1), 5)
    x.copy_(torch.randn(3, 40, generator=cpu(4)))
    want = nearest(x.double().cpu().numpy(), "mxfp4")
    m = rd.mx4_quantize(x, out=rd.MX4Matrix(flat[1024:1024 + 17408], 3, 40))
    same(m.dequantize(out=x), want)


def test_room_is_kept_for_torchs_own_streams_only():
    from recurrent_decode_gb300 import mx
    w, x = rd.mx4_quantize(torch.ones(70, 640, device="cuda")), torch.ones(40, 640, device="cuda")
    own = [torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream(priority=-1)]
    torch.cuda.synchronize()
    for i, s in enumerate(own + [torch.cuda.ExternalStream(own[1].cuda_stream)]):
        vars(mx._kept).clear()
        with torch.cuda.stream(s):
            y = rd.mx4_linear(x, w)
        s.synchronize()
        assert bool((y == 640).all()) and len(vars(mx._kept)) == (1 if i < len(own) else 0)
    rd.mx4_check()


def test_a_refused_launch_leaves_no_error_for_a_slot_call():
    """A call on a stream whose capture broke says so; the next slot call, on a sound
    stream, has no part in it."""
    assert fresh_process("""
import synth
ctx = rd.Rwkv7(synth.Dims("tiny"), 2)
x = torch.ones(4, 64, device="cuda")
m = rd.mx4_quantize(x)
torch.cuda.synchronize()
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        try:
            torch.cuda.current_stream().synchronize()
        except RuntimeError:
            print("broken")
        try:
            rd.mx4_quantize(x, out=m)
        except rd.RWKV7Error as e:
            print(e.code == rd.ECUDA)
except RuntimeError:
    pass
ctx.slot_reset(0)
ctx.synchronize()
print("reset")
""") == ["broken", "True", "reset"]


# ------------------------------------------------------------------ ends of the range
ENDS = [-127, -126, -100, -64, -1, 0, 63, 101, 124, 125]  # 6 * 2^125 is in fp32's range, 6 * 2^126 is not


def powers_apart(x_power, w_power, B=70, N=150):
    """Rows on the grid in blocks of these powers (a 6 in each pins its power), their exact
    values in fp64."""
    g = cpu(50)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    out = []
    for rows, power in ((B, x_power), (N, w_power)):
        v = grid[torch.randint(0, 8, (rows, 32 * len(power)), generator=g)]
        v *= torch.randint(0, 2, v.shape, generator=g) * 2 - 1
        v[:, ::32] = 6.0
        out.append(v * 2.0 ** torch.tensor(power, dtype=torch.float64).repeat_interleave(32))
    return out


@pytest.mark.parametrize("B", [3, 70])
def test_product_of_powers_at_both_ends(B):
    """Blocks of x from 2^-127 to 2^125 against blocks of w of about the inverse: terms of
    ordinary size, their sum as exact as the product's always is."""
    x, w = powers_apart(ENDS, [min(125, -e) for e in ENDS], B)
    assert torch.equal(x.float().double(), x) and torch.equal(w.float().double(), w)
    wq, xq = rd.mx4_quantize(w.float().cuda()), rd.mx4_quantize(x.float().cuda())
    assert torch.equal(wq.dequantize().cpu().double(), w) and torch.equal(xq.dequantize().cpu().double(), x)
    want, off = product(x.numpy(), w.numpy(), None, torch.float32)
    for rows in (x.float().cuda(), xq):
        y = rd.mx4_linear(rows, wq)
        assert (np.abs(y.double().cpu().numpy() - want) <= off).all()
    rd.mx4_check()


@pytest.mark.parametrize("e", [(-127, -127), (-100, -60), (-75, -70), (-127, -1)])
def test_products_below_the_normal_range(e):
    """Within fp32's smallest normal number of the sum, which the bound has in it."""
    x, w = powers_apart([e[0]] * 3, [e[1]] * 3)
    want, off = product(x.numpy(), w.numpy(), None, torch.float32)
    y = rd.mx4_linear(x.float().cuda(), rd.mx4_quantize(w.float().cuda()))
    assert (np.abs(y.double().cpu().numpy() - want) <= off).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_products_past_the_range_are_infinite(dtype):
    x, w = powers_apart([70] * 2, [70] * 2)
    y = rd.mx4_linear(x.abs().float().cuda(), rd.mx4_quantize(w.abs().float().cuda()), out_dtype=dtype)
    assert bool((y == float("inf")).all())
    y = rd.mx4_linear(-x.abs().float().cuda(), rd.mx4_quantize(w.abs().float().cuda()), out_dtype=dtype)
    assert bool((y == float("-inf")).all())


@pytest.mark.parametrize("fmt,part", [("mxint8", 127), ("mxfp4", 5)])
def test_a_state_keeps_its_documented_part(fmt, part):
    """MXINT8: max > 127/64 * 2^(e-1), so half a step, 2^e/128, is below max/127.  MXFP4:
    a value is off by 1/4 at most below 2, by 1/2 at 2.5 and by 1 at 5 (times 2^e), each
    time no more than a fifth of itself or of max > 3 * 2^e.  Down to 2^-126, where e no
    longer follows max, and at the ties themselves."""
    st = tuple(t.cuda() for t in pool(1, 2, 2, 35))
    st[0][0, 0, 0, 0, :32] = 5.0 * 2.0 ** -127  # 5 = a tie between 4 and 6
    st[0][0, 0, 0, 1, :32] = 2.0 ** -126
    st[0][0, 0, 0, 2, :32] = torch.linspace(1, 5, 32, device="cuda") * 2.0 ** 100
    st[0][0, 0, 0, 3, :32] = 3.4 * 2.0 ** 126
    before = st[0][:, 0].double()
    cache = rd.StateCache(1, 2, 1, fmt)
    cache.save(st, ints(0), ints(0))
    cache.load(st, ints(0), ints(1))
    d = (st[0][:, 1].double() - before).view(-1, 32).abs().amax(1)
    assert bool((d * part <= before.view(-1, 32).abs().amax(1)).all())
