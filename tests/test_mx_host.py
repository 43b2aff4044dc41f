"""What the binding of the microscaled operators does on the host: the order of streams,
the memory that calls keep, who makes the error word, indices of the packed prefix
cache.  No GPU: the library, streams and tensors are stand-ins."""
import ctypes as C
import os
import subprocess
import sys
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import recurrent_decode_gb300 as rd
from recurrent_decode_gb300 import mx
from recurrent_decode_gb300.prefix_cache import PackedPrefixStateCache, PrefixStateCache

CUDA0, CUDA1 = torch.device("cuda", 0), torch.device("cuda", 1)


# ------------------------------------------------------------------ streams
class Stream:
    def __init__(self, name, log, device=CUDA0):
        self.name, self.log, self.device, self.cuda_stream = name, log, device, hash(name)

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")


class Tensor:
    def __init__(self, name, log, device=CUDA0):
        self.name, self.log, self.device = name, log, device

    def data_ptr(self):
        return 4096

    def record_stream(self, stream):
        self.log.append(f"{self.name} kept for {stream.name}")


def context(stream, log):
    ctx = rd.Rwkv7.__new__(rd.Rwkv7)
    ctx.h, ctx.stream, ctx.dims = None, stream, SimpleNamespace(n_layer=2, n_head=3)
    ctx.lib = SimpleNamespace(rwkv7_slots_save=lambda *a: log.append("save") or 0,
                              rwkv7_slots_load=lambda *a: log.append("load") or 0)
    return ctx


class Log(list):
    current = None  # stream


@pytest.fixture
def log(monkeypatch):
    log = Log()
    monkeypatch.setattr(mx, "_pair_count", lambda slots, entries, dev: 1)
    monkeypatch.setattr(mx, "_raw_stream", lambda dev: log.current.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: log.current)
    return log


def cache_of(log, device=CUDA0):
    return SimpleNamespace(n_layer=2, n_head=3, n_entries=4, format=1, data=Tensor("cache", log, device))


@pytest.mark.parametrize("what", ["save", "load"])
def test_slots_on_a_stream_of_their_own_follow_the_current_one(log, what):
    log.current = Stream("current", log)
    ctx, cache = context(Stream("own", log), log), cache_of(log)
    a, b = Tensor("a", log), Tensor("b", log)
    (ctx.slots_save if what == "save" else ctx.slots_load)(cache, a, b)
    assert log.index("own waits for current") < log.index(what)
    for name in ("cache", "a", "b"):
        assert f"{name} kept for own" in log


def test_slots_on_the_current_stream_wait_for_nothing(log):
    log.current = Stream("current", log)
    ctx, cache = context(log.current, log), cache_of(log)
    ctx.slots_save(cache, Tensor("a", log), Tensor("b", log))
    assert log == ["save"]


def test_slots_refuse_a_cache_of_another_device(log):
    log.current = Stream("current", log)
    ctx = context(Stream("own", log), log)
    for call in (ctx.slots_save, ctx.slots_load):
        with pytest.raises(ValueError, match="cuda:1"):
            call(cache_of(log, CUDA1), Tensor("a", log, CUDA1), Tensor("b", log, CUDA1))
    assert log == []


# ------------------------------------------------------------------ the error word
def test_threads_that_come_at_once_share_one_error_word(monkeypatch):
    import threading
    import time

    def zeros(*a, **k):
        time.sleep(0.02)  # long enough for all threads to find no word
        return object()
    monkeypatch.setattr(mx, "_err", {})
    monkeypatch.setattr(mx, "_capturing", lambda dev: False)
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: SimpleNamespace(synchronize=lambda: None))
    start, words = threading.Barrier(8), []

    def first_call():
        start.wait()
        words.append(mx._err_word(0))
    threads = [threading.Thread(target=first_call) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(words) == 8 and all(w is mx._err[0] for w in words)


# ------------------------------------------------------------------ memory kept between calls
class Devices:
    """Two devices, each with a current stream, which may be one that is being captured."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.made = 0, set(), []
        self.stream = {0: 0, 1: 0}
        fakes = self

        class device:
            def __init__(self, dev):
                self.dev = dev

            def __enter__(self):
                self.before, fakes.current = fakes.current, self.dev

            def __exit__(self, *a):
                fakes.current = self.before

        def empty(n, dtype, device):
            self.made.append(SimpleNamespace(n=n, device=device))
            return self.made[-1]
        monkeypatch.setattr(mx, "_kept", SimpleNamespace())
        monkeypatch.setattr(mx, "_current_device", lambda: self.current)
        monkeypatch.setattr(mx, "_raw_stream", lambda dev: self.stream[dev])
        monkeypatch.setattr(mx, "_stream_data", lambda dev: (self.stream[dev], dev, 1))
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(mx, "_is_capturing", lambda: self.current in self.capturing)


@pytest.mark.parametrize("dev", [0, 1])
def test_a_graph_of_any_device_gets_room_of_its_own(monkeypatch, dev):
    """Also of a device that is not the current one: room of the device whose stream is
    captured, whatever the current device does."""
    d = Devices(monkeypatch)
    kept = mx._room(100, dev)
    assert mx._room(200, dev) is kept
    d.capturing = {dev}
    assert mx._room(100, dev) is not kept and d.made[-1].n == 100 and d.made[-1].device == f"cuda:{dev}"
    d.capturing = {1 - dev}
    assert mx._room(100, dev) is kept
    assert d.current == 0


def test_the_error_word_is_made_with_a_devices_first_matrix(monkeypatch):
    d = Devices(monkeypatch)
    monkeypatch.setattr(mx, "_err", {})
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: "word of " + k["device"])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: SimpleNamespace(synchronize=lambda: None))
    data = SimpleNamespace(is_cuda=True, get_device=lambda: 1)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: data)
    d.capturing = {1}
    mx.mx4_empty(1, 32, "cuda:1")  # quantised inside a capture: no word yet
    assert mx._err == {}
    with pytest.raises(rd.RWKV7Error, match="before the first capture") as e:
        mx._err_word(1)
    assert e.value.code == rd.ESTATE and mx._err == {}
    d.capturing = {0}
    mx.mx4_empty(1, 32, "cuda:1")
    assert mx._err == {1: "word of cuda:1"}
    d.capturing = {1}
    assert mx._err_word(1) == "word of cuda:1"


def test_the_error_word_is_no_inference_tensor(monkeypatch):
    """It may be made under inference_mode and reset by a check outside."""
    zeros = torch.zeros
    monkeypatch.setattr(mx, "_err", {})
    monkeypatch.setattr(mx, "_capturing", lambda dev: False)
    monkeypatch.setattr(torch, "zeros", lambda *a, dtype, device: zeros(*a, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: SimpleNamespace(synchronize=lambda: None))
    with torch.inference_mode():
        w = mx._err_word(0)
    w.fill_(8)
    w.zero_()
    assert not w.is_inference()


# ------------------------------------------------------------------ memory that calls share
def refused(fn, *args):
    msg = C.c_char_p(b"unset")
    assert fn(*args, None, C.byref(msg)) == rd.EINVAL
    return msg.value.decode()


def test_a_product_refuses_to_write_over_its_matrices():
    """x 2 x 64 fp16 rows 128 apart from 1 << 20, room for them (one tile) from 2 << 20,
    w (8 x 64, one tile) from 3 << 20, y 2 x 8 fp16 rows 8 apart from 4 << 20."""
    rd.build()
    f = rd.load_library().rwkv7_mx4_linear
    X, ROOM, W, Y, TILE = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 17408

    def call(x=X, room=ROOM, w=W, y=Y, ldy=8, B=2):
        return x, 1, 128, room, B, w, 8, 64, y, 1, ldy, 0, 8 << 20
    for bad in (dict(y=W), dict(y=W + TILE - 2), dict(y=W - 30), dict(y=ROOM), dict(y=ROOM + TILE - 16),
                dict(x=None, y=ROOM), dict(y=W - 4096 - 14, ldy=2048), dict(y=W - 4096 + 16, ldy=2048),
                dict(y=W - 10 * 65536 + TILE - 2, ldy=32768, B=11)):
        assert "output overlaps" in refused(f, *call(**bad))
    for bad in (dict(room=W), dict(room=W - TILE + 16), dict(room=W + TILE - 16)):
        assert "room" in refused(f, *call(**bad))


def test_rows_and_their_matrix_do_not_overlap():
    """Four fp32 rows of 32 values and a matrix of one tile."""
    rd.build()
    lib, M, TILE = rd.load_library(), 1 << 20, 17408
    for x, ld in ((M, 32), (M - 508, 32), (M + TILE - 4, 32), (M - 3 * 8192 - 124, 2048), (M - 8192 + 64, 2048)):
        assert "overlap" in refused(lib.rwkv7_mx4_quantize, x, 0, 4, 32, ld, M)
        assert "overlap" in refused(lib.rwkv7_mx4_dequantize, M, 4, 32, x, 0, ld)
    # the room for x
    assert "overlap" in refused(lib.rwkv7_mx4_linear, M, 0, 32, M, 4, 2 * M, 8, 32, 3 * M, 0, 8, 0, 4 * M)


def test_room_is_kept_for_streams_that_cannot_be_destroyed(monkeypatch):
    """By stream, for torch's own; a handle that came from elsewhere may be another
    stream's by the next call."""
    d = Devices(monkeypatch)
    first = mx._room(100, 0)
    d.stream[0] = 3
    second = mx._room(100, 0)
    assert second is not first and mx._room(100, 0) is second
    d.stream[0] = 0
    assert mx._room(100, 0) is first
    d.stream[0] = 0x5580_1234_5670
    a, b = mx._room(100, 0), mx._room(100, 0)
    assert a is not b and a.n == b.n == 100 and not any(k[1] == d.stream[0] for k in vars(mx._kept))


# ------------------------------------------------------------------ imports
def test_a_star_import_needs_no_torch():
    """Nor do the package and its names outside the microscaled operators, which are
    there on first use and listed by dir()."""
    code = """
import sys
sys.modules["torch"] = None  # an import of it raises
from recurrent_decode_gb300 import *
import recurrent_decode_gb300 as rd
assert Rwkv7 is rd.Rwkv7 and "mx4_linear" in dir(rd) and "Rwkv7" in dir(rd)
try:
    rd.mx4_linear
except ImportError:
    print("no torch")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["no", "torch"]
    names = {}
    exec("from recurrent_decode_gb300 import *", names)  # here there is one
    assert all(names[n] is getattr(mx, n) for n in rd._MX)


# ------------------------------------------------------------------ prefix caches
class Slots:
    """A context of two slots that refuses others, as the library does."""
    n_slots, dims, stream = 2, SimpleNamespace(n_layer=2, n_head=3), SimpleNamespace(device=CUDA1)

    def __init__(self):
        self.calls = []

    def slot_copy(self, src, dst):
        if not 0 <= src < self.n_slots + 2:
            raise rd.RWKV7Error(rd.EINVAL, "slot out of range")
        self.calls.append((src, dst))


def contents(cache):
    return (list(cache.entries.items()), list(cache.free), cache.hits, cache.misses, cache.hit_tokens, cache.stores,
            cache.evictions)


def test_a_refused_store_leaves_the_prefix_cache_as_it_was():
    cache = PrefixStateCache(Slots(), [2, 3], block=4)
    a, b, c = (np.full(4, i, np.int32) for i in range(3))
    for have in (a, b, None):  # with two free slots, with one, with none
        before = contents(cache)
        with pytest.raises(rd.RWKV7Error):
            cache.store(c, 9)
        assert contents(cache) == before
        if have is not None:
            cache.store(have, 0)
    assert len(cache) == 2 and cache.lookup(a)[0] == 4 and cache.lookup(c)[0] == 0
    cache.store(c, 1)
    assert cache.evictions == 1 and cache.lookup(b)[0] == 0 and cache.lookup(c)[0] == 4


class PackedSlots(Slots):
    """Moves states as the device does, which leaves a pair out of range out and says so later."""

    def slots_save(self, cache, slots, entries):
        self.calls.append(("save", slots.tolist(), entries.tolist()))

    def slots_load(self, cache, entries, slots):
        self.calls.append(("load", entries.tolist(), slots.tolist()))


@pytest.fixture
def packed(monkeypatch):
    """A packed prefix cache of six entries over a context of two slots."""
    made = []

    def state_cache(n_layer, n_head, n_entries, format="mxint8", device=None):
        made.append((n_layer, n_head, n_entries, format, device))
        return SimpleNamespace(data=SimpleNamespace(device="cpu"))
    monkeypatch.setattr(mx, "StateCache", state_cache)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(synchronize=lambda: None))
    cache = PackedPrefixStateCache(PackedSlots(), 6, "mxfp4", block=4)
    cache.made = made
    return cache


@pytest.mark.parametrize("slot", [-1, 2, 5, 6])
def test_packed_prefix_cache_refuses_a_slot_out_of_range(packed, slot):
    """Also one that is an entry's number, at storing and at restoring."""
    a = np.arange(4, dtype=np.int32)
    packed.store(a, 1)
    assert packed.restore(a, 0) == 4
    assert packed.ctx.calls == [("save", [1], [5]), ("load", [5], [0])]
    before = contents(packed)
    for call in (lambda: packed.store(a + 1, slot), lambda: packed.restore(a, slot)):
        with pytest.raises(rd.RWKV7Error, match="out of range") as e:
            call()
        assert e.value.code == rd.EINVAL
    assert contents(packed) == before and len(packed.ctx.calls) == 2 and packed.lookup(a + 1)[0] == 0


def test_packed_prefix_cache_lies_on_the_contexts_device(packed):
    assert packed.made == [(2, 3, 6, "mxfp4", CUDA1)]
