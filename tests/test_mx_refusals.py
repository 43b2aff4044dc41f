"""The microscaled calls refuse bad arguments before they touch a device, and say
why; sizes of matrices and entries; the plain reference of the formats itself."""
import ctypes as C
import math

import numpy as np
import pytest

import recurrent_decode_gb300 as rd
from _mx_reference import FP4, fp4, nearest, power

P = 4096  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def lib():
    rd.build()
    return rd.load_library()


def refused(fn, *args):
    msg = C.c_char_p(b"unset")
    assert fn(*args, None, C.byref(msg)) == rd.EINVAL
    text = msg.value.decode()
    assert text not in ("", "unset")
    return text


def test_matrix_bytes(lib):
    f = lib.rwkv7_mx4_bytes
    assert f(128, 256) == f(1, 1) == 17408
    assert f(129, 256) == f(128, 257) == 2 * 17408
    assert f(0, 256) == 0 and f(-1, 256) == 0 and f(4, 0) == 0 and f(1 << 25, 32) == 0 and f(4, (1 << 24) + 1) == 0
    assert f(1 << 24, 1 << 24) == (1 << 17) * (1 << 16) * 17408  # past 32 bits


def test_entry_bytes(lib):
    f = lib.rwkv7_state_entry_bytes
    assert f(2, 3, 1) == 6 * (4096 + 128 + 512)
    assert f(2, 3, 0) == 6 * (2048 + 128 + 512)
    for bad in ((0, 3, 1), (2, 0, 1), (-1, 3, 0), (2, 3, 2), (2, 3, -1), (1 << 20, 1 << 20, 0)):
        assert f(*bad) == 0


def test_rows_refused(lib):
    for fn, call in ((lib.rwkv7_mx4_quantize, lambda x, dt, r, c, ld, mx: (x, dt, r, c, ld, mx)),
                     (lib.rwkv7_mx4_dequantize, lambda x, dt, r, c, ld, mx: (mx, r, c, x, dt, ld))):
        assert "rows" in refused(fn, *call(P, 0, -1, 32, 32, P))
        assert "cols" in refused(fn, *call(P, 0, 4, 0, 32, P))
        assert "dtype" in refused(fn, *call(P, 3, 4, 32, 32, P))
        assert "stride" in refused(fn, *call(P, 0, 4, 32, 31, P))
        assert "null" in refused(fn, *call(None, 0, 4, 32, 32, P))
        assert "null" in refused(fn, *call(P, 0, 4, 32, 32, None))
        assert "aligned" in refused(fn, *call(P + 2, 0, 4, 32, 32, P))
        assert "aligned" in refused(fn, *call(P + 1, 1, 4, 32, 32, P))
        assert "aligned" in refused(fn, *call(P, 0, 4, 32, 32, P + 8))
        msg = C.c_char_p()
        assert fn(*call(None, 0, 0, 32, 32, None), None, C.byref(msg)) == rd.OK and msg.value == b""


def test_linear_refused(lib):
    def call(x=P, xt=1, ldx=64, xm=P, B=2, w=P, N=8, K=64, y=P, yt=1, ldy=8, act=0, err=P):
        return x, xt, ldx, xm, B, w, N, K, y, yt, ldy, act, err
    f = lib.rwkv7_mx4_linear
    for bad in (dict(B=-1), dict(N=0), dict(K=0), dict(N=1 << 25), dict(B=1 << 25)):
        assert "at most" in refused(f, *call(**bad))
    assert "too large" in refused(f, *call(B=1 << 24, N=1 << 24, ldy=1 << 24))
    assert "output dtype" in refused(f, *call(yt=7))
    assert "activation" in refused(f, *call(act=2))
    assert "output row stride" in refused(f, *call(ldy=7))
    for bad in (dict(xm=None), dict(w=None), dict(y=None), dict(err=None)):
        assert "null" in refused(f, *call(**bad))
    assert "16-byte" in refused(f, *call(w=P + 8))
    assert "16-byte" in refused(f, *call(xm=P + 8))
    assert "output pointer" in refused(f, *call(y=P + 1))
    assert "output pointer" in refused(f, *call(y=P + 2, yt=0))
    assert "dtype" in refused(f, *call(xt=9))
    assert "stride" in refused(f, *call(ldx=63))
    msg = C.c_char_p()
    assert f(*call(x=None, xm=None, y=None, err=None, B=0), None, C.byref(msg)) == rd.OK


def test_states_refused(lib):
    def call(wkv=P, att=P, ffn=P, L=2, H=3, n_slots=4, slots=P, entries=P, n=2, cache=P, n_entries=4, fmt=1, err=P):
        return wkv, att, ffn, L, H, n_slots, slots, entries, n, cache, n_entries, fmt, err
    for f in (lib.rwkv7_states_save, lib.rwkv7_states_load):
        for bad in (dict(L=0), dict(H=0), dict(n_slots=0), dict(n_entries=0), dict(L=1 << 20, H=1 << 20)):
            assert ">= 1" in refused(f, *call(**bad))
        assert "pairs" in refused(f, *call(n=-1))
        assert "pairs" in refused(f, *call(n=1025))
        assert "format" in refused(f, *call(fmt=2))
        for name in ("wkv", "att", "ffn", "slots", "entries", "cache", "err"):
            assert "null" in refused(f, *call(**{name: None}))
        for name in ("wkv", "att", "ffn", "cache"):
            assert "16-byte" in refused(f, *call(**{name: P + 4}))
        msg = C.c_char_p()
        assert f(*call(n=0), None, C.byref(msg)) == rd.OK
    assert lib.rwkv7_slots_save(None, None, None, 0, None, 1, 1) == rd.EINVAL
    assert lib.rwkv7_slots_load(None, None, None, 0, None, 1, 1) == rd.EINVAL


def test_binding_refuses_what_is_not_on_the_device(lib):
    import torch
    with pytest.raises(TypeError, match="CUDA"):
        rd.mx4_quantize(torch.zeros(2, 32))
    with pytest.raises(TypeError, match="MX4Matrix"):
        rd.mx4_linear(torch.zeros(2, 32), torch.zeros(2, 32))
    with pytest.raises(ValueError, match="format"):
        rd.StateCache(2, 2, 2, "fp8")
    with pytest.raises(rd.RWKV7Error):
        rd.StateCache(0, 2, 2, "mxint8", device="cpu")
    with pytest.raises(rd.RWKV7Error):
        rd.mx4_empty(3, 0, "cpu")


def test_reference_grid():
    for c, v in enumerate(FP4):
        assert fp4(v) == v and fp4(-v) == -v
    ties = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0}
    for t, want in ties.items():
        assert fp4(t) == want
        assert fp4(math.nextafter(t, 9)) >= want >= fp4(math.nextafter(t, -9))
    assert power(6.0, 6.0, -127, 127) == 0 and power(math.nextafter(6.0, 7), 6.0, -127, 127) == 1
    assert power(0.0, 6.0, -127, 127) == -127


def test_reference_blocks():
    x = np.zeros((1, 70))
    x[0, 0], x[0, 40], x[0, 64:] = 96.0, 0.375, [1, 2, 3, 4, 5, 6]
    got = nearest(x, "mxfp4")[0]
    assert got[0] == 96 and got[40] == 0.375 and got[64:].tolist() == [1, 2, 3, 4, 4, 6]
    got = nearest(x, "mxint8")[0]
    assert got[0] == 96 and got[40] == 0.375 and got[64:].tolist() == [1, 2, 3, 4, 5, 6]
    x[0, 5] = np.inf
    got = nearest(x, "mxint8")[0]
    assert np.isnan(got[:32]).all() and np.isfinite(got[32:]).all()
