"""One row of x of more values than the few-row product takes, of any number: its stride stands for
nothing.  Tolerance as in test_gpu_q4.py: |error| <= (K + K / 32 + 1) 2^-23 sum |x w|."""
import ctypes as C

import pytest
import torch

import recurrent_decode_gb300 as rd
from recurrent_decode_gb300 import mx, q4
from _beam_reference import values

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def make(N, K, dtype, off=0):
    g = torch.Generator()
    g.manual_seed(N + K)
    q = torch.randint(0, 16, (N, K), generator=g).to(torch.uint8)
    s = (0.001 + 0.02 * torch.rand(N, -(-K // 128), generator=g)).half()
    z = torch.full(s.shape, 8, dtype=torch.uint8)
    w = torch.from_numpy(values(q.numpy(), s.numpy(), z.numpy(), 128))
    x = torch.empty(1, K + off, dtype=TYPES[dtype], device="cuda")[:, off:]
    x.copy_(torch.randn(1, K, generator=g))
    return rd.q4_pack(q.cuda(), s.cuda(), group=128), w, x


def check(y, x, w):
    x, K = x.double().cpu(), w.shape[1]
    off = (y.double().cpu() - x @ w.t()).abs()
    assert bool((off <= (K + K / 32 + 1) * 2.0 ** -23 * (x.abs() @ w.abs().t())).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [131072, 131073, 131079, 131080, 140001])
@pytest.mark.parametrize("off", [0, 3])
def test_one_long_row(K, off, dtype):
    m, w, x = make(50, K, dtype, off)
    check(rd.q4_linear(x, m, out_dtype=torch.float32), x, w)
    rd.q4_check()


@pytest.mark.parametrize("K", [131080, 131081])
@pytest.mark.parametrize("ldx", [0, 1, -16, 1 << 50])
def test_the_stride_of_one_row_is_free(ldx, K):
    m, w, x = make(20, K, "fp16")
    y, msg = torch.empty(1, 20, device="cuda"), C.c_char_p()
    assert rd.load_library().rwkv7_q4_linear(x.data_ptr(), 1, ldx, 1, m.data.data_ptr(), 20, K, 128, 0, y.data_ptr(), 0, 0, 0,
                                             None, q4._err_word(0).data_ptr(), mx._raw_stream(0), C.byref(msg)) == rd.OK, msg.value
    check(y, x, w)
