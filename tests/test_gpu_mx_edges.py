"""The microscaled operators where a call goes wrong beside its values: repeated and
bad indices, entries that nothing was saved to, tensors and graphs on other streams,
results over their inputs, powers at the ends of their range."""
import pytest
import torch

import recurrent_decode_gb300 as rd
from _mx_reference import nearest
from test_gpu_mx import cpu, ints, pool, same

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
