"""Zeros of a group are four bits, as codes are: of a byte with more the low four count."""
import pytest
import torch

import recurrent_decode_gb300 as rd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [32, 64, 128])
def test_low_four_bits_of_zeros_count(group):
    N, K = 19, 200
    g = torch.Generator()
    g.manual_seed(group)
    q = torch.randint(0, 16, (N, K), generator=g).to(torch.uint8).cuda()
    s = (0.001 + 0.02 * torch.rand(N, -(-K // group), generator=g)).half().cuda()
    z = torch.randint(0, 16, s.shape, generator=g).to(torch.uint8).cuda()
    z[0], z[1] = 0, 15
    want = rd.q4_pack(q, s, z, group=group)
    assert torch.equal(rd.q4_pack(q, s, z + 16, group=group).data, want.data)  # 16 is 0
    x = torch.randn(3, K, generator=g).half().cuda()
    assert torch.equal(rd.q4_linear(x, rd.q4_pack(q, s, z + 240, group=group)), rd.q4_linear(x, want))
