"""Digits that the gated delta rule keeps where large parts of a result cancel."""
import pytest
import torch

from long_convolution_sequence_amd import ops
from tests._parity import say

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("dk", [16, 40, 80, 128])
def test_a_query_for_a_key_that_was_just_overwritten(dk, dtype):
    """y = S^T q + (k . q) b (v - S^T k) with q = k a unit vector and b = 1 is v, whatever the state held.  States
    in [1, 2) of 24 bits and values that are whole multiples of 2^-19 of up to 2^-12: every product and sum is a
    number of 24 bits, so fp32 gives v to the last bit.  A term of the state left out (2^-17) is thirty times the
    step of a 16-bit v there."""
    say(f"case delta overwritten key dk={dk} {dtype}")
    T, B, H, dv, at = 40, 2, 2, 48, 7
    gen = torch.Generator().manual_seed(dk)
    state = 1 + torch.randint(0, 1 << 23, (B, H, dk, dv), generator=gen) * 2.0 ** -23
    v = torch.zeros(T, B, H, dv)
    v[at] = torch.randint(64, 128, (B, H, dv), generator=gen) * 2.0 ** -19
    k = torch.zeros(T, B, H, dk)
    k[at, ..., dk // 3] = 1.0
    gates = torch.zeros(T, B, H, device="cuda")
    k, v, state = k.to(dtype).cuda(), v.to(dtype).cuda(), state.cuda()
    y, final = ops.gated_delta(k, k, v, gates, gates + 1, state, scale=1.0)
    assert torch.equal(y[at], v[at])
    assert torch.equal(final[:, :, dk // 3], v[at].float())
    assert (y[:at] == 0).all() and (y[at + 1:] == 0).all()
