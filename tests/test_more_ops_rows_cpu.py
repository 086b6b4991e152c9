"""What the binding of the gated delta rule takes as rows of heads, without a GPU."""
import pytest
import torch

from long_convolution_sequence_amd import fi, ops


@pytest.mark.parametrize("make", [lambda t: t[..., :1].expand(t.shape), lambda t: t[:5].as_strided((5, *t.shape[1:]), (*t.stride()[:-1], 2)),
                                  lambda t: t[:, :, :1, :1].expand(t.shape)])
def test_channels_that_are_no_neighbours_are_refused(make):
    """Heads one row apart whose channels are not: flattened they would be a copy that nobody keeps, read after its
    memory is free, or written in place of the caller's output."""
    bad = make(torch.zeros(7, 2, 3, 8))
    with pytest.raises(fi.FiError) as e:
        ops._heads(bad, bad.shape, torch.float32, -1, "t")
    assert e.value.status == fi.FI_EINVAL


def test_one_channel_at_any_stride():
    """A single channel's stride says nothing: heads one element apart are packed."""
    t = torch.zeros(6, 2, 30)[..., 4:7].unsqueeze(-1)
    t = t.as_strided(t.shape, (*t.stride()[:-1], 9), t.storage_offset())
    p, pitch = ops._heads(t, t.shape, torch.float32, -1, "t")
    assert (p, pitch) == (t.data_ptr(), 30)
