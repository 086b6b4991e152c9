"""The layer norm's gradients of rows far from zero: the digits that fp32 rows leave."""
import pytest
import torch

from long_convolution_sequence_amd import ops
from tests import _more_ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _bounds(x, weight, da):
    """dx, dweight and bounds that know nothing of the size of the mean but through the sums it is in: the mean
    that is kept is off by U |m|, the mean of the deviations from it takes that away again."""
    U = ref.U
    x, w, da = x.double(), weight.double(), da.double()
    rows, D = x.shape
    mean = lambda t: t.mean(-1, keepdim=True)                                      # noqa: E731
    s = (D / 64 + 24) * U
    m = mean(x)
    v = x - m
    ev = 3 * U * (v.abs() + s * mean(x.abs())) + s * mean(v.abs()) + s ** 2 * mean(x.abs())
    var = mean(v * v) + EPS
    n = 1 / torch.sqrt(var)
    fn = mean(v.abs() * ev) / var + s + 6 * U
    u = v * n
    eu = ev * n + (fn + 2 * U) * u.abs()
    e = da * w
    m1, m2 = mean(e), mean(e * u)
    # mean(e u) is formed as n (mean(e v') - d mean(e)) with v' the deviations from the kept mean, d their mean:
    # both products at magnitudes of |e| (|u| + U |m| n)
    shift = U * m.abs() * n
    e2 = mean(e.abs() * eu) + (s + 6 * U) * mean(e.abs() * (u.abs() + shift))
    big = e.abs() + m1.abs() + (u * m2).abs()
    dx = n * (e - m1 - u * m2)
    edx = n * (s * mean(e.abs()) + eu * m2.abs() + u.abs() * e2) + (fn + 6 * U) * n * big
    terms = (rows / 64 + 1100) * U
    return {"dx": (dx, edx), "dweight": ((da * u).sum(0), (da.abs() * eu + (terms + 2 * U) * (da * u).abs()).sum(0))}


@pytest.mark.parametrize("ratio", [0.0, 1000.0, 30000.0])
@pytest.mark.parametrize("rows,D", [(1, 7), (9, 1000), (5, 864), (40, 5001), (3, 16384), (4, 1024), (2, 9000)])
def test_gradients_of_rows_far_from_zero(rows, D, ratio):
    say(f"case layer far gradients rows={rows} D={D} mean/deviation={ratio}")
    gen = torch.Generator().manual_seed(rows + D)
    r = lambda *s: torch.randn(*s, generator=gen)                                  # noqa: E731
    x = r(rows, D) + ratio * (1 + torch.rand(rows, 1, generator=gen))
    weight = 1 + r(D) / 8
    da = r(rows, D) + (x - x.mean(-1, keepdim=True))         # not at right angles to the row
    c = [t.cuda() for t in (x, weight, da)]
    _, _, saved = ops.layer_norm(c[0], weight=c[1], eps=EPS, save=True)
    got = ops.layer_norm_backward(None, c[2], c[0], None, saved, weight=c[1], eps=EPS)
    for name, (value, tol) in _bounds(x, weight, da).items():
        w = ref.worst(got.x if name == "dx" else got.weight, value, ref.stored(value, tol, torch.float32))
        assert w <= 1.0, f"{name}: {w:.3g} of its bound"
