"""Products in 8-bit integers on the GPU: codes and scales equal to the definition's
bit for bit, products within three roundings of it."""
import pytest
import torch

from long_convolution_sequence_amd import fi, ops
from tests import _more_ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _weight(N, K, gen):
    return (torch.randint(-127, 128, (N, K), generator=gen, dtype=torch.int8), torch.rand(N, generator=gen) * 0.01 + 1e-3,
            torch.randn(N, generator=gen))


def _check(y, x, codes, scales, bias):
    c, s = ref.q8_rows(x)
    value, tol = ref.q8(c, s, codes, scales, bias)
    w = ref.worst(y, value, ref.stored(value, tol, y.dtype))
    assert w <= 1.0, f"{w:.3g} of its bound"


CASES = [(1, 1, 1), (1, 17, 5), (1, 864, 864), (2, 100, 64), (3, 33, 127), (15, 70, 129), (16, 256, 128), (17, 40, 200),
         (31, 129, 300), (33, 16, 1000), (64, 300, 96), (100, 255, 257), (129, 128, 128), (200, 500, 513), (257, 640, 999),
         (513, 129, 2048), (1, 5003, 4999), (8, 2592, 864), (700, 1030, 640), (40, 4000, 1500), (1000, 96, 8192), (300, 10, 70)]


@pytest.mark.parametrize("M,N,K", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_products(M, N, K, dtype):
    say(f"case q8 M={M} N={N} K={K} {dtype}")
    gen = torch.Generator().manual_seed(M + 7 * N + 31 * K)
    codes, scales, bias = _weight(N, K, gen)
    x = torch.randn(M, K, generator=gen).to(dtype)
    w = ops.Q8Weight(codes.cuda(), scales.cuda())
    for b in (None, bias):
        y = ops.q8_product(w, x.cuda(), b.cuda() if b is not None else None)
        assert y.shape == (M, N) and y.dtype == dtype
        _check(y, x, codes, scales, b)


@pytest.mark.parametrize("rows,K", [(1, 1), (5, 130), (16, 64), (17, 1000), (40, 4999), (3, 70001)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_codes_and_scales(rows, K, dtype):
    say(f"case q8 codes rows={rows} K={K} {dtype}")
    gen = torch.Generator().manual_seed(rows + K)
    x = (torch.randn(rows, K, generator=gen) * torch.exp(torch.randn(rows, 1, generator=gen))).to(dtype)
    q = ops.Q8Rows.quantize(x.cuda())
    codes, scales = ref.q8_rows(x)
    assert torch.equal(q.scales.cpu(), scales) and torch.equal(q.codes.cpu(), codes)
    again = ops.Q8Rows(q.codes, q.scales.clone())
    assert torch.equal(again.codes, q.codes) and torch.equal(again.scales, q.scales)


def test_one_quantization_for_several_weights():
    say("case q8 shared rows")
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(70, 300, generator=gen).bfloat16()
    q = ops.Q8Rows.quantize(x.cuda())
    for N in (5, 200):
        codes, scales, bias = _weight(N, 300, gen)
        w = ops.Q8Weight(codes.cuda(), scales.cuda())
        direct = ops.q8_product(w, x.cuda(), bias.cuda())
        assert torch.equal(ops.q8_product(w, q, bias.cuda()), direct)
        _check(ops.q8_product(w, q, bias.cuda(), dtype=F32), x, codes, scales, bias)
        assert torch.equal(ops.q8_product(w, x.cuda(), bias.cuda(), dtype=F32), ops.q8_product(w, q, bias.cuda(), dtype=F32))


@pytest.mark.parametrize("M", [1, 7, 40, 300])
def test_sums_that_no_float_holds(M):
    """The largest codes along the longest k: sums of 2^31 - 2^14, exact to the last bit before they are
    rounded once; codes of -128 count."""
    say(f"case q8 largest sums M={M}")
    K, N = 131071, 33
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1:, 1::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    y = ops.q8_product(ops.Q8Weight(w, one[:N].clone()), ops.Q8Rows(a, one[:M].clone()), dtype=F32)
    want = torch.full((N,), float(65536 * 128 * 128 - 65535 * 128 * 127), dtype=torch.float64)
    want[0] = 131071.0 * 128 * 128
    assert torch.equal(y.cpu(), want.float().expand(M, N))


@pytest.mark.parametrize("M", [3, 40])
def test_rows_of_zeros_and_bad_rows(M):
    """A row of zeros gives the bias; an infinity or NaN gives NaN in its row only."""
    say(f"case q8 zero and bad rows M={M}")
    gen = torch.Generator().manual_seed(5)
    codes, scales, bias = _weight(50, 200, gen)
    w = ops.Q8Weight(codes.cuda(), scales.cuda())
    x = torch.randn(M, 200, generator=gen)
    clean = ops.q8_product(w, x.cuda(), bias.cuda())
    x[0] = 0.0
    x[1, 7] = float("inf")
    x[2, 199] = float("nan")
    y = ops.q8_product(w, x.cuda(), bias.cuda())
    assert torch.equal(y[0].cpu(), bias) and y[1].isnan().all() and y[2].isnan().all()
    assert torch.equal(y[3:], clean[3:])
    tiny = torch.full((M, 200), 1e-45)
    q = ops.Q8Rows.quantize(tiny.cuda())
    assert (q.scales == 0).all() and (q.codes == 0).all()
    small = torch.full((M, 200), 2.0 ** -140)                       # the scale has lost digits: codes stop at 127
    q = ops.Q8Rows.quantize(small.cuda())
    assert (q.codes.abs() <= 127).all() and (q.scales > 0).all()


def test_slices_outputs_and_quantized_weights():
    say("case q8 slices")
    gen = torch.Generator().manual_seed(6)
    wide = torch.randn(50, 400, generator=gen).bfloat16().cuda()
    wf = torch.randn(90, 150, generator=gen).cuda()
    w = ops.Q8Weight.quantize(wf)
    codes, scales = ref.q8_rows(wf.cpu())
    assert torch.equal(w.codes.cpu(), codes) and torch.equal(w.scales.cpu(), scales) and (w.N, w.K) == (90, 150)
    for rows in (1, 50):
        x = wide[:rows, 101:251]
        out = torch.full((rows, 200), 3.0, dtype=BF16, device="cuda")
        y = ops.q8_product(w, x, y=out[:, 7:97])
        assert y.data_ptr() == out[:, 7:97].data_ptr()
        _check(y, x.cpu(), codes, scales, None)
        mask = torch.ones(200, dtype=torch.bool, device="cuda")
        mask[7:97] = False
        assert (out[:, mask] == 3).all()


def test_no_rows():
    say("case q8 no rows")
    w = ops.Q8Weight.quantize(torch.ones(4, 5, device="cuda"))
    assert ops.q8_product(w, torch.zeros(0, 5, device="cuda")).shape == (0, 4)


@pytest.mark.parametrize("M", [1, 16, 90])
def test_side_stream_and_graph(M):
    say(f"case q8 graph M={M}")
    gen = torch.Generator().manual_seed(8)
    codes, scales, bias = _weight(300, 700, gen)
    w = ops.Q8Weight(codes.cuda(), scales.cuda())
    b = bias.cuda()
    x = torch.randn(M, 700, generator=gen).cuda()
    want = ops.q8_product(w, x, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        side = ops.q8_product(w, x, b)
    s.synchronize()
    assert torch.equal(side, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ops.q8_product(w, x, b)
    for _ in range(4):
        new = torch.randn(M, 700, generator=gen).cuda()
        x.copy_(new)
        g.replay()
        eager = ops.q8_product(w, new, b)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_binding_refuses_mismatches():
    say("case q8 refusals")
    w = ops.Q8Weight.quantize(torch.ones(6, 8, device="cuda"))
    x = torch.zeros(3, 8, device="cuda")
    b = torch.zeros(6, device="cuda")
    c = torch.zeros(6, 8, dtype=torch.int8, device="cuda")
    for call in (lambda: ops.q8_product(x, x), lambda: ops.q8_product(w, x[:, :7]), lambda: ops.q8_product(w, x.double()),
                 lambda: ops.q8_product(w, x.cpu()), lambda: ops.q8_product(w, x[0]), lambda: ops.q8_product(w, x, b[:5]),
                 lambda: ops.q8_product(w, x, b.half()), lambda: ops.q8_product(w, x, dtype=torch.int8),
                 lambda: ops.q8_product(w, x, y=torch.zeros(3, 5, device="cuda")),
                 lambda: ops.q8_product(w, x, y=torch.zeros(3, 6, device="cuda").half()),
                 lambda: ops.q8_product(w, ops.Q8Rows.quantize(torch.zeros(3, 9, device="cuda"))),
                 lambda: ops.Q8Weight(c, b[:5]), lambda: ops.Q8Weight(c, b.half()), lambda: ops.Q8Weight(c.float(), b),
                 lambda: ops.Q8Weight(c[0], b), lambda: ops.Q8Weight(c, None), lambda: ops.Q8Rows.quantize(x.double()),
                 lambda: ops.Q8Rows.quantize(torch.zeros(1, 131072, device="cuda")), lambda: ops.Q8Rows.quantize(x[:, ::2])):
        with pytest.raises(fi.FiError) as e:
            call()
        assert e.value.status == fi.FI_EINVAL
