"""4-bit matrix-vector products on the GPU against the 64-bit definition, within
the bound that tests/_ops_ref.py derives, and exactly where fp32 sums are exact."""
import pytest
import torch

from long_convolution_sequence_amd import fi, ops
from tests import _ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _inputs(N, K, B, group, dtype, st, zeros, seed=0):
    gen = torch.Generator().manual_seed(31 * seed + N + 7 * K + B)
    groups = -(-K // group)
    return {"x": torch.randn(B, K, generator=gen).to(dtype),
            "codes": torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8),
            "scales": ((torch.rand(N, groups, generator=gen) + 0.5) * 0.005).to(st),
            "zeros": torch.randint(0, 16, (N, groups), generator=gen, dtype=torch.uint8) if zeros else None}


def _weight(v, group):
    return ops.Q4Weight(v["codes"].cuda(), v["scales"].cuda(), v["zeros"].cuda() if v["zeros"] is not None else None,
                        group=group)


CASES = [(1, 1, 1, 32, F32, F32, False), (16, 128, 1, 128, BF16, BF16, False), (17, 129, 2, 32, F32, BF16, True),
         (33, 300, 3, 64, F16, F16, True), (5, 31, 16, 32, BF16, F32, True), (100, 1000, 5, 128, F32, F16, True),
         (48, 640, 6, 64, F32, F32, False), (257, 513, 8, 32, F16, BF16, True), (64, 2050, 9, 128, F16, BF16, False),
         (31, 4097, 16, 64, F32, BF16, True), (130, 96, 10, 32, F32, F32, True), (2000, 70, 1, 32, BF16, F16, False),
         (40, 9000, 11, 128, F32, BF16, True), (640, 1152, 16, 128, BF16, BF16, True), (18, 20000, 4, 32, F32, BF16, True)]


@pytest.mark.parametrize("N,K,B,group,dtype,st,zeros", CASES)
def test_products(N, K, B, group, dtype, st, zeros):
    say(f"case q4 N={N} K={K} B={B} group={group} {dtype}/{st} zeros={zeros}")
    v = _inputs(N, K, B, group, dtype, st, zeros)
    y = ops.q4_matvec(_weight(v, group), v["x"].cuda())
    want, tol = ref.q4(v["x"], v["codes"], v["scales"], v["zeros"], group)
    assert y.dtype == dtype
    w = ref.worst(y, want, ref.stored(want, tol, dtype))
    assert w <= 1.0, f"{w:.3g} of its bound"


@pytest.mark.parametrize("N,K,B,group", [(37, 333, 1, 32), (64, 1500, 4, 64), (20, 2100, 16, 128), (300, 5000, 7, 32)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_whole_numbers_are_exact(N, K, B, group, dtype):
    """Small whole numbers and scales that are powers of two: every product and partial sum is a
    multiple of 2^-6 below 2^18 in size, so fp32 sums lose nothing, whatever their order."""
    say(f"case q4 exact N={N} K={K} B={B} group={group} {dtype}")
    v = _inputs(N, K, B, group, F32, BF16, True, seed=1)
    gen = torch.Generator().manual_seed(9)
    v["x"] = torch.randint(-1, 2, (B, K), generator=gen).to(dtype)
    v["scales"] = (2.0 ** torch.randint(-6, -3, v["scales"].shape, generator=gen)).to(BF16)
    y = ops.q4_matvec(_weight(v, group), v["x"].cuda())
    want, _ = ref.q4(v["x"], v["codes"], v["scales"], v["zeros"], group)
    assert torch.equal(y.cpu(), want.to(torch.float32).to(dtype))


def test_full_precision_of_the_inputs():
    """One input per output: fp32 values come back to the last bits (three bf16 terms), not rounded."""
    say("case q4 precise inputs")
    K = 64
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(5, K, generator=gen)
    codes = torch.full((K, K), 8, dtype=torch.uint8)
    codes[torch.arange(K), torch.arange(K)] = 9                       # the unit matrix
    w = ops.Q4Weight(codes.cuda(), torch.ones(K, 2, device="cuda"), group=32)
    y = ops.q4_matvec(w, x.cuda()).cpu()
    _, tol = ref.q4(x, codes, torch.ones(K, 2), None, 32)
    assert float(((y - x).double().abs() / tol).max()) <= 1.0
    assert float((y - x).abs().max()) < 2.0 ** -14                    # bf16 alone would be off by 2^-8


@pytest.mark.parametrize("N,B,group", [(50, 1, 32), (70, 5, 64), (40, 9, 128), (33, 16, 32), (12400, 16, 128)])
def test_every_bit_of_the_inputs(N, B, group):
    """One input a group that is not zero, with all 24 significand bits, times a power of two: each of
    its three terms is a product of at most 8 + 5 bits, so every sum is exact and y is the input, bit
    for bit.  Two terms of 8 bits do not hold any of these inputs."""
    say(f"case q4 every bit N={N} B={B} group={group}")
    groups = 5
    K = groups * group
    gen = torch.Generator().manual_seed(N + B)
    at = torch.arange(groups) * group + torch.randint(0, group, (groups,), generator=gen)
    x = torch.zeros(B, K)
    # 24 bits, the lowest of them set; sizes from 2^-20 to 2^20
    bits = torch.randint(1 << 22, 1 << 23, (B, groups), generator=gen) * 2 + 1
    x[:, at] = bits.float() * 2.0 ** torch.randint(-43, -3, (B, groups), generator=gen).float()
    top = (x.view(torch.int32) & -65536).view(torch.float32)
    rest = x - top
    two = top + (rest.view(torch.int32) & -65536).view(torch.float32)
    assert (two != x)[:, at].all()
    mine = torch.arange(N) % groups
    step = torch.tensor([1, -1, 2, -2, 4, -4, -8])[torch.arange(N) % 7]
    codes = torch.full((N, K), 8, dtype=torch.uint8)
    codes[torch.arange(N), at[mine]] = (8 + step).to(torch.uint8)
    for zeros in (None, torch.full((N, groups), 8, dtype=torch.uint8)):
        w = _weight({"codes": codes, "scales": torch.ones(N, groups), "zeros": zeros}, group)
        y = ops.q4_matvec(w, x.cuda()).cpu()
        assert torch.equal(y, x[:, at][:, mine] * step.float())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero,code", [(15, 15), (15, 0), (0, 15), (None, 8), (None, 0), (8, "any")])
def test_largest_inputs(dtype, group, zero, code):
    """Inputs of one sign next to 2^116, the largest that are taken: within a group no partial sum
    passes (32 x 31 + 96 x 15) 2^116 < 2^128, whatever the codes and zeros."""
    say(f"case q4 largest inputs {dtype} group={group} zero={zero} code={code}")
    N, K, B = 40, 300, 6
    v = _inputs(N, K, B, group, dtype, F32, False, seed=12)
    groups = -(-K // group)
    v["x"] = torch.full((B, K), 2.0 ** 116 * (1 - 2.0 ** -23)).to(dtype)
    if dtype is BF16:
        v["x"] = torch.full((B, K), 2.0 ** 116 * (1 - 2.0 ** -8), dtype=BF16)
    v["x"][1::2] *= -1
    if code != "any":
        v["codes"][:] = code
    v["zeros"] = torch.full((N, groups), zero, dtype=torch.uint8) if zero is not None else None
    v["scales"] = v["scales"] * 2.0 ** -30
    want, tol = ref.q4(v["x"], v["codes"], v["scales"], v["zeros"], group)
    y = ops.q4_matvec(_weight(v, group), v["x"].cuda())
    assert ref.worst(y, want, ref.stored(want, tol, dtype)) <= 1.0


@pytest.mark.parametrize("N,K,B", [(5003, 1700, 8), (5003, 1750, 9), (9003, 1500, 16), (9003, 1500, 11), (4807, 1500, 16),
                                   (9003, 1500, 8), (4803, 700, 6), (12270, 900, 10)])
def test_several_rows_between_few_and_many_outputs(N, K, B):
    """fp32 rows and 257 to 767 row tiles, where the number of waves goes down to a multiple of four
    (ten and nine to eight, five to four) or stays as it is, by how many workgroups a CU holds."""
    say(f"case q4 wave counts N={N} K={K} B={B}")
    v = _inputs(N, K, B, 64, F32, BF16, B % 2 == 0, seed=13)
    y = ops.q4_matvec(_weight(v, 64), v["x"].cuda())
    want, tol = ref.q4(v["x"], v["codes"], v["scales"], v["zeros"], 64)
    assert ref.worst(y, want, ref.stored(want, tol, F32)) <= 1.0


def test_tiny_inputs_are_not_dropped():
    """fp16 inputs below the normal numbers, whole scales: exact.  In units of 2^-24 no sum passes
    7 groups x 32 x 200 x 15 x 8 < 2^23, and within a group 32 x 200 x 31 < 2^18."""
    say("case q4 tiny inputs")
    v = _inputs(40, 200, 3, 32, F16, F32, True, seed=6)
    gen = torch.Generator().manual_seed(11)
    v["x"] = (torch.randint(-200, 201, (3, 200), generator=gen).double() * 2.0 ** -24).to(F16)
    v["scales"] = (2.0 ** torch.randint(0, 4, v["scales"].shape, generator=gen)).float()
    y = ops.q4_matvec(_weight(v, 32), v["x"].cuda())
    want, _ = ref.q4(v["x"], v["codes"], v["scales"], v["zeros"], 32)
    assert torch.equal(y.cpu(), want.to(F16))


@pytest.mark.parametrize("dtype,B,group", [(F32, 3, 32), (BF16, 3, 128), (F32, 8, 128), (F32, 16, 64), (F32, 11, 128),
                                           (F16, 16, 32)])
def test_many_outputs_and_a_large_weight(dtype, B, group):
    """More weights than the layout's kernels take in one turn, and row tiles enough for several a
    wave (1057: the last wave's are not all there)."""
    say(f"case q4 large {dtype} B={B} group={group}")
    N, K = 16900, 1100
    v = _inputs(N, K, B, group, dtype, F32, True, seed=7)
    y = ops.q4_matvec(_weight(v, group), v["x"].cuda())
    want, tol = ref.q4(v["x"], v["codes"], v["scales"], v["zeros"], group)
    assert ref.worst(y, want, ref.stored(want, tol, dtype)) <= 1.0


def test_bad_rows_stay_alone():
    say("case q4 bad rows")
    v = _inputs(50, 260, 6, 32, F32, BF16, True, seed=2)
    w = _weight(v, 32)
    clean = ops.q4_matvec(w, v["x"].cuda())
    v["x"][1, 3], v["x"][4, 200] = float("nan"), float("inf")
    y = ops.q4_matvec(w, v["x"].cuda())
    for b in (0, 2, 3, 5):
        assert torch.equal(y[b], clean[b])
    assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[4]).any()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_column_slices(dtype):
    """x and y as column slices (aligned or not); what lies beside y and past its last row stays."""
    say(f"case q4 slices {dtype}")
    N, K, B = 45, 270, 3
    v = _inputs(N, K, B, 64, dtype, BF16, True, seed=3)
    w = _weight(v, 64)
    want, tol = ref.q4(v["x"], v["codes"], v["scales"], v["zeros"], 64)
    for lead in (0, 1, 8):
        wide = torch.full((B, K + 5 + lead), float("nan"), dtype=dtype, device="cuda")
        x = wide[:, lead:lead + K]
        x.copy_(v["x"])
        out = torch.full((B + 2, N + 9 + lead), 7.0, dtype=dtype, device="cuda")
        y = ops.q4_matvec(w, x, y=out[:B, lead + 2:lead + 2 + N])
        assert ref.worst(y, want, ref.stored(want, tol, dtype)) <= 1.0
        y.fill_(7.0)
        assert (out == 7).all()


@pytest.mark.parametrize("wt", [F32, BF16, F16])
@pytest.mark.parametrize("st", [F32, BF16, F16])
@pytest.mark.parametrize("N,K,group", [(3, 40, 32), (20, 300, 64), (7, 256, 128), (900, 1300, 32)])
def test_quantize(wt, st, N, K, group):
    """Scales are max|w| / 7 rounded to their type; codes are the nearest, at most half a scale off
    (more only where the rounded scale cannot reach the largest value)."""
    say(f"case q4 quantize {wt}/{st} N={N} K={K} group={group}")
    gen = torch.Generator().manual_seed(N + K)
    w = torch.randn(N, K, generator=gen).to(wt)
    w[1, :group] = 0.0
    q = ops.Q4Weight.quantize(w.cuda(), group=group, scale_dtype=st)
    groups = -(-K // group)
    pad = torch.zeros(N, groups * group)
    pad[:, :K] = w.float()
    m = pad.reshape(N, groups, group).abs().amax(-1)
    assert torch.equal(q.scales.cpu(), (m / 7).to(st))
    codes, s = q.codes.cpu().double(), q.scales.cpu().double().repeat_interleave(group, 1)[:, :K]
    assert codes.min() >= 1 and codes.max() <= 15 and (codes[1, :group] == 8).all()
    off = ((codes - 8) * s - w.double()).abs()
    reach = (w.double().abs() - 7 * s).clamp(min=0)
    # half a scale, and the quotient's rounding (2^-24 of at most 7.03 scales)
    assert (off <= torch.maximum(s * (0.5 + 8 * ref.U), reach + s * 8 * ref.U)).all()
    x = torch.randn(2, K, generator=gen)
    want, tol = ref.q4(x, q.codes.cpu(), q.scales.cpu(), None, group)
    assert ref.worst(ops.q4_matvec(q, x.cuda()), want, ref.stored(want, tol, F32)) <= 1.0


def test_repeats_streams_and_graphs():
    say("case q4 graph")
    v = _inputs(500, 1300, 8, 32, F32, BF16, False, seed=4)
    w = _weight(v, 32)
    x = v["x"].cuda()
    first = ops.q4_matvec(w, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = ops.q4_matvec(w, x)
    s.synchronize()
    assert torch.equal(first, again)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ops.q4_matvec(w, x)
    for i in range(4):
        x.copy_(torch.randn(8, 1300, generator=torch.Generator().manual_seed(i)))
        g.replay()
        eager = ops.q4_matvec(w, x)
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_binding_refuses_mismatches():
    say("case q4 refusals")
    codes = torch.zeros(20, 70, dtype=torch.uint8, device="cuda")
    sc = torch.ones(20, 3, device="cuda")
    w = ops.Q4Weight(codes, sc, group=32)
    x = torch.zeros(2, 70, device="cuda")
    for call in (lambda: ops.Q4Weight(codes, sc, group=16), lambda: ops.Q4Weight(codes, sc, group=64),
                 lambda: ops.Q4Weight(codes.int(), sc, group=32), lambda: ops.Q4Weight(codes[:, ::2], sc, group=32),
                 lambda: ops.Q4Weight(codes, sc.double(), group=32), lambda: ops.Q4Weight(codes, sc, sc, group=32),
                 lambda: ops.Q4Weight.quantize(codes), lambda: ops.Q4Weight.quantize(x, group=50),
                 lambda: ops.Q4Weight.quantize(x, scale_dtype=torch.float64),
                 lambda: ops.q4_matvec(w, x[:, :69]), lambda: ops.q4_matvec(w, x[0]), lambda: ops.q4_matvec(w, x[:0]),
                 lambda: ops.q4_matvec(w, torch.zeros(17, 70, device="cuda")), lambda: ops.q4_matvec(w, x.double()),
                 lambda: ops.q4_matvec(w, x.cpu()), lambda: ops.q4_matvec(w, x, y=torch.zeros(2, 19, device="cuda")),
                 lambda: ops.q4_matvec(w, x, y=x[:, :20])):
        with pytest.raises(fi.FiError) as e:
            call()
        assert e.value.status == fi.FI_EINVAL
