"""The layer norm with a residual on the GPU against the 64-bit definition, within
the bounds that tests/_more_ops_ref.py derives."""
import pytest
import torch

from long_convolution_sequence_amd import fi, ops
from tests import _more_ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


def _inputs(N, D, dtype, rt, seed=0, shift=0.5):
    gen = torch.Generator().manual_seed(991 * seed + N + 31 * D)
    r = lambda *s: torch.randn(*s, generator=gen)                   # noqa: E731
    return {"x": r(N, D).to(dtype), "res": (2 * r(N, D) + shift).to(rt) if rt else None, "weight": 1 + r(D) / 8,
            "bias": r(D) / 8, "dr": r(N, D).to(rt or dtype), "da": r(N, D).to(dtype)}


def _cuda(v):
    return {k: t.cuda() if t is not None else None for k, t in v.items()}


def _run(c, eps=EPS, **kw):
    w = dict(weight=c["weight"], bias=c["bias"], eps=eps)
    r, a, saved = ops.layer_norm(c["x"], c["res"], save=True, **w)
    g = ops.layer_norm_backward(c["dr"], c["da"], c["x"], c["res"], saved, **w, **kw)
    return {"r": r, "a": a, "dx": g.x, "dres": g.res, "dweight": g.weight, "dbias": g.bias}


def _check(got, v, eps=EPS):
    dtype, rt = v["x"].dtype, v["res"].dtype if v["res"] is not None else v["x"].dtype
    want = ref.layer(v["x"], v["res"], v["weight"], v["bias"], eps, v["dr"], v["da"], back=True)
    types = {"r": rt, "a": dtype, "dx": dtype, "dres": rt}
    for name, g in got.items():
        if g is None:
            continue
        if name not in want:
            assert (g == 0).all(), name
            continue
        value, tol = want[name]
        assert g.shape == value.shape and g.dtype == types.get(name, F32), name
        w = ref.worst(g, value, ref.stored(value, tol, types.get(name, F32)))
        assert w <= 1.0, f"{name}: {w:.3g} of its bound"


CASES = [(1, 1, F32, F32), (1, 864, BF16, F32), (8, 864, BF16, BF16), (3, 7, F16, F16), (5, 64, F32, F32), (33, 100, BF16, F32),
         (17, 255, F16, F32), (70, 256, F32, F32), (9, 257, BF16, None), (4, 1000, F16, F32), (3, 1024, F32, None),
         (6, 1025, BF16, F32), (2, 2050, F32, F32), (3, 4100, F16, F16), (2, 8191, BF16, F32), (2, 16384, F32, F32),
         (3, 16383, F16, F32), (2500, 40, F32, F32), (1300, 96, BF16, F32), (5, 4097, BF16, None), (600, 5001, F16, None),
         (3, 6145, F16, F32), (2, 9000, BF16, BF16), (3, 2, F32, F32)]


@pytest.mark.parametrize("N,D,dtype,rt", CASES)
def test_forward_and_gradients(N, D, dtype, rt):
    say(f"case layer N={N} D={D} {dtype}/{rt}")
    v = _inputs(N, D, dtype, rt)
    got = _run(_cuda(v))
    assert (got["dres"] is None) == (rt is None)
    _check(got, v)


@pytest.mark.parametrize("gone", [("weight",), ("bias",), ("dr",), ("da",), ("weight", "bias"), ("res", "dr"), ("res", "da", "weight")])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_left_out(gone, dtype):
    say(f"case layer without {gone} {dtype}")
    v = _inputs(12, 300, dtype, dtype if "res" in gone else F32, seed=1)
    for k in gone:
        v[k] = None
    got = _run(_cuda(v))
    for name, k in (("dres", "res"), ("dweight", "weight"), ("dbias", "bias")):
        assert (got[name] is None) == (v[k] is None)
    _check(got, v)


def test_without_a_residual_r_is_x():
    say("case layer r is x")
    x = _inputs(5, 70, BF16, None)["x"].cuda()
    r, a = ops.layer_norm(x)
    assert r is x and a.dtype == BF16


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [7, 864, 5001])
def test_an_fp32_stream_into_16_bits(D, dtype):
    """x fp32 without a residual, a of 16 bits; dx fp32."""
    say(f"case layer fp32 into {dtype} D={D}")
    v = _inputs(21, D, dtype, F32, seed=2)
    c = _cuda(v)
    r, a, saved = ops.layer_norm(c["res"], weight=c["weight"], bias=c["bias"], eps=EPS, dtype=dtype, save=True)
    g = ops.layer_norm_backward(c["dr"], c["da"], c["res"], None, saved, weight=c["weight"], bias=c["bias"], eps=EPS,
                                dtype=dtype)
    assert r is c["res"] and g.res is None
    v["x"] = None
    want = ref.layer(None, v["res"], v["weight"], v["bias"], EPS, v["dr"], v["da"], back=True)
    for got, name, t in ((a, "a", dtype), (g.x, "dx", F32), (g.weight, "dweight", F32), (g.bias, "dbias", F32)):
        value, tol = want[name]
        assert got.dtype == t and ref.worst(got, value, ref.stored(value, tol, t)) <= 1.0, name


def test_rows_far_from_zero_and_constant_rows():
    """A mean a thousand times the deviation keeps the digits that fp32 inputs leave; a constant row is
    normed to the bias, a row of zeros too."""
    say("case layer far rows")
    v = _inputs(9, 1000, F32, F32, seed=3, shift=3000.0)
    v["x"][1], v["res"][1] = 0.0, 0.0
    v["x"][2], v["res"][2] = 0.25, 7.5
    got = _run(_cuda(v))
    _check(got, v)
    assert torch.equal(got["a"][2].cpu(), v["bias"]) and torch.equal(got["a"][1].cpu(), v["bias"])


def test_no_rows():
    say("case layer no rows")
    got = _run(_cuda(_inputs(0, 130, BF16, F32)))
    assert got["r"].shape == (0, 130) and got["dx"].shape == (0, 130)
    assert (got["dweight"] == 0).all() and (got["dbias"] == 0).all()


def test_bad_values_stay_in_their_row():
    say("case layer bad rows")
    v = _inputs(6, 200, BF16, F32, seed=4)
    clean = _run(_cuda(v))
    v["x"][2, 5], v["res"][4, 0] = float("nan"), float("inf")
    got = _run(_cuda(v))
    for name in ("r", "a", "dx", "dres"):
        for i in (0, 1, 3, 5):
            assert torch.equal(got[name][i], clean[name][i])
    assert got["a"][2].isnan().any() and not torch.isfinite(got["a"][4]).all()


@pytest.mark.parametrize("D,dtype", [(40, BF16), (864, BF16), (33, F32), (1200, F16)])
def test_column_slices(D, dtype):
    say(f"case layer slices D={D} {dtype}")
    N = 37
    v = _inputs(N, D, dtype, dtype, seed=5)
    c = _cuda(v)
    for lead in (0, 1, 8):
        wide = torch.full((N, 2 * D + 3 + lead), 7.0, dtype=dtype, device="cuda")
        grads = torch.full((N, 2 * D + 3 + lead), 9.0, dtype=dtype, device="cuda")
        cols = (slice(lead, lead + D), slice(lead + D + 2, lead + 2 * D + 2))
        s = dict(c, x=wide[:, cols[0]], res=wide[:, cols[1]])
        s["x"].copy_(c["x"]), s["res"].copy_(c["res"])
        got = _run(s, dx=grads[:, cols[0]], dres=grads[:, cols[1]])
        _check(got, v)
        mask = torch.ones(wide.shape[1], dtype=torch.bool, device="cuda")
        mask[cols[0]] = mask[cols[1]] = False
        assert (wide[:, mask] == 7).all() and (grads[:, mask] == 9).all()


def test_in_place_residual_and_gradient():
    say("case layer in place")
    for D, rt in ((130, F32), (864, BF16), (2000, F32), (9000, F32), (7, BF16), (1037, BF16), (2001, F32), (8195, BF16)):
        v = _inputs(21, D, BF16, rt, seed=6)
        c = _cuda(v)
        want = _run(c)
        dr = c["dr"].clone()
        got = _run(dict(c, dr=dr), dres=dr)
        assert got["dres"] is dr
        assert all(torch.equal(got[k], want[k]) for k in want)
        res = c["res"].clone()
        r, a = ops.layer_norm(c["x"], res, weight=c["weight"], bias=c["bias"], eps=EPS, r=res)
        assert r is res and torch.equal(r, want["r"]) and torch.equal(a, want["a"])


def test_leading_dimensions_repeats_streams_and_graphs():
    say("case layer [T][B][D], side stream, graph")
    v = _inputs(60, 96, BF16, F32, seed=7)
    c = _cuda(v)
    flat = _run(c)
    deep = {k: (t.reshape(20, 3, 96) if t.dim() == 2 else t) for k, t in c.items()}
    got = _run(deep)
    assert got["r"].shape == (20, 3, 96) and all(torch.equal(got[k].reshape(flat[k].shape), flat[k]) for k in flat)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        side = _run(c)
    s.synchronize()
    assert all(torch.equal(side[k], flat[k]) for k in flat)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(c)
    for i in range(4):
        new = _cuda(_inputs(60, 96, BF16, F32, seed=8 + i))
        for k, t in new.items():
            c[k].copy_(t)
        g.replay()
        eager = _run(new)
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], eager[k]) for k in out)


def test_offsets_past_32_bits():
    say("case layer far rows in memory")
    N, D, pitch = 1100, 24, 1 << 21
    v = _inputs(N, D, BF16, BF16, seed=10)
    c = _cuda(v)
    buf = torch.empty(N * pitch, dtype=BF16, device="cuda")
    far = lambda at: buf.as_strided((N, D), (pitch, 1), at)          # noqa: E731
    s = dict(c)
    for i, k in enumerate(("x", "res", "dr", "da")):
        s[k] = far(64 * i)
        s[k].copy_(c[k])
    _check(_run(s, dx=far(512), dres=far(640)), v)


@pytest.mark.parametrize("D,dtype,rt", [(864, BF16, F32), (1001, F16, F16), (256, F32, F32), (5000, BF16, BF16), (40, BF16, F32)])
def test_no_part_of_the_column_sums_is_lost(D, dtype, rt):
    """Inputs past the size from which they are read as streams: rows as in slices below that size, and
    column sums of terms of one sign within less than half of one workgroup's part."""
    N = (1 << 28) // (D * (4 if dtype is F32 else 2) * 2) + 77
    say(f"case layer column parts N={N} D={D} {dtype}/{rt}")
    gen = torch.Generator(device="cuda").manual_seed(D + 1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").clamp_(-3, 3)        # noqa: E731
    x, res = (r(N, D) / 5).to(dtype), r(N, D).to(rt)
    da = (1 + r(N, D) / 5).to(dtype)
    # one sign in every column's sum: da's is that of the normed row, which r's own sign all but fixes
    da = torch.where(res.float() + x.float() < 0, -da.float(), da.float()).to(dtype)
    c = {"x": x, "res": res, "weight": 1 + r(D) / 8, "bias": r(D) / 8, "dr": r(N, D).to(rt), "da": da}
    got = _run(c)
    groups = ops._layer_workspace(N, D, ops._TYPES[dtype], ops._TYPES[rt]) // (8 * D)
    chain = -(-N // groups) + 4 + -(-groups // 16) + 16
    total = torch.zeros(2, D, dtype=torch.float64, device="cuda")
    size = torch.zeros(2, D, dtype=torch.float64, device="cuda")
    step = -(-N // 8)
    for i in range(0, N, step):
        part = {k: t[i:i + step] if t.dim() == 2 else t for k, t in c.items()}
        one = _run(part)
        for k in ("r", "a", "dx", "dres"):
            assert torch.equal(got[k][i:i + step], one[k]), f"{k} rows {i}.."
        R, e = part["x"].double() + part["res"].double(), part["da"].double()
        mean = R.mean(-1, keepdim=True)
        u = (R - mean) * ((R - mean).pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
        total += torch.stack(((e * u).sum(0), e.sum(0)))
        # a term's own error: two means (D / 64 + 24 roundings each) and 60 others
        near = (e * u).abs() * chain + e.abs() * (u.abs() + 1) * (2 * D / 64 + 110)
        size += torch.stack((near.sum(0), (e.abs() * chain).sum(0))) * ref.U
    assert (size[0] < total[0].abs() / (2 * groups)).all(), "the bound says nothing"
    for g, t, s in ((got["dweight"], total[0], size[0]), (got["dbias"], total[1], size[1])):
        assert ((g.double() - t).abs() <= s + ref.U * t.abs()).all()


def test_binding_refuses_mismatches():
    say("case layer refusals")
    x = torch.zeros(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    saved = torch.zeros(2, 4, device="cuda")
    for call in (lambda: ops.layer_norm(x, x[:3]), lambda: ops.layer_norm(x, x.half()), lambda: ops.layer_norm(x.double()),
                 lambda: ops.layer_norm(x, x.cpu()), lambda: ops.layer_norm(x, weight=w[:7]), lambda: ops.layer_norm(x, bias=w.half()),
                 lambda: ops.layer_norm(None), lambda: ops.layer_norm(x, eps=-1.0), lambda: ops.layer_norm(x, a=x),
                 lambda: ops.layer_norm(x, eps="1"), lambda: ops.layer_norm(x, r=x), lambda: ops.layer_norm(x.half(), dtype=F32),
                 lambda: ops.layer_norm(x, x, dtype=BF16), lambda: ops.layer_norm(x, dtype=torch.float64),
                 lambda: ops.layer_norm(torch.zeros(2, 16385, device="cuda")), lambda: ops.layer_norm(x[:, ::2]),
                 lambda: ops.layer_norm_backward(x, x, x, None, None),
                 lambda: ops.layer_norm_backward(x, x, x, None, saved[:, :3]),
                 lambda: ops.layer_norm_backward(x, x[:2], x, None, saved),
                 lambda: ops.layer_norm_backward(x, x, x, None, saved, dres=x),
                 lambda: ops.layer_norm_backward(x, x, x, None, saved, dx=x)):
        with pytest.raises(fi.FiError) as e:
            call()
        assert e.value.status == fi.FI_EINVAL
