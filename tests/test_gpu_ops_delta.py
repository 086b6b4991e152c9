"""The gated delta rule on the GPU against its recurrence in 64 bits, within the
bounds that tests/_more_ops_ref.py derives, and in the 2-norm."""
import math

import pytest
import torch

from long_convolution_sequence_amd import fi, ops
from tests import _more_ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
CHUNK = {F32: 32, BF16: 64, F16: 32}
NAMES = ("q", "k", "v", "g", "beta")


def _inputs(T, B, HK, H, dk, dv, dtype, unit, lengths=None, seed=0, decay=0.2, state=True):
    gen = torch.Generator().manual_seed(1009 * seed + T + 7 * B + 31 * H + 101 * dk + 211 * dv)
    r = lambda *s: torch.randn(*s, generator=gen)                   # noqa: E731
    size = 1.0 if unit else 0.9 / math.sqrt(dk)
    return {"q": (size * r(T, B, HK, dk)).to(dtype), "k": (size * r(T, B, HK, dk)).to(dtype), "v": r(T, B, H, dv).to(dtype),
            "g": -decay * r(T, B, H).abs(), "beta": torch.sigmoid(r(T, B, H)),
            "state": r(B, H, dk, dv) / 2 if state else None,
            "lengths": torch.tensor(lengths, dtype=torch.int32) if lengths else None,
            "dy": r(T, B, H, dv).to(dtype), "dfinal": r(B, H, dk, dv) if state else None}


def _cuda(v):
    return {k: t.cuda() if t is not None else None for k, t in v.items()}


def _run(c, unit, train=True, scale=None, **kw):
    args = [c[n] for n in NAMES]
    if not train:
        y, final = ops.gated_delta(*args, c["state"], c["lengths"], unit=unit, scale=scale)
        return {"y": y, "final": final}
    y, final, saved = ops.gated_delta(*args, c["state"], c["lengths"], unit=unit, scale=scale, save=True)
    d = ops.gated_delta_backward(c["dy"], *args, saved, c["state"], c["lengths"], dfinal=c["dfinal"], unit=unit, scale=scale, **kw)
    return {"y": y, "final": final, "dq": d.q, "dk": d.k, "dv": d.v, "dg": d.decay, "dbeta": d.beta, "dstate": d.state}


def _check(got, v, unit, scale=None):
    T, B, H, dv = v["v"].shape
    dk, dtype = v["q"].shape[-1], v["q"].dtype
    scale = dk ** -0.5 if scale is None else scale
    C = CHUNK[dtype]
    grads = (v["dy"], v["dfinal"]) if "dq" in got else ()
    args = [v[n] for n in NAMES] + [v["state"], v["lengths"], scale, unit]
    want = ref.delta(*args, *grads)
    tol = ref.delta_bounds(*args, C, 3 if dtype is F32 else 2, *grads)
    # in the 2-norm independent roundings add as their squares do: a value's chain is at most four products of
    # dk, dv and the chunk's terms a chunk, each amplified by at most 8 by what cancels
    chain = 8 * ref.U * math.sqrt(4 * (dk + dv + 2 * C) * (1 + T / C))
    for name, g in got.items():
        if g is None:
            continue
        t = dtype if name in ("y", "dq", "dk", "dv") else F32
        assert g.shape == want[name].shape and g.dtype == t, name
        w = ref.worst(g, want[name], ref.stored(want[name], tol[name], t))
        assert w <= 1.0, f"{name}: {w:.3g} of its bound"
        d = float((g.double().cpu() - want[name]).norm())
        n = float(want[name].norm())
        assert d <= (chain + (2.0 ** -16 if t is not F32 else 0.0) + ref.HALF_STEP[t]) * n + 1e-30, f"{name}: {d / n:.3g}"


CASES = [  # T B HK H dk dv dtype unit lengths
    (1, 1, 1, 1, 1, 1, F32, False, None), (1, 2, 1, 2, 16, 33, BF16, True, None), (2, 1, 1, 1, 33, 1, F16, True, None),
    (8, 3, 2, 4, 128, 40, BF16, True, [8, 0, 5]), (9, 1, 1, 1, 16, 20, F32, False, None), (31, 1, 1, 1, 5, 7, F32, True, None),
    (32, 1, 1, 1, 32, 32, F16, False, None), (33, 2, 1, 1, 40, 64, F32, True, [33, 32]), (63, 1, 1, 2, 96, 32, BF16, True, None),
    (64, 2, 1, 2, 32, 32, BF16, False, [64, 1]), (65, 1, 1, 1, 64, 96, BF16, True, None), (100, 1, 2, 2, 7, 130, F16, True, None),
    (130, 3, 2, 4, 72, 41, F16, False, [130, 65, 0]), (129, 2, 1, 3, 128, 128, BF16, True, [129, 64]),
    (200, 2, 3, 3, 64, 96, F32, True, [133, 200]), (192, 1, 1, 1, 128, 16, F32, True, None), (300, 1, 1, 2, 100, 150, BF16, True, None)]


@pytest.mark.parametrize("T,B,HK,H,dk,dv,dtype,unit,lengths", CASES)
def test_forward_and_gradients(T, B, HK, H, dk, dv, dtype, unit, lengths):
    say(f"case delta T={T} B={B} HK={HK} H={H} dk={dk} dv={dv} {dtype} unit={unit} {lengths}")
    v = _inputs(T, B, HK, H, dk, dv, dtype, unit, lengths)
    c = _cuda(v)
    _check(_run(c, unit), v, unit)
    _check(_run(c, unit, train=False), v, unit)


@pytest.mark.parametrize("T,lengths", [(2500, None), (2111, [2111, 900])])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_sequences_in_segments(T, lengths, dtype):
    """Long sequences of few heads, which run in segments that are joined (one of them ends inside one)."""
    say(f"case delta segments T={T} {dtype} {lengths}")
    v = _inputs(T, 2 if lengths else 1, 1, 1, 24, 40, dtype, True, lengths, decay=0.02)
    c = _cuda(v)
    _check(_run(c, True), v, True)
    _check(_run(c, True, train=False), v, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_positions_one_by_one_as_a_sequence(dtype):
    """Steps in place, a short sequence and one in chunks agree within their bounds; an empty slot keeps its state."""
    say(f"case delta steps {dtype}")
    v = _inputs(40, 3, 1, 2, 48, 36, dtype, True)
    c = _cuda(v)
    state = c["state"].clone()
    live = torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda")
    ys = [ops.gated_delta_step(*(c[n][t] for n in NAMES), state, live, unit=True) for t in range(40)]
    w = dict(v, lengths=torch.tensor([40, 40, 0], dtype=torch.int32))
    _check({"y": torch.stack(ys), "final": state}, w, True)
    assert torch.equal(state[2], c["state"][2]) and all((y[2] == 0).all() for y in ys)
    first = {n: (t[:8] if n in NAMES else t) for n, t in v.items()}
    _check(_run(_cuda(first), True, train=False), first, True)


def test_no_state_no_final_gradient_and_a_scale():
    say("case delta left out")
    v = _inputs(70, 2, 1, 2, 20, 24, F32, True, state=False)
    got = _run(_cuda(v), True, scale=-1.5)
    assert got["dstate"] is None
    _check(got, v, True, scale=-1.5)


def test_no_positions():
    say("case delta T=0")
    v = _inputs(0, 2, 1, 2, 20, 24, F32, True)
    c = _cuda(v)
    got = _run(c, True)
    assert torch.equal(got["final"], c["state"]) and torch.equal(got["dstate"], c["dfinal"])
    assert got["y"].shape == (0, 2, 2, 24) and got["dq"].shape == (0, 2, 1, 20)
    c["state"] = c["dfinal"] = None
    assert (_run(c, True)["final"] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decays_that_forget_everything(dtype):
    """-infinity and -1000 at some positions, 0 at others: finite values, nothing before them counts, and the
    positions after a large one keep their digits."""
    say(f"case delta resets {dtype}")
    v = _inputs(150, 1, 1, 2, 24, 16, dtype, True, decay=0.05)
    v["g"][40], v["g"][64], v["g"][100] = float("-inf"), -1000.0, -20000.0
    v["g"][101:110] = 0.0
    w = dict(v, g=v["g"].clamp_min(-1e4))                  # e^-10^4 is 0
    _check(_run(_cuda(v), True), w, True)


def test_strong_writes():
    """Betas up to 2 (eigenvalues down to -1), and zeros."""
    say("case delta beta to 2")
    v = _inputs(140, 1, 1, 1, 32, 32, BF16, True)
    v["beta"] = v["beta"] * 2
    v["beta"][::5] = 0.0
    v["beta"][3::7] = 2.0
    _check(_run(_cuda(v), True), v, True)


def test_like_keys():
    """The same key at many positions: the triangular system is as far from a unit one as it gets."""
    say("case delta like keys")
    for dtype in (BF16, F32):
        v = _inputs(130, 1, 1, 1, 16, 16, dtype, True, decay=0.01)
        v["k"][10:60] = v["k"][10]
        v["beta"][10:60] = 0.999
        _check(_run(_cuda(v), True), v, True)


def test_values_past_a_length_count_for_nothing():
    say("case delta NaN behind the end")
    for dtype in (BF16, F32):
        v = _inputs(100, 2, 1, 2, 24, 20, dtype, True, [70, 33])
        clean = _run(_cuda(v), True)
        for n in (*NAMES, "dy"):
            for b, end in enumerate((70, 33)):
                v[n][end:, b] = float("nan") if b else float("inf")
        got = _run(_cuda(v), True)
        for k in got:
            assert torch.equal(got[k], clean[k]), k
        assert (got["y"][70:, 0] == 0).all() and (got["dq"][33:, 1] == 0).all() and (got["dg"][70:, 0] == 0).all()


def test_bad_values_stay_in_their_head():
    say("case delta bad values")
    v = _inputs(100, 2, 2, 2, 24, 20, BF16, True)
    clean = _run(_cuda(v), True)
    v["v"][80, 1, 0, 3] = float("nan")
    got = _run(_cuda(v), True)
    for k, t in got.items():
        lead = t if k in ("final", "dstate") else t.transpose(0, 1)
        want = clean[k] if k in ("final", "dstate") else clean[k].transpose(0, 1)
        assert torch.equal(lead[0], want[0]), k
    assert torch.equal(got["y"][:64], clean["y"][:64]) and not torch.isfinite(got["y"][80:, 1, 0, 3].float()).any()
    assert torch.equal(got["y"][:, 1, 1], clean["y"][:, 1, 1]) and torch.equal(got["final"][1, 1], clean["final"][1, 1])


def test_slices_of_one_projection():
    """q, k, v, decay and beta as slices of wider tensors, y and the gradients written into others'; no other
    column changes."""
    say("case delta slices")
    T, B, HK, H, dk, dv = 75, 2, 1, 2, 24, 20
    for dtype in (BF16, F32):
        v = _inputs(T, B, HK, H, dk, dv, dtype, True)
        c = _cuda(v)
        want = _run(c, True)
        sizes = [HK * dk, HK * dk, H * dv]
        wide = torch.full((T, B, 3 + sum(sizes)), 7.0, dtype=dtype, device="cuda")
        grads = torch.full_like(wide, 9.0)
        gates = torch.zeros(T, B, 2 * H + 1, device="cuda")
        shapes = [(T, B, HK, dk), (T, B, HK, dk), (T, B, H, dv)]
        cut = lambda t: [x.unflatten(-1, s[2:]) for x, s in zip(torch.split(t[..., 2:-1], sizes, -1), shapes)]   # noqa: E731
        s = dict(c)
        for n, view in zip(("q", "k", "v"), cut(wide)):
            view.copy_(c[n])
            s[n] = view
        s["g"], s["beta"] = gates[..., :H], gates[..., H + 1:]
        s["g"].copy_(c["g"]), s["beta"].copy_(c["beta"])
        dq, dk_, dv_ = cut(grads)
        got = _run(s, True, dq=dq, dk=dk_, dv=dv_)
        assert all(torch.equal(got[k], want[k]) for k in want)
        for t, fill in ((wide, 7), (grads, 9)):
            assert (t[..., :2] == fill).all() and (t[..., -1] == fill).all()
        out = torch.full((T, B, H * dv + 4), 5.0, dtype=dtype, device="cuda")
        y, _ = ops.gated_delta(*(s[n] for n in NAMES), s["state"], unit=True, y=out[..., 1:1 + H * dv].unflatten(-1, (H, dv)))
        assert torch.equal(y, want["y"]) and (out[..., 0] == 5).all() and (out[..., 1 + H * dv:] == 5).all()


def test_in_place_state_repeats_streams_and_graphs():
    say("case delta in place, side stream, graph")
    shape = (700, 1, 1, 2, 40, 24, BF16, True)
    c = _cuda(_inputs(*shape))
    want = _run(c, True)
    for _ in range(3):
        again = _run(c, True)
        assert all(torch.equal(again[k], want[k]) for k in want)
    state = c["state"].clone()
    y, final = ops.gated_delta(*(c[n] for n in NAMES), state, unit=True, final=state)
    plain = _run(c, True, train=False)
    assert final is state and torch.equal(final, plain["final"]) and torch.equal(y, plain["y"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        side = _run(c, True)
    s.synchronize()
    assert all(torch.equal(side[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(c, True)
    for i in range(4):
        new = _cuda(_inputs(*shape, seed=1 + i))
        for k, t in new.items():
            if t is not None:
                c[k].copy_(t)
        g.replay()
        eager = _run(new, True)
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], eager[k]) for k in out)


def test_two_calls_at_once():
    """Two sequences on two streams, workspaces of their own: as one after the other."""
    say("case delta two streams")
    a, b = _cuda(_inputs(1500, 1, 1, 1, 32, 32, BF16, True)), _cuda(_inputs(900, 2, 1, 1, 64, 16, F32, True))
    wa, wb = _run(a, True), _run(b, True)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(sa):
            ga = _run(a, True)
        with torch.cuda.stream(sb):
            gb = _run(b, True)
    torch.cuda.synchronize()
    assert all(torch.equal(ga[k], wa[k]) for k in wa) and all(torch.equal(gb[k], wb[k]) for k in wb)


def test_offsets_past_32_bits():
    say("case delta far rows")
    T, H, dk, dv, pitch = 520, 1, 8, 12, 1 << 22
    v = _inputs(T, 1, 1, H, dk, dv, BF16, True)
    c = _cuda(v)
    buf = torch.empty(T * pitch, dtype=BF16, device="cuda")
    far = lambda at, d: buf.as_strided((T, 1, 1, d), (pitch, pitch, d, 1), at)          # noqa: E731
    s = dict(c)
    for i, (n, d) in enumerate((("q", dk), ("k", dk), ("v", dv), ("dy", dv))):
        s[n] = far(64 * i, d)
        s[n].copy_(c[n])
    got = _run(s, True, dq=far(512, dk), dk=far(640, dk), dv=far(768, dv))
    want = _run(c, True)
    assert all(torch.equal(got[k], want[k]) for k in want)
    _check(got, v, True)


@pytest.mark.parametrize("share", [1, 3])
def test_gradients_against_differences(share):
    """The slope of the kernels' own forward pass along random directions, from wide differences in fp32."""
    say(f"case delta differences share={share}")
    v = _inputs(50, 1, 1, share, 12, 10, F32, True, seed=4)
    c = _cuda(v)
    got = _run(c, True)
    gen = torch.Generator().manual_seed(9)
    grads = {"q": "dq", "k": "dk", "v": "dv", "g": "dg", "beta": "dbeta", "state": "dstate"}

    def loss(w):
        o = _run(w, True, train=False)
        return float((o["y"].double() * c["dy"].double()).sum() + (o["final"].double() * c["dfinal"].double()).sum())
    for n, d in grads.items():
        u = torch.randn(c[n].shape, generator=gen).cuda()
        h = 2.0 ** -7
        slope = (loss(dict(c, **{n: c[n] + h * u})) - loss(dict(c, **{n: c[n] - h * u}))) / (2 * h)
        exact = float((got[d].double() * u.double()).sum())
        # h^2 / 6 of the third derivative (of the gradient's size times a few tens), and the values' rounding
        # of 2^-21 of |y| |dy| over h
        size = float(got[d].double().norm() * u.double().norm())
        loose = float(c["dy"].double().norm() * 10 + c["dfinal"].double().norm() * 10) * 2.0 ** -21 / h
        assert abs(slope - exact) <= 40 * h * h * size + loose, n


def test_binding_refuses_mismatches():
    say("case delta refusals")
    c = _cuda(_inputs(5, 2, 1, 2, 8, 6, F32, True))
    a = [c[n] for n in NAMES]
    q, k, v, g, b = a
    _, _, saved = ops.gated_delta(*a, save=True)
    for call in (lambda: ops.gated_delta(q.half(), k, v, g, b), lambda: ops.gated_delta(q, k[:4], v, g, b),
                 lambda: ops.gated_delta(q, k, v[:, :1], g, b), lambda: ops.gated_delta(q, k, v, g.half(), b),
                 lambda: ops.gated_delta(q, k, v, g, b[..., :1]), lambda: ops.gated_delta(None, k, v, g, b),
                 lambda: ops.gated_delta(q, None, v, g, b), lambda: ops.gated_delta(q, k, v, None, b),
                 lambda: ops.gated_delta(q, k, v, g, None), lambda: ops.gated_delta(q, k, v, g, b, c["state"].half()),
                 lambda: ops.gated_delta(q, k, v, g, b, c["state"][:1]), lambda: ops.gated_delta(q, k, v, g, b, scale="1"),
                 lambda: ops.gated_delta(q, k, v, g, b, scale=float("nan")), lambda: ops.gated_delta(q[..., ::2], k[..., ::2], v, g, b),
                 lambda: ops.gated_delta(q.cpu(), k, v, g, b), lambda: ops.gated_delta(q, k, v, g, b, y=v),
                 lambda: ops.gated_delta(q.expand(5, 2, 1, 8)[:, :, :0], k[:, :, :0], v, g, b),
                 lambda: ops.gated_delta(q.repeat(1, 1, 3, 1), k.repeat(1, 1, 3, 1), v, g, b),
                 lambda: ops.gated_delta(q.repeat(1, 1, 1, 17), k.repeat(1, 1, 1, 17), v, g, b),
                 lambda: ops.gated_delta(*a, lengths=torch.ones(2, device="cuda")),
                 lambda: ops.gated_delta_step(*(t[0] for t in a), None), lambda: ops.gated_delta_step(*a, c["state"]),
                 lambda: ops.gated_delta_backward(None, *a, saved), lambda: ops.gated_delta_backward(c["dy"], *a, None),
                 lambda: ops.gated_delta_backward(c["dy"], *a, saved[:-1]), lambda: ops.gated_delta_backward(c["dy"][:4], *a, saved),
                 lambda: ops.gated_delta_backward(c["dy"], *a, saved, dq=q), lambda: ops.gated_delta_backward(c["dy"], *a, saved, dv=c["dy"])):
        with pytest.raises(fi.FiError) as e:
            call()
        assert e.value.status == fi.FI_EINVAL
