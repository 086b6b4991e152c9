"""The 64-bit references of the gated delta rule and the layer norm against
differences, and the chunked form that the bounds follow against the recurrence."""
import pytest
import torch

from tests import _more_ops_ref as ref


def _slopes(value, v, grads, step):
    for name, d in grads.items():
        g = d.reshape(-1)
        for i in range(0, g.numel(), step):
            h = 1e-5
            lo, hi = ({k: t.clone() if t is not None else None for k, t in v.items()} for _ in range(2))
            lo[name].view(-1)[i] -= h
            hi[name].view(-1)[i] += h
            slope = (value(hi) - value(lo)) / (2 * h)
            # h^2/6 of a third derivative of order 100, and 1e-13 / h of cancellation
            assert abs(slope - float(g[i])) < 1e-7 * (1 + abs(slope)), (name, i)


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("lengths", [None, [5, 0]])
def test_delta_gradients_are_the_slopes(unit, lengths):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)    # noqa: E731
    T, B, HK, H, dk, dv = 6, 2, 1, 2, 3, 4
    v = {"q": r(T, B, HK, dk), "k": r(T, B, HK, dk) * (1.0 if unit else 0.5), "v": r(T, B, H, dv), "g": -r(T, B, H).abs(),
         "beta": torch.sigmoid(r(T, B, H)), "state": r(B, H, dk, dv)}
    dy, df = r(T, B, H, dv), r(B, H, dk, dv)
    n = torch.tensor(lengths) if lengths else None
    args = lambda w: (w["q"], w["k"], w["v"], w["g"], w["beta"], w["state"], n, 0.7, unit)      # noqa: E731

    def value(w):
        o = ref.delta(*args(w))
        return float((o["y"] * dy).sum() + (o["final"] * df).sum())
    o = ref.delta(*args(v), dy, df)
    _slopes(value, v, {"q": o["dq"], "k": o["dk"], "v": o["dv"], "g": o["dg"], "beta": o["dbeta"], "state": o["dstate"]}, 2)


@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("with_da", [False, True])
def test_layer_gradients_are_the_slopes(with_res, with_da):
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)    # noqa: E731
    N, D = 3, 5
    v = {"x": r(N, D), "res": r(N, D) if with_res else None, "weight": r(D), "bias": r(D)}
    dr, da = r(N, D), r(N, D) if with_da else None

    def value(w):
        o = ref.layer(w["x"], w["res"], w["weight"], w["bias"], 1e-3)
        return float((o["r"][0] * dr).sum() + ((o["a"][0] * da).sum() if with_da else 0.0))
    o = ref.layer(v["x"], v["res"], v["weight"], v["bias"], 1e-3, dr, da, back=True)
    _slopes(value, v, {n: o["d" + n][0] for n in v if v[n] is not None and "d" + n in o}, 1)


def test_an_evaluation_in_fp32_stays_within_the_delta_bounds():
    """The recurrence itself in fp32, whose rounding the bounds are to hold as well (it makes fewer sums)."""
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen)                         # noqa: E731
    T, B, H, dk, dv = 150, 1, 2, 24, 10
    q, k, v, g, beta = r(T, B, H, dk), r(T, B, H, dk), r(T, B, H, dv), -0.1 * r(T, B, H).abs(), torch.sigmoid(r(T, B, H))
    S0 = r(B, H, dk, dv)
    want = ref.delta(q, k, v, g, beta, S0, None, 0.2, True)
    tol = ref.delta_bounds(q, k, v, g, beta, S0, None, 0.2, True, 64, 3)
    hq, hk = ref._unit(q, True)[0], ref._unit(k, True)[0]
    S, ys = S0, []
    for t in range(T):
        S = torch.exp(g[t])[..., None, None] * S
        e = v[t] - (hk[t][..., None] * S).sum(-2)
        S = S + hk[t][..., None] * (beta[t][..., None] * e)[..., None, :]
        ys.append(0.2 * (S * hq[t][..., None]).sum(-2))
    assert ref.worst(torch.stack(ys), want["y"], tol["y"]) <= 1.0
    assert ref.worst(S, want["final"], tol["final"]) <= 1.0


def test_a_planted_mistake_passes_no_bound():
    """A decay applied one position late in the oracle: every gradient leaves its bound."""
    gen = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen)                         # noqa: E731
    T, B, H, dk, dv = 70, 1, 1, 16, 8
    q, k, v, g, beta = r(T, B, H, dk), r(T, B, H, dk), r(T, B, H, dv), -0.1 * r(T, B, H).abs(), torch.sigmoid(r(T, B, H))
    S0, dy, df = r(B, H, dk, dv), r(T, B, H, dv), r(B, H, dk, dv)
    want = ref.delta(q, k, v, g, beta, S0, None, 0.25, True, dy, df)
    off = ref.delta(q, k, v, torch.cat((g[1:], g[:1])), beta, S0, None, 0.25, True, dy, df)
    tol = ref.delta_bounds(q, k, v, g, beta, S0, None, 0.25, True, 64, 3, dy, df)
    for name, t in tol.items():
        assert ref.worst(off[name], want[name], t) > 1.0, name
