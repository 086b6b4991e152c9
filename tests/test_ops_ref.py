"""The 64-bit references of the recurrent-block operators against differences:
every gradient formula is the slope of the plain forward definition."""
import pytest
import torch

from tests import _ops_ref as ref


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float64)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("lengths", [None, [7, 0, 4]])
def test_scan_gradients_are_the_slopes(kind, lengths):
    gen = torch.Generator().manual_seed(5 + kind)
    T, B, D = 7, 3, 2
    v = {"x": _rand(gen, T, B, D), "gate": _rand(gen, T, B, D), "bias": _rand(gen, D), "state": _rand(gen, B, D)}
    dy, df = _rand(gen, T, B, D), _rand(gen, B, D)
    n = torch.tensor(lengths) if lengths else None

    def value(w):
        r = ref.scan(w["x"], w["gate"], w["bias"], w["state"], n, kind)
        return float((r["y"][0] * dy).sum() + (r["final"][0] * df).sum())
    grads = ref.scan(v["x"], v["gate"], v["bias"], v["state"], n, kind, dy, df)
    for name in v:
        g = grads["d" + name][0].reshape(-1)
        for i in range(0, g.numel(), 1 if g.numel() < 8 else 5):
            h = 1e-5
            lo, hi = ({k: t.clone() for k, t in v.items()} for _ in range(2))
            lo[name].view(-1)[i] -= h
            hi[name].view(-1)[i] += h
            slope = (value(hi) - value(lo)) / (2 * h)
            # h^2/6 of a third derivative of order 100, and 1e-13 / h of cancellation
            assert abs(slope - float(g[i])) < 1e-7 * (1 + abs(slope)), (name, i)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("with_da", [False, True])
def test_norm_gradients_are_the_slopes(kind, post, with_da):
    gen = torch.Generator().manual_seed(50 + kind)
    N, D = 3, 5
    v = {"o": _rand(gen, N, D), "res": _rand(gen, N, D), "gate": _rand(gen, N, D), "w1": _rand(gen, D),
         "k": _rand(gen, D), "w2": _rand(gen, D)}
    if not post:
        v["w1"] = None
    dr, da = _rand(gen, N, D), _rand(gen, N, D) if with_da else None
    names = {"o": "do", "res": "dres", "gate": "dgate", "w1": "dpost", "k": "dscale", "w2": "dpre"}

    def value(w):
        r = ref.norm(w["o"], w["res"], w["gate"], w["w1"], w["k"], w["w2"], post, kind, 1e-3)
        return float((r["r"][0] * dr).sum() + ((r["a"][0] * da).sum() if with_da else 0.0))
    grads = ref.norm(*(v[n] for n in names), post, kind, 1e-3, dr, da, back=True)
    for name, d in names.items():
        if v[name] is None or d not in grads:
            continue
        g = grads[d][0].reshape(-1)
        for i in range(0, g.numel(), 2):
            h = 1e-5
            lo, hi = ({k: t.clone() if t is not None else None for k, t in v.items()} for _ in range(2))
            lo[name].view(-1)[i] -= h
            hi[name].view(-1)[i] += h
            slope = (value(hi) - value(lo)) / (2 * h)
            assert abs(slope - float(g[i])) < 1e-7 * (1 + abs(slope)), (name, i)
