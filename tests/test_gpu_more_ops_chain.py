"""The gated delta rule, the layer norm and the 8-bit products together, as a user
runs them: a served block beside the library's own mixer, position by position and
over a prompt, and one training step."""
import pytest
import torch

from long_convolution_sequence_amd import fi, ops, workloads
from tests import _more_ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu
F32 = torch.float32


class _Block:
    """norm -> 8-bit projection to [q | k | v | decay, beta] -> delta rule -> norm with the residual."""

    def __init__(self, D, H, seed):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)                   # noqa: E731
        self.D, self.H, self.d = D, H, D // H
        self.w0, self.b0, self.w1, self.b1 = (x.cuda() for x in (1 + r(D) / 10, r(D) / 10, 1 + r(D) / 10, r(D) / 10))
        self.weight = ops.Q8Weight.quantize((r(3 * D + 2 * H, D) / D ** 0.5).cuda())
        self.bias = torch.cat((torch.zeros(3 * D), 2 + r(H), r(H))).cuda()

    def project(self, a):
        """Slices of one projection, decays and strengths made of its last columns."""
        lead, D, H = a.shape[:-1], self.D, self.H
        p = ops.q8_product(self.weight, a.reshape(-1, D), self.bias).reshape(*lead, 3 * D + 2 * H)
        q, k, v = (x.unflatten(-1, (H, self.d)) for x in torch.split(p[..., :3 * D], D, -1))
        return p, q, k, v, -torch.nn.functional.softplus(-p[..., 3 * D:3 * D + H]), torch.sigmoid(p[..., 3 * D + H:])

    def check(self, p, a):
        codes, scales = ref.q8_rows(a.reshape(-1, self.D))
        want, tol = ref.q8(codes, scales, self.weight.codes, self.weight.scales, self.bias)
        assert ref.worst(p.reshape(want.shape), want, ref.stored(want, tol, F32)) <= 1.0


def test_generation_with_a_delta_rule_block():
    """Positions of a two-layer stack in external-block mode, each checked against 64-bit replays of the
    operators' own inputs."""
    w = workloads.custom(M=2, B=3, D=48, L=64, decay=16.0, scale=0.3, seed=7)
    say("case more chain generation M=2 B=3 D=48")
    B, D, M, H = w.B, w.D, w.M, 3
    blocks = [_Block(D, H, 10 + l) for l in range(M)]
    state = torch.zeros(M, B, H, D // H, D // H, device="cuda")
    seen = 0
    with fi.Context(torch.from_numpy(workloads.filters(w)).cuda(), B, map=fi.MAP_EXTERNAL) as ctx:
        x = torch.from_numpy(workloads.x_first(w)).cuda()
        for n in range(20):
            for l, block in enumerate(blocks):
                c = ctx.layer_red(l, x)
                _, a = ops.layer_norm(c, weight=block.w0, bias=block.b0)
                p, q, k, v, g, beta = block.project(a)
                before = state[l].clone()
                y = ops.gated_delta_step(q, k, v, g, beta, state[l], unit=True)
                r, out = ops.layer_norm(y.reshape(B, D), c, weight=block.w1, bias=block.b1)
                value, tol = ref.layer(c, None, block.w0, block.b0, 1e-5)["a"]
                assert ref.worst(a, value, ref.stored(value, tol, F32)) <= 1.0
                block.check(p, a)
                args = [t[None] for t in (q, k, v, g, beta)] + [before, None, (D // H) ** -0.5, True]
                want, bound = ref.delta(*args), ref.delta_bounds(*args, 32, 3)
                assert ref.worst(y[None], want["y"], ref.stored(want["y"], bound["y"], F32)) <= 1.0
                assert ref.worst(state[l], want["final"], ref.stored(want["final"], bound["final"], F32)) <= 1.0
                for name, got in (("r", r), ("a", out)):
                    value, tol = ref.layer(y.reshape(B, D), c, block.w1, block.b1, 1e-5)[name]
                    assert ref.worst(got, value, ref.stored(value, tol, F32)) <= 1.0
                x, seen = out, seen + 1
            ctx.tiles()
            x = torch.tanh(x)
    assert seen == 40


@pytest.mark.parametrize("T", [7, 90])
def test_a_prompt_is_its_positions(T):
    """The block over a prompt of ragged lengths at once, and the same block position by position."""
    say(f"case more chain prompt T={T}")
    B, D, H = 3, 64, 2
    block = _Block(D, H, 3)
    lengths = torch.tensor([T, T // 2, 0], dtype=torch.int32, device="cuda")
    h = torch.randn(T, B, D, generator=torch.Generator().manual_seed(5)).cuda()
    S0 = torch.zeros(B, H, D // H, D // H, device="cuda")

    def block_over(x):
        _, a = ops.layer_norm(x, weight=block.w0, bias=block.b0)
        return block.project(a)[1:]
    y, final = ops.gated_delta(*block_over(h), S0, lengths, unit=True)
    state, ys = S0.clone(), []
    for t in range(T):
        live = (lengths > t).int()
        ys.append(ops.gated_delta_step(*block_over(h[t]), state, live, unit=True))
    args = [*block_over(h), S0, lengths, (D // H) ** -0.5, True]
    bound = ref.delta_bounds(*args, 32, 3)
    want = ref.delta(*args)
    for got in (y, torch.stack(ys)):
        assert ref.worst(got, want["y"], ref.stored(want["y"], bound["y"], F32)) <= 1.0
    for got in (final, state):
        assert ref.worst(got, want["final"], ref.stored(want["final"], bound["final"], F32)) <= 1.0


def test_training_step_of_a_block():
    """Forward and backward through norm, a plain projection, the delta rule and the norm with the residual,
    gradients written straight into the slices of the projection's gradient, against differentiating the
    definition in 64 bits."""
    say("case more chain training T=70 B=2 D=36")
    T, B, D, H = 70, 2, 36, 3
    d = D // H
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen)                    # noqa: E731
    v = {"h": r(T, B, D), "W": r(D, 3 * D) / 6, "w0": 1 + 0.1 * r(D), "b0": 0.1 * r(D), "w1": 1 + 0.1 * r(D), "b1": 0.1 * r(D),
         "g": -0.2 * r(T, B, H).abs(), "beta": torch.sigmoid(r(T, B, H)), "state": r(B, H, d, d)}
    dr, da, df = r(T, B, D), r(T, B, D), r(B, H, d, d)
    c = {k: t.cuda() for k, t in v.items()}

    def step(c, dr, da, df):
        _, a0, s0 = ops.layer_norm(c["h"], weight=c["w0"], bias=c["b0"], save=True)
        p = a0 @ c["W"]
        q, k, x = (t.unflatten(-1, (H, d)) for t in torch.split(p, D, -1))
        y, final, s1 = ops.gated_delta(q, k, x, c["g"], c["beta"], c["state"], unit=True, save=True)
        res, a, s2 = ops.layer_norm(y.flatten(-2), c["h"], weight=c["w1"], bias=c["b1"], save=True)
        g2 = ops.layer_norm_backward(dr, da, y.flatten(-2), c["h"], s2, weight=c["w1"], bias=c["b1"])
        dp = torch.empty_like(p)
        dq, dk, dx = (t.unflatten(-1, (H, d)) for t in torch.split(dp, D, -1))
        g1 = ops.gated_delta_backward(g2.x.unflatten(-1, (H, d)), q, k, x, c["g"], c["beta"], s1, c["state"], dfinal=df, unit=True,
                                      dq=dq, dk=dk, dv=dx)
        dW = a0.reshape(-1, D).t() @ dp.reshape(-1, 3 * D)
        g0 = ops.layer_norm_backward(None, dp @ c["W"].t(), c["h"], None, s0, weight=c["w0"], bias=c["b0"])
        return (res, a, final), {"h": g0.x + g2.res, "W": dW, "w0": g0.weight, "b0": g0.bias, "w1": g2.weight, "b1": g2.bias,
                                 "g": g1.decay, "beta": g1.beta, "state": g1.state}
    outs, got = step(c, dr.cuda(), da.cuda(), df.cuda())

    w = {k: t.double().requires_grad_() for k, t in v.items()}
    norm = lambda t, s, b: torch.nn.functional.layer_norm(t, (D,), s, b, 1e-5)                 # noqa: E731
    p = norm(w["h"], w["w0"], w["b0"]) @ w["W"]
    q, k, x = (t.unflatten(-1, (H, d)) for t in torch.split(p, D, -1))
    q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    S, ys = w["state"], []
    for t in range(T):
        S = torch.exp(w["g"][t])[..., None, None] * S
        e = x[t] - (k[t][..., None] * S).sum(-2)
        S = S + k[t][..., None] * (w["beta"][t][..., None] * e)[..., None, :]
        ys.append(d ** -0.5 * (S * q[t][..., None]).sum(-2))
    R = w["h"] + torch.stack(ys).flatten(-2)
    A = norm(R, w["w1"], w["b1"])
    want = torch.autograd.grad((R * dr.double()).sum() + (A * da.double()).sum() + (S * df.double()).sum(), list(w.values()))
    # a chain of five operators and two products of 36 terms: each adds a relative 2^-24 times at most its
    # length (70 positions, 140 rows, 36 to 108 terms) to the norm of a gradient; the norms' Jacobians amplify
    # by at most their condition of about 2 each, the triangular systems of keys of 12 channels by about 4
    tol = (70 + 140 + 5 * 108) * 16 * ref.U
    for value, t in zip(outs, (R, A, S)):
        assert float((value.double().cpu() - t.detach()).norm() / t.detach().norm()) < tol
    for (name, value), t in zip(((k, got[k]) for k in w), want):
        assert float((value.double().cpu() - t).norm() / t.norm()) < tol, name

    # captured once and replayed, with eager steps between
    into = [t.cuda() for t in (dr, da, df)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _, captured = step(c, *into)
    for i in range(3):
        for t in into:
            t.copy_(torch.randn(t.shape, generator=gen).cuda())
        graph.replay()
        _, eager = step(c, *into)
        torch.cuda.synchronize()
        for k in ("w1", "b1", "g", "beta", "state"):      # what no library product stands behind
            assert torch.equal(captured[k], eager[k]), k
