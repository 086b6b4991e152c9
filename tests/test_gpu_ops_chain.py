"""The recurrent-block operators together, as a user runs them: around the
library's own mixer in external-block mode, and as one training step."""
import numpy as np
import pytest
import torch

from long_convolution_sequence_amd import fi, ops, workloads
from tests import _ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu


def test_generation_with_a_recurrent_block():
    """Positions of a two-layer stack in external-block mode: the long convolution mixes, then the
    caller's block runs on these operators: norm, 4-bit projection to [x | gate | out gate], the
    recurrence's step on a column slice, gated norm with the residual, and the next layer's norm.
    Every position is checked layer by layer against 64-bit replays of the operators' own inputs."""
    w = workloads.custom(M=2, B=3, D=48, L=64, decay=16.0, scale=0.3, seed=5)
    say("case chain generation M=2 B=3 D=48")
    B, D, M = w.B, w.D, w.M
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen)                    # noqa: E731
    proj = [ops.Q4Weight.quantize((0.3 * r(3 * D, D)).cuda(), group=32) for _ in range(M)]
    bias = [1 + r(D).cuda() for _ in range(M)]
    w1, w2, k = ([(1 + 0.1 * r(D)).cuda() for _ in range(M)] for _ in range(3))
    state = torch.zeros(M, B, D, device="cuda")
    seen = []
    with fi.Context(torch.from_numpy(workloads.filters(w)).cuda(), B, map=fi.MAP_EXTERNAL) as ctx:
        x = torch.from_numpy(workloads.x_first(w)).cuda()
        for n in range(24):
            for l in range(M):
                c = ctx.layer_red(l, x)
                p = ops.q4_matvec(proj[l], c)
                before = state[l].clone()
                y = ops.gated_scan_step(p[:, :D], p[:, D:2 * D], state[l], bias[l])
                res, a = ops.block_norm(y, c, p[:, 2 * D:], post_weight=w1[l], scale=k[l], pre_weight=w2[l],
                                        post_norm=True, act=ops.GATE_SILU)
                seen.append((l, c.clone(), p.clone(), before, state[l].clone(), y.clone(), res.clone(), a.clone()))
                x = a
            ctx.tiles()
            x = torch.tanh(x)
    assert len(seen) == 48
    for l, c, p, before, after, y, res, a in seen:
        want, tol = ref.q4(c, proj[l].codes, proj[l].scales, None, 32)
        assert ref.worst(p, want, ref.stored(want, tol, torch.float32)) <= 1.0
        s = ref.scan(p[None, :, :D], p[None, :, D:2 * D], bias[l], before, None, ops.SCAN_CONVEX)
        assert ref.worst(after, s["final"][0], ref.stored(*s["final"], torch.float32)) <= 1.0
        assert torch.equal(y, after)
        b = ref.norm(y, c, p[:, 2 * D:], w1[l], k[l], w2[l], True, 2, 1e-6)
        assert ref.worst(res, b["r"][0], ref.stored(*b["r"], torch.float32)) <= 1.0
        assert ref.worst(a, b["a"][0], ref.stored(*b["a"], torch.float32)) <= 1.0


def _block(v, T, B, D):
    """loss of one block in 64 bits: norm, projection, recurrence, gated norm with residual, norm."""
    rms = lambda t: t * torch.rsqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6)      # noqa: E731
    p = (rms(v["h"]) * v["w0"]) @ v["W"]
    x, z, g = p[..., :D], p[..., D:2 * D] + v["bias"], p[..., 2 * D:]
    s, ys = v["state"], []
    for t in range(T):
        s = torch.sigmoid(z[t]) * s + torch.sigmoid(-z[t]) * x[t]
        ys.append(s)
    y = torch.stack(ys)
    r = v["h"] + v["k"] * (rms(y) * v["w1"]) * torch.nn.functional.silu(g)
    return r, rms(r) * v["w2"], s


def test_training_step_of_a_block():
    """Forward and backward through the operators with plain products between them, gradients written
    straight into the slices of the projection's gradient, against differentiating the definition."""
    say("case chain training T=70 B=2 D=36")
    T, B, D = 70, 2, 36
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen)                    # noqa: E731
    v = {"h": r(T, B, D), "W": r(D, 3 * D) / 6, "w0": 1 + 0.1 * r(D), "w1": 1 + 0.1 * r(D), "w2": 1 + 0.1 * r(D),
         "k": 0.5 + 0.1 * r(D), "bias": 1 + r(D), "state": r(B, D)}
    dr, da, df = r(T, B, D), r(T, B, D), r(B, D)
    c = {k: t.cuda() for k, t in v.items()}

    _, a0, sv0 = ops.block_norm(None, c["h"], pre_weight=c["w0"], save=True)
    p = a0 @ c["W"]
    x, z, g = p[..., :D], p[..., D:2 * D], p[..., 2 * D:]
    y, fin, sv1 = ops.gated_scan(x, z, c["bias"], c["state"], save=True)
    nw = dict(post_weight=c["w1"], scale=c["k"], pre_weight=c["w2"], post_norm=True)
    res, a, sv2 = ops.block_norm(y, c["h"], g, save=True, **nw)
    dp = torch.empty_like(p)
    gr = ops.block_norm_backward(dr.cuda(), da.cuda(), y, c["h"], g, sv2, dgate=dp[..., 2 * D:], **nw)
    _, _, dbias, dstate = ops.gated_scan_backward(gr.o, x, z, sv1, c["bias"], c["state"], dfinal=df.cuda(),
                                                  dx=dp[..., :D], dgate=dp[..., D:2 * D])
    dW = a0.reshape(-1, D).t() @ dp.reshape(-1, 3 * D)
    g0 = ops.block_norm_backward(gr.res, dp @ c["W"].t(), None, c["h"], None, sv0, pre_weight=c["w0"])
    got = {"h": g0.res, "W": dW, "w0": g0.pre_weight, "w1": gr.post_weight, "w2": gr.pre_weight, "k": gr.scale,
           "bias": dbias, "state": dstate}

    v64 = {k: t.double().requires_grad_() for k, t in v.items()}
    R, A, S = _block(v64, T, B, D)
    want = torch.autograd.grad((R * dr.double()).sum() + (A * da.double()).sum() + (S * df.double()).sum(),
                               list(v64.values()))
    # a chain of five operators and two products of 36 terms: each adds a relative 2^-24 times at
    # most its length (70 positions, 140 rows) to the norm of a gradient, the norms' Jacobians
    # amplify by at most their condition of about 2 each
    tol = (70 + 140 + 5 * 36) * 4 * ref.U
    for value, w in ((res, R), (a, A), (fin, S)):
        assert float((value.double().cpu() - w.detach()).norm() / w.detach().norm()) < tol
    for (name, value), w in zip(((k, got[k]) for k in v64), want):
        assert float((value.double().cpu() - w).norm() / w.norm()) < tol, name


def test_many_training_steps_of_the_chain_agree():
    """The same step captured once and replayed gives what eager calls give, with eager steps between."""
    say("case chain captured")
    T, B, D = 300, 2, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")     # noqa: E731
    x, z, g, h, dr = (r(T, B, D) for _ in range(5))
    w, bias = 1 + 0.1 * r(D), 1 + r(D)

    def step():
        y, _, s1 = ops.gated_scan(x, z, bias, save=True)
        res, _, s2 = ops.block_norm(y, h, g, post_weight=w, post_norm=True, save=True)
        gr = ops.block_norm_backward(dr, None, y, h, g, s2, post_weight=w, post_norm=True)
        dx, dz, db, _ = ops.gated_scan_backward(gr.o, x, z, s1, bias)
        return res, gr.gate, gr.post_weight, dx, dz, db
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in (x, z, g, h, dr):
            t.copy_(r(T, B, D))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        assert all(np.isfinite(t.float().sum().item()) for t in out)
