"""Digits that the gated delta rule keeps where large parts of a result cancel."""
import pytest
import torch

from long_convolution_sequence_amd import ops
from tests import _more_ops_ref as ref
from tests._parity import say

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("dk", [16, 40, 80, 128])
def test_a_query_for_a_key_that_was_just_overwritten(dk, dtype):
    """y = S^T q + (k . q) b (v - S^T k) with q = k a unit vector and b = 1 is v, whatever the state held.  States
    in [1, 2) of 24 bits and values that are whole multiples of 2^-19 of up to 2^-12: every product and sum is a
    number of 24 bits, so fp32 gives v to the last bit.  A term of the state left out (2^-17) is thirty times the
    step of a 16-bit v there."""
    say(f"case delta overwritten key dk={dk} {dtype}")
    T, B, H, dv, at = 40, 2, 2, 48, 7
    gen = torch.Generator().manual_seed(dk)
    state = 1 + torch.randint(0, 1 << 23, (B, H, dk, dv), generator=gen) * 2.0 ** -23
    v = torch.zeros(T, B, H, dv)
    v[at] = torch.randint(64, 128, (B, H, dv), generator=gen) * 2.0 ** -19
    k = torch.zeros(T, B, H, dk)
    k[at, ..., dk // 3] = 1.0
    gates = torch.zeros(T, B, H, device="cuda")
    k, v, state = k.to(dtype).cuda(), v.to(dtype).cuda(), state.cuda()
    y, final = ops.gated_delta(k, k, v, gates, gates + 1, state, scale=1.0)
    assert torch.equal(y[at], v[at])
    assert torch.equal(final[:, :, dk // 3], v[at].float())
    assert (y[:at] == 0).all() and (y[at + 1:] == 0).all()


def _decay_bound(v, unit, C, dy, dfinal):
    """Bound of the decays' gradients from what passes through each decay alone.

    Everything is evaluated chunk by chunk on absolute values: a position's part is then the sum of the sizes
    of the terms that carry its decay (|D| a |S|, taken apart into pairs of positions, states and gradients), and
    a stage of the evaluation (a product, a factor) adds its relative error to it.  The inverse M of I + A has
    |M| |I + A| |M| in its place, to which its error is relative; a factor e^(-x) is off by 2 U + 1.5 x U for its
    argument's rounding, so 24 U of e^(-x) (1 + x / 16)."""
    U = ref.U
    q, k, x, g, beta = (v[n].double() for n in ("q", "k", "v", "g", "beta"))
    T, B, H, dv = x.shape
    HK, dk = q.shape[2:]
    q, k = (ref._unit(t, unit)[0].abs() for t in (q, k))
    ef = (dk / 4 + 48) * U
    stage = 2 * ref._sum(dk) + 2 * ref._sum(C) + 4 * ef + (C + 60) * U             # one chunk, in one direction
    last = ref._sum(dv) + ref._sum(dk) + 4 * ef + (C + dk + dv + 60) * U
    eps = 1.01 * (2 * -(-T // C) * stage + last)
    out = torch.zeros(T, B, H, dtype=torch.float64)
    signed = ref._unit(v["k"].double(), unit)[0]
    fade = lambda d: torch.exp(-d) * (1 + d / 16)                                  # noqa: E731
    for b in range(B):
        for h in range(H):
            hk, S, kept = h // (H // HK), v["state"][b, h].double().abs(), []
            spans = [slice(t, min(t + C, T)) for t in range(0, T, C)]
            for sl in spans:
                K, be, G = k[sl, b, hk], beta[sl, b, h][:, None], -g[sl, b, h].clamp_min(-1e4).cumsum(0)
                n = len(G)
                E = torch.tril(fade((G[:, None] - G[None, :]).clamp_min(0.0)))
                A = torch.tril(E * (K @ K.T) * be.T, -1)
                true = torch.tril(torch.exp(-(G[:, None] - G[None, :]).clamp_min(0.0)) * (signed[sl, b, hk] @ signed[sl, b, hk].T) * be.T, -1)
                M = torch.linalg.inv(torch.eye(n, dtype=torch.float64) + true).abs()
                M = M @ (torch.eye(n, dtype=torch.float64) + A) @ M
                rise, fall, end = fade(G)[:, None], fade(G[-1] - G)[:, None], fade(G[-1])
                W = M @ (x[sl, b, h].abs() + rise * (K @ S))
                kept.append((S, W, E, be, rise, fall, end, A))
                S = end * S + (fall * K).T @ (be * W)
            D = dfinal[b, h].double().abs()
            for sl, (S, W, E, be, rise, fall, end, A) in list(zip(spans, kept))[::-1]:
                Q, K, Y = q[sl, b, hk], k[sl, b, hk], dy[sl, b, h].double().abs() * dk ** -0.5
                n = len(be)
                N = (be * E).tril(-1) * (signed[sl, b, hk] @ signed[sl, b, hk].T)
                N = torch.linalg.inv(torch.eye(n, dtype=torch.float64) + N).abs()
                N = N @ (torch.eye(n, dtype=torch.float64) + (be * E).tril(-1) * (K @ K.T)) @ N
                X = N.T @ ((E * (Q @ K.T)).T @ Y + fall * (K @ D))
                Z, bw = be * X, be * W
                P = (E * (Z @ bw.T)).tril(-1) * (K @ K.T) + E * (Y @ bw.T) * (Q @ K.T)
                own = rise[:, 0] * ((Q * (Y @ S.T)).sum(-1) + (K * (Z @ S.T)).sum(-1))
                ends = fall[:, 0] * (K * (bw @ D.T)).sum(-1)
                rect = torch.stack([P[t:, :t].sum() for t in range(n)])
                out[sl, b, h] = eps * (rect + own.flip(0).cumsum(0).flip(0) + ends.cumsum(0) - ends + end * (D * S).sum())
                D = end * D + (rise * Q).T @ Y + (rise * K).T @ Z
    return out


@pytest.mark.parametrize("T,HK,H,dk,dv,unit", [(30, 1, 6, 24, 16, True), (100, 2, 6, 72, 40, True), (150, 3, 6, 128, 64, False),
                                               (70, 6, 6, 40, 33, True)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_gradients_of_decays_that_are_nearly_shut(T, HK, H, dk, dv, unit, dtype):
    """Heads whose decays are about 0.05, 6, 10, 20, 1000 and infinite: each gradient to the digits of what
    passes through its decay, and 0 where nothing does."""
    say(f"case delta shut decays T={T} HK={HK} dk={dk} dv={dv} unit={unit} {dtype}")
    gen = torch.Generator().manual_seed(T + dk)
    r = lambda *s: torch.randn(*s, generator=gen)                                  # noqa: E731
    size = 1.0 if unit else 0.9 / dk ** 0.5
    v = {"q": (size * r(T, 1, HK, dk)).to(dtype), "k": (size * r(T, 1, HK, dk)).to(dtype), "v": r(T, 1, H, dv).to(dtype),
         "beta": torch.sigmoid(r(T, 1, H)), "state": r(1, H, dk, dv)}
    v["g"] = -torch.tensor([0.05, 6.0, 10.0, 20.0, 1000.0, float("inf")]) * (0.75 + torch.rand(T, 1, H, generator=gen) / 2)
    dy, dfinal = r(T, 1, H, dv).to(dtype), r(1, H, dk, dv)
    c = {n: t.cuda() for n, t in v.items()}
    a = [c[n] for n in ("q", "k", "v", "g", "beta")]
    _, _, saved = ops.gated_delta(*a, c["state"], unit=unit, save=True)
    d = ops.gated_delta_backward(dy.cuda(), *a, saved, c["state"], dfinal=dfinal.cuda(), unit=unit)
    w = dict(v, g=v["g"].clamp_min(-1e4))                                          # e^-10^4 is 0
    args = [w[n] for n in ("q", "k", "v", "g", "beta", "state")]
    want = ref.delta(*args, None, dk ** -0.5, unit, dy, dfinal)["dg"]
    tol = _decay_bound(w, unit, 64 if dtype is BF16 else 32, dy, dfinal)
    assert (d.decay[..., 4:] == 0).all()
    for h in range(H):
        worst = ref.worst(d.decay[..., h], want[..., h], ref.stored(want[..., h], tol[..., h], F32))
        assert worst <= 1.0, f"head {h}: {worst:.3g} of its bound"
    # the bound says something: a tenth of most gradients at least, where their own size is not less by chance
    for h in (1, 2, 3):
        assert (tol[..., h] < want[..., h].abs() / 10).float().mean() > 0.5, h
