"""Plain 64-bit implementations of the gated delta rule, the layer norm and the
products in 8-bit integers, with bounds on what 32-bit arithmetic may differ by.

U = 2^-24 is half a step of fp32; a rounding costs U of the magnitude it happens at.
A product's sum of n terms on the matrix units passes through 3 n / 8 sums of steps
(six products of terms, sixteen values each) and 16 within one; cutting both factors
into three terms loses less than 8 U: `_sum(n)` in all.
"""
import torch

from tests._ops_ref import HALF_STEP, TINY, U, stored, worst    # noqa: F401


def _sum(n):
    return (0.375 * n + 30) * U


def _unit(x, unit):
    if not unit:
        return x, torch.ones_like(x[..., :1])
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)
    return x * r, r


def delta(q, k, v, g, beta, state, lengths, scale, unit, dy=None, dfinal=None):
    """The gated delta rule and (with dy) its gradients in fp64, by its recurrence, position after
    position.  Returns {name: value}."""
    q, k, v, g, beta = (x.double().cpu() for x in (q, k, v, g, beta))
    T, B, H, dv = v.shape
    HK, dk = q.shape[2:]
    share = H // HK
    n = [T] * B if lengths is None else [min(max(int(x), 0), T) for x in lengths.tolist()]
    live = torch.arange(T)[:, None] < torch.tensor(n)[None, :]
    q, k, v = (torch.where(live[..., None, None], x, 0.0) for x in (q, k, v))
    g, beta = (torch.where(live[..., None], x, 0.0) for x in (g, beta))
    uq, rq = _unit(q, unit)
    uk, rk = _unit(k, unit)
    hq, hk = uq.repeat_interleave(share, 2), uk.repeat_interleave(share, 2)
    a = torch.exp(g)
    S = state.double().cpu() if state is not None else torch.zeros(B, H, dk, dv, dtype=torch.float64)
    y, before, error = torch.zeros_like(v), [], []
    for t in range(T):
        before.append(S)
        decayed = a[t][..., None, None] * S
        e = v[t] - (hk[t][..., None] * decayed).sum(-2)
        error.append(e)
        S = decayed + hk[t][..., None] * (beta[t][..., None] * e)[..., None, :]
        y[t] = scale * (S * hq[t][..., None]).sum(-2)
    mask = live[..., None, None]
    out = {"y": torch.where(mask, y, 0.0), "final": S}
    if dy is None:
        return out
    dy = torch.where(mask, dy.double().cpu(), 0.0) * scale
    D = dfinal.double().cpu() if dfinal is not None else torch.zeros_like(S)
    dq, dk_, dvv = torch.zeros_like(hq), torch.zeros_like(hk), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(beta)
    after = before[1:] + [S]
    for t in range(T - 1, -1, -1):
        dq[t] = (after[t] * dy[t][..., None, :]).sum(-1)
        D = D + hq[t][..., None] * dy[t][..., None, :]
        du = (D * hk[t][..., None]).sum(-2)
        db[t] = (du * error[t]).sum(-1)
        de = beta[t][..., None] * du
        dvv[t] = de
        decayed = a[t][..., None, None] * before[t]
        dk_[t] = (D * (beta[t][..., None] * error[t])[..., None, :]).sum(-1) - (decayed * de[..., None, :]).sum(-1)
        D = D - hk[t][..., None] * de[..., None, :]
        dg[t] = (D * decayed).sum((-1, -2))
        D = a[t][..., None, None] * D

    def back(u, r, d):
        d = d.unflatten(2, (HK, share)).sum(3)
        return torch.where(mask, r * (d - u * (u * d).sum(-1, keepdim=True)) if unit else d, 0.0)
    out.update(dq=back(uq, rq, dq), dk=back(uk, rk, dk_), dv=torch.where(mask, dvv, 0.0),
               dg=torch.where(live[..., None], dg, 0.0), dbeta=torch.where(live[..., None], db, 0.0), dstate=D)
    return out


def delta_bounds(q, k, v, g, beta, state, lengths, scale, unit, chunk, terms, dy=None, dfinal=None):
    """Bounds of delta's values for an evaluation in chunks: {name: bound}, without the rounding of what
    is stored.

    In a chunk every product's error is bounded element by element by |left| |right| of the matrices that
    are multiplied; the triangular inverse M of I + A is off by (chunk + 40) U |M| |I + A| |M| (substitution,
    row by row; A's own elements carry the errors of a product over dk and of three factors).  From chunk to
    chunk the error of S passes through the chunk's map, whose 2-norm is at most the product over its
    positions of a max(1, |1 - b |k|^2|), so as a Frobenius norm; the gradient's through the same maps'
    transposes.  terms: of what y is made of (2: each factor is off by 2^-17 there)."""
    q, k, v, g, beta = (x.double().cpu() for x in (q, k, v, g, beta))
    T, B, H, dv = v.shape
    HK, dk = q.shape[2:]
    share = H // HK
    n = [T] * B if lengths is None else [min(max(int(x), 0), T) for x in lengths.tolist()]
    ef = (dk / 4 + 24) * U if unit else 12 * U            # of a row's factors: its length, its decay
    rough = 2.0 ** -16 if terms == 2 else 0.0
    back = dy is not None
    names = ("y", "final") + (("dq", "dk", "dv", "dg", "dbeta", "dstate") if back else ())
    out = {"y": torch.zeros_like(v), "final": torch.zeros(B, H, dk, dv, dtype=torch.float64)}
    if back:
        out.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v), dg=torch.zeros_like(g),
                   dbeta=torch.zeros_like(beta), dstate=torch.zeros_like(out["final"]))
    norm = torch.linalg.norm
    uq, rq = _unit(q, unit)
    uk, rk = _unit(k, unit)
    for b in range(B):
        for h in range(H):
            hk = h // share
            S = state[b, h].double().cpu() if state is not None else torch.zeros(dk, dv, dtype=torch.float64)
            eS = 0.0                                       # Frobenius norm of S's error
            parts = []
            for t0 in range(0, n[b], chunk):
                sl = slice(t0, min(t0 + chunk, n[b]))
                Q, K, V = uq[sl, b, hk], uk[sl, b, hk], v[sl, b, h]
                G = g[sl, b, h].clamp_min(-1e4).cumsum(0)
                be = beta[sl, b, h][:, None]
                C = len(G)
                low = torch.tril(torch.ones(C, C, dtype=torch.float64))
                E = torch.exp(torch.where(low > 0, G[:, None] - G[None, :], 0.0)) * low
                kk, akk = K @ K.T, K.abs() @ K.T.abs()
                A = torch.tril(E * kk * be.T, -1)
                eA = torch.tril(E * be.T.abs() * akk, -1) * (_sum(dk) + 2 * ef + 6 * U)
                I = torch.eye(C, dtype=torch.float64)
                M = torch.linalg.inv(I + A)
                eM = M.abs() @ (eA + (C + 40) * U * (I + A).abs()) @ M.abs()
                rise, fall = torch.exp(G)[:, None], torch.exp(G[-1] - G)[:, None]
                KS, aKS = K @ S, K.abs() @ S.abs()
                R = V - rise * KS
                eR = rise * aKS * (_sum(dk) + ef) + 2 * U * (V.abs() + rise * aKS)
                W = M @ R
                eW = M.abs() @ eR + eM @ R.abs() + _sum(C) * M.abs() @ R.abs()
                eW = eW + norm(M @ (rise * K), dim=-1)[:, None] * eS
                bw = be * W
                P, aP = E * (Q @ K.T), E * (Q.abs() @ K.T.abs())
                aY = rise * (Q.abs() @ S.abs()) + aP @ bw.abs()
                eY = aY * (_sum(dk) + _sum(C) + 2 * ef + 8 * U + rough) + aP @ (be.abs() * eW) + norm(rise * Q, dim=-1)[:, None] * eS
                out["y"][sl, b, h] = abs(scale) * eY
                aN = torch.exp(G[-1]) * S.abs() + (fall * K).abs().T @ bw.abs()
                # its own error (w's without what S's error adds, which passes through the map)
                eWl = M.abs() @ eR + eM @ R.abs() + _sum(C) * M.abs() @ R.abs()
                eN = aN * (_sum(C) + ef + 8 * U) + (fall * K).abs().T @ (be.abs() * eWl)
                grow = float(torch.exp(G[-1]) * torch.clamp((1 - be[:, 0] * (K * K).sum(-1)).abs(), min=1.0).prod())
                parts.append((sl, S, eS, W, eW, grow))
                S = torch.exp(G[-1]) * S + (fall * K).T @ bw
                eS = grow * eS + float(norm(eN))
            out["final"][b, h] = eS
            if not back:
                continue
            last, eL = S, eS
            D = dfinal[b, h].double().cpu() if dfinal is not None else torch.zeros(dk, dv, dtype=torch.float64)
            eD = 0.0
            for sl, S, eS, W, eW, grow in reversed(parts):
                Q, K, V = uq[sl, b, hk], uk[sl, b, hk], v[sl, b, h]
                Y = dy[sl, b, h].double().cpu() * scale
                G = g[sl, b, h].clamp_min(-1e4).cumsum(0)
                be = beta[sl, b, h][:, None]
                C = len(G)
                low = torch.tril(torch.ones(C, C, dtype=torch.float64))
                E = torch.exp(torch.where(low > 0, G[:, None] - G[None, :], 0.0)) * low
                A = torch.tril(be * E * (K @ K.T), -1)
                eA = torch.tril(be.abs() * E * (K.abs() @ K.T.abs()), -1) * (_sum(dk) + 2 * ef + 6 * U)
                I = torch.eye(C, dtype=torch.float64)
                N = torch.linalg.inv(I + A)
                eN = N.abs() @ (eA + (C + 40) * U * (I + A).abs()) @ N.abs()
                rise, fall = torch.exp(G)[:, None], torch.exp(G[-1] - G)[:, None]
                P, aP = E * (Q @ K.T), E * (Q.abs() @ K.T.abs())
                F = P.T @ Y + fall * (K @ D)
                aF = aP.T @ Y.abs() + fall * (K.abs() @ D.abs())
                eF = aF * (_sum(dk) + _sum(C) + 2 * ef + 10 * U)
                X = N.T @ F
                eXl = N.T.abs() @ eF + eN.T @ F.abs() + _sum(C) * N.T.abs() @ F.abs()
                eX = eXl + norm(N.T @ (fall * K), dim=-1)[:, None] * eD
                Z, eZ = be * X, be.abs() * eX + 2 * U * (be * X).abs()
                out["dv"][sl, b, h] = eZ
                out["dbeta"][sl, b, h] = (X.abs() * eW + eX * W.abs() + (dv / 4 + 20) * U * (X * W).abs()).sum(-1)
                # pairs, and what is made of them
                bw, ebw = be * W, be.abs() * eW
                XW, YW = Z.abs() @ bw.T.abs(), Y.abs() @ bw.T.abs()
                Hm, Jm = torch.tril(E * (Z @ bw.T), -1).abs(), (E * (Y @ bw.T)).abs()
                up = (_sum(dv) + 2 * ef + 10 * U)
                eH = torch.tril(E * (XW * up + eZ @ bw.T.abs() + Z.abs() @ ebw.T), -1)
                eJ = E * (YW * up + Y.abs() @ ebw.T)
                aq = Jm @ K.abs() + rise * (Y.abs() @ S.T.abs())
                eq = eJ @ K.abs() + aq * (_sum(C) + _sum(dv) + ef + 10 * U) + rise * norm(Y, dim=-1)[:, None] * eS
                Hs, eHs = Hm + Hm.T, eH + eH.T
                ak = Hs @ K.abs() + Jm.T @ Q.abs() + rise * (Z.abs() @ S.T.abs()) + fall * (bw.abs() @ D.T.abs())
                ek = eHs @ K.abs() + eJ.T @ Q.abs() + ak * (_sum(C) + _sum(dv) + ef + 12 * U)
                ek = ek + rise * (eZ @ S.T.abs() + norm(Z, dim=-1)[:, None] * eS)
                ek = ek + fall * (ebw @ D.T.abs() + norm(bw, dim=-1)[:, None] * eD)
                # what decays scale: the state behind the chunk against its gradient, rows of q . dq and v . dv
                rows = (Q.abs() * eq).sum(-1) + (dk / 4 + 20) * U * (Q.abs() * aq).sum(-1) + \
                    (V.abs() * eZ).sum(-1) + (dv / 4 + 20) * U * (V * Z).abs().sum(-1)
                size = (Q.abs() * aq).sum(-1) + (V * Z).abs().sum(-1)
                ends = float((D.abs() * (torch.exp(G[-1]) * S.abs() + (fall * K).abs().T @ bw.abs())).sum())
                tail = rows.flip(0).cumsum(0).flip(0) + 8 * U * size.flip(0).cumsum(0).flip(0)
                out["dg"][sl, b, h] = tail + ends * (_sum(dv) + _sum(C) + (dk * dv / 64 + 40) * U + 2 * ef) + \
                    float(norm(D)) * (eL + float(norm((fall * K).abs().T @ ebw))) + float(norm(last)) * eD
                if unit:
                    for name, u, r, a, e in (("dq", Q, rq[sl, b, hk], aq, eq), ("dk", K, rk[sl, b, hk], ak, ek)):
                        dot = (u.abs() * a).sum(-1, keepdim=True)
                        edot = (u.abs() * e).sum(-1, keepdim=True) + (dk / 4 + 20 + share) * U * dot
                        out[name][sl, b, hk] += r * (e + u.abs() * edot + (3 * ef + 6 * U) * (a + u.abs() * dot))
                else:
                    out["dq"][sl, b, hk] += eq + share * U * aq
                    out["dk"][sl, b, hk] += ek + share * U * ak
                aD = torch.exp(G[-1]) * D.abs() + (rise * Q).abs().T @ Y.abs() + (rise * K).abs().T @ Z.abs()
                eDl = aD * (_sum(2 * C) + ef + 10 * U) + (rise * K).abs().T @ (be.abs() * eXl)
                last, eL = S, eS
                D = torch.exp(G[-1]) * D + (rise * Q).T @ Y - (rise * K).T @ Z
                eD = grow * eD + float(norm(eDl))
            out["dstate"][b, h] = eD
    return {x: out[x] for x in names}


def layer(x, res, weight, bias, eps, dr=None, da=None, back=False):
    """The layer norm with a residual and its gradients in fp64, each with the bound of an fp32
    evaluation.  Returns {name: (value, bound)}; bounds do not hold the rounding of what is stored."""
    c = {n: t.double().cpu() if t is not None else None
         for n, t in (("x", x), ("res", res), ("w", weight), ("b", bias), ("dr", dr), ("da", da))}
    r = (c["x"] if c["x"] is not None else 0.0) + (c["res"] if c["res"] is not None else 0.0)
    D = r.shape[-1]
    mean = lambda t: t.mean(-1, keepdim=True)                            # noqa: E731
    one = torch.ones(D, dtype=torch.float64)
    w, b = c["w"] if c["w"] is not None else one, c["b"] if c["b"] is not None else 0 * one
    sum_err = (D / 64 + 24) * U                 # a sum of D values: D/64 in a lane at most, then the tree
    er = U * r.abs() if c["x"] is not None and c["res"] is not None else 0 * r
    m = mean(r)
    v = r - m
    # r - m0 and its mean, which takes m0's rounding away again
    ev = er + mean(er) + 3 * U * (v.abs() + sum_err * mean(r.abs())) + sum_err * mean(v.abs()) + sum_err ** 2 * mean(r.abs())
    var = mean(v * v) + eps
    n = 1 / torch.sqrt(var)
    fn = mean(v.abs() * ev) / var + sum_err + 6 * U
    u = v * n
    eu = ev * n + (fn + 2 * U) * u.abs()
    out = {"r": (r, er), "a": (u * w + b, eu * w.abs() + 2 * U * ((u * w).abs() + b.abs()))}
    if not back:
        return out
    eu = eu + U * m.abs() * n                    # the mean as it is kept
    dr = c["dr"] if c["dr"] is not None else torch.zeros_like(r)
    if c["da"] is not None:
        e = c["da"] * w
        m1, m2 = mean(e), mean(e * u)
        e1 = sum_err * mean(e.abs())
        e2 = mean(e.abs() * eu) + (sum_err + 3 * U) * mean((e * u).abs())
        big = e.abs() + m1.abs() + (u * m2).abs()
        G = dr + n * (e - m1 - u * m2)
        eG = n * (e1 + eu * m2.abs() + u.abs() * e2) + (fn + 5 * U) * n * big + U * (dr.abs() + n * big)
    else:
        G, eG = dr, torch.zeros_like(dr)
    out["dx"] = out["dres"] = (G, eG)
    if c["da"] is not None:
        rows = r.numel() // D
        terms = (rows / 64 + 1100) * U          # a column's sum: rows of a workgroup, then the workgroups
        lead = tuple(range(r.dim() - 1))
        out["dweight"] = ((c["da"] * u).sum(lead), (c["da"].abs() * eu + (terms + 2 * U) * (c["da"] * u).abs()).sum(lead))
        out["dbias"] = (c["da"].sum(lead), (terms * c["da"].abs()).sum(lead))
    return out


def q8_rows(x):
    """Scales and codes of rows of values, as defined: both quotients in fp32."""
    x = x.float().cpu()
    top = x.abs().amax(-1) if x.shape[-1] else x.new_zeros(x.shape[:-1])
    scale = top / torch.full_like(top, 127.0)
    scale = torch.where(torch.isfinite(top), scale, torch.full_like(scale, float("nan")))
    codes = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x)).round().clamp(-127, 127)
    return codes.to(torch.int8), scale


def q8(codes, scales, wcodes, wscales, bias):
    """The product in fp64 and its bound: the whole sum rounded to fp32, two factors, the bias."""
    y = (codes.cpu().double() @ wcodes.cpu().double().t()) * scales.cpu().double()[:, None] * wscales.cpu().double()
    b = bias.cpu().double() if bias is not None else torch.zeros_like(y[0])
    return y + b, 3 * U * (y.abs() + b.abs()) + TINY[torch.float32]
