"""Plain 64-bit implementations of the recurrent-block operators, with bounds on
what fp32 arithmetic may differ by.

The bounds are worst cases, run along with the definition: U = 2^-24 is half a
step of fp32, a rounding costs U of the magnitude it happens at, the hardware
exp2, reciprocal and square root 2 U.  Magnitudes are majorants (the same
recurrence on absolute values), so they hold for any grouping of the sums.
"""
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def stored(ref, tol, dtype):
    """Bound of a value within tol of ref after its rounding to dtype."""
    return tol + HALF_STEP[dtype] * (ref.abs() + tol) + TINY[dtype]


def worst(got, ref, bound):
    """max |got - ref| / bound (a NaN or infinity in got gives infinity)."""
    d = (got.double().cpu() - ref).abs()
    d = torch.where(torch.isfinite(d), d, torch.full_like(d, float("inf")))
    return float((d / bound).max()) if d.numel() else 0.0


def factor(kind, d, a):
    """e(d) and q with de/dz = -a d q' ... : e, and the slope of e over z."""
    if kind == 0:
        return torch.ones_like(d), torch.zeros_like(d)
    if kind == 1:
        return d, -a * d
    return torch.sqrt(d * (1 + a)), -a * a * torch.sqrt(d / (1 + a))


def scan(x, gate, bias, state, lengths, kind, dy=None, dfinal=None, digits=False):
    """The recurrence and (with dy) its gradients in fp64 on the CPU, by the definition,
    each with the bound of an fp32 evaluation.  Returns {name: (value, bound)}; bounds do
    not hold the rounding of what is stored.

    digits: of an evaluation that keeps the digits of a = 1 - d however small it is (the
    bounds without it allow a an absolute error)."""
    x, gate = x.double().cpu(), gate.double().cpu()
    T, B, D = x.shape
    z = gate + (bias.double().cpu() if bias is not None else 0.0)
    s0 = state.double().cpu() if state is not None else torch.zeros(B, D, dtype=torch.float64)
    n = [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths.tolist()]
    live = torch.arange(T)[:, None, None] < torch.tensor(n)[None, :, None] if T else torch.ones(0, B, 1, dtype=torch.bool)
    live = live.expand(T, B, D)
    d, a = torch.sigmoid(-z), torch.sigmoid(z)
    rel = (3 * z.abs() + 5) * U                 # of d: sum, product and constant at |z| each, exp2, 1 +, rcp
    # e^z passes the largest fp32 at 2^128 and 1 / (1 + e^z) the smallest normal one at 2^-126:
    # from there on d may be 0, a relative error of 1 of a d below 2^-126 (and of its root in e);
    # d / (2 - d), under the root in the slope of e, passes it at d = 2^-125 already
    rel = torch.where(d < 2.0 ** -124.9, torch.ones_like(rel), rel)
    # of a: e^z d where z < 0, off by e^z's and d's errors and a rounding (from 2^-126 on it may be 0);
    # 1 - d where z >= 0, so d (rel + U) of at least 1/2, and d is no more than 1/2
    ra = torch.where(z < 0, 2 * rel + U, rel + 2 * U)
    ra = torch.where(a < 2.0 ** -124.9, torch.ones_like(ra), ra)
    e, slope = factor(kind, d, a)
    zero = torch.zeros_like(x)
    # masked places may hold anything: nothing of theirs is used
    x, d, rel, ra, slope, e = (torch.where(live, v, zero) for v in (x, d, rel, ra, slope, e))
    a = torch.where(live, a, zero + 1)
    s, m, tol = s0.clone(), s0.abs(), torch.zeros_like(s0)
    S, M, E = [s0], [m], [tol]
    for t in range(T):
        b = e[t] * x[t]
        step = (ra[t] + U) * a[t] if digits else (rel[t] + U) * d[t]
        tol = a[t] * tol + step * m + (rel[t] + 6 * U) * b.abs()
        s, m = a[t] * s + b, a[t] * m + b.abs()
        tol = tol + 3 * U * torch.where(live[t], m, zero[t])
        S.append(s), M.append(m), E.append(tol)
    S, M, E = torch.stack(S), torch.stack(M), torch.stack(E)
    E = E + 10 * U * M                          # joining of chunks
    out = {"y": (torch.where(live, S[1:], zero), torch.where(live, E[1:], zero)), "final": (S[T], E[T])}
    if dy is None:
        return out
    g = torch.where(live, dy.double().cpu(), zero)
    c = dfinal.double().cpu() if dfinal is not None else torch.zeros_like(s0)
    mc, tc = c.abs(), torch.zeros_like(c)
    dx, dz = torch.zeros_like(x), torch.zeros_like(x)
    bx, bz, mz = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T - 1, -1, -1):
        G, mg, tg = g[t] + c, g[t].abs() + mc, tc + U * (g[t].abs() + mc)
        tg10 = tg + 10 * U * mg
        dx[t], bx[t] = e[t] * G, e[t] * tg10 + (rel[t] + 7 * U) * e[t] * mg
        k = a[t] * d[t] * S[t] + slope[t] * x[t]
        mk = a[t] * d[t] * M[t] + slope[t].abs() * x[t].abs()
        q = torch.sqrt(d[t] / (2 - d[t])) if kind == 2 else zero[t]
        dk = d[t] * (rel[t] + 4 * U) * (M[t] + x[t].abs()) + a[t] * d[t] * E[t] + 3 * x[t].abs() * q * (rel[t] + 6 * U)
        if digits:        # the factors' errors, each of its term
            dk = (2 * ra[t] + rel[t] + 10 * U) * mk + a[t] * d[t] * E[t]
        dk = torch.where(live[t], dk, zero[t])
        dz[t], bz[t], mz[t] = G * k, mg * dk + mk * tg10 + 3 * U * mg * mk, mg * mk
        c, mc = a[t] * G, a[t] * mg
        step = (ra[t] + U) * a[t] if digits else (rel[t] + U) * d[t]
        tc = a[t] * tg + torch.where(live[t], step * mg + U * mc, zero[t])
    dx, dz, bx, bz = (torch.where(live, v, zero) for v in (dx, dz, bx, bz))
    out.update(dx=(dx, bx), dgate=(dz, bz), dstate=(c, tc + 10 * U * mc))
    terms = 300 + (T // 64 + 2) * B             # roundings on a term's way into the sum
    out["dbias"] = (dz.sum((0, 1)), (bz + terms * U * torch.where(live, mz, zero)).sum((0, 1)) if T else
                    torch.zeros(D, dtype=torch.float64))
    return out


def act(kind, g):
    """act(g) and its derivative."""
    if kind == 0:
        return g, torch.ones_like(g)
    s, rest = torch.sigmoid(g), torch.sigmoid(-g)      # 1 - s would be 0 from g = 37 on, also in fp64
    if kind == 1:
        return s, s * rest
    return g * s, s * (1 + g * rest)


def norm(o, res, gate, w1, k, w2, post, kind, eps, dr=None, da=None, back=False):
    """The norms around a block and their gradients in fp64, with the bounds of an fp32
    evaluation.  Roundings are counted per factor: f is the relative error of a product's
    factors so far; sums carry the majorant of their terms."""
    c = {"o": o, "res": res, "gate": gate, "w1": w1, "k": k, "w2": w2, "dr": dr, "da": da}
    c = {n: (v.double().cpu() if v is not None else None) for n, v in c.items()}
    first = c["o"] if c["o"] is not None else c["res"]
    D = first.shape[-1]
    one = torch.ones(D, dtype=torch.float64)
    w1, k, w2 = (c[n] if c[n] is not None else one for n in ("w1", "k", "w2"))
    sum_err = (D / 64 + 24) * U                 # a sum of D squares: D/64 in a lane at most, then the tree
    res = c["res"] if c["res"] is not None else torch.zeros_like(first)
    if c["o"] is not None:
        q = 1 / torch.sqrt((c["o"] ** 2).mean(-1, keepdim=True) + eps) if post else torch.ones_like(first[..., :1])
        unit = c["o"] * q
        if c["gate"] is not None:
            A, As = act(kind, c["gate"])
            fa = (3 * c["gate"].abs() + 8) * U if kind else torch.zeros_like(first)
            fa = torch.minimum(fa, fa * 0 + 1)
        else:
            A, As, fa = torch.ones_like(first), torch.zeros_like(first), torch.zeros_like(first)
        m = unit * w1 * A
        fq = (sum_err + 6 * U) if post else 0.0
        fm = fq + fa + 3 * U                     # relative error of m
        r = res + k * m
        er = (fm + 2 * U) * (k * m).abs() + 2 * U * (res.abs() + (k * m).abs())
    else:
        unit = A = As = m = torch.zeros_like(first)
        fq, fm, fa = 0.0, torch.zeros_like(first), torch.zeros_like(first)
        q = torch.ones_like(first[..., :1])
        r, er = res, torch.zeros_like(res)
    ms = (r ** 2).mean(-1, keepdim=True) + eps
    n = 1 / torch.sqrt(ms)
    fn = (2 * r.abs() * er).mean(-1, keepdim=True) / (2 * ms) + sum_err + 6 * U
    ru = r * n
    eru = er * n + (fn + U) * ru.abs()
    out = {"r": (r, er), "a": (ru * w2, (eru + U * ru.abs()) * w2.abs())}
    if not back:
        return out
    dr = c["dr"] if c["dr"] is not None else torch.zeros_like(r)
    if c["da"] is not None:
        u = c["da"] * w2
        mean2 = (u * ru).mean(-1, keepdim=True)
        e2 = (u.abs() * eru).mean(-1, keepdim=True) + (sum_err + 3 * U) * (u * ru).abs().mean(-1, keepdim=True)
        inner = u - ru * mean2
        big = u.abs() + (ru * mean2).abs()
        ei = eru * mean2.abs() + ru.abs() * e2 + 2 * U * big
        G = dr + n * inner
        eG = n * ei + (fn + 2 * U) * n * big + U * (dr.abs() + n * big)
    else:
        G, eG = dr, torch.zeros_like(dr)
    out["dres"] = (G, eG)
    dm, edm = G * k, eG * k.abs() + U * (G * k).abs()
    dv, edv = dm * A, edm * A.abs() + (fa + U) * (dm * A).abs()
    v = unit * w1
    # act' of silu is a sum of two terms: its error is of their size, not of its own
    slope_big = torch.sigmoid(c["gate"]) * (1 + c["gate"].abs()) if c["gate"] is not None and kind == 2 else As.abs()
    out["dgate"] = (dm * v * As, edm * (v * As).abs() + (fq + 4 * U) * (dm * v * As).abs() +
                    2 * (fa + 3 * U) * (dm * v).abs() * slope_big)
    w, ew = dv * w1, edv * w1.abs() + U * (dv * w1).abs()
    if post:
        mean1 = (w * unit).mean(-1, keepdim=True)
        e1 = (ew * unit.abs() + (fq + sum_err + 3 * U) * (w * unit).abs()).mean(-1, keepdim=True)
        big = w.abs() + (unit * mean1).abs()
        ei = ew + unit.abs() * e1 + (fq + U) * (unit * mean1).abs() + 2 * U * big
        out["do"] = (q * (w - unit * mean1), q * ei + (fq + 2 * U) * q * big)
    else:
        out["do"] = (w, ew)
    rows = first.numel() // D
    terms = (rows / 64 + 1100) * U              # a column's sum: rows of a workgroup, then the workgroups

    def column(value, err):
        lead = tuple(range(value.dim() - 1))
        return value.sum(lead), (err + (terms + 2 * U) * value.abs()).sum(lead)
    out["dpost"] = column(dv * unit, edv * unit.abs() + (fq + U) * (dv * unit).abs())
    out["dscale"] = column(m * G, fm * (m * G).abs() + m.abs() * eG)
    if c["da"] is not None:
        out["dpre"] = column(c["da"] * ru, c["da"].abs() * eru)
    return out


def q4(x, codes, scales, zeros, group):
    """The product in fp64 and its bound: a group's fp32 sum runs over (16 + code) x and loses
    (16 + zero) sum(x), every partial sum below 31 sum|x|; the groups' sums follow."""
    x, s = x.double().cpu(), scales.double().cpu()
    codes = codes.cpu().long()
    N, K = codes.shape
    zero = zeros.cpu().double() if zeros is not None else torch.full_like(s, 8.0)
    g = torch.arange(K) // group
    y = torch.zeros(x.shape[0], N, dtype=torch.float64)
    bound = torch.zeros_like(y)
    groups = s.shape[1]
    for j in range(groups):
        at = g == j
        part, big = x[:, at], x[:, at].abs().sum(-1, keepdim=True)
        y += s[:, j] * (part @ codes[:, at].double().t() - zero[:, j] * part.sum(-1, keepdim=True))
        bound += s[:, j].abs() * (31 * (group + 4) + 31 * 8 + 31 * (groups + 20)) * U * big
    return y, bound
