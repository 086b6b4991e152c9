"""More operators of a recurrent block: what is measured, and their plain forms.

Three operators, in the layouts of the library (sequences [T][B][...], rows [..., D]):

* delta: the gated delta rule, a recurrence whose state is a matrix [dk][dv] for each head.
  S_t = e^{g_t} (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T, y_t = scale S_t^T q_t with scale = 1 / sqrt(dk); with
  "unit" q and k are divided by their length, k / sqrt(sum k^2 + 1e-6).  Groups of value heads share a query and key
  head.  Rows past a sequence's length give y = 0 and leave the state.
* layer: the layer norm with a residual.  r = res + x, a = (r - mean(r)) / sqrt(var(r) + eps) * weight + bias.
* q8: products in 8-bit integers.  Every row of x gets a scale s = max|x| / 127 and codes c = round(x / s), the
  quotients in 32 bits; every output n has its own scale; y[m][n] = s[m] sw[n] sum_k c[m][k] w[n][k] + bias[n].

``direction`` "train" is a training step's share: the forward pass, then the gradients of everything that has one.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
UNIT_EPS = 1e-6


def listed():
    return [
        # one position of a batch of eight sequences: what a serving loop pays for each token
        {"name": "delta step", "op": "delta", "direction": "forward", "T": 1, "B": 8, "HK": 9, "H": 9, "dk": 96,
         "dv": 96, "dtype": "bf16", "unit": True, "ragged": False},
        # the longest prompt of the library's benchmark at its width, one sequence: parallelism comes from the length
        {"name": "delta long prompt", "op": "delta", "direction": "forward", "T": 131072, "B": 1, "HK": 9, "H": 9,
         "dk": 96, "dv": 96, "dtype": "bf16", "unit": True, "ragged": False},
        # a padded batch of prompts with shared key heads, one slot of it empty
        {"name": "delta padded prompts", "op": "delta", "direction": "forward", "T": 4096, "B": 8, "HK": 6, "H": 12,
         "dk": 64, "dv": 128, "dtype": "f32", "unit": True, "ragged": True},
        # a training batch at the block workload's width
        {"name": "delta train", "op": "delta", "direction": "train", "T": 8192, "B": 4, "HK": 6, "H": 6, "dk": 128,
         "dv": 128, "dtype": "bf16", "unit": True, "ragged": False},
        # odd sizes, unequal lengths and shared key heads in training
        {"name": "delta train odd", "op": "delta", "direction": "train", "T": 1999, "B": 3, "HK": 2, "H": 4, "dk": 72,
         "dv": 41, "dtype": "f16", "unit": False, "ragged": True},
        # one position of a batch of eight
        {"name": "layer step", "op": "layer", "direction": "forward", "rows": 8, "D": 864, "dtype": "bf16",
         "res": "f32"},
        # a long prompt: every row once
        {"name": "layer prompt", "op": "layer", "direction": "forward", "rows": 131072, "D": 864, "dtype": "bf16",
         "res": "f32"},
        # a training batch, float residual stream around 16-bit blocks
        {"name": "layer train", "op": "layer", "direction": "train", "rows": 131072, "D": 768, "dtype": "bf16",
         "res": "f32"},
        # wide odd rows, no residual
        {"name": "layer train odd", "op": "layer", "direction": "train", "rows": 1999, "D": 5001, "dtype": "f16",
         "res": "none"},
        # one token against a wide layer: the weights' bytes alone count
        {"name": "q8 token", "op": "q8", "rows": 1, "N": 28672, "K": 8192, "dtype": "bf16", "bias": False},
        # a prompt against a wide layer: the products count
        {"name": "q8 prompt", "op": "q8", "rows": 16384, "N": 8192, "K": 4096, "dtype": "bf16", "bias": True},
        # a batch of a few hundred rows at odd sizes
        {"name": "q8 odd", "op": "q8", "rows": 333, "N": 2593, "K": 4999, "dtype": "f16", "bias": True},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], uniform in its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("delta", "layer", "q8"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    if op == "q8":
        K = _spread(rng, 64, 16384)
        N = _spread(rng, 16, min(32768, (1 << 28) // K))
        rows = _spread(rng, 1, max(1, min(16384, (1 << 38) // (K * N), (1 << 27) // max(K, N))))
        return {"op": op, "rows": rows, "N": N, "K": K, "dtype": dtype, "bias": rng.random() < 0.5}
    direction = rng.choice(("forward", "train"))
    if op == "delta":
        dk = rng.choice((64, 96, 128, rng.randint(16, 128)))
        dv = rng.choice((64, 96, 128, rng.randint(16, 160)))
        HK = rng.choice((1, 2, 3, 6, 9))
        H = HK * rng.choice((1, 1, 2))
        B = rng.choice((1, 2, 3, 4, 8))
        most = (100_000_000 if direction == "forward" else 25_000_000) // (B * H * max(dk, dv))
        T = _spread(rng, 1, max(1, min(131072 if direction == "forward" else 8192, most)))
        return {"op": op, "direction": direction, "T": T, "B": B, "HK": HK, "H": H, "dk": dk, "dv": dv,
                "dtype": dtype, "unit": rng.random() < 0.7, "ragged": B > 1 and rng.random() < 0.4}
    D = rng.choice((256, 768, 864, _spread(rng, 64, 8192)))
    rows = _spread(rng, 1, 60_000_000 // D)
    return {"op": op, "direction": direction, "rows": rows, "D": D, "dtype": dtype,
            "res": rng.choice(("f32", dtype, "none"))}


def _lengths(case):
    """Unequal lengths from T down to 0: the last slot of a padded batch is empty."""
    T, B = case["T"], case["B"]
    return [T - b * T // (B - 1) for b in range(B)]


class _Inputs:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=self.gen, device="cuda") * scale + shift).to(dtype)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.gen, device="cuda")

    def codes(self, *shape):
        return torch.randint(-127, 128, shape, generator=self.gen, device="cuda", dtype=torch.int8)


def prepare(case, seed):
    r = _Inputs(seed)
    s = {"case": case}
    t = TYPES[case["dtype"]]
    if case["op"] == "delta":
        T, B, HK, H, dk, dv = (case[n] for n in ("T", "B", "HK", "H", "dk", "dv"))
        # keys and queries that are not divided by their length come near to length one
        size = 1.0 if case["unit"] else 0.9 / math.sqrt(dk)
        s["q"] = r.normal(T, B, HK, dk, dtype=t, scale=size)
        s["k"] = r.normal(T, B, HK, dk, dtype=t, scale=size)
        s["v"] = r.normal(T, B, H, dv, dtype=t)
        # decay times from 2 to 4096 positions, moved about by the data
        times = 2.0 * torch.exp(r.uniform(H) * math.log(2048.0))
        s["g"] = -torch.exp(r.normal(T, B, H, scale=0.5)) / times
        s["beta"] = 1 / (1 + torch.exp(-r.normal(T, B, H)))
        s["state"] = r.normal(B, H, dk, dv, scale=0.3)
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if case["direction"] == "train":
            s["dy"] = r.normal(T, B, H, dv, dtype=t)
            s["dfinal"] = r.normal(B, H, dk, dv)
    elif case["op"] == "layer":
        N, D = case["rows"], case["D"]
        rt = TYPES[case["res"]] if case["res"] != "none" else t
        s["x"] = r.normal(N, D, dtype=t, shift=0.25)
        s["res"] = r.normal(N, D, dtype=rt, scale=2.0, shift=0.5) if case["res"] != "none" else None
        s["weight"], s["bias"] = r.normal(D, scale=0.1, shift=1.0), r.normal(D, scale=0.1)
        if case["direction"] == "train":
            s["dr"] = r.normal(N, D, dtype=rt) if s["res"] is not None else None
            s["da"] = r.normal(N, D, dtype=t)
    else:
        N, K = case["N"], case["K"]
        s["x"] = r.normal(case["rows"], K, dtype=t)
        s["codes"] = r.codes(N, K)
        # steps of weights of about 0.02, as the block's are
        s["scales"] = (r.uniform(N) + 0.5) * 0.0003
        s["bias"] = r.normal(N) if case["bias"] else None
        if own:
            from long_convolution_sequence_amd import ops
            s["weight"] = ops.Q8Weight(s["codes"], s["scales"])
    return s


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "q8":
        N, K, M = case["N"], case["K"], case["rows"]
        return {"bytes": N * K + 4 * N + (4 * N if case["bias"] else 0) + M * (K + N) * es, "flops": 2 * M * N * K}
    if case["op"] == "delta":
        T, B, HK, H, dk, dv = (case[n] for n in ("T", "B", "HK", "H", "dk", "dv"))
        live, rows = sum(_lengths(case)) if case["ragged"] else T * B, T * B
        state = 4 * B * H * dk * dv
        qk, v, gates = 2 * HK * dk * es, H * dv * es, 8 * H
        if case["direction"] == "forward":
            return {"bytes": live * (qk + v + gates) + rows * v + 2 * state, "flops": 7 * live * H * dk * dv}
        # q, k, v, g, beta, dy in; y and the gradients out; states and their gradients
        return {"bytes": live * (qk + 2 * v + gates) + rows * (2 * v + qk + gates) + 4 * state,
                "flops": 21 * live * H * dk * dv}
    n, D = case["rows"] * case["D"], case["D"]
    rs = SIZE[case["res"]] if case["res"] != "none" else 0
    forward = n * (2 * es + 2 * rs) + 8 * D
    if case["direction"] == "forward":
        return {"bytes": forward, "flops": 8 * n}
    # dr and da in, the gradients of x and res, which are one tensor's values, out
    return {"bytes": forward + n * (2 * es + 2 * rs) + 8 * D, "flops": 24 * n}


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"delta": _plain_delta, "layer": _plain_layer, "q8": _plain_q8}[c["op"]](s, c)


def _run_own(s, c):
    from long_convolution_sequence_amd import ops
    if c["op"] == "q8":
        return {"y": ops.q8_product(s["weight"], s["x"], s["bias"])}
    if c["op"] == "delta":
        args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
        if c["direction"] == "forward":
            y, final = ops.gated_delta(*args, s["state"], s["lengths"], unit=c["unit"])
            return {"y": y, "final": final}
        y, final, saved = ops.gated_delta(*args, s["state"], s["lengths"], unit=c["unit"], save=True)
        d = ops.gated_delta_backward(s["dy"], *args, saved, s["state"], s["lengths"], dfinal=s["dfinal"],
                                     unit=c["unit"])
        return {"y": y, "final": final, "dq": d.q, "dk": d.k, "dv": d.v, "dg": d.decay, "dbeta": d.beta,
                "dstate": d.state}
    weights = {"weight": s["weight"], "bias": s["bias"], "eps": EPS}
    if c["direction"] == "forward":
        r, a = ops.layer_norm(s["x"], s["res"], **weights)
        return {"r": r, "a": a} if s["res"] is not None else {"a": a}
    r, a, saved = ops.layer_norm(s["x"], s["res"], save=True, **weights)
    d = ops.layer_norm_backward(s["dr"], s["da"], s["x"], s["res"], saved, **weights)
    out = {"a": a, "dx": d.x, "dweight": d.weight, "dbias": d.bias}
    return {**out, "r": r, "dres": d.res} if s["res"] is not None else out


# ---- plain forms: elementary operations in 32 bits, rounded once at the end ----------------------------------------

CHUNK = 64


def _chunks(x, H):
    """[T][B][HK][d] as [chunk][B][H][CHUNK][d] in 32 bits, zeros behind the end, shared heads repeated."""
    T, B, HK, d = x.shape
    n = -(-T // CHUNK)
    full = torch.zeros((n * CHUNK, B, HK, d), dtype=torch.float32, device=x.device)
    full[:T] = x
    return full.view(n, CHUNK, B, HK, d).permute(0, 2, 3, 1, 4).repeat_interleave(H // HK, 2).contiguous()


def _rows_of(x, T):
    """The way back: [chunk][B][H][CHUNK][d] as [T][B][H][d]."""
    n, B, H, _, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(n * CHUNK, B, H, d)[:T]


def _plain_delta(s, c):
    """Chunk by chunk.  With G the sum of g from the chunk's start, E_ij = e^(G_i - G_j) (i >= j), L_ij = b_i E_ij k_i.k_j
    (i > j) and N = (I + L)^-1: R = V - e^G K S, U = N (b R), Y = scale (e^G Q S + (E o Q K^T) U),
    S' = e^(G_end) S + sum_j e^(G_end - G_j) k_j u_j^T."""
    T, HK, H, dk, dv = (c[n] for n in ("T", "HK", "H", "dk", "dv"))
    t = s["q"].dtype
    scale = 1 / math.sqrt(dk)
    q, k = s["q"].float(), s["k"].float()
    rq, rk = ((1 / torch.sqrt((x * x).sum(-1, keepdim=True) + UNIT_EPS) if c["unit"] else torch.ones_like(x[..., :1]))
              for x in (q, k))
    hq, hk = q * rq, k * rk
    live = None
    g, beta, v = s["g"], s["beta"], s["v"].float()
    if s["lengths"] is not None:
        live = (torch.arange(T, device=q.device)[:, None] < s["lengths"][None, :])[..., None]
        g, beta = torch.where(live, g, 0.0), torch.where(live, beta, 0.0)
        live = live[..., None]
        hq, hk, v = torch.where(live, hq, 0.0), torch.where(live, hk, 0.0), torch.where(live, v, 0.0)
    Q, K, V = _chunks(hq, H), _chunks(hk, H), _chunks(v, H)
    G = _chunks(g[..., None], H)[..., 0].double().cumsum(-1)
    b = _chunks(beta[..., None], H)
    index = torch.arange(CHUNK, device=q.device)
    below, upto = index[:, None] > index[None, :], index[:, None] >= index[None, :]
    E = torch.exp(torch.where(upto, G[..., :, None] - G[..., None, :], 0.0)).float()
    KT = K.transpose(-1, -2).contiguous()
    kk, qk = K @ KT, Q @ KT
    L = torch.where(below, b * E * kk, 0.0)
    # (I + L)^-1 = (I - L)(I + L^2)(I + L^4) ...: in 64 bits, since powers of L may grow before they vanish
    power = -L.double()
    N = torch.eye(CHUNK, dtype=torch.float64, device=q.device) + power
    for _ in range(5):
        power = power @ power
        N = N + N @ power
    N = N.float()
    P = torch.where(upto, E * qk, 0.0)
    eG, eE = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    last = eG[..., -1:, :]
    KE = (K * eE).transpose(-1, -2).contiguous()
    KG, Nb = K * eG, N * b.transpose(-1, -2)
    NV, NK = Nb @ V, Nb @ KG
    state, states, U = s["state"], [], []
    for i in range(Q.shape[0]):
        states.append(state)
        u = NV[i] - NK[i] @ state
        U.append(u)
        state = last[i] * state + KE[i] @ u
    S, U, final = torch.stack(states), torch.stack(U), state
    y = _rows_of(scale * (eG * (Q @ S) + P @ U), T).to(t)
    if c["direction"] == "forward":
        return {"y": y, "final": final}

    dy = s["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    dY = scale * _chunks(dy, H)
    PT, NT = P.transpose(-1, -2).contiguous(), N.transpose(-1, -2).contiguous()
    D0, dS0 = PT @ dY, (Q * eG).transpose(-1, -2).contiguous() @ dY
    KGT, KEr = KG.transpose(-1, -2).contiguous(), K * eE
    dstate, ends, X = s["dfinal"], [], []
    for i in range(Q.shape[0] - 1, -1, -1):
        ends.append(dstate)
        x = NT[i] @ (D0[i] + KEr[i] @ dstate)
        X.append(x)
        dstate = last[i] * dstate + dS0[i] - KGT[i] @ (b[i] * x)
    dE, X = torch.stack(ends[::-1]), torch.stack(X[::-1])
    Z = b * X
    UT, ST = U.transpose(-1, -2).contiguous(), S.transpose(-1, -2).contiguous()
    XU = torch.where(below, E * (X @ UT), 0.0)
    Hm = -b * XU
    J = torch.where(upto, E * (dY @ UT), 0.0)
    fromq, fromk, toend = eG * (dY @ ST), eG * (Z @ ST), eE * (U @ dE.transpose(-1, -2).contiguous())
    dQ = J @ K + fromq
    dK = Hm @ K + Hm.transpose(-1, -2).contiguous() @ K + J.transpose(-1, -2).contiguous() @ Q - fromk + toend
    R = V - KG @ S
    dbeta = (R * X).sum(-1) - (XU * kk).sum(-1)
    pairs = (Hm * kk + J * qk).double()
    ends = (K * toend).sum(-1).double()
    dG = pairs.sum(-1) - pairs.sum(-2) + ((Q * fromq).sum(-1) - (K * fromk).sum(-1)).double() - ends
    dG[..., -1] += ends.sum(-1) + (last.double()[..., 0, 0] * (dE * S).double().sum((-1, -2)))
    dg = dG.flip(-1).cumsum(-1).flip(-1).float()

    def back(hat, r, d):
        d = d.reshape(d.shape[0], d.shape[1], HK, H // HK, dk).sum(3)
        return r * (d - hat * (hat * d).sum(-1, keepdim=True)) if c["unit"] else d
    dq, dkk = back(hq, rq, _rows_of(dQ, T)), back(hk, rk, _rows_of(dK, T))
    dvv, dg, dbeta = _rows_of(Z, T), _rows_of(dg[..., None], T)[..., 0], _rows_of(dbeta[..., None], T)[..., 0]
    if live is not None:
        dq, dkk, dvv = torch.where(live, dq, 0.0), torch.where(live, dkk, 0.0), torch.where(live, dvv, 0.0)
        dg, dbeta = torch.where(live[..., 0], dg, 0.0), torch.where(live[..., 0], dbeta, 0.0)
    return {"y": y, "final": final, "dq": dq.to(t), "dk": dkk.to(t), "dv": dvv.to(t), "dg": dg.contiguous(),
            "dbeta": dbeta.contiguous(), "dstate": dstate}


def _plain_layer(s, c):
    t = s["x"].dtype
    r = s["x"].float()
    if s["res"] is not None:
        r = s["res"].float() + r
    centred = r - r.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((centred * centred).mean(-1, keepdim=True) + EPS)
    unit = centred * rstd
    out = {"a": (unit * s["weight"] + s["bias"]).to(t)}
    if s["res"] is not None:
        out["r"] = r.to(s["res"].dtype)
    if c["direction"] == "forward":
        return out
    da = s["da"].float()
    u = da * s["weight"]
    d = rstd * (u - u.mean(-1, keepdim=True) - unit * (u * unit).mean(-1, keepdim=True))
    if s["res"] is not None:
        d = d + s["dr"].float()
        out["dres"] = d.to(s["res"].dtype)
    return {**out, "dx": d.to(t), "dweight": (da * unit).sum(0, dtype=torch.float64).float(),
            "dbias": da.sum(0, dtype=torch.float64).float()}


def _plain_q8(s, c):
    x = s["x"].float()
    # a quotient by a tensor: by a number, torch multiplies by its rounded reciprocal
    scale = x.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=x.device)
    codes = torch.round(torch.where(scale > 0, x / scale, 0.0))
    y = (codes @ s["codes"].float().t()) * scale * s["scales"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype)}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "layer": _exact_layer, "q8": _exact_q8}[case["op"]](s, case)


def _exact_delta(s, c):
    """Position by position, forwards and then backwards (from states kept every so often)."""
    T, B, HK, H, dk, dv = (c[n] for n in ("T", "B", "HK", "H", "dk", "dv"))
    scale, share = dk ** -0.5, H // HK
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    nq, nk = ((x.square().sum(-1, keepdim=True) + UNIT_EPS).sqrt() if c["unit"] else torch.ones_like(x[..., :1])
              for x in (q, k))
    q, k = q / nq, k / nk
    qh, kh = (x.repeat_interleave(share, 2).unsqueeze(-1) for x in (q, k))       # [T][B][H][dk][1]
    a, beta, v = s["g"].double().exp(), s["beta"].double(), v.unsqueeze(-2)      # v [T][B][H][1][dv]
    dead = None
    if s["lengths"] is not None:
        dead = torch.arange(T, device=q.device)[:, None] >= s["lengths"][None, :]
        a, beta = a.masked_fill(dead[..., None], 1.0), beta.masked_fill(dead[..., None], 0.0)
    a, beta = a[..., None, None], beta[..., None, None]

    def step(S, t):
        decayed = a[t] * S
        error = v[t] - (kh[t] * decayed).sum(-2, keepdim=True)
        return decayed, error, torch.addcmul(decayed, kh[t], beta[t] * error)

    train = c["direction"] == "train"
    S, every, kept = s["state"].double(), 64, []
    y = torch.empty((T, B, H, dv), dtype=torch.float64, device=q.device)
    for t in range(T):
        if train and t % every == 0:
            kept.append(S)
        S = step(S, t)[2]
        torch.sum(S * qh[t], -2, out=y[t])
    y *= scale
    if dead is not None:
        y.masked_fill_(dead[..., None, None], 0.0)
    out = {"y": y, "final": S}
    if not train:
        return out
    dy = s["dy"].double() * scale
    if dead is not None:
        dy = dy.masked_fill(dead[..., None, None], 0.0)
    dy = dy.unsqueeze(-2)
    dq, dkey = (torch.empty((T, B, H, dk), dtype=torch.float64, device=q.device) for _ in range(2))
    dval = torch.empty((T, B, H, dv), dtype=torch.float64, device=q.device)
    dg, dbeta = (torch.empty((T, B, H), dtype=torch.float64, device=q.device) for _ in range(2))
    D = s["dfinal"].double()
    for first in range((T - 1) // every * every, -1, -every):
        S, seen = kept[first // every], []
        for t in range(first, min(T, first + every)):
            seen.append(step(S, t))
            S = seen[-1][2]
        for t in range(min(T, first + every) - 1, first - 1, -1):
            decayed, error, S = seen[t - first]
            dq[t] = (S * dy[t]).sum(-1)
            D = torch.addcmul(D, qh[t], dy[t])
            du = (D * kh[t]).sum(-2, keepdim=True)
            dbeta[t] = (du * error).sum((-1, -2))
            de = beta[t] * du
            dval[t] = de[..., 0, :]
            dkey[t] = (D * (beta[t] * error) - decayed * de).sum(-1)
            D = torch.addcmul(D, kh[t], de, value=-1)
            dg[t] = (D * decayed).sum((-1, -2))
            D = a[t] * D

    def back(hat, norm, d):
        d = d.unflatten(2, (HK, share)).sum(3)
        return (d - hat * (hat * d).sum(-1, keepdim=True)) / norm if c["unit"] else d
    out.update(dq=back(q, nq, dq), dk=back(k, nk, dkey), dv=dval, dg=dg, dbeta=dbeta, dstate=D)
    if dead is not None:
        for n in ("dq", "dk", "dv"):
            out[n] = out[n].masked_fill(dead[..., None, None], 0.0)
        for n in ("dg", "dbeta"):
            out[n] = out[n].masked_fill(dead[..., None], 0.0)
    return out


def _exact_layer(s, c):
    """The definition, its gradients by differentiating it."""
    train = c["direction"] == "train"
    names = [n for n in ("x", "res", "weight", "bias") if s[n] is not None]
    v = {n: s[n].double().requires_grad_(train) for n in names}
    with torch.set_grad_enabled(train):
        r = v["x"] + v["res"] if "res" in v else v["x"]
        mean = r.mean(-1, keepdim=True)
        a = (r - mean) * torch.rsqrt((r - mean).pow(2).mean(-1, keepdim=True) + EPS) * v["weight"] + v["bias"]
        if train:
            outs = (r, a) if "res" in v else (a,)
            into = (s["dr"].double(), s["da"].double()) if "res" in v else (s["da"].double(),)
            g = torch.autograd.grad(outs, [v[n] for n in names], into)
    out = {"a": a.detach()}
    if "res" in v:
        out["r"] = r.detach()
    if train:
        out.update({"d" + n: x for n, x in zip(names, g)})
    return out


def _exact_q8(s, c):
    """Output by output in groups; scales and codes are by definition those of a quotient in 32 bits."""
    x = s["x"].float()
    scale = x.abs().amax(-1, keepdim=True)
    scale = scale.div(torch.full_like(scale, 127.0))
    codes = x.div(scale).nan_to_num(0.0).round().double()
    scale = scale.double()
    y = torch.empty((c["rows"], c["N"]), dtype=torch.float64, device=x.device)
    for n in range(0, c["N"], 4096):
        y[:, n:n + 4096] = scale * (codes @ s["codes"][n:n + 4096].double().t()) * s["scales"][n:n + 4096].double()
    return {"y": y + s["bias"].double() if s["bias"] is not None else y}
