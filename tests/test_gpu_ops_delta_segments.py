"""The gated delta rule in segments: sequences of few heads that are cut, run at the same
time and joined, at every width of the keys, with workgroups of more than one group of
columns, and in the ways in which one segment is tested elsewhere."""
import pytest
import torch

from long_convolution_sequence_amd import fi, ops
from tests import test_gpu_ops_delta as one
from tests._parity import say

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _segments(v):
    """Segments of a call, from the maps [segments][B][H][dk][dk] that it keeps beside the states before its
    chunks and its rows of w."""
    T, B, HK, dk = v["q"].shape
    H, dv = v["v"].shape[2:]
    C = one.CHUNK[v["v"].dtype]
    up = lambda n: -(-n // 256) * 256                                              # noqa: E731
    d = ops._pack(ops._DELTA_DESC, T, B, HK, H, dk, dv, ops._TYPES[v["v"].dtype], 1, 1.0, *([0] * 12))
    chunks = -(-T // C) * B * H
    maps = fi.load_library().fi_delta_saved_bytes(d) - up(chunks * dk * dv * 4) - up(chunks * C * dv * 4) - 256
    return maps // (B * H * dk * dk * 4)


CASES = [  # chunks B HK H dk dv unit lengths (of T) extra positions
    (40, 1, 1, 1, 40, 41, True, None, 0), (33, 2, 1, 2, 72, 150, True, (1.0, 0.4), 5), (48, 1, 2, 2, 96, 128, True, None, 17),
    (36, 2, 1, 2, 128, 128, True, (0.7, 1.0), 1), (34, 1, 1, 1, 128, 1, False, None, 20), (41, 2, 1, 1, 100, 200, True, (0.0, 1.0), 9),
    (64, 1, 1, 1, 64, 260, True, None, 31), (35, 1, 1, 3, 5, 33, False, None, 3)]


@pytest.mark.parametrize("chunks,B,HK,H,dk,dv,unit,parts,extra", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_joined_segments(chunks, B, HK, H, dk, dv, unit, parts, extra, dtype):
    T = chunks * one.CHUNK[dtype] + extra
    say(f"case delta segments T={T} B={B} HK={HK} H={H} dk={dk} dv={dv} {dtype} unit={unit} {parts}")
    v = one._inputs(T, B, HK, H, dk, dv, dtype, unit, [int(p * T) for p in parts] if parts else None, decay=0.03)
    assert _segments(v) >= 4
    c = one._cuda(v)
    one._check(one._run(c, unit), v, unit)
    one._check(one._run(c, unit, train=False), v, unit)


@pytest.mark.parametrize("dk,dv,dtype", [(72, 40, BF16), (128, 150, BF16), (96, 96, F32), (40, 20, F16)])
def test_in_place_state_repeats_streams_and_graphs(dk, dv, dtype):
    say(f"case delta segments in place, side stream, graph dk={dk} dv={dv} {dtype}")
    shape = (40 * one.CHUNK[dtype] + 11, 1, 1, 2, dk, dv, dtype, True)
    v = one._inputs(*shape)
    assert _segments(v) >= 4
    c = one._cuda(v)
    want = one._run(c, True)
    for _ in range(3):
        again = one._run(c, True)
        assert all(torch.equal(again[k], want[k]) for k in want)
    state = c["state"].clone()
    y, final = ops.gated_delta(*(c[n] for n in one.NAMES), state, unit=True, final=state)
    assert final is state and torch.equal(final, want["final"]) and torch.equal(y, want["y"])
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:                                    # two calls at once, workspaces of their own
        with torch.cuda.stream(s):
            outs.append(one._run(c, True))
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[k]) for o in outs for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = one._run(c, True)
    for i in range(3):
        new = one._cuda(one._inputs(*shape, seed=1 + i))
        for k, t in new.items():
            if t is not None:
                c[k].copy_(t)
        g.replay()
        eager = one._run(new, True)
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], eager[k]) for k in out)


def test_a_bad_value_reaches_its_own_head_from_its_chunk_on():
    """A NaN in one segment of one head: the chunks before its own, and the other head, as without it."""
    say("case delta segments bad value")
    v = one._inputs(2600, 1, 1, 2, 72, 40, BF16, True, decay=0.03)
    assert _segments(v) >= 4
    clean = one._run(one._cuda(v), True, train=False)
    v["v"][1500, 0, 1, 3] = float("nan")
    got = one._run(one._cuda(v), True, train=False)
    assert torch.equal(got["y"][:, :, 0], clean["y"][:, :, 0]) and torch.equal(got["final"][:, 0], clean["final"][:, 0])
    start = 1500 // 64 * 64
    assert torch.equal(got["y"][:start], clean["y"][:start]) and got["y"][1500:, 0, 1, 3].isnan().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_left_out_states_and_slices(dtype):
    """No state and no gradient of the last one; q, k, v, gates, outputs and gradients as columns of wider tensors,
    in segments: as packed, and no other column changes."""
    say(f"case delta segments left out and slices {dtype}")
    T, HK, H, dk, dv = 36 * one.CHUNK[dtype] + 7, 1, 2, 40, 52
    v = one._inputs(T, 1, HK, H, dk, dv, dtype, True, state=False, decay=0.03)
    assert _segments(v) >= 4
    c = one._cuda(v)
    want = one._run(c, True, scale=0.3)
    assert want["dstate"] is None
    one._check(want, v, True, scale=0.3)
    sizes, shapes = [HK * dk, HK * dk, H * dv], [(HK, dk), (HK, dk), (H, dv)]
    wide = torch.full((T, 1, 3 + sum(sizes)), 7.0, dtype=dtype, device="cuda")
    grads, gates = torch.full_like(wide, 9.0), torch.zeros(T, 1, 2 * H + 1, device="cuda")
    cut = lambda t: [x.unflatten(-1, s) for x, s in zip(torch.split(t[..., 2:-1], sizes, -1), shapes)]   # noqa: E731
    s = dict(c)
    for n, view in zip(("q", "k", "v"), cut(wide)):
        view.copy_(c[n])
        s[n] = view
    s["g"], s["beta"] = gates[..., :H], gates[..., H + 1:]
    s["g"].copy_(c["g"]), s["beta"].copy_(c["beta"])
    dq, dk_, dv_ = cut(grads)
    got = one._run(s, True, scale=0.3, dq=dq, dk=dk_, dv=dv_)
    assert all(torch.equal(got[k], want[k]) for k in want if want[k] is not None)
    for t, fill in ((wide, 7), (grads, 9)):
        assert (t[..., :2] == fill).all() and (t[..., -1] == fill).all()


def test_gradients_after_a_state_in_place():
    """The state overwritten by the last one: the gradients need what was kept, not the state."""
    say("case delta segments gradients after a state in place")
    v = one._inputs(2400, 1, 1, 1, 72, 40, BF16, True, decay=0.03)
    c = one._cuda(v)
    want = one._run(c, True)
    state = c["state"].clone()
    a = [c[n] for n in one.NAMES]
    _, _, saved = ops.gated_delta(*a, state, unit=True, save=True, final=state)
    d = ops.gated_delta_backward(c["dy"], *a, saved, state, dfinal=c["dfinal"], unit=True)
    assert all(torch.equal(x, want[n]) for n, x in (("dq", d.q), ("dk", d.k), ("dg", d.decay), ("dstate", d.state)))
