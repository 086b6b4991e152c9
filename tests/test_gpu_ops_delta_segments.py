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
