"""Refusals of the recurrent-block operators, without a GPU: every bad argument
is an error before anything is launched, at the C entries and in the binding."""
import ctypes
import warnings

import pytest
import torch

from long_convolution_sequence_amd import fi, ops

class ScanDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("batch", ctypes.c_int), ("channels", ctypes.c_int), ("dtype", ctypes.c_int),
                ("input", ctypes.c_int), ("ld_x", ctypes.c_int64), ("ld_gate", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_dy", ctypes.c_int64), ("ld_dx", ctypes.c_int64),
                ("ld_dgate", ctypes.c_int64), ("reserved", ctypes.c_int * 4)]


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int), ("dtype", ctypes.c_int),
                ("res_dtype", ctypes.c_int), ("post_norm", ctypes.c_int), ("act", ctypes.c_int),
                ("eps", ctypes.c_float)] + \
        [(n, ctypes.c_int64) for n in ("ld_o", "ld_gate", "ld_res", "ld_r", "ld_a", "ld_dr", "ld_da", "ld_do",
                                       "ld_dgate", "ld_dres")] + [("reserved", ctypes.c_int * 4)]


class Q4Desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("K", ctypes.c_int), ("group", ctypes.c_int), ("scale_dtype", ctypes.c_int),
                ("has_zeros", ctypes.c_int), ("reserved", ctypes.c_int * 3)]


P = 0x100000          # made-up device addresses: nothing below reaches a launch
STEP = 0x1000000


@pytest.fixture(scope="module")
def lib():
    return fi.load_library()


def _ptrs(n):
    return [P + i * STEP for i in range(n)]


def _scan(T=300, B=2, D=5, dtype=ops.F32, input=ops.SCAN_CONVEX, **kw):
    q = ScanDesc()
    q.T, q.batch, q.channels, q.dtype, q.input = T, B, D, dtype, input
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def _scan_args(**kw):
    names = ["x", "gate", "bias", "state", "lengths", "y", "final", "saved", "workspace"]
    a = dict(zip(names, _ptrs(len(names))))
    a.update(kw)
    return [a[k] for k in names] + [None]


def _back_args(**kw):
    names = ["x", "gate", "bias", "state", "lengths", "saved", "dy", "dfinal", "dx", "dgate", "dbias", "dstate",
             "workspace"]
    a = dict(zip(names, _ptrs(len(names))))
    a.update(kw)
    return [a[k] for k in names] + [None]


def _refused(lib, status, why):
    assert status == fi.FI_EINVAL
    assert why in lib.fi_op_last_error().decode()


@pytest.mark.parametrize("kw,why", [
    (dict(T=-1), "T >= 0"), (dict(B=0), "batch >= 1"), (dict(D=0), "channels >= 1"), (dict(dtype=3), "dtype"),
    (dict(dtype=-1), "dtype"), (dict(input=3), "input"), (dict(input=-1), "input"), (dict(ld_x=4), "pitch"),
    (dict(ld_gate=-5), "pitch"), (dict(ld_y=4), "pitch"), (dict(ld_dy=1), "pitch"), (dict(ld_dx=1), "pitch"),
    (dict(ld_dgate=1), "pitch"), (dict(B=1 << 13, D=1 << 12), "2^24"), (dict(T=(1 << 23) + 1), "2^23"),
    (dict(T=1 << 23, B=1, D=8193), "too large"), (dict(T=1 << 23, B=2049, D=1), "too large"),
    (dict(T=1 << 23, B=683, D=3), "too large")])
def test_scan_descriptors_are_checked(lib, kw, why):
    q = _scan(**kw)
    assert lib.fi_scan_saved_bytes(ctypes.byref(q)) == 0
    assert lib.fi_scan_workspace_bytes(ctypes.byref(q), 0) == 0
    assert lib.fi_scan_workspace_bytes(ctypes.byref(q), 1) == 0
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args()), why)
    _refused(lib, lib.fi_scan_backward(ctypes.byref(q), *_back_args()), why)


def test_scan_reserved_and_null_descriptors_are_refused(lib):
    q = _scan()
    q.reserved[2] = 1
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args()), "reserved")
    _refused(lib, lib.fi_scan_forward(None, *_scan_args()), "null descriptor")
    _refused(lib, lib.fi_scan_backward(None, *_back_args()), "null descriptor")
    assert lib.fi_scan_saved_bytes(None) == 0 and lib.fi_scan_workspace_bytes(None, 1) == 0


@pytest.mark.parametrize("missing", ["x", "gate", "y", "workspace"])
def test_scan_forward_needs_its_tensors(lib, missing):
    q = _scan(T=70000)
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args(**{missing: None})), "required")


@pytest.mark.parametrize("missing", ["x", "gate", "saved", "dy", "dx", "dgate"])
def test_scan_backward_needs_its_tensors(lib, missing):
    q = _scan(T=70000)
    _refused(lib, lib.fi_scan_backward(ctypes.byref(q), *_back_args(**{missing: None})), "required")


@pytest.mark.parametrize("T,B,D", [(10, 2, 5), (200, 2, 32), (256, 1, 64), (300, 1, 1), (300, 2, 5)])
def test_which_scans_need_a_workspace(lib, T, B, D):
    """Forwards a workspace of 256 bytes may be left out (the call gets as far as the next check);
    backwards none may, also where 256 bytes are all there is."""
    q = _scan(T=T, B=B, D=D)
    forward = lib.fi_scan_workspace_bytes(ctypes.byref(q), 0)
    why = "aligned" if forward == 256 else "required"
    assert (forward == 256) == (T <= 256)
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args(workspace=None, bias=P + 2 * STEP + 1)), why)
    _refused(lib, lib.fi_scan_backward(ctypes.byref(q), *_back_args(workspace=None, bias=P + 2 * STEP + 1)), "required")


@pytest.mark.parametrize("kw", [dict(y=P + 4), dict(y=P + STEP), dict(final=P), dict(final=P + 3 * STEP + 4),
                                dict(saved=P + 5 * STEP), dict(workspace=P + 256), dict(final=P + 5 * STEP),
                                dict(state=P + 5 * STEP, final=P + 5 * STEP)])
def test_scan_outputs_may_not_overlap(lib, kw):
    q = _scan(T=2000)
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args(**kw)), "shares memory")


def test_scan_slices_of_one_tensor_may_interleave_but_not_overlap(lib):
    """x, gate and y as thirds of one [T*B][15] tensor pass the overlap check (then a
    misaligned workspace stops the call); a y that begins inside the gate does not."""
    q = _scan(ld_x=15, ld_gate=15, ld_y=15)
    bad_ws = dict(workspace=P + 8 * STEP + 4)
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args(gate=P + 20, y=P + 40, **bad_ws)), "256")
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args(gate=P + 20, y=P + 36)), "shares memory")
    q.ld_y = 16                # another pitch over the same memory
    _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args(gate=P + 20, y=P + 40)), "shares memory")


@pytest.mark.parametrize("kw", [dict(dx=P), dict(dgate=P + 8 * STEP), dict(dbias=P + 2 * STEP), dict(dstate=P + 3 * STEP),
                                dict(dstate=P + 7 * STEP), dict(dx=P + 5 * STEP), dict(workspace=P + 9 * STEP)])
def test_scan_backward_outputs_may_not_overlap(lib, kw):
    q = _scan(T=2000)
    _refused(lib, lib.fi_scan_backward(ctypes.byref(q), *_back_args(**kw)), "shares memory")


def _norm(rows=7, D=9, dtype=ops.BF16, res_dtype=ops.F32, post_norm=1, act=ops.GATE_SILU, eps=1e-6, **kw):
    q = NormDesc()
    q.rows, q.channels, q.dtype, q.res_dtype, q.post_norm, q.act, q.eps = rows, D, dtype, res_dtype, post_norm, act, eps
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def _norm_args(**kw):
    names = ["o", "gate", "res", "w1", "k", "w2", "r", "a", "saved"]
    a = dict(zip(names, _ptrs(len(names))))
    a.update(kw)
    return [a[k] for k in names] + [None]


def _norm_back_args(**kw):
    names = ["o", "gate", "res", "w1", "k", "w2", "saved", "dr", "da", "do", "dgate", "dres", "dpost", "dscale",
             "dpre", "workspace"]
    a = dict(zip(names, _ptrs(len(names))))
    a.update(kw)
    return [a[k] for k in names] + [None]


@pytest.mark.parametrize("kw,why", [
    (dict(rows=-1), "rows"), (dict(D=0), "channels"), (dict(D=16385), "channels"), (dict(dtype=5), "dtype"),
    (dict(dtype=ops.BF16, res_dtype=ops.F16), "res_dtype"), (dict(dtype=ops.F32, res_dtype=ops.BF16), "res_dtype"),
    (dict(post_norm=2), "post_norm"), (dict(act=3), "act"), (dict(eps=-1e-6), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(ld_o=8), "pitch"), (dict(ld_gate=8), "pitch"), (dict(ld_res=8), "pitch"), (dict(ld_r=8), "pitch"),
    (dict(ld_a=8), "pitch"), (dict(ld_dr=8), "pitch"), (dict(ld_da=8), "pitch"), (dict(ld_do=8), "pitch"),
    (dict(ld_dgate=8), "pitch"), (dict(ld_dres=-9), "pitch")])
def test_norm_descriptors_are_checked(lib, kw, why):
    q = _norm(**kw)
    assert lib.fi_norm_workspace_bytes(ctypes.byref(q)) == 0
    _refused(lib, lib.fi_norm_forward(ctypes.byref(q), *_norm_args()), why)
    _refused(lib, lib.fi_norm_backward(ctypes.byref(q), *_norm_back_args()), why)


def test_norm_inputs_that_do_not_go_together_are_refused(lib):
    q = ctypes.byref(_norm())
    _refused(lib, lib.fi_norm_forward(q, *_norm_args(o=None, res=None)), "o or res")
    _refused(lib, lib.fi_norm_forward(q, *_norm_args(o=None)), "need o")
    keep = _norm(post_norm=0)
    q0 = ctypes.byref(keep)
    _refused(lib, lib.fi_norm_forward(q0, *_norm_args()), "post_weight needs post_norm")
    _refused(lib, lib.fi_norm_forward(q0, *_norm_args(o=None, w1=None, k=None)), "need o")
    _refused(lib, lib.fi_norm_forward(q0, *_norm_args(o=None, w1=None, gate=None)), "need o")
    for kw in (dict(gate=None), dict(res=None), dict(da=None)):
        keep = _norm()
        _refused(lib, lib.fi_norm_backward(ctypes.byref(keep), *_norm_back_args(**kw)), "is not given")
    _refused(lib, lib.fi_norm_backward(q0, *_norm_back_args(w1=None)), "is not given")          # dpost, no norm
    for kw in (dict(saved=None), dict(workspace=None), dict(workspace=P + 15 * STEP + 8)):
        keep = _norm()
        _refused(lib, lib.fi_norm_backward(ctypes.byref(keep), *_norm_back_args(**kw)), "required")


@pytest.mark.parametrize("kw", [dict(r=P), dict(a=P), dict(r=P + 2 * STEP + 4), dict(a=P + 2 * STEP), dict(a=P + 6 * STEP),
                                dict(saved=P + 7 * STEP), dict(a=P + 5 * STEP)])
def test_norm_outputs_may_not_overlap(lib, kw):
    keep = _norm(rows=50)
    _refused(lib, lib.fi_norm_forward(ctypes.byref(keep), *_norm_args(**kw)), "shares memory")


def test_norm_in_place_needs_the_same_pitch(lib):
    keep = _norm(rows=50, ld_r=10)
    _refused(lib, lib.fi_norm_forward(ctypes.byref(keep), *_norm_args(r=P + 2 * STEP)), "shares memory")


@pytest.mark.parametrize("kw", [dict(do=P), dict(dgate=P + STEP), dict(dres=P + 2 * STEP), dict(dres=P + 7 * STEP + 4),
                                dict(do=P + 8 * STEP), dict(dpre=P + 12 * STEP), dict(workspace=P + 6 * STEP),
                                dict(do=P + 7 * STEP)])
def test_norm_backward_outputs_may_not_overlap(lib, kw):
    keep = _norm(rows=50)
    _refused(lib, lib.fi_norm_backward(ctypes.byref(keep), *_norm_back_args(**kw)), "shares memory")


def _q4(N=20, K=70, group=32, scale_dtype=ops.BF16, has_zeros=0):
    q = Q4Desc()
    q.N, q.K, q.group, q.scale_dtype, q.has_zeros = N, K, group, scale_dtype, has_zeros
    return q


@pytest.mark.parametrize("kw,why", [(dict(N=0), "N and K"), (dict(K=0), "N and K"), (dict(N=(1 << 20) + 1), "N and K"),
                                    (dict(group=16), "group"), (dict(group=48), "group"), (dict(scale_dtype=3), "scale"),
                                    (dict(has_zeros=2), "has_zeros")])
def test_q4_descriptors_are_checked(lib, kw, why):
    q = _q4(**kw)
    assert lib.fi_q4_packed_bytes(ctypes.byref(q)) == 0
    _refused(lib, lib.fi_q4_pack(ctypes.byref(q), P, P + STEP, None, P + 2 * STEP, None), why)
    _refused(lib, lib.fi_q4_quantize(ctypes.byref(q), 0, P, 0, P + STEP, P + 2 * STEP, None), why)
    _refused(lib, lib.fi_q4_matvec(ctypes.byref(q), P, 1, 0, P + STEP, 0, P + 2 * STEP, 0, None), why)


def test_q4_packed_bytes(lib):
    """Tiles of 16 x 128 codes (1 KB), 16 scales and 16 four-bit zeros per group of the padded sizes."""
    up = lambda v: (v + 255) // 256 * 256                       # noqa: E731
    for N, K, group, st, z in ((1, 1, 32, ops.F32, 0), (20, 70, 32, ops.BF16, 1), (33, 300, 128, ops.F16, 1)):
        q = _q4(N, K, group, st, z)
        tiles, kt = -(-N // 16), -(-K // 128)
        groups = kt * (128 // group)
        want = tiles * kt * 1024 + up(tiles * groups * 16 * (4 if st == ops.F32 else 2)) + z * up(tiles * groups * 8)
        assert lib.fi_q4_packed_bytes(ctypes.byref(q)) == want


def test_q4_arguments_are_checked(lib):
    keep, zeros = _q4(), _q4(has_zeros=1)
    q, qz = ctypes.byref(keep), ctypes.byref(zeros)
    _refused(lib, lib.fi_q4_pack(q, None, P, None, P + STEP, None), "required")
    _refused(lib, lib.fi_q4_pack(q, P, P + STEP, None, P + 2 * STEP + 8, None), "required")
    _refused(lib, lib.fi_q4_pack(q, P, P + STEP, P + 2 * STEP, P + 3 * STEP, None), "has_zeros")
    _refused(lib, lib.fi_q4_pack(qz, P, P + STEP, None, P + 3 * STEP, None), "has_zeros")
    _refused(lib, lib.fi_q4_pack(q, P, P + STEP, None, P, None), "shares memory")
    _refused(lib, lib.fi_q4_quantize(qz, 0, P, 0, P + STEP, P + 2 * STEP, None), "symmetric")
    _refused(lib, lib.fi_q4_quantize(q, 9, P, 0, P + STEP, P + 2 * STEP, None), "w_dtype")
    _refused(lib, lib.fi_q4_quantize(q, 0, P, 69, P + STEP, P + 2 * STEP, None), "pitch")
    _refused(lib, lib.fi_q4_quantize(q, 0, P, 0, P + STEP, P + 4, None), "shares memory")
    mv = lib.fi_q4_matvec
    _refused(lib, mv(q, P, 0, 0, P + STEP, 0, P + 2 * STEP, 0, None), "rows")
    _refused(lib, mv(q, P, 17, 0, P + STEP, 0, P + 2 * STEP, 0, None), "rows")
    _refused(lib, mv(q, P, 1, 7, P + STEP, 0, P + 2 * STEP, 0, None), "dtype")
    _refused(lib, mv(q, P + 4, 1, 0, P + STEP, 0, P + 2 * STEP, 0, None), "required")
    _refused(lib, mv(q, P, 1, 0, None, 0, P + 2 * STEP, 0, None), "required")
    _refused(lib, mv(q, P, 2, 0, P + STEP, 69, P + 2 * STEP, 0, None), "pitch")
    _refused(lib, mv(q, P, 2, 0, P + STEP, 0, P + 2 * STEP, 19, None), "pitch")
    _refused(lib, mv(q, P, 2, 0, P + STEP, 0, P + STEP + 4, 0, None), "shares memory")


def test_misaligned_pointers_are_refused(lib):
    q = _scan(T=2000)
    for name in ("x", "gate", "y", "bias", "state", "lengths", "final"):
        a = dict(zip(["x", "gate", "bias", "state", "lengths", "y", "final", "saved", "workspace"], _ptrs(9)))
        _refused(lib, lib.fi_scan_forward(ctypes.byref(q), *_scan_args(**{name: a[name] + 2})), "aligned")
    names = ["x", "gate", "bias", "state", "lengths", "saved", "dy", "dfinal", "dx", "dgate", "dbias", "dstate", "workspace"]
    a = dict(zip(names, _ptrs(13)))
    for name in ("x", "dy", "dfinal", "dx", "dgate", "dbias", "dstate"):
        _refused(lib, lib.fi_scan_backward(ctypes.byref(q), *_back_args(**{name: a[name] + 2})), "aligned")
    n = _norm(rows=50)
    names = ["o", "gate", "res", "w1", "k", "w2", "r", "a", "saved"]
    for name, off in zip(names, (1, 1, 2, 2, 2, 2, 2, 1, 2)):
        at = dict(zip(names, _ptrs(9)))[name] + off
        _refused(lib, lib.fi_norm_forward(ctypes.byref(n), *_norm_args(**{name: at})), "aligned")
    names = ["o", "gate", "res", "w1", "k", "w2", "saved", "dr", "da", "do", "dgate", "dres", "dpost", "dscale", "dpre"]
    for name in ("dr", "da", "do", "dgate", "dres", "dpost", "dscale", "dpre"):
        at = dict(zip(names, _ptrs(15)))[name] + 1
        _refused(lib, lib.fi_norm_backward(ctypes.byref(n), *_norm_back_args(**{name: at})), "aligned")
    w = _q4()
    _refused(lib, lib.fi_q4_pack(ctypes.byref(w), P, P + STEP + 1, None, P + 2 * STEP, None), "aligned")
    _refused(lib, lib.fi_q4_quantize(ctypes.byref(w), 0, P + 2, 0, P + STEP, P + 2 * STEP, None), "aligned")
    _refused(lib, lib.fi_q4_matvec(ctypes.byref(w), P, 1, 0, P + STEP + 2, 0, P + 2 * STEP, 0, None), "aligned")


def test_huge_pitches_do_not_wrap_the_overlap_check(lib):
    """2^40 rows at 2^40 elements: the extents pass 64 bits, and still overlap."""
    n = _norm(rows=1 << 40, ld_o=1 << 40, ld_a=(1 << 40) - 64)
    _refused(lib, lib.fi_norm_forward(ctypes.byref(n), *_norm_args()), "shares memory")


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 2, 8)
    for call in (lambda: ops.gated_scan(x, x), lambda: ops.gated_scan_step(x[0], x[0], x[0]),
                 lambda: ops.gated_scan_backward(x, x, x, x), lambda: ops.block_norm(x),
                 lambda: ops.block_norm_backward(x, x, x, None, None, x), lambda: ops.block_norm(None),
                 lambda: ops.Q4Weight(torch.zeros(4, 4, dtype=torch.uint8), x[0]), lambda: ops.Q4Weight.quantize(x[0]),
                 lambda: ops.q4_matvec(x, x), lambda: ops.gated_scan(None, x), lambda: ops.gated_scan([1], x)):
        with pytest.raises(fi.FiError) as e:
            call()
        assert e.value.status == fi.FI_EINVAL


def test_binding_warns_where_autograd_would_be_expected():
    """A forward call on a tensor that requires gradients says that it is not recorded (and then
    refuses the host tensor); under no_grad, or without such a tensor, it does not."""
    x = torch.zeros(4, 2, 8)
    w = torch.ones(8, requires_grad=True)
    q = object.__new__(ops.Q4Weight)
    q._index = 0
    calls = {"gated_scan": lambda: ops.gated_scan(x, x, w), "gated_scan_step": lambda: ops.gated_scan_step(x[0], x[0], x[0], w),
             "block_norm": lambda: ops.block_norm(x, pre_weight=w),
             "q4_matvec": lambda: ops.q4_matvec(q, x[0].requires_grad_())}
    for name, call in calls.items():
        with pytest.warns(UserWarning, match=f"{name}: autograd does not see"), pytest.raises(fi.FiError):
            call()
        with warnings.catch_warnings(), torch.no_grad(), pytest.raises(fi.FiError):
            warnings.simplefilter("error")
            call()
    with warnings.catch_warnings(), pytest.raises(fi.FiError):
        warnings.simplefilter("error")
        ops.gated_scan(x, x, w.detach())
    for call in (lambda: ops.gated_scan(x, x, w, save=True), lambda: ops.block_norm(x, pre_weight=w, save=True)):
        with warnings.catch_warnings(), pytest.raises(fi.FiError):       # the gradients are asked for explicitly
            warnings.simplefilter("error")
            call()


def test_binding_refuses_values_past_a_descriptors_fields():
    for values in ((1 << 70, 1, 1, 0, 0), (1, 1 << 40, 1, 0, 0), (1, 1, 1, 0, 0.5), (1, 1, None, 0, 0)):
        with pytest.raises(fi.FiError) as e:
            ops._scan_sizes(*values)
        assert e.value.status == fi.FI_EINVAL


def test_largest_scans_fit_a_launch(lib):
    """The largest sizes that are taken: less than 2^23 workgroups, so less than 2^32 threads."""
    for T, B, D in ((1 << 23, 1, 8192), (1 << 23, 1638, 5), (1 << 23, 2048, 1), (1 << 23, 682, 3), (257, 1 << 24, 1),
                    (1 << 20, 1 << 14, 1)):
        assert lib.fi_scan_workspace_bytes(ctypes.byref(_scan(T=T, B=B, D=D)), 0) > 0
        c = 4 if D >= 4 else 1
        groups = (B * -(-D // c) + 15) // 16
        assert -(-T // 256) * groups < 1 << 23


def test_row_pitches():
    """What the binding takes as rows at one pitch, and what it refuses."""
    cpu = -1
    wide = torch.zeros(6, 2, 24)
    assert ops._rows(wide, wide.shape, torch.float32, cpu, "t")[1] == 0
    assert ops._rows(wide[..., 8:16], (6, 2, 8), torch.float32, cpu, "t")[1] == 24
    assert ops._rows(wide[:, :1, :8], (6, 1, 8), torch.float32, cpu, "t")[1] == 48
    assert ops._rows(wide[:1, :1, :8], (1, 1, 8), torch.float32, cpu, "t")[1] == 0
    assert ops._rows(wide[:1, :, :8], (1, 2, 8), torch.float32, cpu, "t")[1] == 24
    for bad in (wide[:, :, ::2], wide.transpose(0, 1), wide[:, :1].expand(6, 2, 24), wide[::2, :, :8],
                wide[:1].expand(6, 2, 24)):
        with pytest.raises(fi.FiError):
            ops._rows(bad, bad.shape, torch.float32, cpu, "t")
