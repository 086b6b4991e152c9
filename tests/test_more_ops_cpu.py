"""Refusals of the gated delta rule, the layer norm and the 8-bit products, without
a GPU: every bad argument is an error before anything is launched, at the C entries
and in the binding."""
import ctypes
import warnings

import pytest
import torch

from long_convolution_sequence_amd import fi, ops

P = 0x100000          # made-up device addresses: nothing below reaches a launch
STEP = 0x10000000


class LayerDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("channels", ctypes.c_int), ("dtype", ctypes.c_int), ("res_dtype", ctypes.c_int),
                ("eps", ctypes.c_float)] + \
        [(n, ctypes.c_int64) for n in ("ld_x", "ld_res", "ld_r", "ld_a", "ld_dr", "ld_da", "ld_dx", "ld_dres")] + \
        [("reserved", ctypes.c_int * 4)]


class DeltaDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64)] + [(n, ctypes.c_int) for n in ("batch", "key_heads", "heads", "dk", "dv", "dtype", "unit")] + \
        [("scale", ctypes.c_float)] + \
        [(n, ctypes.c_int64) for n in ("ld_q", "ld_k", "ld_v", "ld_decay", "ld_beta", "ld_y", "ld_dy", "ld_dq", "ld_dk", "ld_dv",
                                       "ld_ddecay", "ld_dbeta")] + [("reserved", ctypes.c_int * 4)]


@pytest.fixture(scope="module")
def lib():
    return fi.load_library()


def _fill(q, kw, **first):
    for k, v in {**first, **kw}.items():
        setattr(q, k, v)
    return q


def _layer(**kw):
    return _fill(LayerDesc(), kw, rows=10, channels=64, dtype=ops.BF16, res_dtype=ops.F32, eps=1e-5)


def _delta(**kw):
    return _fill(DeltaDesc(), kw, T=100, batch=2, key_heads=2, heads=4, dk=16, dv=24, dtype=ops.BF16, unit=1, scale=0.25)


def _args(names, kw):
    a = {n: P + i * STEP for i, n in enumerate(names)}
    a.update(kw)
    return [a[n] for n in names] + [None]


LAYER = ["x", "res", "weight", "bias", "r", "a", "saved"]
LAYER_BACK = ["x", "res", "weight", "saved", "dr", "da", "dx", "dres", "dweight", "dbias", "workspace"]
DELTA = ["q", "k", "v", "decay", "beta", "state", "lengths", "y", "final", "saved", "workspace"]
DELTA_BACK = ["q", "k", "v", "decay", "beta", "state", "lengths", "saved", "dy", "dfinal", "dq", "dk", "dv", "ddecay", "dbeta",
              "dstate", "workspace"]


def _refused(lib, status, why):
    assert status == fi.FI_EINVAL
    assert why in lib.fi_op_last_error().decode(), lib.fi_op_last_error()


def _layer_refused(lib, desc, why, forward=True, backward=True, **kw):
    ref = ctypes.byref(desc) if desc is not None else None
    if forward:
        _refused(lib, lib.fi_layer_forward(ref, *_args(LAYER, {k: v for k, v in kw.items() if k in LAYER})), why)
    if backward:
        _refused(lib, lib.fi_layer_backward(ref, *_args(LAYER_BACK, {k: v for k, v in kw.items() if k in LAYER_BACK})), why)


def _delta_refused(lib, desc, why, forward=True, backward=True, **kw):
    ref = ctypes.byref(desc) if desc is not None else None
    if forward:
        _refused(lib, lib.fi_delta_forward(ref, *_args(DELTA, {k: v for k, v in kw.items() if k in DELTA})), why)
    if backward:
        _refused(lib, lib.fi_delta_backward(ref, *_args(DELTA_BACK, {k: v for k, v in kw.items() if k in DELTA_BACK})), why)


@pytest.mark.parametrize("kw,why", [
    (dict(rows=-1), "rows"), (dict(rows=(1 << 40) + 1), "rows"), (dict(channels=0), "channels"), (dict(channels=16385), "channels"),
    (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(res_dtype=2), "res_dtype"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(ld_x=63), "pitch"), (dict(ld_res=-1), "pitch"), (dict(ld_r=1), "pitch"),
    (dict(ld_a=63), "pitch"), (dict(ld_dr=2), "pitch"), (dict(ld_da=1), "pitch"), (dict(ld_dx=1), "pitch"),
    (dict(ld_dres=(1 << 40) + 1), "pitch")])
def test_layer_descriptors_are_checked(lib, kw, why):
    q = _layer(**kw)
    assert lib.fi_layer_workspace_bytes(ctypes.byref(q)) == 0
    _layer_refused(lib, q, why)


def test_layer_arguments_are_checked(lib):
    _layer_refused(lib, None, "null descriptor")
    q = _layer()
    q.reserved[1] = 1
    _layer_refused(lib, q, "reserved")
    q = _layer()
    _layer_refused(lib, q, "x or res", x=None, res=None)
    for kw in (dict(x=None), dict(res=None), dict(da=None)):
        _layer_refused(lib, q, "is not given", forward=False, **kw)
    for kw in (dict(saved=None), dict(workspace=None), dict(workspace=P + 100 * STEP + 8)):
        _layer_refused(lib, q, "required", forward=False, **kw)
    for name, off in (("x", 1), ("res", 2), ("weight", 2), ("bias", 1), ("r", 2), ("a", 1), ("saved", 2)):
        _layer_refused(lib, q, "aligned", backward=False, **{name: P + LAYER.index(name) * STEP + off})
    for name, off in (("dr", 2), ("da", 1), ("dx", 1), ("dres", 2), ("dweight", 2), ("dbias", 1)):
        _layer_refused(lib, q, "aligned", forward=False, **{name: P + LAYER_BACK.index(name) * STEP + off})
    for kw in (dict(r=P), dict(a=P + 2), dict(a=P + STEP), dict(r=P + STEP + 4), dict(saved=P + 5 * STEP), dict(r=P + 5 * STEP),
               dict(a=P + 2 * STEP)):
        _layer_refused(lib, q, "shares memory", backward=False, **kw)
    for kw in (dict(dx=P), dict(dres=P + STEP), dict(dx=P + 5 * STEP), dict(dres=P + 4 * STEP + 4), dict(dweight=P + 9 * STEP),
               dict(dbias=P + 2 * STEP), dict(dx=P + 4 * STEP), dict(workspace=P + 256)):
        _layer_refused(lib, q, "shares memory", forward=False, **kw)


@pytest.mark.parametrize("kw,why", [
    (dict(T=-1), "T is"), (dict(T=(1 << 23) + 1), "T is"), (dict(batch=0), "batch"), (dict(key_heads=0), "key_heads"),
    (dict(heads=0), "heads"), (dict(heads=3), "multiple"), (dict(dk=0), "dk"), (dict(dk=129), "dk"), (dict(dv=0), "dv"),
    (dict(dv=1025), "dv"), (dict(dtype=3), "dtype"), (dict(dtype=-1), "dtype"), (dict(unit=2), "unit"),
    (dict(scale=float("nan")), "scale"), (dict(batch=1 << 19), "2^20"), (dict(T=1 << 23, batch=64), "too large"),
    (dict(ld_q=31), "pitch"), (dict(ld_k=-1), "pitch"), (dict(ld_v=95), "pitch"), (dict(ld_decay=3), "pitch"),
    (dict(ld_beta=1), "pitch"), (dict(ld_y=95), "pitch"), (dict(ld_dy=1), "pitch"), (dict(ld_dq=1), "pitch"), (dict(ld_dk=1), "pitch"),
    (dict(ld_v=(1 << 23) + 1), "2^24"), (dict(ld_dq=1 << 40), "2^24"), (dict(dv=1024, heads=16384), "2^24"), (dict(ld_dv=1), "pitch"), (dict(ld_ddecay=1), "pitch"), (dict(ld_dbeta=3), "pitch")])
def test_delta_descriptors_are_checked(lib, kw, why):
    q = _delta(**kw)
    assert lib.fi_delta_saved_bytes(ctypes.byref(q)) == 0
    assert lib.fi_delta_workspace_bytes(ctypes.byref(q), 0) == 0 and lib.fi_delta_workspace_bytes(ctypes.byref(q), 1) == 0
    _delta_refused(lib, q, why)


def test_delta_arguments_are_checked(lib):
    _delta_refused(lib, None, "null descriptor")
    q = _delta()
    q.reserved[3] = 1
    _delta_refused(lib, q, "reserved")
    q = _delta()
    for name in ("q", "k", "v", "decay", "beta", "workspace"):
        _delta_refused(lib, q, "required", **{name: None})
    _delta_refused(lib, q, "required", backward=False, y=None)
    for name in ("saved", "dy", "dq", "dk", "dv", "ddecay", "dbeta"):
        _delta_refused(lib, q, "required", forward=False, **{name: None})
    for name in DELTA[:9]:
        _delta_refused(lib, q, "aligned", backward=False, **{name: P + DELTA.index(name) * STEP + 1})
    for name in ("saved", "workspace"):
        _delta_refused(lib, q, "aligned", backward=False, **{name: P + DELTA.index(name) * STEP + 128})
    for name in [n for n in DELTA_BACK if n not in ("saved", "workspace")]:
        _delta_refused(lib, q, "aligned", forward=False, **{name: P + DELTA_BACK.index(name) * STEP + 1})
    for kw in (dict(y=P), dict(y=P + 2 * STEP), dict(final=P + 5 * STEP + 4), dict(final=P + 3 * STEP), dict(saved=P + 7 * STEP),
               dict(workspace=P), dict(y=P + 6 * STEP), dict(final=P + 7 * STEP)):
        _delta_refused(lib, q, "shares memory", backward=False, **kw)
    for kw in (dict(dq=P), dict(dk=P + 2 * STEP), dict(dv=P + 8 * STEP), dict(ddecay=P + 3 * STEP), dict(dbeta=P + 13 * STEP),
               dict(dstate=P + 9 * STEP), dict(dstate=P + 5 * STEP), dict(workspace=P + 7 * STEP), dict(dq=P + 11 * STEP)):
        _delta_refused(lib, q, "shares memory", forward=False, **kw)


def test_few_positions_need_no_workspace(lib):
    """Up to 14 positions that save nothing: the call gets as far as the next check."""
    for T, why in ((14, "aligned"), (15, "required")):
        _delta_refused(lib, _delta(T=T), why, backward=False, workspace=None, saved=None, final=P + 1)
    assert ops._DELTA_STEPS == 14
    _delta_refused(lib, _delta(T=14), "required", backward=False, workspace=None)


def test_q8_arguments_are_checked(lib):
    for rows, K in ((-1, 5), ((1 << 24) + 1, 5), (5, 0), (5, 131072)):
        assert lib.fi_q8_bytes(rows, K) == 0
        why = "rows" if K == 5 else "K is"
        _refused(lib, lib.fi_q8_pack(rows, K, P, P + STEP, P + 2 * STEP, None), why)
        _refused(lib, lib.fi_q8_quantize(rows, K, 0, P, 0, P + STEP, None), why)
        _refused(lib, lib.fi_q8_product(rows, 8, K, P, P + STEP, None, 0, P + 2 * STEP, 0, None), why)
    assert lib.fi_q8_bytes(17, 129) == 32 * 256 + 256
    pack, quant, mul = lib.fi_q8_pack, lib.fi_q8_quantize, lib.fi_q8_product
    for a in ((None, P + STEP, P + 2 * STEP), (P, None, P + 2 * STEP), (P, P + STEP, None), (P, P + STEP, P + 2 * STEP + 16)):
        _refused(lib, pack(5, 9, *a, None), "required")
    _refused(lib, pack(5, 9, P, P + STEP + 2, P + 2 * STEP, None), "aligned")
    _refused(lib, pack(5, 9, P, P + STEP, P + STEP, None), "shares memory")
    _refused(lib, quant(5, 9, 4, P, 0, P + STEP, None), "dtype")
    _refused(lib, quant(5, 9, 1, P, 8, P + STEP, None), "pitch")
    _refused(lib, quant(5, 9, 1, None, 0, P + STEP, None), "required")
    _refused(lib, quant(5, 9, 1, P, 0, P + STEP + 8, None), "required")
    _refused(lib, quant(5, 9, 1, P + 1, 0, P + STEP, None), "aligned")
    _refused(lib, quant(5, 9, 1, P, 0, P, None), "shares memory")
    y = P + 3 * STEP
    _refused(lib, mul(5, 0, 9, P, P + STEP, None, 1, y, 0, None), "N is")
    _refused(lib, mul(5, (1 << 24) + 1, 9, P, P + STEP, None, 1, y, 0, None), "N is")
    _refused(lib, mul(1 << 24, 1 << 24, 9, P, P + STEP, None, 1, y, 0, None), "2^42")
    _refused(lib, mul(5, 8, 9, P, P + STEP, None, 7, y, 0, None), "dtype")
    _refused(lib, mul(5, 8, 9, P, P + STEP, None, 1, y, 7, None), "pitch")
    for a, w, o in ((None, P + STEP, y), (P, None, y), (P, P + STEP, None), (P + 8, P + STEP, y), (P, P + STEP + 64, y)):
        _refused(lib, mul(5, 8, 9, a, w, None, 1, o, 0, None), "required")
    _refused(lib, mul(5, 8, 9, P, P + STEP, P + 2 * STEP + 2, 1, y, 0, None), "aligned")
    _refused(lib, mul(5, 8, 9, P, P + STEP, None, 1, y + 1, 0, None), "aligned")
    for o in (P, P + STEP, P + 2 * STEP):
        _refused(lib, mul(5, 8, 9, P, P + STEP, P + 2 * STEP, 1, o, 0, None), "shares memory")


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 8)
    h = torch.zeros(4, 2, 1, 8)
    for call in (lambda: ops.layer_norm(x), lambda: ops.layer_norm(None), lambda: ops.layer_norm([1]),
                 lambda: ops.layer_norm_backward(x, x, x, None, x), lambda: ops.Q8Rows.quantize(x[0]),
                 lambda: ops.Q8Weight(torch.zeros(4, 4, dtype=torch.int8), x[0, 0]), lambda: ops.q8_product(x, x),
                 lambda: ops.gated_delta(h, h, h, x[..., :1], x[..., :1]), lambda: ops.gated_delta(h, h, None, x, x),
                 lambda: ops.gated_delta_step(h[0], h[0], h[0], x[0, :, :1], x[0, :, :1], h),
                 lambda: ops.gated_delta_backward(h, h, h, h, x, x, x)):
        with pytest.raises(fi.FiError) as e:
            call()
        assert e.value.status == fi.FI_EINVAL


def test_binding_warns_where_autograd_would_be_expected():
    x = torch.zeros(4, 2, 8)
    h = torch.zeros(4, 2, 1, 8)
    w = torch.ones(8, requires_grad=True)
    g = torch.zeros(4, 2, 1, requires_grad=True)
    q = object.__new__(ops.Q8Weight)
    q._index = 0
    calls = {"layer_norm": lambda: ops.layer_norm(x, weight=w), "gated_delta": lambda: ops.gated_delta(h, h, h, g, g),
             "gated_delta_step": lambda: ops.gated_delta_step(h[0], h[0], h[0], g[0], g[0], h),
             "q8_product": lambda: ops.q8_product(q, x[0], w)}
    for name, call in calls.items():
        with pytest.warns(UserWarning, match=f"{name}: autograd does not see"), pytest.raises(fi.FiError):
            call()
        with warnings.catch_warnings(), torch.no_grad(), pytest.raises(fi.FiError):
            warnings.simplefilter("error")
            call()
    for call in (lambda: ops.layer_norm(x, weight=w, save=True), lambda: ops.gated_delta(h, h, h, g, g, save=True)):
        with warnings.catch_warnings(), pytest.raises(fi.FiError):       # the gradients are asked for explicitly
            warnings.simplefilter("error")
            call()


def test_rows_of_heads():
    """What the binding takes as rows of packed heads at one pitch, and what it refuses."""
    cpu = -1
    wide = torch.zeros(6, 2, 40)
    t = wide[..., 8:32].unflatten(-1, (3, 8))
    assert ops._heads(t, t.shape, torch.float32, cpu, "t")[1] == 40
    assert ops._heads(t[:, :, :1], (6, 2, 1, 8), torch.float32, cpu, "t")[1] == 40
    packed = torch.zeros(6, 2, 3, 8)
    assert ops._heads(packed, packed.shape, torch.float32, cpu, "t")[1] == 0
    for bad in (packed[:, :, :, ::2], packed.transpose(2, 3), packed[..., :4], packed.transpose(0, 1), packed[:, :, ::2]):
        with pytest.raises(fi.FiError):
            ops._heads(bad, bad.shape, torch.float32, cpu, "t")
