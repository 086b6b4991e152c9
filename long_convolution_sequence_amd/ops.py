"""Binding of the operators of a recurrent block in ``include/fi.h``: the gated
linear recurrence and the gated delta rule, the norms fused with gate and
residual and the layer norm, 4-bit and 8-bit products.

For a caller that runs its own block between the mixers (``fi.Context`` with
``MAP_EXTERNAL``) or trains one.  As in ``fi``: argument marshalling only, no
CPU path; a mismatch raises ``FiError(FI_EINVAL)`` before anything is
launched.  Every call runs on the current torch stream of its tensors' device,
waits for nothing and can be captured into a graph; workspaces and outputs
that are not given come from torch's allocator on that stream.  Gradients are
explicit calls: nothing here records itself for autograd, and a forward call on
tensors that require gradients warns, unless it saves what the backward call
takes or stands under ``torch.no_grad()``.

Tensors need contiguous rows at one pitch (a column slice of a wider tensor
is fine; a row of heads is all of them); states, weights and ``lengths`` are
densely packed.  Sequences are ``[T][B][D]`` as in ``fi.Context.prefill``, with
heads ``[T][B][heads][d]``.
"""
from __future__ import annotations

import functools
import struct
import warnings
from typing import NamedTuple, Optional

import torch

from .fi import FI_EINVAL, FI_OK, FiError, load_library

F32, BF16, F16 = 0, 1, 2
SCAN_PLAIN, SCAN_CONVEX, SCAN_ENERGY = 0, 1, 2
SCAN_INPUTS = {"plain": SCAN_PLAIN, "convex": SCAN_CONVEX, "energy": SCAN_ENERGY}
GATE_LINEAR, GATE_SIGMOID, GATE_SILU = 0, 1, 2

_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


# The descriptors of include/fi.h, packed (reserved fields zero).
_SCAN_DESC = struct.Struct("=q4i6q16x")       # T batch channels dtype input ld_x ld_gate ld_y ld_dy ld_dx ld_dgate
_NORM_DESC = struct.Struct("=q5if10q16x")     # rows channels dtype res_dtype post_norm act eps ld_o .. ld_dres
_DELTA_DESC = struct.Struct("=q7if12q16x")     # T batch key_heads heads dk dv dtype unit scale ld_q .. ld_dbeta
_LAYER_DESC = struct.Struct("=q3if8q16x")      # rows channels dtype res_dtype eps ld_x .. ld_dres
_Q4_DESC = struct.Struct("=5i12x")            # N K group scale_dtype has_zeros


def _bad(what):
    raise FiError(FI_EINVAL, what)


def _pack(desc, *values):
    try:
        return desc.pack(*values)
    except (struct.error, TypeError, OverflowError) as e:      # a size past its field, an eps that is no number
        raise FiError(FI_EINVAL, str(e)) from None


def _check(status):
    if status != FI_OK:
        msg = load_library().fi_op_last_error()
        raise FiError(status, msg.decode() if msg else "")


def _device(t, name):
    """Index of the device that every tensor of a call has to be on: that of its first one."""
    if not isinstance(t, torch.Tensor):
        _bad(f"{name}: expected a torch tensor, got {type(t).__name__}")
    index = t.get_device()
    if index < 0:
        _bad(f"{name}: not a device tensor")
    return index


def _type(t, name):
    d = _TYPES.get(t.dtype)
    if d is None:
        _bad(f"{name}: dtype {t.dtype}, expected float32, bfloat16 or float16")
    return d


def _fits(t, shape, dtype, device, name):
    """Check a tensor's shape, dtype and device (an index, -1 the host)."""
    if not isinstance(t, torch.Tensor):
        _bad(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.shape != shape:
        _bad(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        _bad(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.get_device() != device:
        _bad(f"{name}: on {t.device}, expected the call's device {device}")


def _packed(t, shape, dtype, device):
    return (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == device and
            t.is_contiguous())


def _rows(t, shape, dtype, device, name):
    """(pointer, row pitch) of a tensor of that exact shape, dtype and device
    with contiguous rows at one pitch (0: densely packed); (None, 0) for None."""
    if t is None:
        return None, 0
    if _packed(t, shape, dtype, device):
        return t.data_ptr(), 0
    _fits(t, shape, dtype, device, name)
    if t.stride(-1) != 1 and shape[-1] != 1:
        _bad(f"{name}: its rows are not contiguous")
    pitch, step = None, 0
    for i in range(t.dim() - 2, -1, -1):
        if shape[i] == 1:
            continue
        if pitch is None:
            pitch = t.stride(i)
            if pitch < shape[-1]:
                _bad(f"{name}: its rows overlap")
        elif t.stride(i) != step:
            _bad(f"{name}: its rows are not at one pitch")
        step = t.stride(i) * shape[i]
    return t.data_ptr(), pitch or 0


def _dense(t, shape, dtype, device, name):
    """Pointer of a densely packed tensor, or None."""
    if t is None:
        return None
    if _packed(t, shape, dtype, device):
        return t.data_ptr()
    _fits(t, shape, dtype, device, name)
    _bad(f"{name}: not contiguous")


_any_requires_grad = torch._C._any_requires_grad


def _not_recorded(call):
    """Warn where autograd would be expected to see a call: its outputs carry no graph."""
    if torch.is_grad_enabled():
        warnings.warn(f"{call}: autograd does not see this call, its outputs carry no gradients (the gradients are "
                      f"calls of their own; torch.no_grad() silences this)", stacklevel=3)


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream      # the hipStream_t of a device's current stream


def _call(device, fn, *args):
    """Run one C call on the device's current stream (its last argument)."""
    if device != _current_device():
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(device))
    else:
        status = fn(*args, _current_stream(device))
    if status != FI_OK:
        _check(status)


def _like(t):
    """A new packed tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _bytes(n, like):
    return torch.empty(n, dtype=torch.uint8, device=like.device)


# ---- gated linear recurrence ---------------------------------------------------

@functools.lru_cache(maxsize=256)
def _scan_sizes(T, B, D, dtype, input):
    """Bytes of the forward pass's workspace, the backward pass's, and the saved states."""
    lib = load_library()
    d = _pack(_SCAN_DESC, T, B, D, dtype, input, 0, 0, 0, 0, 0, 0)
    return lib.fi_scan_workspace_bytes(d, 0), lib.fi_scan_workspace_bytes(d, 1), lib.fi_scan_saved_bytes(d)


def _scan_inputs(x, gate, bias, state, lengths, input, positions=True):
    device = _device(x, "x")
    shape = x.shape
    T, B, D = shape if positions and len(shape) == 3 else (1, *shape) if not positions and len(shape) == 2 else (0, 0, 0)
    if B < 1 or D < 1:
        _bad(f"x: shape {tuple(shape)}, expected {'[T]' if positions else ''}[B][D]")
    if input not in (SCAN_PLAIN, SCAN_CONVEX, SCAN_ENERGY):
        _bad(f"input: {input!r}, expected SCAN_PLAIN, SCAN_CONVEX or SCAN_ENERGY")
    dtype = x.dtype
    head = (T, B, D, _type(x, "x"), input)
    px, ldx = _rows(x, shape, dtype, device, "x")
    if gate is None:
        _bad("gate: required")
    pg, ldg = _rows(gate, shape, dtype, device, "gate")
    return (device, shape, dtype, head, (ldx, ldg),
            (px, pg, _dense(bias, (D,), torch.float32, device, "bias"),
             _dense(state, (B, D), torch.float32, device, "state"),
             _dense(lengths, (B,), torch.int32, device, "lengths")))


def gated_scan(x, gate, bias=None, state=None, lengths=None, *, input=SCAN_CONVEX, save=False, y=None, final=None):
    """The gated linear recurrence over a sequence (fi_scan_forward).

    z = gate + bias, d = 1 - sigmoid(z), s_t = (1 - d_t) s_{t-1} + e(d_t) x_t, y_t = s_t with e = 1
    (SCAN_PLAIN), d (SCAN_CONVEX) or sqrt(d (2 - d)) (SCAN_ENERGY).

    x, gate [T][B][D] of one type; bias [D], state [B][D] fp32 (the state before the first position)
    or None for zeros; lengths [B] int32 or None: rows past a sequence's length count for nothing, give
    y = 0 and leave the state.  Returns (y, final [B][D] fp32), with save=True also what
    gated_scan_backward needs.  final may be given as the state itself.  Autograd does not see it."""
    if not save and _any_requires_grad(x, gate, bias, state):
        _not_recorded("gated_scan")
    device, shape, dtype, head, ld, args = _scan_inputs(x, gate, bias, state, lengths, input)
    if y is None:
        y = _like(x)
        py, ldy = y.data_ptr(), 0
    else:
        py, ldy = _rows(y, shape, dtype, device, "y")
    if final is None:
        final = _like(state) if state is not None else x.new_empty(shape[1:], dtype=torch.float32)
        pf = final.data_ptr()
    else:
        pf = _dense(final, shape[1:], torch.float32, device, "final")
    work, _, kept = _scan_sizes(*head)
    work = _bytes(work, x) if work > 256 else None
    saved = _bytes(kept, x) if save else None
    _call(device, load_library().fi_scan_forward, _pack(_SCAN_DESC, *head, *ld, ldy, 0, 0, 0), *args, py, pf,
          saved.data_ptr() if save else None, work.data_ptr() if work is not None else None)
    return (y, final, saved) if save else (y, final)


def gated_scan_step(x, gate, state, bias=None, lengths=None, *, input=SCAN_CONVEX, y=None):
    """One position: x, gate [B][D]; state [B][D] fp32 is updated in place.  lengths [B] int32 or None:
    a row with 0 is an empty slot (y = 0, its state stays).  Returns y.  Autograd does not see it."""
    if _any_requires_grad(x, gate, state, bias):
        _not_recorded("gated_scan_step")
    device, shape, dtype, head, ld, args = _scan_inputs(x, gate, bias, state, lengths, input, positions=False)
    if state is None:
        _bad("state: required")
    if y is None:
        y = _like(x)
        py, ldy = y.data_ptr(), 0
    else:
        py, ldy = _rows(y, shape, dtype, device, "y")
    _call(device, load_library().fi_scan_forward, _pack(_SCAN_DESC, *head, *ld, ldy, 0, 0, 0), *args, py, args[3], None,
          None)
    return y


def gated_scan_backward(dy, x, gate, saved, bias=None, state=None, lengths=None, *, dfinal=None, input=SCAN_CONVEX,
                        dx=None, dgate=None):
    """Gradients of gated_scan (fi_scan_backward): the forward call's arguments, its `saved`, and the
    gradients dy [T][B][D] and dfinal [B][D] fp32 (or None) of its outputs.  Returns (dx, dgate,
    dbias, dstate); dbias and dstate are None where bias and state are."""
    device, shape, dtype, head, ld, args = _scan_inputs(x, gate, bias, state, lengths, input)
    if dy is None or saved is None:
        _bad("dy and saved are required")
    pdy, lddy = _rows(dy, shape, dtype, device, "dy")
    pdf = _dense(dfinal, shape[1:], torch.float32, device, "dfinal")
    dx = _like(x) if dx is None else dx
    dgate = _like(gate) if dgate is None else dgate
    pdx, lddx = _rows(dx, shape, dtype, device, "dx")
    pdg, lddg = _rows(dgate, shape, dtype, device, "dgate")
    dbias = _like(bias) if bias is not None else None
    dstate = _like(state) if state is not None else None
    _, work, kept = _scan_sizes(*head)
    psv = _dense(saved, (kept,), torch.uint8, device, "saved")
    work = _bytes(work, x)
    _call(device, load_library().fi_scan_backward, _pack(_SCAN_DESC, *head, *ld, 0, lddy, lddx, lddg), *args, psv, pdy,
          pdf, pdx, pdg, dbias.data_ptr() if dbias is not None else None,
          dstate.data_ptr() if dstate is not None else None, work.data_ptr())
    return dx, dgate, dbias, dstate


# ---- gated delta rule ------------------------------------------------------------

class DeltaGradients(NamedTuple):
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    decay: torch.Tensor
    beta: torch.Tensor
    state: Optional[torch.Tensor]


@functools.lru_cache(maxsize=256)
def _delta_sizes(*head):
    """Bytes of the forward pass's workspace, the backward pass's, and of what is saved."""
    lib = load_library()
    d = _pack(_DELTA_DESC, *head, 0.0, *([0] * 12))
    return lib.fi_delta_workspace_bytes(d, 0), lib.fi_delta_workspace_bytes(d, 1), lib.fi_delta_saved_bytes(d)


_DELTA_STEPS = 14          # positions up to which a forward call that saves nothing takes no workspace


def _heads(t, shape, dtype, device, name):
    """As _rows of a tensor [T][B][heads][d]: a row is all its heads."""
    if t is None:
        _bad(f"{name}: required")
    if _packed(t, shape, dtype, device):
        return t.data_ptr(), 0
    _fits(t, shape, dtype, device, name)
    # a head's channels side by side too: flattening anything else would make a copy
    if shape[-2] != 1 and (t.stride(-2) != shape[-1] or (t.stride(-1) != 1 and shape[-1] != 1)):
        _bad(f"{name}: the heads of a row are not packed")
    return _rows(t.flatten(-2) if shape[-2] != 1 else t.squeeze(-2), (*shape[:-2], shape[-2] * shape[-1]), dtype, device,
                 name)


def _delta_inputs(q, k, v, decay, beta, state, lengths, scale, unit, positions=True):
    device = _device(v, "v")
    dtype = v.dtype
    dt = _type(v, "v")
    if not positions:
        q, k, v, decay, beta = (t.unsqueeze(0) if isinstance(t, torch.Tensor) else t for t in (q, k, v, decay, beta))
    dims = "[T][B]" if positions else "[B]"
    if v.dim() != 4 or not v.shape[1] or not v.shape[2] or not v.shape[3]:
        _bad(f"v: shape {tuple(v.shape)}, expected {dims}[heads][dv]")
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or not q.shape[2] or not q.shape[3]:
        _bad(f"q: expected a tensor {dims}[key heads][dk]")
    T, B, H, dv = v.shape
    HK, dk = q.shape[2:]
    scale = dk ** -0.5 if scale is None else scale
    keys = (T, B, HK, dk)
    pq, ldq = _heads(q, keys, dtype, device, "q")
    pk, ldk = _heads(k, keys, dtype, device, "k")
    pv, ldv = _heads(v, v.shape, dtype, device, "v")
    pg, ldg = _rows(decay, (T, B, H), torch.float32, device, "decay")
    pb, ldb = _rows(beta, (T, B, H), torch.float32, device, "beta")
    if decay is None or beta is None:
        _bad("decay and beta: required")
    return (device, dtype, keys, v.shape, (T, B, HK, H, dk, dv, dt, int(bool(unit))), scale, (ldq, ldk, ldv, ldg, ldb),
            (pq, pk, pv, pg, pb, _dense(state, (B, H, dk, dv), torch.float32, device, "state"),
             _dense(lengths, (B,), torch.int32, device, "lengths")))


def gated_delta(q, k, v, decay, beta, state=None, lengths=None, *, scale=None, unit=False, save=False, y=None, final=None):
    """The gated delta rule over a sequence (fi_delta_forward).

    S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T with a_t = e^decay_t, y_t = scale S_t^T q_t.
    unit: k and q are divided by their lengths (k / sqrt(sum k^2 + 1e-6)); scale None: 1 / sqrt(dk).

    q, k [T][B][key heads][dk] and v [T][B][heads][dv] of one type, heads a multiple of key heads (groups
    of neighbouring heads share one); decay (a logarithm, at most 0) and beta [T][B][heads] fp32; state
    [B][heads][dk][dv] fp32 (before the first position) or None for zeros; lengths as in gated_scan.  dk
    up to 128, dv to 1024.  Returns (y like v, final like state), with save=True also what
    gated_delta_backward needs.  final may be given as the state itself.  Autograd does not see it."""
    if not save and _any_requires_grad(q, k, v, decay, beta, state):
        _not_recorded("gated_delta")
    device, dtype, _, shape, head, scale, ld, args = _delta_inputs(q, k, v, decay, beta, state, lengths, scale, unit)
    if y is None:
        y = _like(v)
        py, ldy = y.data_ptr(), 0
    else:
        py, ldy = _heads(y, shape, dtype, device, "y")
    T, B, _, H, dk, dv = head[:6]
    if final is None:
        final = _like(state) if state is not None else v.new_empty((B, H, dk, dv), dtype=torch.float32)
        pf = final.data_ptr()
    else:
        pf = _dense(final, (B, H, dk, dv), torch.float32, device, "final")
    work, _, kept = _delta_sizes(*head)
    work = _bytes(work, v) if save or T > _DELTA_STEPS else None
    saved = _bytes(kept, v) if save else None
    _call(device, load_library().fi_delta_forward, _pack(_DELTA_DESC, *head, scale, *ld, ldy, 0, 0, 0, 0, 0, 0), *args, py,
          pf, saved.data_ptr() if save else None, work.data_ptr() if work is not None else None)
    return (y, final, saved) if save else (y, final)


def gated_delta_step(q, k, v, decay, beta, state, lengths=None, *, scale=None, unit=False, y=None):
    """One position: q, k [B][key heads][dk], v [B][heads][dv], decay, beta [B][heads]; state
    [B][heads][dk][dv] fp32 is updated in place.  lengths [B] int32 or None: a row with 0 is an empty slot
    (y = 0, its state stays).  Returns y.  Autograd does not see it."""
    if _any_requires_grad(q, k, v, decay, beta, state):
        _not_recorded("gated_delta_step")
    device, dtype, _, shape, head, scale, ld, args = _delta_inputs(q, k, v, decay, beta, state, lengths, scale, unit,
                                                                   positions=False)
    if state is None:
        _bad("state: required")
    if y is None:
        y = _like(v)
        py, ldy = y.data_ptr(), 0
    else:
        if not isinstance(y, torch.Tensor):
            _bad(f"y: expected a torch tensor, got {type(y).__name__}")
        py, ldy = _heads(y.unsqueeze(0), shape, dtype, device, "y")
    _call(device, load_library().fi_delta_forward, _pack(_DELTA_DESC, *head, scale, *ld, ldy, 0, 0, 0, 0, 0, 0), *args, py,
          args[5], None, None)
    return y


def gated_delta_backward(dy, q, k, v, decay, beta, saved, state=None, lengths=None, *, dfinal=None, scale=None, unit=False,
                         dq=None, dk=None, dv=None):
    """Gradients of gated_delta (fi_delta_backward): the forward call's arguments, its `saved`, and the
    gradients dy like v and dfinal like state (or None) of its outputs.  Returns DeltaGradients; state's
    is None where state is."""
    device, dtype, keys, shape, head, scale, ld, args = _delta_inputs(q, k, v, decay, beta, state, lengths, scale, unit)
    if dy is None or saved is None:
        _bad("dy and saved are required")
    T, B, _, H = head[:4]
    pdy, lddy = _heads(dy, shape, dtype, device, "dy")
    pdf = _dense(dfinal, (B, H, *head[4:6]), torch.float32, device, "dfinal")
    dq = _like(q) if dq is None else dq
    dk = _like(k) if dk is None else dk
    dv = _like(v) if dv is None else dv
    pdq, lddq = _heads(dq, keys, dtype, device, "dq")
    pdk, lddk = _heads(dk, keys, dtype, device, "dk")
    pdv, lddv = _heads(dv, shape, dtype, device, "dv")
    ddecay, dbeta = (v.new_empty((T, B, H), dtype=torch.float32) for _ in range(2))
    dstate = _like(state) if state is not None else None
    _, work, kept = _delta_sizes(*head)
    psv = _dense(saved, (kept,), torch.uint8, device, "saved")
    work = _bytes(work, v)
    _call(device, load_library().fi_delta_backward,
          _pack(_DELTA_DESC, *head, scale, *ld, 0, lddy, lddq, lddk, lddv, 0, 0), *args, psv, pdy, pdf, pdq, pdk, pdv,
          ddecay.data_ptr(), dbeta.data_ptr(), dstate.data_ptr() if dstate is not None else None, work.data_ptr())
    return DeltaGradients(dq, dk, dv, ddecay, dbeta, dstate)


# ---- norms around a block --------------------------------------------------------

class NormGradients(NamedTuple):
    o: Optional[torch.Tensor]
    res: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    post_weight: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    pre_weight: Optional[torch.Tensor]


def _norm_inputs(o, res, gate, post_weight, scale, pre_weight, post_norm, act, eps):
    first = o if o is not None else res
    if first is None:
        _bad("o or res is required")
    device = _device(first, "o" if o is not None else "res")
    shape, dtype = first.shape, first.dtype
    if len(shape) < 1 or shape[-1] < 1:
        _bad(f"o: shape {tuple(shape)}, expected [..., D]")
    if act not in (GATE_LINEAR, GATE_SIGMOID, GATE_SILU):
        _bad(f"act: {act!r}, expected GATE_LINEAR, GATE_SIGMOID or GATE_SILU")
    D = shape[-1]
    rows = first.numel() // D
    rt = res.dtype if isinstance(res, torch.Tensor) else dtype
    if rt is not dtype and rt is not torch.float32:
        _bad(f"res: dtype {rt}, expected {dtype} or torch.float32")
    po, ldo = _rows(o, shape, dtype, device, "o")
    pg, ldg = _rows(gate, shape, dtype, device, "gate")
    pr, ldr = _rows(res, shape, rt, device, "res")
    head = (rows, D, _type(first, "o"), _TYPES[rt], int(bool(post_norm)), act, eps, ldo, ldg, ldr)
    return (first, device, shape, dtype, rt, rows, head,
            (po, pg, pr, _dense(post_weight, (D,), torch.float32, device, "post_weight"),
             _dense(scale, (D,), torch.float32, device, "scale"),
             _dense(pre_weight, (D,), torch.float32, device, "pre_weight")))


def block_norm(o, res=None, gate=None, *, post_weight=None, scale=None, pre_weight=None, post_norm=False,
               act=GATE_SILU, eps=1e-6, save=False, r=None, a=None):
    """The norms around a block with its gate, residual and residual scale (fi_norm_forward).

    v = o / rms(o) * post_weight (post_norm; else v = o), m = v * act(gate), r = res + scale * m,
    a = r / rms(r) * pre_weight; what is None is left out.  o None: the norm before a first block
    (r = res; then a has res's type).  o, gate, a [..., D] of one type; res, r of that type or
    fp32; weights and scale fp32 [D].  r may be given as res itself.  Returns (r, a), with
    save=True also what block_norm_backward needs.  Autograd does not see it."""
    if not save and _any_requires_grad(o, res, gate, post_weight, scale, pre_weight):
        _not_recorded("block_norm")
    first, device, shape, dtype, rt, rows, head, args = _norm_inputs(o, res, gate, post_weight, scale, pre_weight,
                                                                     post_norm, act, eps)
    if r is None:
        r = _like(res) if res is not None else _like(o)
        pr, ldr = r.data_ptr(), 0
    else:
        pr, ldr = _rows(r, shape, rt, device, "r")
    if a is None:
        a = _like(first)
        pa, lda = a.data_ptr(), 0
    else:
        pa, lda = _rows(a, shape, dtype, device, "a")
    saved = torch.empty((2, rows), dtype=torch.float32, device=first.device) if save else None
    _call(device, load_library().fi_norm_forward, _pack(_NORM_DESC, *head, ldr, lda, 0, 0, 0, 0, 0), *args, pr, pa,
          saved.data_ptr() if save else None)
    return (r, a, saved) if save else (r, a)


@functools.lru_cache(maxsize=256)
def _norm_workspace(rows, D, dtype, res_dtype):
    return load_library().fi_norm_workspace_bytes(_pack(_NORM_DESC, rows, D, dtype, res_dtype, 0, 0, 0.0, *([0] * 10)))


def block_norm_backward(dr, da, o, res, gate, saved, *, post_weight=None, scale=None, pre_weight=None,
                        post_norm=False, act=GATE_SILU, eps=1e-6, do=None, dres=None, dgate=None):
    """Gradients of block_norm (fi_norm_backward) from those of r and a (either may be None): the
    forward call's arguments and its `saved`.  Returns NormGradients, None where the input is None.
    dres may be given as dr itself."""
    first, device, shape, dtype, rt, rows, head, args = _norm_inputs(o, res, gate, post_weight, scale, pre_weight,
                                                                     post_norm, act, eps)
    if saved is None:
        _bad("saved: required")
    psv = _dense(saved, (2, rows), torch.float32, device, "saved")
    pdr, lddr = _rows(dr, shape, rt, device, "dr")
    pda, ldda = _rows(da, shape, dtype, device, "da")

    do, dres, dgate = [_like(t) if t is not None and given is None else given
                       for given, t in ((do, o), (dres, res), (dgate, gate))]
    pdo, lddo = _rows(do, shape, dtype, device, "do")
    pdres, lddres = _rows(dres, shape, rt, device, "dres")
    pdg, lddg = _rows(dgate, shape, dtype, device, "dgate")
    D = shape[-1]
    cols = torch.empty((3, D), dtype=torch.float32, device=first.device)
    w = [cols[i] if t is not None else None for i, t in enumerate((post_weight, scale, pre_weight))]
    ptr = [t.data_ptr() if t is not None else None for t in w]
    if da is None and w[2] is not None:
        w[2].zero_()
        ptr[2] = None
    work = _bytes(_norm_workspace(rows, D, head[2], head[3]), first)
    _call(device, load_library().fi_norm_backward, _pack(_NORM_DESC, *head, 0, 0, lddr, ldda, lddo, lddg, lddres), *args,
          psv, pdr, pda, pdo, pdg, pdres, *ptr, work.data_ptr())
    return NormGradients(do, dres, dgate, *w)


# ---- layer norm --------------------------------------------------------------------

class LayerGradients(NamedTuple):
    x: torch.Tensor
    res: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]


def _layer_inputs(x, res, weight, bias, eps, dtype):
    """As the C call takes them: without a residual, an fp32 x that is normed into another type is its `res`."""
    device = _device(x, "x")
    shape = x.shape
    if len(shape) < 1 or shape[-1] < 1:
        _bad(f"x: shape {tuple(shape)}, expected [..., D]")
    D = shape[-1]
    dt = x.dtype if dtype is None else dtype
    if dt not in _TYPES:
        _bad(f"dtype: {dtype}, expected float32, bfloat16 or float16")
    alone = None
    if dt is not x.dtype:
        if res is not None or x.dtype is not torch.float32:
            _bad(f"dtype: {dt}, expected x's {x.dtype} (only an fp32 x without res is normed into another type)")
        alone, x, res = x, None, x
    rt = res.dtype if isinstance(res, torch.Tensor) else dt
    if rt is not dt and rt is not torch.float32:
        _bad(f"res: dtype {rt}, expected {dt} or torch.float32")
    px, ldx = _rows(x, shape, dt, device, "x")
    pr, ldr = _rows(res, shape, rt, device, "res")
    rows = (x if x is not None else res).numel() // D
    _type(x if x is not None else res, "x")
    head = (rows, D, _TYPES[dt], _TYPES[rt], eps, ldx, ldr)
    return (device, shape, dt, rt, rows, alone, head,
            (px, pr, _dense(weight, (D,), torch.float32, device, "weight")),
            _dense(bias, (D,), torch.float32, device, "bias"))


def layer_norm(x, res=None, *, weight=None, bias=None, eps=1e-5, dtype=None, save=False, r=None, a=None):
    """The layer norm with a residual (fi_layer_forward).

    r = res + x, a = (r - mean(r)) / sqrt(mean((r - mean(r))^2) + eps) * weight + bias; what is None is
    left out.  x, a [..., D] of one type; res, r of that type or fp32; weight and bias fp32 [D].
    Without res an fp32 x can be normed into 16 bits (dtype).  r may be given as res itself.  Returns
    (r, a), r being x where there is no res; with save=True also what layer_norm_backward needs.
    Autograd does not see it."""
    if not save and _any_requires_grad(x, res, weight, bias):
        _not_recorded("layer_norm")
    device, shape, dt, rt, rows, alone, head, args, pb = _layer_inputs(x, res, weight, bias, eps, dtype)
    if res is None:
        if r is not None:
            _bad("r: without res it is x itself")
        pr, ldr, r = None, 0, x
    elif r is None:
        r = _like(res)
        pr, ldr = r.data_ptr(), 0
    else:
        pr, ldr = _rows(r, shape, rt, device, "r")
    if a is None:
        a = _like(x) if alone is None else x.new_empty(shape, dtype=dt)
        pa, lda = a.data_ptr(), 0
    else:
        pa, lda = _rows(a, shape, dt, device, "a")
    saved = torch.empty((2, rows), dtype=torch.float32, device=x.device) if save else None
    _call(device, load_library().fi_layer_forward, _pack(_LAYER_DESC, *head, ldr, lda, 0, 0, 0, 0), *args, pb, pr, pa,
          saved.data_ptr() if save else None)
    return (r, a, saved) if save else (r, a)


@functools.lru_cache(maxsize=256)
def _layer_workspace(rows, D, dtype, res_dtype):
    return load_library().fi_layer_workspace_bytes(_pack(_LAYER_DESC, rows, D, dtype, res_dtype, 0.0, *([0] * 8)))


def layer_norm_backward(dr, da, x, res, saved, *, weight=None, bias=None, eps=1e-5, dtype=None, dx=None, dres=None):
    """Gradients of layer_norm (fi_layer_backward) from those of r and a (either may be None): the
    forward call's arguments and its `saved`.  Returns LayerGradients, None where the input is None (x
    and res have the same gradient, each in its type).  dres may be given as dr itself."""
    device, shape, dt, rt, rows, alone, head, args, _ = _layer_inputs(x, res, weight, bias, eps, dtype)
    if saved is None:
        _bad("saved: required")
    psv = _dense(saved, (2, rows), torch.float32, device, "saved")
    pdr, lddr = _rows(dr, shape, rt, device, "dr")
    pda, ldda = _rows(da, shape, dt, device, "da")
    if res is None and dres is not None:
        _bad("dres: without res there is none")
    if alone is not None:                        # x's gradient is the C call's dres
        dx = _like(x) if dx is None else dx
        (pdx, lddx), (pdres, lddres) = (None, 0), _rows(dx, shape, rt, device, "dx")
    else:
        dx = _like(x) if dx is None else dx
        dres = _like(res) if res is not None and dres is None else dres
        pdx, lddx = _rows(dx, shape, dt, device, "dx")
        pdres, lddres = _rows(dres, shape, rt, device, "dres")
    D = shape[-1]
    cols = torch.empty((2, D), dtype=torch.float32, device=x.device)
    w = [cols[i] if t is not None else None for i, t in enumerate((weight, bias))]
    ptr = [t.data_ptr() if t is not None else None for t in w]
    if da is None:
        for t in w:
            if t is not None:
                t.zero_()
        ptr = [None, None]
    work = _bytes(_layer_workspace(rows, D, head[2], head[3]), x)
    _call(device, load_library().fi_layer_backward, _pack(_LAYER_DESC, *head, 0, 0, lddr, ldda, lddx, lddres), *args, psv,
          pdr, pda, pdx, pdres, *ptr, work.data_ptr())
    return LayerGradients(dx, dres, *w)


# ---- 4-bit products ----------------------------------------------------------------

class Q4Weight:
    """A weight matrix [N][K] in 4 bits, laid out once for q4_matvec (fi_q4_pack).

    codes [N][K] uint8 (0..15), scales [N][ceil(K/group)] fp32, bf16 or fp16 (kept in their type),
    zeros [N][ceil(K/group)] uint8 (0..15) or None (8 everywhere):
    w[n][k] = scales[n][k // group] * (codes[n][k] - zeros[n][k // group]), group 32, 64 or 128.
    Q4Weight.quantize makes the codes and scales from a matrix."""

    def __init__(self, codes, scales, zeros=None, *, group=128):
        device = _device(codes, "codes")
        if codes.dim() != 2 or codes.shape[0] < 1 or codes.shape[1] < 1:
            _bad(f"codes: shape {tuple(codes.shape)}, expected [N][K]")
        if not isinstance(scales, torch.Tensor):
            _bad(f"scales: expected a torch tensor, got {type(scales).__name__}")
        self.N, self.K = codes.shape
        self.group, self.device, self._index = group, codes.device, device
        self._desc = _pack(_Q4_DESC, self.N, self.K, group, _type(scales, "scales"), int(zeros is not None))
        lib = load_library()
        n = lib.fi_q4_packed_bytes(self._desc)
        if n == 0:
            _bad(f"unsupported N={self.N} K={self.K} group={group}")
        shape = (self.N, -(-self.K // group))
        pc = _dense(codes, codes.shape, torch.uint8, device, "codes")
        ps = _dense(scales, shape, scales.dtype, device, "scales")
        pz = _dense(zeros, shape, torch.uint8, device, "zeros")
        self.packed = _bytes(n, codes)
        _call(device, lib.fi_q4_pack, self._desc, pc, ps, pz, self.packed.data_ptr())

    @classmethod
    def quantize(cls, w, *, group=128, scale_dtype=torch.bfloat16):
        """From a matrix w [N][K]: scale = max|w| / 7 of each group, codes rounded to nearest, zeros 8.
        The codes and scales are kept as .codes and .scales."""
        device = _device(w, "w")
        if w.dim() != 2 or w.shape[0] < 1 or w.shape[1] < 1:
            _bad(f"w: shape {tuple(w.shape)}, expected [N][K]")
        if scale_dtype not in _TYPES:
            _bad(f"scale_dtype: {scale_dtype}, expected float32, bfloat16 or float16")
        if group not in (32, 64, 128):
            _bad(f"group: {group}, expected 32, 64 or 128")
        N, K = w.shape
        wt = _type(w, "w")
        pw, ld = _rows(w, w.shape, w.dtype, device, "w")
        codes = torch.empty((N, K), dtype=torch.uint8, device=w.device)
        scales = torch.empty((N, -(-K // group)), dtype=scale_dtype, device=w.device)
        _call(device, load_library().fi_q4_quantize, _pack(_Q4_DESC, N, K, group, _TYPES[scale_dtype], 0), wt, pw, ld,
              codes.data_ptr(), scales.data_ptr())
        out = cls(codes, scales, group=group)
        out.codes, out.scales = codes, scales
        return out


def q4_matvec(w, x, y=None):
    """y [B][N] = x [B][K] times a Q4Weight, 1 <= B <= 16 rows (fi_q4_matvec); y has x's type, |x| < 2^116.
    Autograd does not see it."""
    if _any_requires_grad(x):
        _not_recorded("q4_matvec")
    if not isinstance(w, Q4Weight):
        _bad(f"w: expected a Q4Weight, got {type(w).__name__}")
    device = _device(x, "x")
    if device != w._index:
        _bad(f"x: on {x.device}, expected {w.device}")
    if x.dim() != 2:
        _bad(f"x: shape {tuple(x.shape)}, expected [B][{w.K}]")
    dtype = x.dtype
    dt = _type(x, "x")
    rows = x.shape[0]
    px, ldx = _rows(x, (rows, w.K), dtype, device, "x")
    if y is None:
        y = x.new_empty((rows, w.N))
        py, ldy = y.data_ptr(), 0
    else:
        py, ldy = _rows(y, (rows, w.N), dtype, device, "y")
    _call(device, load_library().fi_q4_matvec, w._desc, w.packed.data_ptr(), rows, dt, px, ldx, py, ldy)
    return y


# ---- 8-bit products ----------------------------------------------------------------

class Q8Rows:
    """A matrix [rows][K] in 8-bit integers with an fp32 scale a row, laid out for q8_product
    (fi_q8_pack): activations, or a weight [N][K].

    codes [rows][K] int8, scales [rows] fp32; Q8Rows.quantize makes them from values."""

    def __init__(self, codes, scales):
        self._make(codes, "codes")
        rows, K = codes.shape
        pc = _dense(codes, codes.shape, torch.int8, self._index, "codes")
        ps = _dense(scales, (rows,), torch.float32, self._index, "scales")
        if ps is None:
            _bad("scales: required")
        _call(self._index, load_library().fi_q8_pack, rows, K, pc, ps, self.packed.data_ptr())

    def _make(self, t, name):
        device = _device(t, name)
        if t.dim() != 2 or t.shape[1] < 1:
            _bad(f"{name}: shape {tuple(t.shape)}, expected [rows][K]")
        rows, K = t.shape
        if rows > 1 << 24 or K > 131071:
            _bad(f"unsupported rows={rows} K={K}")
        self.rows, self.K, self.device, self._index = rows, K, t.device, device
        self.packed = _bytes(load_library().fi_q8_bytes(rows, K), t)

    @classmethod
    def quantize(cls, x):
        """From values x [rows][K]: scale = max|x| / 127 of each row, codes rounded to nearest."""
        out = cls.__new__(cls)
        out._make(x, "x")
        dt = _type(x, "x")
        px, ld = _rows(x, x.shape, x.dtype, out._index, "x")
        _call(out._index, load_library().fi_q8_quantize, out.rows, out.K, dt, px, ld, out.packed.data_ptr())
        return out

    @property
    def codes(self):
        """The codes [rows][K] int8 (a copy in their plain order)."""
        r, k = -(-self.rows // 16), -(-self.K // 128) * 2
        c = self.packed[:r * 16 * k * 64].view(torch.int8).view(r, k, 4, 16, 16).permute(0, 3, 1, 2, 4)
        return c.reshape(r * 16, k * 64)[:self.rows, :self.K].contiguous()

    @property
    def scales(self):
        """The scales [rows] fp32 (a view)."""
        r, k = -(-self.rows // 16) * 16, -(-self.K // 128) * 128
        at = -(-r * k // 256) * 256
        return self.packed[at:at + 4 * self.rows].view(torch.float32)


class Q8Weight(Q8Rows):
    """A weight matrix [N][K] in 8-bit integers with a scale an output."""

    @property
    def N(self):
        return self.rows


def q8_product(w, x, bias=None, *, dtype=None, y=None):
    """y [rows][N] = x [rows][K] times a Q8Weight, plus bias [N] fp32 (fi_q8_product).  x is a tensor,
    which is brought to 8 bits with a scale a row first, or Q8Rows (one quantization for several weights).
    dtype: of y; None for x's, with Q8Rows bfloat16.  Autograd does not see it."""
    if not isinstance(w, Q8Rows):
        _bad(f"w: expected a Q8Weight, got {type(w).__name__}")
    if isinstance(x, Q8Rows):
        dt = torch.bfloat16 if dtype is None else dtype
    else:
        if _any_requires_grad(x, bias):
            _not_recorded("q8_product")
        device = _device(x, "x")
        if device != w._index:
            _bad(f"x: on {x.device}, expected {w.device}")
        if x.dim() != 2 or x.shape[1] != w.K:
            _bad(f"x: shape {tuple(x.shape)}, expected [rows][{w.K}]")
        dt = x.dtype if dtype is None else dtype
        x = Q8Rows.quantize(x)
    if dt not in _TYPES:
        _bad(f"dtype: {dt}, expected float32, bfloat16 or float16")
    device = w._index
    if x._index != device or x.K != w.K:
        _bad(f"x: [{x.rows}][{x.K}] on {x.device}, expected [rows][{w.K}] on {w.device}")
    pb = _dense(bias, (w.rows,), torch.float32, device, "bias")
    if y is None:
        y = torch.empty((x.rows, w.rows), dtype=dt, device=w.device)
        py, ldy = y.data_ptr(), 0
    else:
        py, ldy = _rows(y, (x.rows, w.rows), dt, device, "y")
    _call(device, load_library().fi_q8_product, x.rows, w.rows, w.K, x.packed.data_ptr(), w.packed.data_ptr(), pb,
          _TYPES[dt], py, ldy)
    return y
