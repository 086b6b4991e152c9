"""Binding of the operators of a recurrent block in ``include/fi.h``: the gated
linear recurrence, the norms fused with gate and residual, 4-bit products.

For a caller that runs its own block between the mixers (``fi.Context`` with
``MAP_EXTERNAL``) or trains one.  As in ``fi``: argument marshalling only, no
CPU path; a mismatch raises ``FiError(FI_EINVAL)`` before anything is
launched.  Every call runs on the current torch stream of its tensors' device,
waits for nothing and can be captured into a graph; workspaces and outputs
that are not given come from torch's allocator on that stream.  Gradients are
explicit calls: nothing here records itself for autograd.

Tensors need contiguous rows at one pitch (a column slice of a wider tensor
is fine); states, weights and ``lengths`` are densely packed.  Sequences are
``[T][B][D]`` as in ``fi.Context.prefill``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .fi import FI_EDEVICE, FI_EINVAL, FI_OK, FiError, load_library

F32, BF16, F16 = 0, 1, 2
SCAN_PLAIN, SCAN_CONVEX, SCAN_ENERGY = 0, 1, 2
SCAN_INPUTS = {"plain": SCAN_PLAIN, "convex": SCAN_CONVEX, "energy": SCAN_ENERGY}
GATE_LINEAR, GATE_SIGMOID, GATE_SILU = 0, 1, 2

_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


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


def _bad(what):
    raise FiError(FI_EINVAL, what)


def _check(status):
    if status != FI_OK:
        msg = load_library().fi_op_last_error()
        raise FiError(status, msg.decode() if msg else "")


def _device(t, name):
    """The device every tensor of a call has to be on: that of its first one."""
    if not isinstance(t, torch.Tensor):
        _bad(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if not t.is_cuda:
        _bad(f"{name}: not a device tensor")
    return t.device


def _type(t, name):
    d = _TYPES.get(t.dtype)
    if d is None:
        _bad(f"{name}: dtype {t.dtype}, expected float32, bfloat16 or float16")
    return d


def _rows(t, shape, dtype, device, name):
    """(pointer, row pitch) of a tensor of that exact shape, dtype and device
    with contiguous rows at one pitch; (None, 0) for None."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        _bad(f"{name}: expected a torch tensor, got {type(t).__name__}")
    if t.shape != shape:
        _bad(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        _bad(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        _bad(f"{name}: on {t.device}, expected {device}")
    if t.is_contiguous():
        return t.data_ptr(), 0
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
    p, _ = _rows(t, shape, dtype, device, name)
    if not t.is_contiguous():
        _bad(f"{name}: not contiguous")
    return p


def _call(device, fn, *args):
    """Run one C call on the device's current stream (its last argument)."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            _check(fn(*args, torch.cuda.current_stream(device).cuda_stream))
    else:
        _check(fn(*args, torch.cuda.current_stream(device).cuda_stream))


def _bytes(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device)


# ---- gated linear recurrence ---------------------------------------------------

def _scan_desc(x, input):
    device = _device(x, "x")
    if x.dim() != 3 or x.shape[1] < 1 or x.shape[2] < 1:
        _bad(f"x: shape {tuple(x.shape)}, expected [T][B][D]")
    q = ScanDesc()
    q.T, q.batch, q.channels = x.shape
    q.dtype, q.input = _type(x, "x"), input
    return q, device


def _scan_inputs(q, x, gate, bias, state, lengths, device):
    B, D = q.batch, q.channels
    px, q.ld_x = _rows(x, x.shape, x.dtype, device, "x")
    if gate is None:
        _bad("gate: required")
    pg, q.ld_gate = _rows(gate, x.shape, x.dtype, device, "gate")
    return (px, pg, _dense(bias, (D,), torch.float32, device, "bias"),
            _dense(state, (B, D), torch.float32, device, "state"),
            _dense(lengths, (B,), torch.int32, device, "lengths"))


def gated_scan(x, gate, bias=None, state=None, lengths=None, *, input=SCAN_CONVEX, save=False, y=None, final=None):
    """The gated linear recurrence over a sequence (fi_scan_forward).

    z = gate + bias, d = 1 - sigmoid(z), s_t = (1 - d_t) s_{t-1} + e(d_t) x_t, y_t = s_t with e = 1
    (SCAN_PLAIN), d (SCAN_CONVEX) or sqrt(d (2 - d)) (SCAN_ENERGY).

    x, gate [T][B][D] of one type; bias [D], state [B][D] fp32 (the state before the first position)
    or None for zeros; lengths [B] int32 or None: rows past a sequence's length are not read, give
    y = 0 and leave the state.  Returns (y, final [B][D] fp32), with save=True also what
    gated_scan_backward needs.  final may be given as the state itself."""
    q, device = _scan_desc(x, input)
    args = _scan_inputs(q, x, gate, bias, state, lengths, device)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=device)
    py, q.ld_y = _rows(y, x.shape, x.dtype, device, "y")
    if final is None:
        final = torch.empty((q.batch, q.channels), dtype=torch.float32, device=device)
    pf = _dense(final, (q.batch, q.channels), torch.float32, device, "final")
    lib = load_library()
    desc = ctypes.addressof(q)
    n = lib.fi_scan_workspace_bytes(desc, 0)
    work = _bytes(n, device) if n > 256 else None
    saved = _bytes(lib.fi_scan_saved_bytes(desc), device) if save else None
    _call(device, lib.fi_scan_forward, desc, *args, py, pf, saved.data_ptr() if save else None,
          work.data_ptr() if work is not None else None)
    return (y, final, saved) if save else (y, final)


def gated_scan_step(x, gate, state, bias=None, lengths=None, *, input=SCAN_CONVEX, y=None):
    """One position: x, gate [B][D]; state [B][D] fp32 is updated in place.  lengths [B] int32 or None:
    a row with 0 is an empty slot (y = 0, its state stays).  Returns y."""
    _device(x, "x")
    if x.dim() != 2 or not isinstance(gate, torch.Tensor) or state is None:
        _bad("x and gate [B][D] and state [B][D] are required")
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif not isinstance(y, torch.Tensor):
        _bad(f"y: expected a torch tensor, got {type(y).__name__}")
    gated_scan(x.unsqueeze(0), gate.unsqueeze(0), bias, state, lengths, input=input, y=y.unsqueeze(0), final=state)
    return y


def gated_scan_backward(dy, x, gate, saved, bias=None, state=None, lengths=None, *, dfinal=None, input=SCAN_CONVEX,
                        dx=None, dgate=None):
    """Gradients of gated_scan (fi_scan_backward): the forward call's arguments, its `saved`, and the
    gradients dy [T][B][D] and dfinal [B][D] fp32 (or None) of its outputs.  Returns (dx, dgate,
    dbias, dstate); dbias and dstate are None where bias and state are."""
    q, device = _scan_desc(x, input)
    px, pg, pb, ps, pl = _scan_inputs(q, x, gate, bias, state, lengths, device)
    if dy is None:
        _bad("dy: required")
    pdy, q.ld_dy = _rows(dy, x.shape, x.dtype, device, "dy")
    B, D = q.batch, q.channels
    pdf = _dense(dfinal, (B, D), torch.float32, device, "dfinal")
    dx = torch.empty(x.shape, dtype=x.dtype, device=device) if dx is None else dx
    dgate = torch.empty(x.shape, dtype=x.dtype, device=device) if dgate is None else dgate
    pdx, q.ld_dx = _rows(dx, x.shape, x.dtype, device, "dx")
    pdg, q.ld_dgate = _rows(dgate, x.shape, x.dtype, device, "dgate")
    dbias = torch.empty((D,), dtype=torch.float32, device=device) if bias is not None else None
    dstate = torch.empty((B, D), dtype=torch.float32, device=device) if state is not None else None
    lib = load_library()
    desc = ctypes.addressof(q)
    n = lib.fi_scan_saved_bytes(desc)
    psv = _dense(saved, (n,), torch.uint8, device, "saved")
    if psv is None:
        _bad("saved: required")
    work = _bytes(lib.fi_scan_workspace_bytes(desc, 1), device)
    _call(device, lib.fi_scan_backward, desc, px, pg, pb, ps, pl, psv, pdy, pdf, pdx, pdg,
          dbias.data_ptr() if dbias is not None else None, dstate.data_ptr() if dstate is not None else None,
          work.data_ptr())
    return dx, dgate, dbias, dstate


# ---- norms around a block --------------------------------------------------------

class NormGradients(NamedTuple):
    o: Optional[torch.Tensor]
    res: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    post_weight: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    pre_weight: Optional[torch.Tensor]


def _norm_desc(o, res, post_norm, act, eps):
    first = o if o is not None else res
    if first is None:
        _bad("o or res is required")
    device = _device(first, "o" if o is not None else "res")
    if first.dim() < 1 or first.shape[-1] < 1:
        _bad(f"o: shape {tuple(first.shape)}, expected [..., D]")
    q = NormDesc()
    q.channels = first.shape[-1]
    q.rows = first.numel() // q.channels
    q.dtype = _type(first, "o")
    q.post_norm, q.act, q.eps = int(bool(post_norm)), act, eps
    return q, device, first.shape, first.dtype


def _norm_inputs(q, o, res, gate, post_weight, scale, pre_weight, device, shape, dtype):
    rt = res.dtype if isinstance(res, torch.Tensor) else dtype
    if rt != dtype and rt != torch.float32:
        _bad(f"res: dtype {rt}, expected {dtype} or torch.float32")
    q.res_dtype = _TYPES[rt]
    D = (q.channels,)
    po, q.ld_o = _rows(o, shape, dtype, device, "o")
    pg, q.ld_gate = _rows(gate, shape, dtype, device, "gate")
    pr, q.ld_res = _rows(res, shape, rt, device, "res")
    return rt, (po, pg, pr, _dense(post_weight, D, torch.float32, device, "post_weight"),
                _dense(scale, D, torch.float32, device, "scale"),
                _dense(pre_weight, D, torch.float32, device, "pre_weight"))


def block_norm(o, res=None, gate=None, *, post_weight=None, scale=None, pre_weight=None, post_norm=False,
               act=GATE_SILU, eps=1e-6, save=False, r=None, a=None):
    """The norms around a block with its gate, residual and residual scale (fi_norm_forward).

    v = o / rms(o) * post_weight (post_norm; else v = o), m = v * act(gate), r = res + scale * m,
    a = r / rms(r) * pre_weight; what is None is left out.  o None: the norm before a first block
    (r = res; then a has res's type).  o, gate, a [..., D] of one type; res, r of that type or
    fp32; weights and scale fp32 [D].  r may be given as res itself.  Returns (r, a), with
    save=True also what block_norm_backward needs."""
    q, device, shape, dtype = _norm_desc(o, res, post_norm, act, eps)
    rt, args = _norm_inputs(q, o, res, gate, post_weight, scale, pre_weight, device, shape, dtype)
    r = torch.empty(shape, dtype=rt, device=device) if r is None else r
    a = torch.empty(shape, dtype=dtype, device=device) if a is None else a
    pr, q.ld_r = _rows(r, shape, rt, device, "r")
    pa, q.ld_a = _rows(a, shape, dtype, device, "a")
    saved = torch.empty((2, q.rows), dtype=torch.float32, device=device) if save else None
    _call(device, load_library().fi_norm_forward, ctypes.addressof(q), *args, pr, pa,
          saved.data_ptr() if save else None)
    return (r, a, saved) if save else (r, a)


def block_norm_backward(dr, da, o, res, gate, saved, *, post_weight=None, scale=None, pre_weight=None,
                        post_norm=False, act=GATE_SILU, eps=1e-6, do=None, dres=None, dgate=None):
    """Gradients of block_norm (fi_norm_backward) from those of r and a (either may be None): the
    forward call's arguments and its `saved`.  Returns NormGradients, None where the input is None.
    dres may be given as dr itself."""
    q, device, shape, dtype = _norm_desc(o, res, post_norm, act, eps)
    rt, args = _norm_inputs(q, o, res, gate, post_weight, scale, pre_weight, device, shape, dtype)
    psv = _dense(saved, (2, q.rows), torch.float32, device, "saved")
    if psv is None:
        _bad("saved: required")
    pdr, q.ld_dr = _rows(dr, shape, rt, device, "dr")
    pda, q.ld_da = _rows(da, shape, dtype, device, "da")

    def like(given, want, dt):
        return torch.empty(shape, dtype=dt, device=device) if want is not None and given is None else given
    do, dres, dgate = like(do, o, dtype), like(dres, res, rt), like(dgate, gate, dtype)
    pdo, q.ld_do = _rows(do, shape, dtype, device, "do")
    pdres, q.ld_dres = _rows(dres, shape, rt, device, "dres")
    pdg, q.ld_dgate = _rows(dgate, shape, dtype, device, "dgate")
    if pre_weight is not None and da is None:
        cols = torch.zeros((3, q.channels), dtype=torch.float32, device=device)
    else:
        cols = torch.empty((3, q.channels), dtype=torch.float32, device=device)
    w = [cols[i] if t is not None else None for i, t in enumerate((post_weight, scale, pre_weight))]
    ptr = [t.data_ptr() if t is not None else None for t in w]
    if da is None:
        ptr[2] = None
    lib = load_library()
    desc = ctypes.addressof(q)
    work = _bytes(lib.fi_norm_workspace_bytes(desc), device)
    _call(device, lib.fi_norm_backward, desc, *args, psv, pdr, pda, pdo, pdg, pdres, *ptr, work.data_ptr())
    return NormGradients(do, dres, dgate, *w)


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
        q = Q4Desc()
        q.N, q.K = codes.shape
        q.group, q.scale_dtype, q.has_zeros = group, _type(scales, "scales"), int(zeros is not None)
        self.N, self.K, self.group, self.device = q.N, q.K, group, device
        lib = load_library()
        self._desc = q
        n = lib.fi_q4_packed_bytes(ctypes.addressof(q))
        if n == 0:
            _bad(f"unsupported N={q.N} K={q.K} group={group}")
        shape = (q.N, -(-q.K // group))
        pc = _dense(codes, codes.shape, torch.uint8, device, "codes")
        ps = _dense(scales, shape, scales.dtype, device, "scales")
        pz = _dense(zeros, shape, torch.uint8, device, "zeros")
        self.packed = _bytes(n, device)
        _call(device, lib.fi_q4_pack, ctypes.addressof(q), pc, ps, pz, self.packed.data_ptr())

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
        q = Q4Desc()
        q.N, q.K = w.shape
        q.group, q.scale_dtype = group, _TYPES[scale_dtype]
        wt = _type(w, "w")
        pw, ld = _rows(w, w.shape, w.dtype, device, "w")
        codes = torch.empty(w.shape, dtype=torch.uint8, device=device)
        scales = torch.empty((q.N, -(-q.K // group)), dtype=scale_dtype, device=device)
        _call(device, load_library().fi_q4_quantize, ctypes.addressof(q), wt, pw, ld, codes.data_ptr(),
              scales.data_ptr())
        out = cls(codes, scales, group=group)
        out.codes, out.scales = codes, scales
        return out


def q4_matvec(w, x, y=None):
    """y [B][N] = x [B][K] times a Q4Weight, 1 <= B <= 16 rows (fi_q4_matvec); y has x's type."""
    if not isinstance(w, Q4Weight):
        _bad(f"w: expected a Q4Weight, got {type(w).__name__}")
    device = _device(x, "x")
    if device != w.device:
        _bad(f"x: on {device}, expected {w.device}")
    if x.dim() != 2:
        _bad(f"x: shape {tuple(x.shape)}, expected [B][{w.K}]")
    dt = _type(x, "x")
    rows = x.shape[0]
    px, ldx = _rows(x, (rows, w.K), x.dtype, device, "x")
    if y is None:
        y = torch.empty((rows, w.N), dtype=x.dtype, device=device)
    py, ldy = _rows(y, (rows, w.N), x.dtype, device, "y")
    _call(device, load_library().fi_q4_matvec, ctypes.addressof(w._desc), w.packed.data_ptr(), rows, dt, px, ldx, py,
          ldy)
    return y
