"""Binding of the operators around a recurrent layer: the short convolution, the selective scan, the norms.

As in ``sq``: argument marshalling and checks only, everything else is the HIP library's.  The functions keep
the ABI's names and take tensors or raw device pointers; the classes hold a layer's sizes and workspaces and check
the tensors that they are given.  Tensors are on the current device; calls that may overlap (on several
streams) need an object each where the object has a workspace.
"""
from __future__ import annotations

import ctypes

from . import sq as _sq
from .sq import SQ_BF16, SQ_F32, _bytes, _check, _data, _ptr, _stream

SQ_ACT_NONE, SQ_ACT_SILU, SQ_ACT_SIGMOID = 0, 1, 2
ACTS = {None: SQ_ACT_NONE, "none": SQ_ACT_NONE, "silu": SQ_ACT_SILU, "sigmoid": SQ_ACT_SIGMOID}

_i32, _i64, _int, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_int, ctypes.c_float


class _ConvDesc(ctypes.Structure):
    _fields_ = [("n_seq", _i32), ("n_channels", _i32), ("width", _i32), ("n_tokens", _i64), ("act", _int), ("dtype", _int),
                ("x_stride", _i64)]


class _ScanDesc(ctypes.Structure):
    _fields_ = [("n_seq", _i32), ("n_heads", _i32), ("n_groups", _i32), ("d_state", _i32), ("d_head", _i32), ("n_tokens", _i64),
                ("softplus", _i32), ("in_dtype", _int), ("y_dtype", _int), ("x_stride", _i64), ("dt_stride", _i64),
                ("b_stride", _i64), ("c_stride", _i64), ("dx_stride", _i64), ("ddt_stride", _i64), ("db_stride", _i64),
                ("dc_stride", _i64)]


class _GateDesc(ctypes.Structure):
    _fields_ = [("n_tokens", _i64), ("n_groups", _i32), ("d", _i32), ("shared_weight", _i32), ("gate_first", _i32), ("act", _int),
                ("eps", _f32), ("dtype", _int), ("x_stride", _i64), ("z_stride", _i64), ("dx_stride", _i64), ("dz_stride", _i64)]


class _ResidualDesc(ctypes.Structure):
    _fields_ = [("n_rows", _i64), ("d", _i32), ("eps", _f32), ("dtype", _int), ("res_dtype", _int)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = _sq.lib()
        vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        psize = ctypes.POINTER(sz)
        conv, scan, gate, res = (ctypes.POINTER(d) for d in (_ConvDesc, _ScanDesc, _GateDesc, _ResidualDesc))
        for name, args in (
                ("sq_conv_bytes", [conv, psize]),
                ("sq_conv_forward", [conv] + [vp] * 7 + [vp]),
                ("sq_conv_backward", [conv] + [vp] * 12 + [sz, vp]),
                ("sq_conv_step", [conv, vp, _i32, vp, _i32] + [vp] * 4 + [vp]),
                ("sq_scan_bytes", [scan, psize, psize]),
                ("sq_scan_forward", [scan] + [vp] * 12 + [sz, vp, sz, vp]),
                ("sq_scan_backward", [scan] + [vp] * 11 + [sz] + [vp] * 9 + [sz, vp]),
                ("sq_scan_step", [scan, vp, _i32, vp, _i32] + [vp] * 8 + [vp]),
                ("sq_gated_norm_bytes", [gate, psize]),
                ("sq_gated_norm_forward", [gate] + [vp] * 4 + [vp]),
                ("sq_gated_norm_backward", [gate] + [vp] * 8 + [sz, vp]),
                ("sq_residual_norm_bytes", [res, psize]),
                ("sq_residual_norm_forward", [res] + [vp] * 7 + [vp]),
                ("sq_residual_norm_backward", [res] + [vp] * 13 + [sz, vp])):
            f = getattr(L, name)
            f.restype, f.argtypes = st, args
        _bound = L
    return _bound


# ------------------------------------------------------------------ the ABI's functions
def conv_desc(n_seq, n_tokens, n_channels, width, act, dtype, x_stride=0) -> _ConvDesc:
    return _ConvDesc(int(n_seq), int(n_channels), int(width), int(n_tokens), int(act), int(dtype), int(x_stride))


def _one_size(name, desc) -> int:
    out = ctypes.c_size_t(0)
    _check(getattr(_lib(), name)(ctypes.byref(desc), ctypes.byref(out)), name)
    return out.value


def sq_conv_bytes(desc) -> int:
    return _one_size("sq_conv_bytes", desc)


def sq_conv_forward(desc, cu, x, weight, bias, S0, y, S_out, stream=None) -> None:
    _check(_lib().sq_conv_forward(ctypes.byref(desc), _ptr(cu), _data(x), _ptr(weight), _ptr(bias), _ptr(S0), _ptr(y), _ptr(S_out),
                                  _stream(stream)), "sq_conv_forward")


def sq_conv_backward(desc, cu, x, weight, bias, S0, dy, dS_out, dx, dweight, dbias, dS0, work, work_bytes=None, stream=None) -> None:
    _check(_lib().sq_conv_backward(ctypes.byref(desc), _ptr(cu), _data(x), _ptr(weight), _ptr(bias), _ptr(S0), _ptr(dy), _ptr(dS_out),
                                   _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(dS0), _ptr(work), _bytes(work, work_bytes),
                                   _stream(stream)), "sq_conv_backward")


def sq_conv_step(desc, pool, n_slots, slot_idx, n, x, weight, bias, y, stream=None) -> None:
    _check(_lib().sq_conv_step(ctypes.byref(desc), _ptr(pool), int(n_slots), _ptr(slot_idx), int(n), _data(x), _ptr(weight), _ptr(bias),
                               _ptr(y), _stream(stream)), "sq_conv_step")


def scan_desc(n_seq, n_tokens, n_heads, d_head, d_state, n_groups=1, softplus=True, in_dtype=SQ_BF16, y_dtype=SQ_BF16, x_stride=0,
              dt_stride=0, b_stride=0, c_stride=0, dx_stride=0, ddt_stride=0, db_stride=0, dc_stride=0) -> _ScanDesc:
    return _ScanDesc(int(n_seq), int(n_heads), int(n_groups), int(d_state), int(d_head), int(n_tokens), int(softplus), int(in_dtype),
                     int(y_dtype), int(x_stride), int(dt_stride), int(b_stride), int(c_stride), int(dx_stride), int(ddt_stride),
                     int(db_stride), int(dc_stride))


def sq_scan_bytes(desc, train: bool = False):
    """Bytes of `work` for sq_scan_forward; train: (work, save), for the backward pass too."""
    work, save = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(_lib().sq_scan_bytes(ctypes.byref(desc), ctypes.byref(work), ctypes.byref(save) if train else None), "sq_scan_bytes")
    return (work.value, save.value) if train else work.value


def sq_scan_forward(desc, cu, x, raw, A, B, C, D, dt_bias, S0, y, S_out, save, work, save_bytes=None, work_bytes=None,
                    stream=None) -> None:
    _check(_lib().sq_scan_forward(ctypes.byref(desc), _ptr(cu), _data(x), _data(raw), _ptr(A), _data(B), _data(C), _ptr(D),
                                  _ptr(dt_bias), _ptr(S0), _ptr(y), _ptr(S_out), _ptr(save), _bytes(save, save_bytes), _ptr(work),
                                  _bytes(work, work_bytes), _stream(stream)), "sq_scan_forward")


def sq_scan_backward(desc, cu, x, raw, A, B, C, D, dt_bias, dy, dS_out, save, dx, draw, dA, dB, dC, dD, ddt_bias, dS0, work,
                     save_bytes=None, work_bytes=None, stream=None) -> None:
    _check(_lib().sq_scan_backward(ctypes.byref(desc), _ptr(cu), _data(x), _data(raw), _ptr(A), _data(B), _data(C), _ptr(D),
                                   _ptr(dt_bias), _ptr(dy), _ptr(dS_out), _ptr(save), _bytes(save, save_bytes), _data(dx), _data(draw),
                                   _ptr(dA), _data(dB), _data(dC), _ptr(dD), _ptr(ddt_bias), _ptr(dS0), _ptr(work),
                                   _bytes(work, work_bytes), _stream(stream)), "sq_scan_backward")


def sq_scan_step(desc, state_pool, n_slots, slot_idx, n, x, raw, A, B, C, D, dt_bias, y, stream=None) -> None:
    _check(_lib().sq_scan_step(ctypes.byref(desc), _ptr(state_pool), int(n_slots), _ptr(slot_idx), int(n), _data(x), _data(raw), _ptr(A),
                               _data(B), _data(C), _ptr(D), _ptr(dt_bias), _ptr(y), _stream(stream)), "sq_scan_step")


def gated_norm_desc(n_tokens, n_groups, d, shared_weight=True, gate_first=False, act=SQ_ACT_SILU, eps=1e-6, dtype=SQ_BF16, x_stride=0,
                    z_stride=0, dx_stride=0, dz_stride=0) -> _GateDesc:
    return _GateDesc(int(n_tokens), int(n_groups), int(d), int(shared_weight), int(gate_first), int(act), float(eps), int(dtype),
                     int(x_stride), int(z_stride), int(dx_stride), int(dz_stride))


def sq_gated_norm_bytes(desc) -> int:
    return _one_size("sq_gated_norm_bytes", desc)


def sq_gated_norm_forward(desc, x, z, weight, y, stream=None) -> None:
    _check(_lib().sq_gated_norm_forward(ctypes.byref(desc), _data(x), _data(z), _ptr(weight), _ptr(y), _stream(stream)),
           "sq_gated_norm_forward")


def sq_gated_norm_backward(desc, x, z, weight, dy, dx, dz, dweight, work, work_bytes=None, stream=None) -> None:
    _check(_lib().sq_gated_norm_backward(ctypes.byref(desc), _data(x), _data(z), _ptr(weight), _ptr(dy), _data(dx), _data(dz),
                                         _ptr(dweight), _ptr(work), _bytes(work, work_bytes), _stream(stream)),
           "sq_gated_norm_backward")


def residual_norm_desc(n_rows, d, eps=1e-6, dtype=SQ_BF16, res_dtype=SQ_BF16) -> _ResidualDesc:
    return _ResidualDesc(int(n_rows), int(d), float(eps), int(dtype), int(res_dtype))


def sq_residual_norm_bytes(desc) -> int:
    return _one_size("sq_residual_norm_bytes", desc)


def sq_residual_norm_forward(desc, o, r, post_weight, scale, weight, r_out, h, stream=None) -> None:
    _check(_lib().sq_residual_norm_forward(ctypes.byref(desc), _ptr(o), _ptr(r), _ptr(post_weight), _ptr(scale), _ptr(weight),
                                           _ptr(r_out), _ptr(h), _stream(stream)), "sq_residual_norm_forward")


def sq_residual_norm_backward(desc, o, r, post_weight, scale, weight, dh, dr_out, d_o, dr, dpost_weight, dscale, dweight, work,
                              work_bytes=None, stream=None) -> None:
    _check(_lib().sq_residual_norm_backward(ctypes.byref(desc), _ptr(o), _ptr(r), _ptr(post_weight), _ptr(scale), _ptr(weight), _ptr(dh),
                                            _ptr(dr_out), _ptr(d_o), _ptr(dr), _ptr(dpost_weight), _ptr(dscale), _ptr(dweight),
                                            _ptr(work), _bytes(work, work_bytes), _stream(stream)), "sq_residual_norm_backward")


# ------------------------------------------------------------------ checks of tensors
_torch = None


def _load():
    """torch, once an object or a call needs it (the binding itself imports without)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _type(t, what):
    code = {_torch.float32: SQ_F32, _torch.bfloat16: SQ_BF16}.get(t)
    if code is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (what, t))
    return code


def _home(t):
    """The number of the device of a call's tensors, which has to be the current one."""
    dev = t.get_device()
    if dev >= 0 and dev != _torch.cuda.current_device():
        raise ValueError("the tensors are on cuda:%d, but the current device is cuda:%d" % (dev, _torch.cuda.current_device()))
    return dev


def _fits(name, t, shape, dtype, dev):
    if not isinstance(t, _torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError("%s must be a device tensor, on the device of the others" % name)
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def _tensor(name, t, shape, dtype, dev):
    """The address of a dense tensor of this shape and type on the call's device."""
    try:
        if t.is_cuda and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _fits(name, t, shape, dtype, dev)
    raise ValueError("%s must be contiguous" % name)


def _maybe(name, t, shape, dtype, dev):
    return None if t is None else _tensor(name, t, shape, dtype, dev)


def _tokens(name, t, shape, dtype, dev):
    """The address and the token stride (0: dense) of a tensor whose rows [1:] are dense, a part of a wider one at most."""
    try:
        if t.is_cuda and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr(), 0
    except AttributeError:
        pass
    _fits(name, t, shape, dtype, dev)
    row, strides = 1, t.stride()
    for i in range(len(shape) - 1, 0, -1):
        if shape[i] > 1 and strides[i] != row:
            raise ValueError("the rows of %s must be dense" % name)
        row *= shape[i]
    if shape[0] < 2:
        return t.data_ptr(), 0
    if strides[0] < row:  # an expanded tensor's 0 would mean dense
        raise ValueError("the tokens of %s must not overlap" % name)
    return t.data_ptr(), strides[0]


def _room(nbytes, device):
    return _torch.empty(max(256, nbytes), dtype=_torch.uint8, device=device)


def _span(buf, dev):
    """Address and size of an object's workspace, which has to be on the device of the call's tensors."""
    if buf is None:
        return None, 0
    if buf.get_device() != dev:
        raise ValueError("the object's workspace is on %s, not on the device of the tensors" % buf.device)
    return buf.data_ptr(), buf.numel()


def _copy(desc):
    """A call's own descriptor: the object's may be in use by another thread."""
    return type(desc).from_buffer_copy(desc)


# ------------------------------------------------------------------ short convolution
class ShortConv:
    """A causal convolution of every channel with `width` taps of its own, and SiLU, over ragged sequences.

    For batches of up to n_seq sequences and n_tokens tokens in all; with train=True it holds the
    workspace of backward.  x [tokens, n_channels] may be part of a wider tensor, everything else is
    dense; weight [n_channels, width], bias [n_channels] and their gradients are fp32."""

    def __init__(self, n_seq: int, n_tokens: int, n_channels: int, width: int, act="silu", dtype=None, device="cuda", train=False):
        torch = _load()
        self.dtype = torch.bfloat16 if dtype is None else dtype
        self.n_seq, self.n_tokens, self.n_channels, self.width = int(n_seq), int(n_tokens), int(n_channels), int(width)
        self.act = ACTS[act]
        self._desc = conv_desc(n_seq, n_tokens, n_channels, width, self.act, _type(self.dtype, "dtype"))
        nbytes = sq_conv_bytes(self._desc)
        self.work = _room(nbytes, device) if train else None

    def _args(self, x, weight, cu, bias, S0):
        f32, n, n_seq, c = _torch.float32, x.shape[0], cu.numel() - 1, self.n_channels
        dev, desc = _home(x), _copy(self._desc)
        if n_seq < 0:
            raise ValueError("cu needs one entry more than there are sequences")
        desc.n_seq, desc.n_tokens = n_seq, n
        at = _tensor("cu", cu, (n_seq + 1,), _torch.int32, dev)
        px, desc.x_stride = _tokens("x", x, (n, c), self.dtype, dev)
        return (desc, at, px, _tensor("weight", weight, (c, self.width), f32, dev), _maybe("bias", bias, (c,), f32, dev),
                _maybe("S0", S0, (n_seq, self.width - 1, c), self.dtype, dev)), dev, (n, c), (n_seq, self.width - 1, c)

    def forward(self, x, weight, cu, y, bias=None, S0=None, S_out=None, stream=None):
        """y [tokens, n_channels]; S0, S_out [n_seq, width - 1, n_channels]: the inputs before each sequence, and its
        last ones; cu: int32 [n_seq + 1], the tokens at which the sequences begin and end."""
        args, dev, tokens, state = self._args(x, weight, cu, bias, S0)
        sq_conv_forward(*args, _tensor("y", y, tokens, self.dtype, dev), _maybe("S_out", S_out, state, self.dtype, dev), stream)

    def backward(self, x, weight, cu, dy, dx, dweight, bias=None, dbias=None, S0=None, dS_out=None, dS0=None, stream=None):
        """Gradients for the inputs of a forward call; dweight and dbias are written, not added to."""
        if self.work is None:
            raise ValueError("backward needs train=True")
        args, dev, tokens, state = self._args(x, weight, cu, bias, S0)
        c, f32, dt = self.n_channels, _torch.float32, self.dtype
        sq_conv_backward(*args, _tensor("dy", dy, tokens, dt, dev), _maybe("dS_out", dS_out, state, dt, dev), _tensor("dx", dx, tokens, dt, dev),
                         _tensor("dweight", dweight, (c, self.width), f32, dev), _maybe("dbias", dbias, (c,), f32, dev),
                         _maybe("dS0", dS0, state, dt, dev), *_span(self.work, dev), stream)


def conv_step(pool, slot_idx, x, weight, y, bias=None, act="silu", stream=None) -> None:
    """One token per request on a pool [n_slots, width - 1, n_channels] of the last inputs, in place on the
    listed slots, which are distinct; x, y [n, n_channels].  Requests whose slot is outside the pool are left out."""
    torch = _load()
    n_slots, before, c = pool.shape
    n, dt, f32, dev = slot_idx.numel(), pool.dtype, torch.float32, _home(pool)
    px, stride = _tokens("x", x, (n, c), dt, dev)
    sq_conv_step(conv_desc(0, 0, c, before + 1, ACTS[act], _type(dt, "pool"), stride), _tensor("pool", pool, (n_slots, before, c), dt, dev), n_slots,
                 _tensor("slot_idx", slot_idx, (n,), torch.int32, dev), n, px, _tensor("weight", weight, (c, before + 1), f32, dev),
                 _maybe("bias", bias, (c,), f32, dev), _tensor("y", y, (n, c), dt, dev), stream)


# ------------------------------------------------------------------ selective scan
class SelectiveScan:
    """The state-space recurrence S_t = exp(dt A) S_{t-1} + dt B x^T, y = S_t^T C + D x over ragged sequences, with its
    workspace; dt = softplus(dt + dt_bias), without softplus: dt + dt_bias.

    For batches of up to n_seq sequences and n_tokens tokens in all.  With train=True, also what backward needs
    of the last forward call, which it belongs to: a second forward takes the first one's place, and
    backward refuses the number of any call but the last (a replayed graph's calls have no number: give a graph an object
    of its own).  x [tokens, n_heads, d_head], dt [tokens, n_heads], B and C
    [tokens, n_groups, d_state] and their gradients may be parts of wider tensors; A, D, dt_bias and their gradients
    are fp32 [n_heads], states fp32 [n_seq, n_heads, d_state, d_head]."""

    def __init__(self, n_seq: int, n_tokens: int, n_heads: int, d_head: int, d_state: int, n_groups: int = 1, softplus=True, dtype=None,
                 y_dtype=None, device="cuda", train=False):
        torch = _load()
        self.dtype = torch.bfloat16 if dtype is None else dtype
        self.y_dtype = self.dtype if y_dtype is None else y_dtype
        self.n_seq, self.n_tokens = int(n_seq), int(n_tokens)
        self.n_heads, self.n_groups, self.d_head, self.d_state = int(n_heads), int(n_groups), int(d_head), int(d_state)
        self.softplus = bool(softplus)
        self._desc = scan_desc(n_seq, n_tokens, n_heads, d_head, d_state, n_groups, self.softplus, _type(self.dtype, "dtype"),
                               _type(self.y_dtype, "y_dtype"))
        sizes = sq_scan_bytes(self._desc, train=bool(train))
        work, save = sizes if train else (sizes, None)
        self.calls, self._sizes = 0, None  # forward calls so far, and the last one's batch
        self.work = _room(work, device)
        self.save = None if save is None else _room(save, device)

    def _inputs(self, x, dt, A, B, C, cu, D, dt_bias, S0):
        f32, n, n_seq, h, to = _torch.float32, x.shape[0], cu.numel() - 1, self.n_heads, self.dtype
        dev, keys, desc = _home(x), (n, self.n_groups, self.d_state), _copy(self._desc)
        if n_seq < 0:
            raise ValueError("cu needs one entry more than there are sequences")
        desc.n_seq, desc.n_tokens = n_seq, n
        at = _tensor("cu", cu, (n_seq + 1,), _torch.int32, dev)
        px, desc.x_stride = _tokens("x", x, (n, h, self.d_head), to, dev)
        pt, desc.dt_stride = _tokens("dt", dt, (n, h), to, dev)
        pb, desc.b_stride = _tokens("B", B, keys, to, dev)
        pc, desc.c_stride = _tokens("C", C, keys, to, dev)
        state = (n_seq, h, self.d_state, self.d_head)
        return (desc, at, px, pt, _tensor("A", A, (h,), f32, dev), pb, pc, _maybe("D", D, (h,), f32, dev),
                _maybe("dt_bias", dt_bias, (h,), f32, dev)), _maybe("S0", S0, state, f32, dev), dev, n, state

    def forward(self, x, dt, A, B, C, cu, y, D=None, dt_bias=None, S0=None, S_out=None, stream=None):
        """y [tokens, n_heads, d_head] and, where given, the final states S_out; cu: int32 [n_seq + 1] on the device, the
        tokens at which the sequences begin and end.  Returns the call's number, for backward."""
        args, start, dev, n, state = self._inputs(x, dt, A, B, C, cu, D, dt_bias, S0)
        py = _tensor("y", y, (n, self.n_heads, self.d_head), self.y_dtype, dev)
        save, save_bytes = _span(self.save, dev)
        work, work_bytes = _span(self.work, dev)
        sq_scan_forward(*args, start, py, _maybe("S_out", S_out, state, _torch.float32, dev), save, work, save_bytes, work_bytes, stream)
        self.calls, self._sizes = self.calls + 1, (state[0], n)
        return self.calls

    def backward(self, x, dt, A, B, C, cu, dy, dx, ddt, dA, dB, dC, D=None, dt_bias=None, dD=None, ddt_bias=None, S0=None, dS_out=None,
                 dS0=None, call=None, stream=None):
        """Gradients of the last forward call, which had the same inputs; dy dense and in `dtype`; dA, dD and ddt_bias
        are written, not added to.  call: what that forward returned; raises RuntimeError where another one came
        after it."""
        if self.save is None:
            raise ValueError("backward needs train=True")
        args, _, dev, n, state = self._inputs(x, dt, A, B, C, cu, D, dt_bias, S0)
        if self.calls == 0 or (call is not None and call != self.calls):
            raise RuntimeError("backward of forward call %s, but the saved states are of call %d" % (
                "?" if call is None else call, self.calls))
        if self._sizes != (state[0], n):
            raise RuntimeError("the last forward call had %d sequences of %d tokens, not %d of %d" % (*self._sizes, state[0], n))
        f32, to, h, desc = _torch.float32, self.dtype, self.n_heads, args[0]
        wide, keys = (n, h, self.d_head), (n, self.n_groups, self.d_state)
        pdx, desc.dx_stride = _tokens("dx", dx, wide, to, dev)
        pdt, desc.ddt_stride = _tokens("ddt", ddt, (n, h), to, dev)
        pdb, desc.db_stride = _tokens("dB", dB, keys, to, dev)
        pdc, desc.dc_stride = _tokens("dC", dC, keys, to, dev)
        save, save_bytes = _span(self.save, dev)
        work, work_bytes = _span(self.work, dev)
        sq_scan_backward(*args, _tensor("dy", dy, wide, to, dev), _maybe("dS_out", dS_out, state, f32, dev), save, pdx, pdt,
                         _tensor("dA", dA, (h,), f32, dev), pdb, pdc, _maybe("dD", dD, (h,), f32, dev), _maybe("ddt_bias", ddt_bias, (h,), f32, dev),
                         _maybe("dS0", dS0, state, f32, dev), work, save_bytes, work_bytes, stream)


def scan_step(pool, slot_idx, x, dt, A, B, C, y, D=None, dt_bias=None, softplus=True, stream=None) -> None:
    """One token per request on an fp32 pool [n_slots, n_heads, d_state, d_head], in place on the listed slots, which
    are distinct: x, y [n, n_heads, d_head], dt [n, n_heads], B, C [n, n_groups, d_state].  Requests whose slot is outside the
    pool are left out."""
    torch = _load()
    n_slots, h, ns, p = pool.shape
    n, dev, f32, to = slot_idx.numel(), _home(pool), torch.float32, x.dtype
    if B.dim() != 3:
        raise ValueError("B must be [n, n_groups, d_state]")
    keys = (n, B.shape[1], ns)
    px, xs = _tokens("x", x, (n, h, p), to, dev)
    pt, ts = _tokens("dt", dt, (n, h), to, dev)
    pb, bs = _tokens("B", B, keys, to, dev)
    pc, cs = _tokens("C", C, keys, to, dev)
    sq_scan_step(scan_desc(0, 0, h, p, ns, keys[1], softplus, _type(to, "x"), _type(y.dtype, "y"), xs, ts, bs, cs),
                 _tensor("pool", pool, (n_slots, h, ns, p), f32, dev), n_slots, _tensor("slot_idx", slot_idx, (n,), torch.int32, dev), n, px, pt,
                 _tensor("A", A, (h,), f32, dev), pb, pc, _maybe("D", D, (h,), f32, dev), _maybe("dt_bias", dt_bias, (h,), f32, dev),
                 _tensor("y", y, (n, h, p), y.dtype, dev), stream)


# ------------------------------------------------------------------ norms
class GatedNorm:
    """The norm behind a layer, with its gate: rms(x) * weight * act(z), or, with gate_first, rms(x * act(z)) * weight, over rows
    of d (each of n_groups of a token).  act: "silu", "sigmoid", or None for a norm without a gate.

    x, z and their gradients [tokens, n_groups, d] may be parts of wider tensors; y and dy are dense; weight is
    fp32 [d], without shared_weight [n_groups, d], or None for ones.  Any number of tokens; train=True: n_tokens
    at most, for backward's workspace (None: the most that it ever takes)."""

    def __init__(self, n_groups: int, d: int, act="silu", gate_first=False, shared_weight=True, eps=1e-6, dtype=None, device="cuda",
                 train=False, n_tokens=None):
        torch = _load()
        self.dtype = torch.bfloat16 if dtype is None else dtype
        self.n_groups, self.d, self.act, self.eps = int(n_groups), int(d), ACTS[act], float(eps)
        self.gate_first, self.shared_weight = bool(gate_first), bool(shared_weight)
        most = (1 << 31) // max(1, self.n_groups) - 1
        self._desc = gated_norm_desc(most if n_tokens is None else n_tokens, n_groups, d, self.shared_weight, self.gate_first, self.act,
                                     self.eps, _type(self.dtype, "dtype"))
        nbytes = sq_gated_norm_bytes(self._desc)
        self.work = _room(nbytes, device) if train else None
        self._wide = (self.d,) if self.shared_weight else (self.n_groups, self.d)

    def _args(self, x, z, weight):
        dev, shape, desc = _home(x), (x.shape[0], self.n_groups, self.d), _copy(self._desc)
        desc.n_tokens = shape[0]
        px, desc.x_stride = _tokens("x", x, shape, self.dtype, dev)
        if (z is None) != (self.act == SQ_ACT_NONE):
            raise ValueError("z is needed with a gate, and only then")
        pz, desc.z_stride = (None, 0) if z is None else _tokens("z", z, shape, self.dtype, dev)
        return desc, px, pz, _maybe("weight", weight, self._wide, _torch.float32, dev), dev, shape

    def forward(self, x, z, weight, y, stream=None):
        desc, px, pz, pw, dev, shape = self._args(x, z, weight)
        sq_gated_norm_forward(desc, px, pz, pw, _tensor("y", y, shape, self.dtype, dev), stream)

    def backward(self, x, z, weight, dy, dx, dz, dweight=None, stream=None):
        """Gradients for the inputs of a forward call; dweight is written, not added to."""
        desc, px, pz, pw, dev, shape = self._args(x, z, weight)
        pdy = _tensor("dy", dy, shape, self.dtype, dev)
        pdx, desc.dx_stride = _tokens("dx", dx, shape, self.dtype, dev)
        if (dz is None) != (z is None):
            raise ValueError("dz is needed with a gate, and only then")
        pdz, desc.dz_stride = (None, 0) if dz is None else _tokens("dz", dz, shape, self.dtype, dev)
        pdw = _maybe("dweight", dweight, self._wide, _torch.float32, dev)
        if pdw is not None and self.work is None:
            raise ValueError("dweight needs train=True")
        sq_gated_norm_backward(desc, px, pz, pw, pdy, pdx, pdz, pdw, *_span(None if pdw is None else self.work, dev), stream)


class ResidualNorm:
    """Between two blocks, over rows of d: r_out = r + scale * a with a = o or rms(o) * post_weight, and h = rms(r_out) * weight.

    o, h and their gradients [..., d] in dtype, r and r_out and theirs in res_dtype, all dense; the parameters and their
    gradients fp32 [d].  train=True holds backward's workspace."""

    def __init__(self, d: int, eps=1e-6, dtype=None, res_dtype=None, device="cuda", train=False):
        torch = _load()
        self.dtype = torch.bfloat16 if dtype is None else dtype
        self.res_dtype = self.dtype if res_dtype is None else res_dtype
        self.d, self.eps = int(d), float(eps)
        self._desc = residual_norm_desc((1 << 31) - 1, d, eps, _type(self.dtype, "dtype"), _type(self.res_dtype, "res_dtype"))
        nbytes = sq_residual_norm_bytes(self._desc)
        self.work = _room(nbytes, device) if train else None

    def _args(self, o, r, post_weight, scale, weight):
        dev, shape, desc, row, f32 = _home(o), o.shape, _copy(self._desc), (self.d,), _torch.float32
        if o.dim() < 1 or shape[-1] != self.d:
            raise ValueError("o has shape %s, expected [..., %d]" % (tuple(shape), self.d))
        desc.n_rows = o.numel() // self.d
        return (desc, _tensor("o", o, shape, self.dtype, dev), _maybe("r", r, shape, self.res_dtype, dev), _maybe("post_weight", post_weight, row, f32, dev),
                _maybe("scale", scale, row, f32, dev), _maybe("weight", weight, row, f32, dev)), dev, shape

    def forward(self, o, r, r_out, weight=None, h=None, post_weight=None, scale=None, stream=None):
        """r None: zeros; h None: the sum alone; r_out may be r."""
        args, dev, shape = self._args(o, r, post_weight, scale, weight)
        sq_residual_norm_forward(*args, _tensor("r_out", r_out, shape, self.res_dtype, dev), _maybe("h", h, shape, self.dtype, dev), stream)

    def backward(self, o, r, dh, dr_out, do, dr, weight=None, dweight=None, post_weight=None, dpost_weight=None, scale=None, dscale=None,
                 stream=None):
        """Gradients from o and r as the forward call had them (so not from an r that r_out took the place of); dh, dr_out, dr
        and the parameters' gradients may be None; the latter are written, not added to."""
        args, dev, shape = self._args(o, r, post_weight, scale, weight)
        row, f32 = (self.d,), _torch.float32
        pdo = _tensor("do", do, shape, self.dtype, dev)
        grads = [_maybe(name, t, row, f32, dev) for name, t in (("dpost_weight", dpost_weight), ("dscale", dscale), ("dweight", dweight))]
        sums = any(g is not None for g in grads)
        if sums and self.work is None:
            raise ValueError("gradients of parameters need train=True")
        sq_residual_norm_backward(*args, _maybe("dh", dh, shape, self.dtype, dev), _maybe("dr_out", dr_out, shape, self.res_dtype, dev), pdo,
                                  _maybe("dr", dr, shape, self.res_dtype, dev), *grads, *_span(self.work if sums else None, dev), stream)
