"""Thin ctypes binding of the C ABI in include/sq.h.

Argument marshalling only: every step of the decode path runs in the HIP
library ``libsq.so``.  There is no CPU fallback; if the library is missing
or fails to load, every entry point raises.

Tensors are torch tensors (device memory and streams only); raw integer
device pointers are accepted too.  Functions keep the ABI's names.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
# the in-tree build; SQ_LIBRARY may name another build of the same sources
# (the instrumented timeline build, libsq_timeline.so)
LIB_PATH = os.environ.get("SQ_LIBRARY") or os.path.join(HERE, "libsq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "sq.h")

SQ_OK, SQ_EINVAL, SQ_EUNSUPPORTED, SQ_ENOMEM, SQ_EHIP = 0, 1, 2, 3, 4
SQ_GATE_GDN, SQ_GATE_KDA = 0, 1
SQ_F32, SQ_BF16 = 0, 1
STATUS_NAMES = {0: "SQ_OK", 1: "SQ_EINVAL", 2: "SQ_EUNSUPPORTED", 3: "SQ_ENOMEM", 4: "SQ_EHIP"}

_lib = None


class SQError(RuntimeError):
    def __init__(self, status: int, func: str, text: str):
        super().__init__("%s -> %s: %s" % (func, STATUS_NAMES.get(status, status), text))
        self.status = status
        self.func = func
        self.text = text


class _Desc(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("head_bits", ctypes.POINTER(ctypes.c_uint8)), ("gate", ctypes.c_int)]


class _SeqDesc(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_key_heads", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("n_tokens", ctypes.c_int64), ("gate", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


def lib():
    """Load libsq.so (built in-tree).  Raises if it is missing: no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("library not built at %s: run __graft_entry__.build() or "
                              "python quantized_gated_delta_amd/build.py" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        st = ctypes.c_int
        pdesc = ctypes.POINTER(_Desc)
        L.sq_pool_bytes.restype = st
        L.sq_pool_bytes.argtypes = [pdesc, ctypes.POINTER(ctypes.c_size_t)]
        L.sq_pool_create.restype = st
        L.sq_pool_create.argtypes = [pdesc, vp, ctypes.c_size_t, ctypes.POINTER(vp)]
        L.sq_pool_bytes_rows.restype = st
        L.sq_pool_bytes_rows.argtypes = [pdesc, vp, ctypes.POINTER(ctypes.c_size_t)]
        L.sq_pool_create_rows.restype = st
        L.sq_pool_create_rows.argtypes = [pdesc, vp, vp, ctypes.c_size_t, ctypes.POINTER(vp)]
        L.sq_pool_destroy.restype = st
        L.sq_pool_destroy.argtypes = [vp]
        L.sq_pool_layout.restype = st
        L.sq_pool_layout.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                     ctypes.POINTER(i64)]
        L.sq_pool_set_row_impact.restype = st
        L.sq_pool_set_row_impact.argtypes = [vp, vp]
        L.sq_quant_state.restype = st
        L.sq_quant_state.argtypes = [vp, vp, i32, vp, vp]
        L.sq_dequant_state.restype = st
        L.sq_dequant_state.argtypes = [vp, vp, i32, vp, vp]
        L.sq_decode_step.restype = st
        L.sq_decode_step.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, ctypes.c_int, vp,
                                     ctypes.c_int, vp]
        L.sq_decode_update.restype = st
        L.sq_decode_update.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, ctypes.c_int, vp,
                                       ctypes.c_int, vp, vp]
        L.sq_split_step_noalloc.restype = st
        L.sq_split_step_noalloc.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, ctypes.c_int, vp,
                                            ctypes.c_int, vp]
        L.sq_f32_decode_step.restype = st
        L.sq_f32_decode_step.argtypes = [vp, i32, i32, i32, i32, ctypes.c_int, vp, i32, vp, vp,
                                         vp, vp, vp, ctypes.c_int, vp, ctypes.c_int, vp]
        L.sq_check_slots.restype = st
        L.sq_check_slots.argtypes = [vp, vp, i32, vp]
        L.sq_arith_selfcheck.restype = st
        L.sq_arith_selfcheck.argtypes = [vp, vp]
        L.sq_device_copy.restype = st
        L.sq_device_copy.argtypes = [vp, vp, ctypes.c_size_t, vp]
        L.sq_issue_probe.restype = st
        L.sq_issue_probe.argtypes = [ctypes.c_int, vp, vp]
        pseq, psize = ctypes.POINTER(_SeqDesc), ctypes.POINTER(ctypes.c_size_t)
        L.sq_chunk_bytes.restype = st
        sz = ctypes.c_size_t
        L.sq_chunk_bytes.argtypes = [pseq, psize, psize]
        L.sq_chunk_forward.restype = st
        L.sq_chunk_forward.argtypes = [pseq] + [vp] * 10 + [sz, vp, sz, vp]
        L.sq_chunk_backward.restype = st
        L.sq_chunk_backward.argtypes = [pseq] + [vp] * 9 + [sz] + [vp] * 7 + [sz, vp]
        L.sq_window_update.restype = st
        L.sq_window_update.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp,
                                       ctypes.c_int, vp, ctypes.c_int, vp, vp]
        L.sq_f32_window_update.restype = st
        L.sq_f32_window_update.argtypes = [vp, i32, i32, i32, i32, i32, ctypes.c_int, vp, i32,
                                           i32, vp, vp, vp, vp, vp, vp, ctypes.c_int, vp,
                                           ctypes.c_int, vp, vp]
        L.sq_verify_bytes.restype = st
        L.sq_verify_bytes.argtypes = [i32, i32, psize]
        L.sq_verify_draft.restype = st
        L.sq_verify_draft.argtypes = [i32, i32, i32, vp, i64, vp, i64, ctypes.c_int, vp, vp, vp, vp,
                                      ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp]
        L.sq_last_error.restype = ctypes.c_char_p
        L.sq_last_error.argtypes = []
        L.sq_version.restype = ctypes.c_char_p
        L.sq_version.argtypes = []
        _lib = L
    return _lib


def header_symbols() -> list:
    """Names of the functions include/sq.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(sq_[a-z0-9_]+)\s*\(", text)))


def _check(status: int, func: str):
    if status != SQ_OK:
        raise SQError(status, func, lib().sq_last_error().decode(errors="replace"))


def _ptr(x) -> Optional[int]:
    """Raw pointer of an int, a ctypes array or a torch tensor.  Tensors must
    be contiguous: the library reads them as dense row-major arrays."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "is_contiguous") and not x.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return x.data_ptr()


def _need(t, name, numel, dtypes):
    """Shape / dtype / device check of one tensor argument (marshalling only)."""
    if getattr(t, "is_cuda", False) and t.dtype in dtypes and t.numel() == numel:
        return
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.numel() != numel:
        raise ValueError("%s has %d elements, expected %d" % (name, t.numel(), numel))
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return SQ_F32
    if t.dtype == torch.bfloat16:
        return SQ_BF16
    raise TypeError("tensor dtype must be float32 or bfloat16, got %s" % t.dtype)


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        # without the Stream object that torch.cuda.current_stream() builds: 0.3 us for 2.9
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        return raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _desc(n_slots, n_heads, d_k, d_v, head_bits: Sequence[int], gate):
    hb = (ctypes.c_uint8 * max(1, len(head_bits)))(*[int(b) for b in head_bits])
    d = _Desc(int(n_slots), int(n_heads), int(d_k), int(d_v),
              ctypes.cast(hb, ctypes.POINTER(ctypes.c_uint8)), int(gate))
    return d, hb


def version() -> str:
    return lib().sq_version().decode()


def sq_last_error() -> str:
    return lib().sq_last_error().decode(errors="replace")


def _row_bits(row_bits):
    if row_bits is None:
        return None
    flat = [int(b) for row in row_bits for b in row]
    return (ctypes.c_uint8 * max(1, len(flat)))(*flat)


def sq_pool_bytes(n_slots, n_heads, d_k, d_v, head_bits, gate, row_bits=None) -> int:
    """row_bits: [n_heads][d_k] key-row widths for heads with head_bits 0 (else None)."""
    d, keep = _desc(n_slots, n_heads, d_k, d_v, head_bits, gate)
    rb = _row_bits(row_bits)
    out = ctypes.c_size_t(0)
    if rb is None:
        _check(lib().sq_pool_bytes(ctypes.byref(d), ctypes.byref(out)), "sq_pool_bytes")
    else:
        _check(lib().sq_pool_bytes_rows(ctypes.byref(d), rb, ctypes.byref(out)),
               "sq_pool_bytes_rows")
    return out.value


def sq_pool_create(n_slots, n_heads, d_k, d_v, head_bits, gate, dev_buf, nbytes=None,
                   row_bits=None) -> int:
    """Wrap a caller-owned device buffer (tensor or pointer); returns the handle."""
    d, keep = _desc(n_slots, n_heads, d_k, d_v, head_bits, gate)
    rb = _row_bits(row_bits)
    if nbytes is None:
        nbytes = dev_buf.numel() * dev_buf.element_size()
    h = ctypes.c_void_p(0)
    if rb is None:
        _check(lib().sq_pool_create(ctypes.byref(d), _ptr(dev_buf), int(nbytes),
                                    ctypes.byref(h)), "sq_pool_create")
    else:
        _check(lib().sq_pool_create_rows(ctypes.byref(d), rb, _ptr(dev_buf), int(nbytes),
                                         ctypes.byref(h)), "sq_pool_create_rows")
    return h.value


def sq_pool_destroy(handle) -> None:
    _check(lib().sq_pool_destroy(handle), "sq_pool_destroy")


def sq_pool_layout(handle, n_heads: int):
    stride = ctypes.c_int64(0)
    off = (ctypes.c_int64 * n_heads)()
    rec = (ctypes.c_int64 * n_heads)()
    _check(lib().sq_pool_layout(handle, ctypes.byref(stride), off, rec), "sq_pool_layout")
    return stride.value, list(off), list(rec)


def sq_quant_state(handle, slot_idx, n: int, S, stream=None) -> None:
    _check(lib().sq_quant_state(handle, _ptr(slot_idx), int(n), _ptr(S), _stream(stream)),
           "sq_quant_state")


def sq_dequant_state(handle, slot_idx, n: int, S, stream=None) -> None:
    _check(lib().sq_dequant_state(handle, _ptr(slot_idx), int(n), _ptr(S), _stream(stream)),
           "sq_dequant_state")


def sq_decode_step(handle, slot_idx, n: int, q, k, v, beta, g, y, in_dtype=None, y_dtype=None,
                   stream=None) -> None:
    in_dtype = _dtype_code(q) if in_dtype is None else in_dtype
    y_dtype = _dtype_code(y) if y_dtype is None else y_dtype
    _check(lib().sq_decode_step(handle, _ptr(slot_idx), int(n), _ptr(q), _ptr(k), _ptr(v),
                                _ptr(beta), _ptr(g), in_dtype, _ptr(y), y_dtype,
                                _stream(stream)), "sq_decode_step")


def sq_pool_set_row_impact(handle, impact) -> None:
    """impact: device tensor [n_heads, d_k] fp32 (kept alive by the caller), or None."""
    _check(lib().sq_pool_set_row_impact(handle, _ptr(impact)), "sq_pool_set_row_impact")


def sq_decode_update(handle, slot_idx, n: int, q, k, v, beta, g, y, S_out, in_dtype=None,
                     y_dtype=None, stream=None) -> None:
    in_dtype = _dtype_code(q) if in_dtype is None else in_dtype
    y_dtype = _dtype_code(y) if y_dtype is None else y_dtype
    _check(lib().sq_decode_update(handle, _ptr(slot_idx), int(n), _ptr(q), _ptr(k), _ptr(v),
                                  _ptr(beta), _ptr(g), in_dtype, _ptr(y), y_dtype, _ptr(S_out),
                                  _stream(stream)), "sq_decode_update")


def sq_split_step_noalloc(handle, slot_idx, n: int, q, k, v, beta, g, y, in_dtype=None,
                          y_dtype=None, stream=None) -> None:
    in_dtype = _dtype_code(q) if in_dtype is None else in_dtype
    y_dtype = _dtype_code(y) if y_dtype is None else y_dtype
    _check(lib().sq_split_step_noalloc(handle, _ptr(slot_idx), int(n), _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(beta), _ptr(g), in_dtype, _ptr(y), y_dtype,
                                       _stream(stream)), "sq_split_step_noalloc")


def sq_f32_decode_step(state, n_slots, n_heads, d_k, d_v, gate, slot_idx, n, q, k, v, beta, g,
                       y, in_dtype=None, y_dtype=None, stream=None) -> None:
    in_dtype = _dtype_code(q) if in_dtype is None else in_dtype
    y_dtype = _dtype_code(y) if y_dtype is None else y_dtype
    _check(lib().sq_f32_decode_step(_ptr(state), int(n_slots), int(n_heads), int(d_k), int(d_v),
                                    int(gate), _ptr(slot_idx), int(n), _ptr(q), _ptr(k), _ptr(v),
                                    _ptr(beta), _ptr(g), in_dtype, _ptr(y), y_dtype,
                                    _stream(stream)), "sq_f32_decode_step")


def sq_check_slots(handle, slot_idx, n: int, stream=None) -> None:
    _check(lib().sq_check_slots(handle, _ptr(slot_idx), int(n), _stream(stream)),
           "sq_check_slots")


def sq_device_copy(src, dst, nbytes: int, stream=None) -> None:
    """Streaming copy of nbytes between two device buffers (measurement helper)."""
    _check(lib().sq_device_copy(_ptr(src), _ptr(dst), int(nbytes), _stream(stream)),
           "sq_device_copy")


# Opcode classes of sq_issue_probe and the operations one launch performs.
SQ_PROBE_FMA_F32, SQ_PROBE_MUL_F32, SQ_PROBE_MAX3_F32, SQ_PROBE_CVT_BYTE = 0, 1, 2, 3
SQ_PROBE_BFE, SQ_PROBE_ALIGNBIT, SQ_PROBE_FMA_F64, SQ_PROBE_FMA_CVT_PAIR = 4, 5, 6, 7
SQ_PROBE_COUNT = 8
SQ_PROBE_OPS_PER_LAUNCH = 17179869184
SQ_SPLIT_SCRATCH_BYTES = 64 << 20   # the static per-GPU buffer of sq_split_step_noalloc


def sq_issue_probe(op: int, sink, stream=None) -> None:
    """One launch of the issue-rate probe of opcode class op (measurement
    helper); sink: a device tensor of at least 4 bytes, never written in
    practice."""
    _check(lib().sq_issue_probe(int(op), _ptr(sink), _stream(stream)), "sq_issue_probe")


def sq_arith_selfcheck(counts, stream=None) -> None:
    """counts: a device tensor of 4 int64 that receives the mismatch counts."""
    _check(lib().sq_arith_selfcheck(_ptr(counts), _stream(stream)), "sq_arith_selfcheck")


def seq_desc(n_seq, n_tokens, n_heads, d, gate, in_dtype, y_dtype, n_key_heads=None, q_stride=0,
             k_stride=0, v_stride=0) -> _SeqDesc:
    """The descriptor of the sequence calls (gate and dtypes: the ABI's codes)."""
    return _SeqDesc(int(n_seq), int(n_heads), int(n_key_heads or n_heads), int(d), int(d),
                    int(n_tokens), int(gate), int(in_dtype), int(y_dtype), int(q_stride),
                    int(k_stride), int(v_stride))


def sq_chunk_bytes(desc, train: bool = False):
    """Bytes of `work` for sq_chunk_forward; train: (work, save), for the backward pass too."""
    work, save = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().sq_chunk_bytes(ctypes.byref(desc), ctypes.byref(work),
                                ctypes.byref(save) if train else None), "sq_chunk_bytes")
    return (work.value, save.value) if train else work.value


def _bytes(x, given) -> int:
    return int(given) if given is not None else 0 if x is None else x.numel() * x.element_size()


def sq_chunk_forward(desc, cu, q, k, v, beta, g, S0, y, S_out, save, work, save_bytes=None,
                     work_bytes=None, stream=None) -> None:
    """q, k, v: pointers, or tensors whose token strides the descriptor holds."""
    _check(lib().sq_chunk_forward(ctypes.byref(desc), _ptr(cu), _data(q), _data(k), _data(v),
                                  _ptr(beta), _ptr(g), _ptr(S0), _ptr(y), _ptr(S_out), _ptr(save),
                                  _bytes(save, save_bytes), _ptr(work), _bytes(work, work_bytes),
                                  _stream(stream)), "sq_chunk_forward")


def sq_chunk_backward(desc, cu, q, k, v, beta, g, dy, dS_out, save, dq, dk, dv, dbeta, dg, dS0,
                      work, save_bytes=None, work_bytes=None, stream=None) -> None:
    _check(lib().sq_chunk_backward(ctypes.byref(desc), _ptr(cu), _data(q), _data(k), _data(v),
                                   _ptr(beta), _ptr(g), _ptr(dy), _ptr(dS_out), _ptr(save),
                                   _bytes(save, save_bytes), _ptr(dq), _ptr(dk), _ptr(dv),
                                   _ptr(dbeta), _ptr(dg), _ptr(dS0), _ptr(work),
                                   _bytes(work, work_bytes), _stream(stream)),
           "sq_chunk_backward")


def _data(x) -> Optional[int]:
    """Raw pointer of an int or of a tensor of any strides."""
    return x if x is None or isinstance(x, int) else x.data_ptr()


def sq_window_update(handle, slot_idx, n: int, length: int, lens, n_key_heads: int, q, k, v, beta,
                     g, y, S_out, in_dtype=None, y_dtype=None, stream=None) -> None:
    in_dtype = _dtype_code(k) if in_dtype is None else in_dtype
    y_dtype = (in_dtype if y is None else _dtype_code(y)) if y_dtype is None else y_dtype
    _check(lib().sq_window_update(handle, _ptr(slot_idx), int(n), int(length), _ptr(lens),
                                  int(n_key_heads), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                  _ptr(g), in_dtype, _ptr(y), y_dtype, _ptr(S_out),
                                  _stream(stream)), "sq_window_update")


def sq_f32_window_update(state, n_slots, n_heads, n_key_heads, d_k, d_v, gate, slot_idx, n, length,
                         lens, q, k, v, beta, g, y, S_out, in_dtype=None, y_dtype=None,
                         stream=None) -> None:
    in_dtype = _dtype_code(k) if in_dtype is None else in_dtype
    y_dtype = (in_dtype if y is None else _dtype_code(y)) if y_dtype is None else y_dtype
    _check(lib().sq_f32_window_update(_ptr(state), int(n_slots), int(n_heads), int(n_key_heads),
                                      int(d_k), int(d_v), int(gate), _ptr(slot_idx), int(n),
                                      int(length), _ptr(lens), _ptr(q), _ptr(k), _ptr(v),
                                      _ptr(beta), _ptr(g), in_dtype, _ptr(y), y_dtype,
                                      _ptr(S_out), _stream(stream)), "sq_f32_window_update")


SQ_WINDOW_MAX = 16


def _window_need(slot_idx, q, k, v, beta, g, y, S_out, lens, H, d, kda):
    """Shapes of a window's tensors; returns n, length and the key heads."""
    import torch
    n = slot_idx.numel()
    if k.dim() != 4 or k.shape[0] != n:
        raise ValueError("k must be [n, length, n_key_heads, d]")
    length, hk, dt = k.shape[1], k.shape[2], (k.dtype,)
    if k.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("k must be float32 or bfloat16")
    _need(slot_idx, "slot_idx", n, (torch.int32,))
    _need(k, "k", n * length * hk * d, dt)
    if y is not None:
        _need(q, "q", n * length * hk * d, dt)
        _need(y, "y", n * length * H * d, (torch.float32, torch.bfloat16))
    _need(v, "v", n * length * H * d, dt)
    _need(beta, "beta", n * length * H, dt)
    _need(g, "g", n * length * H * (d if kda else 1), dt)
    if S_out is not None:
        _need(S_out, "S_out", n * H * d * d, (torch.float32,))
    if lens is not None:
        _need(lens, "lens", n, (torch.int32,))
    return n, length, hk


def f32_window_update(state, slot_idx, q, k, v, beta, g, y=None, S_out=None, lens=None, gate="gdn",
                      stream=None) -> None:
    """A window of tokens per request on an fp32 state pool [n_slots, n_heads, d, d], which is
    only read; see StatePool.window_update."""
    import torch
    n_slots, H, d, _ = state.shape
    _need(state, "state", n_slots * H * d * d, (torch.float32,))
    n, length, hk = _window_need(slot_idx, q, k, v, beta, g, y, S_out, lens, H, d, gate == "kda")
    sq_f32_window_update(state, n_slots, H, hk, d, d, SQ_GATE_KDA if gate == "kda" else SQ_GATE_GDN,
                         slot_idx, n, length, lens, q, k, v, beta, g, y, S_out, stream=stream)


class ChunkedDelta:
    """The gated Delta rule over whole sequences, with its workspace.

    Holds a workspace for batches of up to n_seq sequences and n_tokens tokens
    in all; a call may bring fewer.  With train=True, also what backward needs
    of the last forward call, which it belongs to: a second forward takes the
    first one's place, and backward refuses the number of any call but the last.
    Calls that may overlap (on several streams) need an object each.  q, k: [tokens, n_key_heads, d] and
    v: [tokens, n_heads, d] may be parts of one wider tensor; every other tensor
    is contiguous."""

    def __init__(self, n_seq: int, n_tokens: int, n_heads: int, d: int, gate: str = "gdn",
                 n_key_heads=None, dtype=None, y_dtype=None, device="cuda", train=False):
        import torch
        codes = {torch.float32: SQ_F32, torch.bfloat16: SQ_BF16}
        self.dtype = torch.bfloat16 if dtype is None else dtype
        self.y_dtype = self.dtype if y_dtype is None else y_dtype
        if self.dtype not in codes or self.y_dtype not in codes:
            raise TypeError("dtype and y_dtype must be float32 or bfloat16")
        self.n_seq, self.n_tokens = int(n_seq), int(n_tokens)
        self.n_heads, self.d = int(n_heads), int(d)
        self.n_key_heads = int(n_key_heads or n_heads)
        self.gate = SQ_GATE_KDA if gate == "kda" else SQ_GATE_GDN
        self._codes = (codes[self.dtype], codes[self.y_dtype])
        work, save = sq_chunk_bytes(self._desc(n_seq, n_tokens), train=True)
        if not train:
            work, save = sq_chunk_bytes(self._desc(n_seq, n_tokens)), None
        self.calls, self._sizes = 0, None  # forward calls so far, and the last one's batch
        self.work = torch.empty(max(256, work), dtype=torch.uint8, device=device)
        self.save = None if save is None else torch.empty(max(256, save), dtype=torch.uint8,
                                                          device=device)

    def _desc(self, n_seq, n_tokens, qs=0, ks=0, vs=0):
        return seq_desc(n_seq, n_tokens, self.n_heads, self.d, self.gate, self._codes[0],
                        self._codes[1], self.n_key_heads, qs, ks, vs)

    def _tokens(self, name, t, n, heads):
        """Token stride of q, k or v: [n, heads, d] with dense heads."""
        if t.shape != (n, heads, self.d) or not t.is_cuda or t.dtype != self.dtype:
            raise ValueError("%s must be a %s device tensor of shape %s, got %s %s" % (
                name, self.dtype, (n, heads, self.d), t.dtype, tuple(t.shape)))
        if t.stride(2) != 1 or (heads > 1 and t.stride(1) != self.d):
            raise ValueError("the heads of %s must be dense" % name)
        if n > 1 and t.stride(0) < heads * self.d:  # an expanded tensor's 0 would mean dense
            raise ValueError("the tokens of %s must not overlap" % name)
        return t.stride(0) if n > 1 else 0

    def _args(self, q, k, v, beta, g, cu, S0):
        import torch
        n_seq, n, H, d = cu.numel() - 1, q.shape[0], self.n_heads, self.d
        if n_seq < 0:
            raise ValueError("cu needs one entry more than there are sequences")
        desc = self._desc(n_seq, n, self._tokens("q", q, n, self.n_key_heads),
                          self._tokens("k", k, n, self.n_key_heads), self._tokens("v", v, n, H))
        _need(cu, "cu", n_seq + 1, (torch.int32,))
        _need(beta, "beta", n * H, (self.dtype,))
        _need(g, "g", n * H * (d if self.gate == SQ_GATE_KDA else 1), (self.dtype,))
        if S0 is not None:
            _need(S0, "S0", n_seq * H * d * d, (torch.float32,))
        return desc, n_seq, n

    def forward(self, q, k, v, beta, g, cu, y, S0=None, S_out=None, stream=None):
        """y and, where given, the final states S_out [n_seq, n_heads, d, d]; cu: int32
        [n_seq + 1] on the device, the tokens at which the sequences begin and end.
        Returns the call's number, for backward."""
        import torch
        desc, n_seq, n = self._args(q, k, v, beta, g, cu, S0)
        _need(y, "y", n * self.n_heads * self.d, (self.y_dtype,))
        if S_out is not None:
            _need(S_out, "S_out", n_seq * self.n_heads * self.d * self.d, (torch.float32,))
        sq_chunk_forward(desc, cu, q, k, v, beta, g, S0, y, S_out, self.save, self.work,
                         stream=stream)
        self.calls, self._sizes = self.calls + 1, (n_seq, n)
        return self.calls

    def backward(self, q, k, v, beta, g, cu, dy, dq, dk, dv, dbeta, dg, S0=None, dS_out=None,
                 dS0=None, call=None, stream=None):
        """Gradients of the last forward call, which had the same inputs; dy and every gradient in
        `dtype` and contiguous, dS_out and dS0 [n_seq, n_heads, d, d] fp32 or None.  call: what
        that forward returned; raises RuntimeError where another one came after it."""
        import torch
        if self.save is None:
            raise ValueError("backward needs train=True")
        desc, n_seq, n = self._args(q, k, v, beta, g, cu, S0)
        if self.calls == 0 or (call is not None and call != self.calls):
            raise RuntimeError("backward of forward call %s, but the saved states are of call %d" % (
                "?" if call is None else call, self.calls))
        if self._sizes != (n_seq, n):
            raise RuntimeError("the last forward call had %d sequences of %d tokens, not %d of %d" % (
                *self._sizes, n_seq, n))
        H, hk, d, dt = self.n_heads, self.n_key_heads, self.d, (self.dtype,)
        for name, t, numel in (("dy", dy, n * H * d), ("dq", dq, n * hk * d), ("dk", dk, n * hk * d),
                               ("dv", dv, n * H * d), ("dbeta", dbeta, n * H),
                               ("dg", dg, n * H * (d if self.gate == SQ_GATE_KDA else 1))):
            _need(t, name, numel, dt)
        for name, t in (("dS_out", dS_out), ("dS0", dS0)):
            if t is not None:
                _need(t, name, n_seq * H * d * d, (torch.float32,))
        sq_chunk_backward(desc, cu, q, k, v, beta, g, dy, dS_out, self.save, dq, dk, dv, dbeta, dg,
                          dS0, self.work, stream=stream)


SQ_DRAFT_MAX = 32


def sq_verify_bytes(n: int, m: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().sq_verify_bytes(int(n), int(m), ctypes.byref(out)), "sq_verify_bytes")
    return out.value


def sq_verify_draft(n, m, vocab, target, target_stride, draft, draft_stride, tokens, lens, accept_u,
                    sample_e, temperature, accepted, next_token, work, work_bytes=None,
                    logits_dtype=None, stream=None) -> None:
    """target, draft: pointers, or tensors whose row strides the arguments hold."""
    logits_dtype = _dtype_code(target) if logits_dtype is None else logits_dtype
    if work_bytes is None:
        work_bytes = work.numel() * work.element_size()
    _check(lib().sq_verify_draft(int(n), int(m), int(vocab), _data(target), int(target_stride),
                                 _data(draft), int(draft_stride), logits_dtype, _ptr(tokens),
                                 _ptr(lens), _ptr(accept_u), _ptr(sample_e), float(temperature),
                                 _ptr(accepted), _ptr(next_token), _ptr(work), int(work_bytes),
                                 _stream(stream)), "sq_verify_draft")


class DraftVerifier:
    """sq_verify_draft with its workspace, for up to n requests of up to m drafted tokens.
    Calls that may overlap (on several streams) need an object each."""

    def __init__(self, n: int, m: int, vocab: int, device="cuda"):
        import torch
        self.n, self.m, self.vocab = int(n), int(m), int(vocab)
        self.work = torch.empty(max(256, sq_verify_bytes(n, m)), dtype=torch.uint8, device=device)

    def _rows(self, name, t, n, m, dtype):
        """Stride of the rows of logits [n, m, vocab], whose rows may be padded."""
        if t.shape != (n, m, self.vocab) or not t.is_cuda or t.dtype != dtype:
            raise ValueError("%s must be a %s device tensor of shape %s, got %s %s" % (
                name, dtype, (n, m, self.vocab), t.dtype, tuple(t.shape)))
        stride = t.stride(1) if m > 1 else t.stride(0)
        if (self.vocab > 1 and t.stride(2) != 1) or (n > 1 and m > 1 and t.stride(0) != m * stride):
            raise ValueError("the rows of %s must be evenly spaced and dense" % name)
        if n * m > 1 and stride < self.vocab:  # an expanded tensor's 0 would mean dense
            raise ValueError("the rows of %s must not overlap" % name)
        return stride if n * m > 1 else 0

    def verify(self, target, tokens, accepted, next_token, draft=None, accept_u=None,
               sample_e=None, lens=None, temperature=1.0, stream=None):
        """target: logits [n, m + 1, vocab]; tokens: int32 [n, m]; accepted, next_token: int32 [n],
        the outputs; the rest as sq_verify_draft."""
        import torch
        f32, i32 = (torch.float32,), (torch.int32,)
        if target.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("target must be float32 or bfloat16")
        n, m = target.shape[0], target.shape[1] - 1
        ts = self._rows("target", target, n, m + 1, target.dtype)
        ds = 0 if draft is None else self._rows("draft", draft, n, m, target.dtype)
        _need(tokens, "tokens", n * m, i32)
        _need(accepted, "accepted", n, i32)
        _need(next_token, "next_token", n, i32)
        if lens is not None:
            _need(lens, "lens", n, i32)
        if temperature:
            _need(accept_u, "accept_u", n * m, f32)
            _need(sample_e, "sample_e", n * self.vocab, f32)
        sq_verify_draft(n, m, self.vocab, target, ts, draft, ds, tokens, lens, accept_u, sample_e,
                        temperature, accepted, next_token, self.work, stream=stream)


class StatePool:
    """A packed state pool in a torch-owned device buffer.

    Convenience wrapper: allocates ``sq_pool_bytes`` bytes with torch on the
    given device, creates the pool handle and exposes the ABI calls."""

    def __init__(self, n_slots: int, n_heads: int, d: int, head_bits, gate: str = "gdn",
                 device="cuda", row_bits=None):
        """row_bits: [n_heads][d] key-row widths for the heads whose head_bits is 0."""
        import torch
        self.n_slots, self.n_heads, self.d = int(n_slots), int(n_heads), int(d)
        self.head_bits = [int(b) for b in head_bits]
        self.row_bits = None if row_bits is None else [[int(b) for b in r] for r in row_bits]
        self.gate = SQ_GATE_KDA if gate == "kda" else SQ_GATE_GDN
        nbytes = sq_pool_bytes(n_slots, n_heads, d, d, self.head_bits, self.gate, self.row_bits)
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.handle = sq_pool_create(n_slots, n_heads, d, d, self.head_bits, self.gate, self.buf,
                                     nbytes, self.row_bits)
        self.slot_stride, self.head_off, self.record_bytes = sq_pool_layout(self.handle, n_heads)

    def _step_args(self, slot_idx, q, k, v, beta, g, y):
        import torch
        n, H, d = slot_idx.numel(), self.n_heads, self.d
        _need(slot_idx, "slot_idx", n, (torch.int32,))
        dt = (q.dtype,)
        if q.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("q must be float32 or bfloat16")
        for name, t in (("q", q), ("k", k), ("v", v)):
            _need(t, name, n * H * d, dt)
        _need(beta, "beta", n * H, dt)
        _need(g, "g", n * H * (d if self.gate == SQ_GATE_KDA else 1), dt)
        _need(y, "y", n * H * d, (torch.float32, torch.bfloat16))

    def quant_state(self, slot_idx, S, stream=None):
        import torch
        n = slot_idx.numel()
        _need(slot_idx, "slot_idx", n, (torch.int32,))
        _need(S, "S", n * self.n_heads * self.d * self.d, (torch.float32,))
        sq_quant_state(self.handle, slot_idx, n, S, stream)

    def dequant_state(self, slot_idx, S=None, stream=None):
        import torch
        n = slot_idx.numel()
        if S is None:
            S = torch.empty((n, self.n_heads, self.d, self.d), dtype=torch.float32,
                            device=self.buf.device)
        _need(slot_idx, "slot_idx", n, (torch.int32,))
        _need(S, "S", n * self.n_heads * self.d * self.d, (torch.float32,))
        sq_dequant_state(self.handle, slot_idx, n, S, stream)
        return S

    def decode_step(self, slot_idx, q, k, v, beta, g, y, stream=None):
        self._step_args(slot_idx, q, k, v, beta, g, y)
        sq_decode_step(self.handle, slot_idx, slot_idx.numel(), q, k, v, beta, g, y,
                       stream=stream)

    def set_row_impact(self, impact):
        """Requantize with the key-row-aware fit from now on (impact: [H, d_k]
        fp32 device tensor, > 0), or with the closed rule (None)."""
        if impact is not None:
            impact = impact.contiguous()
            assert impact.shape == (self.n_heads, self.d) and impact.is_cuda
        self.impact = impact  # the library keeps only the pointer
        sq_pool_set_row_impact(self.handle, impact)

    def decode_update(self, slot_idx, q, k, v, beta, g, y, S_out, stream=None):
        """Split step, first half: y and S' (fp32) out, pool unchanged; store
        with quant_state(slot_idx, S_out) afterwards."""
        import torch
        self._step_args(slot_idx, q, k, v, beta, g, y)
        _need(S_out, "S_out", slot_idx.numel() * self.n_heads * self.d * self.d, (torch.float32,))
        sq_decode_update(self.handle, slot_idx, slot_idx.numel(), q, k, v, beta, g, y, S_out,
                         stream=stream)

    def split_step_noalloc(self, slot_idx, q, k, v, beta, g, y, stream=None):
        """Split step with S' in the library's static buffer: no allocation."""
        self._step_args(slot_idx, q, k, v, beta, g, y)
        sq_split_step_noalloc(self.handle, slot_idx, slot_idx.numel(), q, k, v, beta, g, y,
                              stream=stream)

    def window_update(self, slot_idx, q, k, v, beta, g, y=None, S_out=None, lens=None,
                      stream=None):
        """A window of up to SQ_WINDOW_MAX tokens per request, the pool only read.

        q, k: [n, length, n_key_heads, d], v: [n, length, H, d]; y: the read-outs, S_out: the
        fp32 states after each request's first lens tokens (all of them where lens is None);
        store them with quant_state(slot_idx, S_out).  Either of y and S_out may be None (q too
        where y is)."""
        n, length, hk = _window_need(slot_idx, q, k, v, beta, g, y, S_out, lens, self.n_heads,
                                     self.d, self.gate == SQ_GATE_KDA)
        sq_window_update(self.handle, slot_idx, n, length, lens, hk, q, k, v, beta, g, y, S_out,
                         stream=stream)

    def check_slots(self, slot_idx, stream=None):
        sq_check_slots(self.handle, slot_idx, slot_idx.numel(), stream)

    def close(self):
        if getattr(self, "handle", None):
            sq_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
