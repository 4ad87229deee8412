"""Argument checks of the short convolution, the selective scan and the norms: every call here is
refused on the host (or is a no-op) before any work is enqueued, so no GPU is needed."""
import math

import pytest

import quantized_gated_delta_amd as Q
from quantized_gated_delta_amd import block as B

P = 0x7F0000000000   # 256-byte aligned, never dereferenced on the host
STEP = 1 << 36       # apart from each other
BIG = 1 << 40


def at(i):
    return P + i * STEP


def refused(status, text, fn, *args, **kw):
    with pytest.raises(Q.SQError) as e:
        fn(*args, **kw)
    assert e.value.status == status, (e.value.status, e.value.text)
    assert text in e.value.text, e.value.text


# ------------------------------------------------------------------ convolution
def conv_desc(**kw):
    return Q.conv_desc(**{**dict(n_seq=2, n_tokens=100, n_channels=64, width=4, act=Q.SQ_ACT_SILU, dtype=Q.SQ_BF16, x_stride=0), **kw})


def conv_forward(dsc=None, **kw):
    a = dict(cu=at(0), x=at(1), weight=at(2), bias=at(3), S0=at(4), y=at(5), S_out=at(6))
    Q.sq_conv_forward(dsc or conv_desc(), stream=0, **{**a, **kw})


def conv_backward(dsc=None, **kw):
    a = dict(cu=at(0), x=at(1), weight=at(2), bias=at(3), S0=at(4), dy=at(5), dS_out=at(6), dx=at(7), dweight=at(8), dbias=at(9), dS0=at(10), work=at(11), work_bytes=BIG)
    Q.sq_conv_backward(dsc or conv_desc(), stream=0, **{**a, **kw})


def conv_step(dsc=None, **kw):
    a = dict(pool=at(0), n_slots=9, slot_idx=at(1), n=4, x=at(2), weight=at(3), bias=at(4), y=at(5))
    Q.sq_conv_step(dsc or conv_desc(), stream=0, **{**a, **kw})


@pytest.mark.parametrize("kw,status,text", [
    (dict(n_seq=-1), Q.SQ_EINVAL, "n_seq"), (dict(n_tokens=-1), Q.SQ_EINVAL, "n_tokens"), (dict(n_tokens=(1 << 31) - 1), Q.SQ_EUNSUPPORTED, "n_tokens"),
    (dict(n_channels=0), Q.SQ_EINVAL, "n_channels"), (dict(width=1), Q.SQ_EUNSUPPORTED, "width"), (dict(width=5), Q.SQ_EUNSUPPORTED, "width"),
    (dict(act=Q.SQ_ACT_SIGMOID), Q.SQ_EUNSUPPORTED, "act"), (dict(dtype=7), Q.SQ_EINVAL, "dtype"), (dict(x_stride=63), Q.SQ_EINVAL, "x_stride"),
    (dict(x_stride=-64), Q.SQ_EINVAL, "x_stride"), (dict(x_stride=(1 << 24) + 1), Q.SQ_EINVAL, "x_stride"),
    (dict(n_channels=(1 << 23) + 1), Q.SQ_EINVAL, "n_channels"), (dict(n_tokens=1 << 30), Q.SQ_EUNSUPPORTED, "grid"),
    (dict(n_seq=1 << 24), Q.SQ_EUNSUPPORTED, "grid")], ids=str)
def test_conv_descriptor(kw, status, text):
    refused(status, text, Q.sq_conv_bytes, conv_desc(**kw))
    refused(status, text, conv_forward, conv_desc(**kw))
    refused(status, text, conv_backward, conv_desc(**kw))


@pytest.mark.parametrize("call,required,optional", [
    (conv_forward, ["cu", "x", "weight", "y"], ["bias", "S0", "S_out"]),
    (conv_backward, ["cu", "x", "weight", "dy", "dx", "dweight", "work"], ["bias", "S0", "dS_out", "dbias", "dS0"]),
    (conv_step, ["pool", "slot_idx", "x", "weight", "y"], ["bias"])], ids=["forward", "backward", "step"])
def test_conv_pointers(call, required, optional):
    for name in required:
        refused(Q.SQ_EINVAL, name, call, **{name: None})
    for name in required + optional:
        refused(Q.SQ_EINVAL, name, call, **{name: P + 63 * STEP + 1})


def test_conv_overlaps():
    refused(Q.SQ_EINVAL, "overlap", conv_forward, y=at(1))
    refused(Q.SQ_EINVAL, "overlap", conv_forward, y=at(1) + 2 * 64 * 99)
    refused(Q.SQ_EINVAL, "overlap", conv_forward, S_out=at(4))
    refused(Q.SQ_EINVAL, "overlap", conv_backward, dx=at(5))
    refused(Q.SQ_EINVAL, "overlap", conv_backward, dS0=at(6))
    refused(Q.SQ_EINVAL, "overlap", conv_step, y=at(0))
    refused(Q.SQ_EINVAL, "overlap", conv_step, y=at(0) + 2 * 9 * 3 * 64 - 4)


def test_conv_sizes():
    need = Q.sq_conv_bytes(conv_desc())
    refused(Q.SQ_ENOMEM, "work", conv_backward, work_bytes=need - 1)
    most = Q.sq_conv_bytes(conv_desc(n_tokens=100000, n_seq=50))
    assert all(Q.sq_conv_bytes(conv_desc(n_tokens=t, n_seq=s)) <= most for t in (0, 1, 63, 100, 5000, 99999) for s in (0, 1, 49))
    for kw, text in ((dict(n_slots=0), "n_slots"), (dict(n=-1), "n must")):
        refused(Q.SQ_EINVAL, text, conv_step, **kw)
    refused(Q.SQ_EUNSUPPORTED, "grid", conv_step, n=1 << 27)


@pytest.mark.parametrize("width", [2, 4])
@pytest.mark.parametrize("channels", [64, 2048, 8192, 10240, 65536, 1 << 21], ids=str)
def test_the_largest_batchs_convolution_workspace_serves_smaller_ones(channels, width):
    """Also where a batch's blocks of 128 tokens are just more than one, two or three turns of the workgroups."""
    size = lambda t, s: Q.sq_conv_bytes(conv_desc(n_tokens=t, n_seq=s, n_channels=channels, width=width))  # noqa: E731
    turn = max(1, 4096 // (-(-channels // 256)))
    for slots in (turn - 1, turn, turn + 1, 2 * turn, 2 * turn + 1, 3 * turn + 2):
        most = size(slots * 128, 4)
        for t in {0, 1, 5000} | {(k * turn + j) * 128 for k in (1, 2, 3) for j in (-5, -4, -1, 0, 1)}:
            for s in (0, 1, 3, 4):
                if 0 <= t <= slots * 128:
                    assert size(t, s) <= most, (slots, t, s)
        for s in (1, turn // 2, turn, turn + 1, slots):  # as many short sequences
            assert size(0, min(s, slots)) <= size(0, slots), (slots, s)


def test_conv_no_ops():
    none = conv_desc(n_seq=0, n_tokens=0)
    conv_forward(none, cu=None, x=None, y=None)
    conv_backward(none, cu=None, x=None, dy=None, dx=None, dweight=None, dbias=None, work=None)
    conv_step(n=0, pool=None, slot_idx=None, x=None, y=None)


# ------------------------------------------------------------------ scan
def scan_desc(**kw):
    return Q.scan_desc(**{**dict(n_seq=2, n_tokens=100, n_heads=4, d_head=64, d_state=128, n_groups=2), **kw})


def scan_forward(dsc=None, **kw):
    a = dict(cu=at(0), x=at(1), raw=at(2), A=at(3), B=at(4), C=at(5), D=at(6), dt_bias=at(7), S0=at(8), y=at(9), S_out=at(10), save=at(11), work=at(12),
             save_bytes=BIG, work_bytes=BIG)
    Q.sq_scan_forward(dsc or scan_desc(), stream=0, **{**a, **kw})


def scan_backward(dsc=None, **kw):
    a = dict(cu=at(0), x=at(1), raw=at(2), A=at(3), B=at(4), C=at(5), D=at(6), dt_bias=at(7), dy=at(8), dS_out=at(9), save=at(10), dx=at(11), draw=at(12), dA=at(13),
             dB=at(14), dC=at(15), dD=at(16), ddt_bias=at(17), dS0=at(18), work=at(19), save_bytes=BIG, work_bytes=BIG)
    Q.sq_scan_backward(dsc or scan_desc(), stream=0, **{**a, **kw})


def scan_step(dsc=None, **kw):
    a = dict(state_pool=at(0), n_slots=9, slot_idx=at(1), n=4, x=at(2), raw=at(3), A=at(4), B=at(5), C=at(6), D=at(7), dt_bias=at(8), y=at(9))
    Q.sq_scan_step(dsc or scan_desc(), stream=0, **{**a, **kw})


@pytest.mark.parametrize("kw,status,text", [
    (dict(n_seq=-1), Q.SQ_EINVAL, "n_seq"), (dict(n_tokens=-1), Q.SQ_EINVAL, "n_tokens"), (dict(n_tokens=(1 << 31) - 1), Q.SQ_EUNSUPPORTED, "n_tokens"),
    (dict(n_heads=0), Q.SQ_EINVAL, "n_heads"), (dict(n_heads=16385, n_groups=1), Q.SQ_EINVAL, "n_heads"), (dict(n_groups=3), Q.SQ_EINVAL, "n_groups"),
    (dict(n_groups=0), Q.SQ_EINVAL, "n_groups"), (dict(d_state=16), Q.SQ_EUNSUPPORTED, "d_state"), (dict(d_head=32), Q.SQ_EUNSUPPORTED, "d_head"),
    (dict(softplus=2), Q.SQ_EINVAL, "softplus"), (dict(in_dtype=5), Q.SQ_EINVAL, "in_dtype"), (dict(y_dtype=5), Q.SQ_EINVAL, "y_dtype"),
    (dict(x_stride=255), Q.SQ_EINVAL, "x_stride"), (dict(x_stride=260), Q.SQ_EINVAL, "x_stride"), (dict(b_stride=252), Q.SQ_EINVAL, "b_stride"),
    (dict(c_stride=1 << 25), Q.SQ_EINVAL, "c_stride"), (dict(dt_stride=3), Q.SQ_EINVAL, "dt_stride"), (dict(dx_stride=257), Q.SQ_EINVAL, "dx_stride"),
    (dict(ddt_stride=-1), Q.SQ_EINVAL, "ddt_stride"), (dict(db_stride=257), Q.SQ_EINVAL, "db_stride"), (dict(dc_stride=257), Q.SQ_EINVAL, "dc_stride"),
    (dict(n_tokens=1 << 30, n_heads=16384), Q.SQ_EUNSUPPORTED, "grid"), (dict(n_seq=1 << 22), Q.SQ_EUNSUPPORTED, "grid")], ids=str)
def test_scan_descriptor(kw, status, text):
    refused(status, text, Q.sq_scan_bytes, scan_desc(**kw))
    refused(status, text, scan_forward, scan_desc(**kw))
    refused(status, text, scan_backward, scan_desc(**kw))


@pytest.mark.parametrize("call,required,optional", [
    (scan_forward, ["cu", "x", "raw", "A", "B", "C", "y", "work"], ["D", "dt_bias", "S0", "S_out", "save"]),
    (scan_backward, ["cu", "x", "raw", "A", "B", "C", "dy", "save", "dx", "draw", "dA", "dB", "dC", "work"], ["D", "dt_bias", "dS_out", "dD", "ddt_bias", "dS0"]),
    (scan_step, ["state_pool", "slot_idx", "x", "raw", "A", "B", "C", "y"], ["D", "dt_bias"])], ids=["forward", "backward", "step"])
def test_scan_pointers(call, required, optional):
    for name in required:
        refused(Q.SQ_EINVAL, name.replace("state_", ""), call, **{name: None})
    for name in required + optional:
        refused(Q.SQ_EINVAL, name, call, **{name: P + 63 * STEP + 1})


def test_scan_overlaps():
    refused(Q.SQ_EINVAL, "overlap", scan_forward, y=at(1))
    refused(Q.SQ_EINVAL, "overlap", scan_forward, S_out=at(8) + 256)
    refused(Q.SQ_EINVAL, "overlap", scan_backward, dx=at(8))
    refused(Q.SQ_EINVAL, "overlap", scan_backward, dC=at(14) + 2 * 128)
    refused(Q.SQ_EINVAL, "overlap", scan_step, y=at(0))


def test_parts_of_one_tensor_do_not_overlap():
    """x, B and C and their gradients as parts of one wider tensor: refused for the last pair of arguments alone."""
    wide = 256 + 2 * 256
    s = dict(x_stride=wide, b_stride=wide, c_stride=wide, dx_stride=wide, db_stride=wide, dc_stride=wide)
    parts = dict(x=at(1), B=at(1) + 512, C=at(1) + 1024, dx=at(11), dB=at(11) + 512, dC=at(11) + 1024)
    refused(Q.SQ_EINVAL, "dS0 and work overlap", scan_backward, scan_desc(**s), **parts, dS0=at(19))
    refused(Q.SQ_EINVAL, "dB and dC overlap", scan_backward, scan_desc(**s), **{**parts, "dC": at(11) + 1024 - 16})
    refused(Q.SQ_EINVAL, "dx and dB overlap", scan_backward, scan_desc(**s), **{**parts, "dB": at(11) + 512 - 16})


def test_scan_sizes():
    work, save = Q.sq_scan_bytes(scan_desc(), train=True)
    refused(Q.SQ_ENOMEM, "work", scan_backward, work_bytes=work - 1)
    refused(Q.SQ_ENOMEM, "save", scan_backward, save_bytes=save - 1)
    refused(Q.SQ_ENOMEM, "work", scan_forward, work_bytes=Q.sq_scan_bytes(scan_desc()) - 1)
    refused(Q.SQ_ENOMEM, "save", scan_forward, save_bytes=save - 1)


@pytest.mark.parametrize("heads,groups", [(1, 1), (4, 2), (64, 1), (64, 8), (600, 1), (2048, 4)], ids=str)
def test_the_largest_batchs_buffers_serve_smaller_ones(heads, groups):
    size = lambda t, s: Q.sq_scan_bytes(scan_desc(n_tokens=t, n_seq=s, n_heads=heads, n_groups=groups), train=True)  # noqa: E731
    for most in (300, 5000, 70000):
        work, save = size(most, 20)
        for t in (0, 1, 64, 255, 256, 257, 511, 1023, 4097, 8191, 8192, 8193, 33000, 65537):
            if t <= most:
                for s in (0, 1, 19):
                    w, k = size(t, s)
                    assert w <= work and k <= save, (most, t, s)


def test_scan_no_ops():
    none = scan_desc(n_seq=0, n_tokens=0)
    scan_forward(none, cu=None, x=None, y=None, work=None)
    scan_backward(none, cu=None, x=None, dy=None, dx=None, work=None, dA=None, dD=None, ddt_bias=None)
    scan_step(n=0, state_pool=None, slot_idx=None, x=None, y=None)


def test_outputs_over_the_list_of_sequences():
    """A kernel that still reads cu while another workgroup writes over it would see a wrong list."""
    for out in ("y", "S_out"):
        refused(Q.SQ_EINVAL, "cu and %s overlap" % out, conv_forward, **{out: at(0)})
        refused(Q.SQ_EINVAL, "cu and %s overlap" % out, scan_forward, **{out: at(0)})
    for out in ("dx", "dweight", "dbias", "dS0", "work"):
        refused(Q.SQ_EINVAL, "cu and %s overlap" % out, conv_backward, cu=at(40) + 8, **{out: at(40)})
    for out in ("dx", "draw", "dA", "dB", "dC", "dD", "ddt_bias", "dS0", "work"):
        refused(Q.SQ_EINVAL, "cu and %s overlap" % out, scan_backward, cu=at(40) + 12, **{out: at(40)})
    for out in ("save", "work"):
        refused(Q.SQ_EINVAL, "cu and %s overlap" % out, scan_forward, cu=at(40) + 252, **{out: at(40)})


# ------------------------------------------------------------------ norms
def gate_desc(**kw):
    return Q.gated_norm_desc(**{**dict(n_tokens=10, n_groups=2, d=64), **kw})


def gate_forward(dsc=None, **kw):
    Q.sq_gated_norm_forward(dsc or gate_desc(), stream=0, **{**dict(x=at(0), z=at(1), weight=at(2), y=at(3)), **kw})


def gate_backward(dsc=None, **kw):
    a = dict(x=at(0), z=at(1), weight=at(2), dy=at(3), dx=at(4), dz=at(5), dweight=at(6), work=at(7), work_bytes=BIG)
    Q.sq_gated_norm_backward(dsc or gate_desc(), stream=0, **{**a, **kw})


@pytest.mark.parametrize("kw,status,text", [
    (dict(d=0), Q.SQ_EUNSUPPORTED, "d must"), (dict(d=16385), Q.SQ_EUNSUPPORTED, "d must"), (dict(n_groups=0), Q.SQ_EINVAL, "n_groups"),
    (dict(n_groups=65536, d=1), Q.SQ_EINVAL, "n_groups"), (dict(n_tokens=-1), Q.SQ_EINVAL, "n_tokens"), (dict(n_tokens=1 << 31), Q.SQ_EINVAL, "n_tokens"),
    (dict(eps=-1.0), Q.SQ_EINVAL, "eps"), (dict(eps=math.nan), Q.SQ_EINVAL, "eps"), (dict(eps=math.inf), Q.SQ_EINVAL, "eps"), (dict(act=9), Q.SQ_EINVAL, "act"),
    (dict(dtype=9), Q.SQ_EINVAL, "dtype"), (dict(x_stride=127), Q.SQ_EINVAL, "x_stride"), (dict(z_stride=1), Q.SQ_EINVAL, "z_stride"),
    (dict(dx_stride=-1), Q.SQ_EINVAL, "dx_stride"), (dict(dz_stride=1 << 25), Q.SQ_EINVAL, "dz_stride"), (dict(n_groups=2048, d=16384, n_tokens=1), Q.SQ_EUNSUPPORTED, "2^24")],
    ids=str)
def test_gated_descriptor(kw, status, text):
    refused(status, text, Q.sq_gated_norm_bytes, gate_desc(**kw))
    refused(status, text, gate_forward, gate_desc(**kw))
    refused(status, text, gate_backward, gate_desc(**kw))


def test_gated_pointers():
    for name in ("x", "z", "y"):
        refused(Q.SQ_EINVAL, name, gate_forward, **{name: None})
    for name in ("x", "z", "dy", "dx", "dz", "work"):
        refused(Q.SQ_EINVAL, name, gate_backward, **{name: None})
    for name in ("x", "z", "weight", "dy", "dx", "dz", "dweight", "work"):
        refused(Q.SQ_EINVAL, name, gate_backward, **{name: P + 63 * STEP + 1})
    refused(Q.SQ_EINVAL, "z", gate_forward, gate_desc(act=Q.SQ_ACT_NONE))
    refused(Q.SQ_EINVAL, "dz", gate_backward, gate_desc(act=Q.SQ_ACT_NONE), z=None)
    refused(Q.SQ_EINVAL, "overlap", gate_forward, y=at(1))
    refused(Q.SQ_EINVAL, "overlap", gate_forward, y=at(0) + 2)
    refused(Q.SQ_EINVAL, "overlap", gate_backward, dz=at(3))
    refused(Q.SQ_EINVAL, "overlap", gate_backward, gate_desc(dx_stride=136), dx=at(3))
    refused(Q.SQ_ENOMEM, "work", gate_backward, work_bytes=Q.sq_gated_norm_bytes(gate_desc()) - 1)
    gate_forward(gate_desc(n_tokens=0), x=None, z=None, y=None)


def res_forward(dsc=None, **kw):
    a = dict(o=at(0), r=at(1), post_weight=at(2), scale=at(3), weight=at(4), r_out=at(5), h=at(6))
    Q.sq_residual_norm_forward(dsc or Q.residual_norm_desc(10, 64), stream=0, **{**a, **kw})


def res_backward(dsc=None, **kw):
    a = dict(o=at(0), r=at(1), post_weight=at(2), scale=at(3), weight=at(4), dh=at(5), dr_out=at(6), d_o=at(7), dr=at(8), dpost_weight=at(9), dscale=at(10),
             dweight=at(11), work=at(12), work_bytes=BIG)
    Q.sq_residual_norm_backward(dsc or Q.residual_norm_desc(10, 64), stream=0, **{**a, **kw})


@pytest.mark.parametrize("args,status,text", [((10, 0), Q.SQ_EUNSUPPORTED, "d must"), ((10, 16385), Q.SQ_EUNSUPPORTED, "d must"), ((-1, 64), Q.SQ_EINVAL, "n_rows"),
                                              ((1 << 31, 64), Q.SQ_EINVAL, "n_rows"), ((10, 64, -1.0), Q.SQ_EINVAL, "eps"), ((10, 64, 1e-6, 9), Q.SQ_EINVAL, "dtype"),
                                              ((10, 64, 1e-6, 1, 9), Q.SQ_EINVAL, "res_dtype")], ids=str)
def test_residual_descriptor(args, status, text):
    d = Q.residual_norm_desc(*args)
    refused(status, text, Q.sq_residual_norm_bytes, d)
    refused(status, text, res_forward, d)
    refused(status, text, res_backward, d)


def test_residual_pointers():
    for name in ("o", "r_out"):
        refused(Q.SQ_EINVAL, name, res_forward, **{name: None})
    for name in ("o", "d_o", "work"):
        refused(Q.SQ_EINVAL, name, res_backward, **{name: None})
    for name in ("o", "r", "post_weight", "scale", "weight", "dh", "dr_out", "d_o", "dr", "dpost_weight", "dscale", "dweight", "work"):
        refused(Q.SQ_EINVAL, name, res_backward, **{name: P + 63 * STEP + 1})
    refused(Q.SQ_EINVAL, "dpost_weight", res_backward, post_weight=None)
    refused(Q.SQ_EINVAL, "overlap", res_forward, h=at(0))
    refused(Q.SQ_EINVAL, "overlap", res_forward, r_out=at(1) + 2)
    refused(Q.SQ_EINVAL, "overlap", res_backward, dr=at(1))
    refused(Q.SQ_EINVAL, "overlap", res_backward, d_o=at(6))
    refused(Q.SQ_EINVAL, "overlap", res_backward, dscale=at(11))
    refused(Q.SQ_ENOMEM, "work", res_backward, work_bytes=Q.sq_residual_norm_bytes(Q.residual_norm_desc(10, 64)) - 1)
    res_forward(Q.residual_norm_desc(0, 64), o=None, r_out=None)


def test_a_workspace_that_no_call_uses_is_not_held_against_it():
    """Without gradients of parameters the norms' backward pass writes no workspace: one of another size, which other tensors
    lie right behind, is no overlap.  Each call is refused for a later pair of arguments alone."""
    rows = 4000  # with gradients of parameters: 512 rows of partial sums
    behind = dict(work=at(20), work_bytes=256)
    refused(Q.SQ_EINVAL, "dy and dz overlap", gate_backward, gate_desc(n_tokens=rows), dweight=None, x=at(20) + 256, dz=at(3), **behind)
    refused(Q.SQ_EINVAL, "dr_out and d_o overlap", res_backward, Q.residual_norm_desc(rows, 64), dweight=None, dscale=None, dpost_weight=None, o=at(20) + 256,
            d_o=at(6), **behind)
    # with them it has to be large enough, which is said first
    refused(Q.SQ_ENOMEM, "work", gate_backward, gate_desc(n_tokens=rows), dy=at(20) + 256, **behind)
    refused(Q.SQ_ENOMEM, "work", res_backward, Q.residual_norm_desc(rows, 64), dh=at(20) + 256, **behind)


def test_null_descriptors():
    L = B._lib()
    for name in ("sq_conv_bytes", "sq_gated_norm_bytes", "sq_residual_norm_bytes"):
        assert getattr(L, name)(None, None) == Q.SQ_EINVAL
    assert L.sq_scan_bytes(None, None, None) == Q.SQ_EINVAL
