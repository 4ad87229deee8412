"""What the Python classes of the short convolution, the selective scan and the norms refuse before anything is
enqueued.  The tensors lie in host memory and say that they are on the device, so no GPU is needed."""
import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def device(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def bad(t):
    """Tensors that stand for t but are not: another type, one row less, a host tensor, no gaps between rows, all rows the same."""
    yield "type", t.to(torch.float16).as_subclass(OnDevice)
    yield "shape", t[:-1]
    yield "host", torch.zeros(t.shape, dtype=t.dtype)
    if t.dim() > 1:
        yield "strided", torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2].as_subclass(OnDevice)
        yield "expanded", t[:1].expand(t.shape).as_subclass(OnDevice)


def check(call, args, first, may_be_none=()):
    """Every tensor of the call in every bad form; `first` sets the sizes, so another shape of it blames another tensor."""
    for name, t in args.items():
        if t is None:
            continue
        for kind, wrong in bad(t):
            if kind == "shape" and name == "pool":  # a pool with a slot less
                continue
            match = None if kind == "shape" and name in (first, "cu", "slot_idx", "pool", "B") else name
            if kind == "type" and name in ("pool", "y", "x"):
                match = None
            with pytest.raises((ValueError, TypeError), match=match):
                call(**{**args, name: wrong})
        if name not in may_be_none:
            with pytest.raises((ValueError, TypeError, AttributeError)):
                call(**{**args, name: None})


def test_short_conv():
    layer = Q.ShortConv(2, 20, 24, 4, device="cpu", train=True)
    args = dict(x=device(20, 24), weight=device(24, 4, dtype=F32), cu=device(3, dtype=I32), bias=device(24, dtype=F32), S0=device(2, 3, 24))
    forward = dict(args, y=device(20, 24), S_out=device(2, 3, 24))
    check(lambda **k: layer.forward(stream=0, **k), forward, "x", ("bias", "S0", "S_out"))
    back = dict(args, dy=device(20, 24), dx=device(20, 24), dweight=device(24, 4, dtype=F32), dbias=device(24, dtype=F32), dS_out=device(2, 3, 24), dS0=device(2, 3, 24))
    check(lambda **k: layer.backward(stream=0, **k), back, "x", ("bias", "S0", "dbias", "dS_out", "dS0"))
    with pytest.raises(ValueError, match="train"):
        Q.ShortConv(2, 20, 24, 4, device="cpu").backward(stream=0, **back)
    with pytest.raises(TypeError):
        Q.ShortConv(2, 20, 24, 4, dtype=torch.float16, device="cpu")
    with pytest.raises(ValueError, match="cu"):
        layer.forward(stream=0, **dict(forward, cu=device(0, dtype=I32)))
    step = dict(pool=device(5, 3, 24), slot_idx=device(4, dtype=I32), x=device(4, 24), weight=device(24, 4, dtype=F32), y=device(4, 24), bias=device(24, dtype=F32))
    check(lambda **k: Q.conv_step(stream=0, **k), step, "pool", ("bias",))


def scan_tensors(n=20, H=4, G=2, P=64, N=64):
    return dict(x=device(n, H, P), dt=device(n, H), A=device(H, dtype=F32), B=device(n, G, N), C=device(n, G, N), cu=device(3, dtype=I32), D=device(H, dtype=F32),
                dt_bias=device(H, dtype=F32), S0=device(2, H, N, P, dtype=F32))


def test_selective_scan():
    layer = Q.SelectiveScan(2, 20, 4, 64, 64, 2, device="cpu", train=True)
    args = scan_tensors()
    forward = dict(args, y=device(20, 4, 64), S_out=device(2, 4, 64, 64, dtype=F32))
    check(lambda **k: layer.forward(stream=0, **k), forward, "x", ("D", "dt_bias", "S0", "S_out"))
    back = dict(args, dy=device(20, 4, 64), dx=device(20, 4, 64), ddt=device(20, 4), dA=device(4, dtype=F32), dB=device(20, 2, 64), dC=device(20, 2, 64),
                dD=device(4, dtype=F32), ddt_bias=device(4, dtype=F32), dS_out=device(2, 4, 64, 64, dtype=F32), dS0=device(2, 4, 64, 64, dtype=F32))
    with pytest.raises(RuntimeError, match="forward"):
        layer.backward(stream=0, **back)
    layer.calls, layer._sizes = 3, (2, 20)
    check(lambda **k: layer.backward(stream=0, **k), back, "x", ("D", "dt_bias", "S0", "dD", "ddt_bias", "dS_out", "dS0"))
    with pytest.raises(RuntimeError, match="call 2"):
        layer.backward(stream=0, call=2, **back)
    layer._sizes = (2, 19)
    with pytest.raises(RuntimeError, match="19"):
        layer.backward(stream=0, call=3, **back)
    with pytest.raises(ValueError, match="train"):
        Q.SelectiveScan(2, 20, 4, 64, 64, 2, device="cpu").backward(stream=0, **back)
    step = dict({k: v for k, v in scan_tensors(n=3).items() if k not in ("cu", "S0")}, pool=device(5, 4, 64, 64, dtype=F32), slot_idx=device(3, dtype=I32), y=device(3, 4, 64))
    check(lambda **k: Q.scan_step(stream=0, **k), step, "pool", ("D", "dt_bias"))


def test_gated_norm():
    layer = Q.GatedNorm(2, 40, device="cpu", train=True)
    args = dict(x=device(6, 2, 40), z=device(6, 2, 40), weight=device(40, dtype=F32))
    check(lambda **k: layer.forward(stream=0, **k), dict(args, y=device(6, 2, 40)), "x", ("weight",))
    back = dict(args, dy=device(6, 2, 40), dx=device(6, 2, 40), dz=device(6, 2, 40), dweight=device(40, dtype=F32))
    check(lambda **k: layer.backward(stream=0, **k), back, "x", ("weight", "dweight"))
    with pytest.raises(ValueError, match="train"):
        Q.GatedNorm(2, 40, device="cpu").backward(stream=0, **back)
    with pytest.raises(ValueError, match="z"):
        Q.GatedNorm(2, 40, act=None, device="cpu").forward(stream=0, **dict(args, y=device(6, 2, 40)))
    with pytest.raises(KeyError):
        Q.GatedNorm(2, 40, act="relu", device="cpu")


def test_residual_norm():
    layer = Q.ResidualNorm(40, res_dtype=F32, device="cpu", train=True)
    w = lambda: device(40, dtype=F32)  # noqa: E731
    args = dict(o=device(6, 40), r=device(6, 40, dtype=F32), weight=w(), post_weight=w(), scale=w())
    forward = dict(args, r_out=device(6, 40, dtype=F32), h=device(6, 40))
    optional = ("r", "weight", "post_weight", "scale", "h", "dh", "dr_out", "dr", "dweight", "dpost_weight", "dscale")
    check(lambda **k: layer.forward(stream=0, **k), forward, "o", optional)
    back = dict(args, dh=device(6, 40), dr_out=device(6, 40, dtype=F32), do=device(6, 40), dr=device(6, 40, dtype=F32), dweight=w(), dpost_weight=w(), dscale=w())
    check(lambda **k: layer.backward(stream=0, **k), back, "o", optional)
    with pytest.raises(ValueError, match="train"):
        Q.ResidualNorm(40, res_dtype=F32, device="cpu").backward(stream=0, **back)


class Elsewhere(OnDevice):
    """A device tensor that says that it is on another device than the call's."""
    get_device = lambda self: 1  # noqa: E731


def test_workspaces_of_another_device():
    """An object's workspaces lie where it was made: a call with tensors of another device would hand their addresses to that one."""
    conv, back, scan, gate, res = (Q.ShortConv(2, 20, 24, 4, device="cpu", train=True), Q.SelectiveScan(2, 20, 4, 64, 64, 2, device="cpu", train=True),
                                   Q.SelectiveScan(2, 20, 4, 64, 64, 2, device="cpu"), Q.GatedNorm(2, 40, device="cpu", train=True), Q.ResidualNorm(40, device="cpu", train=True))
    for layer in (conv, back, scan, gate, res):
        layer.work = layer.work.as_subclass(Elsewhere)
    there = pytest.raises(ValueError, match="workspace")
    tokens, taps = (lambda: device(20, 24)), device(24, 4, dtype=F32)
    with there:
        conv.backward(tokens(), taps, device(3, dtype=I32), tokens(), tokens(), device(24, 4, dtype=F32), stream=0)
    args, out = scan_tensors(), dict(dy=device(20, 4, 64), dx=device(20, 4, 64), ddt=device(20, 4), dA=device(4, dtype=F32), dB=device(20, 2, 64), dC=device(20, 2, 64))
    with there:
        scan.forward(y=device(20, 4, 64), stream=0, **args)
    back.calls, back._sizes = 1, (2, 20)
    for name in ("work", "save"):
        with there:
            back.forward(y=device(20, 4, 64), stream=0, **args)
        with there:
            back.backward(stream=0, **args, **out)
        back.work, back.save = back.work.as_subclass(OnDevice), back.save.as_subclass(Elsewhere)
    rows, w = (lambda: device(6, 2, 40)), lambda: device(40, dtype=F32)  # noqa: E731
    with there:
        gate.backward(rows(), rows(), w(), rows(), rows(), rows(), w(), stream=0)
    row = lambda: device(6, 40)  # noqa: E731
    with there:
        res.backward(row(), row(), row(), row(), row(), row(), weight=w(), dweight=w(), stream=0)
