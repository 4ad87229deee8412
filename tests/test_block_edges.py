"""Calls of the operators around a layer at the ends of what their documentation allows: elements behind 2^31, the largest strides,
wrong lists, a second pass back, unlike types, rates that grow, gradients as parts of wider tensors.  Results are held to the same call
on small dense tensors, to the bit, or by the tests' own formulas and tolerances."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_block_norms as norms  # noqa: E402
import test_scan as scan  # noqa: E402
import test_short_conv as conv  # noqa: E402

import quantized_gated_delta_amd as Q  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def give_back():
    """Some tests take up to 90 GB."""
    yield
    torch.cuda.empty_cache()


def equal(got, want):
    for k in want:
        assert torch.equal(got[k], want[k]), k


def spread(t, stride, at=0):
    """t's tokens with `stride` elements between them, in a tensor whose other elements are left as they are."""
    n, row = t.shape[0], t[0].numel()
    flat = torch.empty((n - 1) * stride + at + row, dtype=t.dtype, device=DEV)
    out = torch.as_strided(flat, t.shape, (stride, *t.contiguous().stride()[1:]), at)
    return out.copy_(t)


# ------------------------------------------------------------------ strides and sizes
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_largest_strides(dtype):
    """2^24 elements from token to token, 140 tokens: offsets behind 2^31 from the tensor, and up to 2^32 bytes within a chunk."""
    wide = 1 << 24
    b = conv.batch(lens=(100, 40), C=72, dtype=dtype)
    equal(conv.run(dict(b, x=spread(b["x"], wide))), conv.run(b))
    b = scan.batch(lens=(100, 40), H=2, dtype=dtype)
    want = scan.run(b)
    out = dict(want, **{k: spread(torch.full_like(want[k], 7.0), wide) for k in ("dx", "ddt", "dB", "dC")}, y=torch.empty_like(want["y"]), S=torch.empty_like(want["S"]),
               **{k: torch.empty_like(want[k]) for k in ("dA", "dD", "dbias", "dS0")})
    scan.run(dict(b, **{k: spread(b[k], wide) for k in ("x", "dt", "B", "C")}), out=out)
    equal(out, want)
    b = norms.gate_batch(T=140, G=3, d=128, dtype=dtype)
    want = norms.gate_run(b)
    out = {k: spread(torch.empty_like(v), wide) if k in ("dx", "dz") else torch.empty_like(v) for k, v in want.items()}
    norms.gate_run(dict(b, x=spread(b["x"], wide), z=spread(b["z"], wide)), out=out)
    equal(out, want)


def test_more_elements_than_32_bits_convolution():
    T, C, tail = (1 << 31) // 8192 + 300, 8192, 200
    b = conv.batch(lens=(tail,), C=C)
    want = conv.run(b)
    long = dict(case=dict(b["case"], lens=[T - tail, tail]), x=torch.zeros(T, C, dtype=BF, device=DEV), weight=b["weight"], bias=b["bias"], dy=torch.zeros(T, C, dtype=BF, device=DEV),
                S0=b["S0"].repeat(2, 1, 1), dS=b["dS"].repeat(2, 1, 1), cu=torch.tensor([0, T - tail, T], dtype=torch.int32, device=DEV))
    long["x"][-tail:], long["dy"][-tail:] = b["x"], b["dy"]
    out = conv.run(long)
    equal({k: out[k][-tail:] for k in ("y", "dx")}, {k: want[k] for k in ("y", "dx")})
    equal({k: out[k][1:] for k in ("S", "dS0")}, {k: want[k] for k in ("S", "dS0")})


def test_more_elements_than_32_bits_norms():
    d, T, tail = 4096, (1 << 19) + 200, 150
    b = norms.gate_batch(T=tail, G=1, d=d)
    want = norms.gate_run(b)
    whole = dict(b, case=dict(b["case"], T=T), **{k: torch.ones(T, 1, d, dtype=BF, device=DEV) for k in ("x", "z", "dy")})
    for k in ("x", "z", "dy"):
        whole[k][-tail:] = b[k]
    out = norms.gate_run(whole)
    equal({k: out[k][-tail:] for k in ("y", "dx", "dz")}, {k: want[k] for k in ("y", "dx", "dz")})
    del whole, out
    b = norms.res_batch(T=tail, d=d, res=F32)
    want = norms.res_run(b)
    whole = dict(b, case=dict(b["case"], T=T), **{k: torch.ones(T, d, dtype=b[k].dtype, device=DEV) for k in ("o", "r", "dh", "dr_out")})
    for k in ("o", "r", "dh", "dr_out"):
        whole[k][-tail:] = b[k]
    out = norms.res_run(whole)
    equal({k: out[k][-tail:] for k in ("r_out", "h", "do", "dr")}, {k: want[k] for k in ("r_out", "h", "do", "dr")})


def test_more_elements_than_32_bits_scan():
    """States and their gradients of 1027 chunks of 256 heads, one group each: the last sequence as it is alone."""
    T, tail, H = 65600, 70, 256
    b = scan.batch(lens=(tail,), H=H, G=H)
    want = scan.run(b)
    zeros = lambda t: torch.zeros(T, *t.shape[1:], dtype=BF, device=DEV)  # noqa: E731
    long = dict(b, case=dict(b["case"], lens=[T - tail, tail]), **{k: zeros(b[k]) for k in ("x", "dt", "B", "C", "dy")}, S0=b["S0"].repeat(2, 1, 1, 1), dS=b["dS"].repeat(2, 1, 1, 1),
                cu=torch.tensor([0, T - tail, T], dtype=torch.int32, device=DEV))
    for k in ("x", "dt", "B", "C", "dy"):
        long[k][-tail:] = b[k]
    out = scan.run(long)
    rows, states = ("y", "dx", "ddt", "dB", "dC"), ("S", "dS0")
    equal({k: out[k][-tail:] for k in rows}, {k: want[k] for k in rows})
    equal({k: out[k][1:] for k in states}, {k: want[k] for k in states})


def test_steps_on_slots_behind_32_bits():
    slots = torch.tensor([0, 2099, 5, 2060], dtype=torch.int32, device=DEV)
    b = scan.batch(lens=(1,) * 4, H=64, P=128)
    small = b["S0"].clone()
    y, far = (torch.empty(4, 64, 128, dtype=BF, device=DEV) for _ in range(2))
    args = [b[k] for k in ("x", "dt", "A", "B", "C")]
    Q.scan_step(small, torch.arange(4, dtype=torch.int32, device=DEV), *args, y, D=b["D"], dt_bias=b["bias"])
    pool = torch.empty(2100, 64, 128, 128, device=DEV)
    pool[slots.long()] = b["S0"]
    Q.scan_step(pool, slots, *args, far, D=b["D"], dt_bias=b["bias"])
    assert torch.equal(y, far) and torch.equal(pool[slots.long()], small)
    del pool
    slots = torch.tensor([0, 89999, 5, 88000], dtype=torch.int32, device=DEV)
    b = conv.batch(lens=(1,) * 4, C=8192)
    small, pool = b["S0"].clone(), torch.empty(90000, 3, 8192, dtype=BF, device=DEV)
    pool[slots.long()] = b["S0"]
    y, far = (torch.empty(4, 8192, dtype=BF, device=DEV) for _ in range(2))
    Q.conv_step(small, torch.arange(4, dtype=torch.int32, device=DEV), b["x"], b["weight"], y, bias=b["bias"])
    Q.conv_step(pool, slots, b["x"], b["weight"], far, bias=b["bias"])
    assert torch.equal(y, far) and torch.equal(pool[slots.long()], small)


# ------------------------------------------------------------------ wrong lists
def framed(t, pad=256):
    """A tensor like t between two strips of `pad` elements, and the whole of it."""
    whole = torch.full((t.numel() + 2 * pad,), 7.0, dtype=t.dtype, device=DEV)
    return whole[pad:pad + t.numel()].view(t.shape), whole


@pytest.mark.parametrize("lists", [[90, 10, 300, 10], [-50, 400, 0, 300], [300, 200, 100, 0], [0, 300, 0, 300]], ids=["down", "outside", "back", "twice"])
def test_wrong_lists_stay_inside_the_tensors(lists):
    """Lists that decrease or point outside: what comes out is undefined, but nothing beside the outputs is written (spans are held
    inside the tokens, and block numbers inside the slots, whatever the list says)."""
    cu = torch.tensor(lists, dtype=torch.int32, device=DEV)
    b = dict(conv.batch(lens=(100, 100, 100), C=64), cu=cu)
    out, frames = {}, []
    for k, v in conv.run(dict(b, cu=torch.tensor([0, 100, 200, 300], dtype=torch.int32, device=DEV))).items():
        out[k], whole = framed(v)
        frames.append(whole)
    conv.run(b, out=out)
    b = dict(scan.batch(lens=(100, 100, 100), H=2, N=64), cu=cu)
    out = {}
    for k, v in scan.run(dict(b, cu=torch.tensor([0, 100, 200, 300], dtype=torch.int32, device=DEV))).items():
        out[k], whole = framed(v.contiguous())
        frames.append(whole)
    scan.run(b, out=out)
    for whole in frames:
        assert (whole[:256] == 7).all() and (whole[-256:] == 7).all()


# ------------------------------------------------------------------ other calls
def test_a_second_pass_back_of_one_forward():
    """Backward leaves what the forward saved as it is, also with other calls of other objects between."""
    for lens in ((70, 3), (900, 300)):
        b = scan.batch(lens=lens, H=4, G=2, N=64)
        layer = scan.make(b)
        want = scan.run(b, layer=layer)
        scan.run(scan.batch(lens=lens, H=4, G=2, N=64, seed=3))
        again = scan.gradients(b)
        layer.backward(*(b[k] for k in ("x", "dt", "A", "B", "C", "cu")), b["dy"], *(again[k] for k in ("dx", "ddt", "dA", "dB", "dC")), D=b["D"], dt_bias=b["bias"],
                       dD=again["dD"], ddt_bias=again["dbias"], S0=b["S0"], dS_out=b["dS"], dS0=again["dS0"], call=1)
        equal(again, {k: want[k] for k in again})


@pytest.mark.parametrize("case", [dict(lens=(70, 200)), dict(lens=(600,), N=64, P=128)], ids=str)
def test_bf16_output_of_fp32_inputs(case):
    b = scan.batch(dtype=F32, **case)
    scan.check(b, scan.run(b, y_dtype=BF))
    n, c = 5, b["case"]
    one = scan.batch(lens=(1,) * n, H=2, N=c["N"], P=c["P"], dtype=F32)
    pool, y = one["S0"].clone(), torch.empty(n, 2, c["P"], dtype=BF, device=DEV)
    Q.scan_step(pool, torch.arange(n, dtype=torch.int32, device=DEV), one["x"], one["dt"], one["A"], one["B"], one["C"], y, D=one["D"], dt_bias=one["bias"])
    scan.check(one, dict(y=y, S=pool))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rates_that_grow(dtype):
    """A above 0: the state grows, by up to e^8 over a chunk."""
    b = scan.batch(lens=(150, 300), H=3, rate=(-0.9, -0.1), step=(0.05, 0.1), dtype=dtype)
    assert (b["A"] > 0).all()
    scan.check(b, scan.run(b))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("wide", [16, 3], ids=["aligned", "odd"])
def test_gated_gradients_as_parts_of_one_tensor(wide, dtype):
    """dx and dz beside each other in one gradient, as x and z are in a projection's output."""
    b = norms.gate_batch(T=37, G=2, d=96, dtype=dtype)
    want = norms.gate_run(b)
    grad = torch.full((37, 2 * 192 + wide), 7.0, dtype=dtype, device=DEV)
    both = torch.empty(37, 2 * 192 + wide, dtype=dtype, device=DEV)
    x, z = both[:, :192].view(37, 2, 96), both[:, 192 + wide:].view(37, 2, 96)
    x.copy_(b["x"])
    z.copy_(b["z"])
    out = dict(y=torch.empty_like(want["y"]), dx=grad[:, :192].view(37, 2, 96), dz=grad[:, 192 + wide:].view(37, 2, 96), dweight=torch.empty_like(want["dweight"]))
    norms.near(norms.gate_run(dict(b, x=x, z=z), out=out), norms.gate_plain(b), norms.gate_plain(b, size=True), 74)
    assert (grad[:, 192:192 + wide] == 7).all()


def test_residual_norm_without_rows_and_without_gradients():
    layer, e = Q.ResidualNorm(40, train=True), torch.empty(0, 40, dtype=BF, device=DEV)
    w, dw = torch.ones(40, device=DEV), [torch.full((40,), 7.0, device=DEV) for _ in range(3)]
    layer.forward(e, e, e.clone(), weight=w, h=e.clone())
    layer.backward(e, e, e, e, e.clone(), e.clone(), weight=w, dweight=dw[0], post_weight=w, dpost_weight=dw[1], scale=w, dscale=dw[2])
    assert all((v == 0).all() for v in dw)
    b = norms.res_batch(T=9, d=40)
    do, dr = (torch.full((9, 40), 7.0, dtype=BF, device=DEV) for _ in range(2))
    layer.backward(b["o"], b["r"], None, None, do, dr, weight=b["weight"], dweight=dw[0], post_weight=b["post"], scale=b["scale"])
    assert (do == 0).all() and (dr == 0).all() and (dw[0] == 0).all()


def test_one_object_in_two_graphs():
    """Two captured training steps that share an object's workspace, replayed one after another."""
    layer = Q.ShortConv(2, 400, 64, 4, train=True)
    bs = [conv.batch(lens=lens, C=64, seed=s) for s, lens in enumerate(((90, 300), (200, 17)))]
    outs = [conv.run(b, layer=layer) for b in bs]
    want = [{k: v.clone() for k, v in o.items()} for o in outs]
    torch.cuda.synchronize()
    graphs = []
    for b, o in zip(bs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            conv.run(b, layer=layer, out=o)
    for turn in range(4):
        for o in outs:
            for v in o.values():
                v.zero_()
        for g in (graphs if turn % 2 else graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            equal(o, w)
