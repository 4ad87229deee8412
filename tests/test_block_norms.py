"""The norms around a block on the GPU against their formulas in 64 bits.

Tolerances.  A row's mean square is a sum of d squares, 8 or 16 to a thread and then by halves: at most 16 + 10 + 16
additions, each half a step of 2^-24; everything else is a few roundings and one exponential and reciprocal (2^-21). With
"size" the sum of the absolute values of a result's terms: 2^-19 size in fp32, and 2^-8 of the value more in bf16.
Gradients of parameters sum over the rows, a workgroup's rows one by one and then 512 partial sums in four
lists: (rows / 512 + 256) 2^-24 size more.
"""
import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def near(out, want, size, rows):
    for k, got in out.items():
        assert torch.isfinite(got).all(), k
        bound = 2.0 ** -19 * size[k] + 1e-30
        if k in ("dweight", "dpost_weight", "dscale"):
            bound = bound + (rows / 512 + 256) * 2.0 ** -24 * size[k]
        if got.dtype == BF:
            bound = bound + 2.0 ** -8 * want[k].abs()
        over = ((got.to(F64) - want[k]).abs() / bound).max()
        assert over <= 1, (k, float(over))


def norm_back(n, rstd, dn, size=False):
    m = (dn * n).mean(-1, keepdim=True)
    return rstd * (dn + n * m if size else dn - n * m)


# ------------------------------------------------------------------ gated
def gate_batch(T=5, G=2, d=128, act="silu", first=False, shared=True, dtype=BF, wide=0, seed=0, weight=True, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    part = lambda: (scale * randn(T, G * d + wide)).to(dtype)[:, wide:].view(T, G, d)  # noqa: E731
    return dict(case=dict(T=T, G=G, d=d, act=act, first=first, shared=shared), x=part(), z=part() if act else None, dy=randn(T, G, d).to(dtype),
                weight=1 + 0.3 * randn(*([d] if shared else [G, d])) if weight else None)


def gate_plain(b, size=False):
    c = b["case"]
    ab = lambda v: v.abs() if size else v  # noqa: E731
    x, dy = b["x"].to(F64), ab(b["dy"].to(F64))
    w = torch.ones(c["d"], dtype=F64, device=DEV) if b["weight"] is None else ab(b["weight"].to(F64))
    if c["act"]:
        z = b["z"].to(F64)
        s = torch.sigmoid(z)
        act, slope = (z * s, s * (1 + z * (1 - s))) if c["act"] == "silu" else (s, s * (1 - s))
        act, slope = ab(act), s + (z * s).abs() if size else slope
    else:
        act, slope = torch.ones_like(x), torch.zeros_like(x)
    u = x * act if c["first"] else x
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-6)
    n, x = ab(u * rstd), ab(x)
    over = (0, 1) if c["shared"] else (0,)
    if c["first"]:
        du = norm_back(n, rstd, dy * w, size)
        return dict(y=n * w, dx=du * act, dz=du * x * slope, dweight=(dy * n).sum(over))
    return dict(y=n * w * act, dx=norm_back(n, rstd, dy * w * act, size), dz=dy * n * w * slope, dweight=(dy * act * n).sum(over))


def gate_run(b, layer=None, out=None, backward=True):
    c, dt = b["case"], b["x"].dtype
    layer = layer or Q.GatedNorm(c["G"], c["d"], act=c["act"], gate_first=c["first"], shared_weight=c["shared"], dtype=dt, train=True)
    if out is None:
        out = dict(y=torch.empty(b["dy"].shape, dtype=dt, device=DEV), dx=torch.empty(b["dy"].shape, dtype=dt, device=DEV),
                   dz=torch.empty(b["dy"].shape, dtype=dt, device=DEV) if c["act"] else None,
                   dweight=torch.empty([c["d"]] if c["shared"] else [c["G"], c["d"]], device=DEV))
    layer.forward(b["x"], b["z"], b["weight"], out["y"])
    if backward:
        layer.backward(b["x"], b["z"], b["weight"], b["dy"], out["dx"], out["dz"], out["dweight"])
    return {k: v for k, v in out.items() if v is not None}


GATES = [dict(T=1, G=1, d=1), dict(T=3, G=2, d=7), dict(T=70, G=3, d=64), dict(T=600, G=4, d=128), dict(T=9, G=1, d=520), dict(T=5, G=2, d=1024), dict(T=4, G=1, d=4096),
         dict(T=3, G=1, d=5000), dict(T=700, G=1, d=2048), dict(T=2, G=1, d=9001), dict(T=2, G=1, d=16384), dict(T=33, G=2, d=96, wide=24), dict(T=33, G=2, d=96, wide=3),
         dict(T=40, G=600, d=16)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", [dict(), dict(first=True, shared=False), dict(act="sigmoid", shared=False), dict(act=None, weight=False)], ids=["after", "first", "sigmoid", "none"])
@pytest.mark.parametrize("case", GATES, ids=lambda c: "-".join("%s%s" % kv for kv in c.items()))
def test_gated(case, kind, dtype):
    b = gate_batch(dtype=dtype, **case, **kind)
    near(gate_run(b), gate_plain(b), gate_plain(b, size=True), case["T"] * case["G"])


@pytest.mark.parametrize("scale", [1e-12, 1e12], ids=str)
def test_gated_of_tiny_and_huge_rows(scale):
    """Where eps is all there is, and where it is nothing."""
    b = gate_batch(T=6, G=2, d=64, act=None, dtype=F32, scale=scale)
    near(gate_run(b), gate_plain(b), gate_plain(b, size=True), 12)


def test_gated_strong_gates():
    """Gates far below and above 0: act goes to 0 and to z, and nothing overflows."""
    b = gate_batch(T=4, G=1, d=64, dtype=F32)
    b["z"][0], b["z"][1], b["z"][2] = -200.0, 200.0, 1e30
    out = gate_run(b)
    assert all(torch.isfinite(v).all() for v in out.values())
    assert (out["y"][0].abs() < 1e-30).all() and (out["dz"][0].abs() < 1e-30).all()


def test_gated_in_place_and_no_tokens():
    b = gate_batch(T=40, G=3, d=64)
    want = gate_run(b)
    layer = Q.GatedNorm(3, 64, train=True)
    x, dy = b["x"].clone(), b["dy"].clone()
    dz, dw = torch.empty_like(dy), torch.empty(64, device=DEV)
    layer.backward(x, b["z"], b["weight"], dy, dy, dz, dw)
    layer.forward(x, b["z"], b["weight"], x)
    for got, k in ((x, "y"), (dy, "dx"), (dz, "dz"), (dw, "dweight")):
        assert torch.equal(got, want[k]), k
    e = torch.empty(0, 3, 64, dtype=BF, device=DEV)
    layer.forward(e, e, b["weight"], e.clone())
    layer.backward(e, e, b["weight"], e, e.clone(), e.clone(), dw)
    assert (dw == 0).all()


# ------------------------------------------------------------------ residual
def res_batch(T=5, d=128, dtype=BF, res=None, post=True, scale=True, weight=True, r=True, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    res = res or dtype
    w = lambda on: 1 + 0.3 * randn(d) if on else None  # noqa: E731
    return dict(case=dict(T=T, d=d, res=res), o=randn(T, d).to(dtype), r=(2 * randn(T, d)).to(res) if r else None, weight=w(weight), post=w(post), scale=w(scale),
                dh=randn(T, d).to(dtype), dr_out=randn(T, d).to(res))


def res_plain(b, size=False):
    ab = lambda v: v.abs() if size else v  # noqa: E731
    one = torch.ones(b["case"]["d"], dtype=F64, device=DEV)
    o, r = b["o"].to(F64), torch.zeros_like(b["o"], dtype=F64) if b["r"] is None else b["r"].to(F64)
    weight, post, scale = (one if b[k] is None else b[k].to(F64) for k in ("weight", "post", "scale"))
    ro = torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6) if b["post"] is not None else torch.ones_like(o[:, :1])
    no = o * ro
    a = no * post
    out = r + scale * a
    rs = torch.rsqrt(out.square().mean(-1, keepdim=True) + 1e-6)
    big = r.abs() + (scale * a).abs() if size else out  # the sum's terms
    n = big * rs
    got = dict(r_out=big, h=n * ab(weight))
    if b["dh"] is not None:
        dn = ab(b["dh"].to(F64) * weight)
        total = norm_back(n, rs, dn, size)
        got["dweight"] = (ab(b["dh"].to(F64)) * n).sum(0)
    else:
        total = torch.zeros_like(o)
        got["dweight"] = torch.zeros_like(one)
    if b["dr_out"] is not None:
        total = total + ab(b["dr_out"].to(F64))
    a, no = ab(a), ab(no)
    da = total * ab(scale)
    got.update(dr=total, dscale=(total * a).sum(0), dpost_weight=(da * no).sum(0), do=norm_back(no, ro, da * ab(post), size) if b["post"] is not None else da)
    return got


def res_run(b, layer=None):
    c, dt = b["case"], b["o"].dtype
    layer = layer or Q.ResidualNorm(c["d"], dtype=dt, res_dtype=c["res"], train=True)
    new = lambda t, on=True: torch.empty(b["o"].shape, dtype=t, device=DEV) if on else None  # noqa: E731
    p = lambda k: torch.empty(c["d"], device=DEV) if b[k] is not None else None  # noqa: E731
    out = dict(r_out=new(c["res"]), h=new(dt), do=new(dt), dr=new(c["res"]), dweight=p("weight"), dpost_weight=p("post"), dscale=p("scale"))
    layer.forward(b["o"], b["r"], out["r_out"], weight=b["weight"], h=out["h"], post_weight=b["post"], scale=b["scale"])
    layer.backward(b["o"], b["r"], b["dh"], b["dr_out"], out["do"], out["dr"], weight=b["weight"], dweight=out["dweight"], post_weight=b["post"],
                   dpost_weight=out["dpost_weight"], scale=b["scale"], dscale=out["dscale"])
    return {k: v for k, v in out.items() if v is not None}


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "mixed", "f32"])
@pytest.mark.parametrize("kind", [dict(), dict(post=False), dict(scale=False), dict(post=False, scale=False, weight=False, r=False)], ids=["all", "no-post", "no-scale", "bare"])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (70, 64), (5, 520), (600, 128), (4, 4096), (3, 5001), (2, 8200), (2, 16384), (1300, 2048)], ids=str)
def test_residual(T, d, kind, types):
    b = res_batch(T=T, d=d, dtype=types[0], res=types[1], **kind)
    near(res_run(b), res_plain(b), res_plain(b, size=True), T)


def test_residual_without_some_gradients():
    for gone in ("dh", "dr_out"):
        b = dict(res_batch(T=30, d=200), **{gone: None})
        near(res_run(b), res_plain(b), res_plain(b, size=True), 30)


def test_residual_in_place_and_the_sum_alone():
    b = res_batch(T=50, d=256)
    want = res_run(b)
    layer = Q.ResidualNorm(256, train=True)
    args = dict(weight=b["weight"], post_weight=b["post"], scale=b["scale"])
    dh, dr = b["dh"].clone(), b["dr_out"].clone()
    layer.backward(b["o"], b["r"], dh, dr, dh, dr, **args)
    r, h = b["r"].clone(), torch.empty_like(b["o"])
    layer.forward(b["o"], r, r, h=h, **args)
    alone = torch.empty_like(r)
    layer.forward(b["o"], b["r"], alone, post_weight=b["post"], scale=b["scale"])
    for got, k in ((dh, "do"), (dr, "dr"), (r, "r_out"), (h, "h"), (alone, "r_out")):
        assert torch.equal(got, want[k]), k


@pytest.mark.parametrize("which", ["gated", "residual"])
def test_equal_inputs_give_equal_bits_and_graphs_replay(which):
    make, go = (lambda s: gate_batch(T=900, G=2, d=128, seed=s), gate_run) if which == "gated" else (lambda s: res_batch(T=900, d=384, seed=s), res_run)
    b = make(0)
    first, again = go(b), go(b)
    for k in first:
        assert torch.equal(first[k], again[k]), k
    layer = Q.GatedNorm(2, 128, train=True) if which == "gated" else Q.ResidualNorm(384, train=True)
    go(b, layer)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go(b, layer)
    for seed in range(1, 5):
        new = make(seed)
        for k, v in new.items():
            if torch.is_tensor(v):
                b[k].copy_(v)
        graph.replay()
        want = go(new)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (seed, k)


def test_gradients_against_differences():
    gen = torch.Generator(device=DEV).manual_seed(5)
    b = gate_batch(T=7, G=2, d=48, dtype=F32)
    out = gate_run(b)
    for k, g in dict(x="dx", z="dz", weight="dweight").items():
        d = torch.randn(b[k].shape, generator=gen, device=DEV, dtype=F64)
        loss = lambda h: (gate_plain(dict(b, **{k: b[k].to(F64) + h * d}))["y"] * b["dy"].to(F64)).sum()  # noqa: B023, E731
        diff = (loss(1e-6) - loss(-1e-6)) / 2e-6
        assert abs((out[g].to(F64) * d).sum() - diff) <= 1e-4 * (out[g].to(F64) * d).abs().sum(), k
    b = res_batch(T=7, d=48, dtype=F32)
    out = res_run(b)
    for k, g in dict(o="do", r="dr", weight="dweight", post="dpost_weight", scale="dscale").items():
        d = torch.randn(b[k].shape, generator=gen, device=DEV, dtype=F64)

        def loss(h):
            got = res_plain(dict(b, **{k: b[k].to(F64) + h * d}))
            return (got["h"] * b["dh"].to(F64)).sum() + (got["r_out"] * b["dr_out"].to(F64)).sum()
        diff = (loss(1e-6) - loss(-1e-6)) / 2e-6
        assert abs((out[g].to(F64) * d).sum() - diff) <= 1e-4 * (out[g].to(F64) * d).abs().sum(), k


# ------------------------------------------------------------------ gates far from 0
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gates_are_accurate_relative_to_themselves(act, dtype):
    """Gates and slopes of any size, not against the largest.  Rows of +1 and -1 and no eps, so that y and dz are the gate and its
    slope with x's sign.  Tolerances, in 2^-24: the exponential 2 and its argument's rounding, which is put back to |z| / 22 (ln 2 as a
    float) with 1 for the step, so under 7; 1 + e^-z and its reciprocal 1 and 2 more; the product with z 1: under 11, so 2^-20 for the
    gate.  What is left to 1, e^-z times the gate's 10, has under 18; a slope is a product of the two or their sum: under 30, 2^-19 of
    its terms' absolute values.  bf16: the argument's rounding stays, 80 in the gate and 160 in what is left: 2^-17 and 2^-16, and 2^-8
    of the value at the end."""
    z = torch.linspace(-80, 80, 8 * 4001, device=DEV).view(-1, 1, 8).to(dtype)
    x = torch.ones_like(z)
    x[..., ::2] = -1
    y, dx, dz = (torch.empty_like(z) for _ in range(3))
    layer = Q.GatedNorm(1, 8, act=act, eps=0.0, dtype=dtype)
    layer.forward(x, z, None, y)
    layer.backward(x, z, None, torch.ones_like(z), dx, dz)
    v, x = z.to(F64), x.to(F64)
    s, rest = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
    gate, slope, size = (v * s, s * (1 + v * rest), s * (1 + v.abs() * rest)) if act == "silu" else (s, s * rest, s * rest)
    for got, want, big, fine, coarse in ((y, gate, gate.abs(), 2.0 ** -20, 2.0 ** -17), (dz, slope, size, 2.0 ** -19, 2.0 ** -16)):
        bound = fine * big if dtype == F32 else coarse * big + 2.0 ** -8 * want.abs()
        over = float(((got.to(F64) - x * want).abs() / bound.clamp_min(1e-300)).max())
        assert over <= 1, over


def test_gates_beyond_the_exponentials_range():
    """Behind 87 the exponential leaves fp32's range: the gate goes to 0 or z all the same, NaN stays NaN."""
    z = torch.tensor([-89.0, -150.0, -3e38, -float("inf"), 89.0, 150.0, 3e38, float("nan")], device=DEV).view(1, 1, 8)
    x, y = torch.ones_like(z), torch.empty_like(z)
    dx, dz = torch.empty_like(z), torch.empty_like(z)
    layer = Q.GatedNorm(1, 8, act="sigmoid", eps=0.0, dtype=F32)
    layer.forward(x, z, None, y)
    layer.backward(x, z, None, torch.ones_like(z), dx, dz)
    for v in (y, dz):
        assert (v[0, 0, :4].abs() < 1e-37).all() and torch.isnan(v[0, 0, 7])
    assert (y[0, 0, 4:7] == 1).all() and (dz[0, 0, 4:7].abs() < 1e-37).all()
    z[0, 0, 3] = -88.0
    z[0, 0, 7] = 88.0
    Q.GatedNorm(1, 8, eps=0.0, dtype=F32).forward(x, z, None, y)
    assert (y[0, 0, :4].abs() < 1e-35).all() and torch.equal(y[0, 0, 4:], z[0, 0, 4:])


# ------------------------------------------------------------------ rows in several turns
# A forward pass has up to 2048 workgroups of 256 threads (one row of 2048 each), 1024 of 512 or 512 of 1024, a pass back 512: more
# rows, and a workgroup walks over several, the last one's fewer.
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("first,shared", [(False, True), (True, False)], ids=["after", "first"])
@pytest.mark.parametrize("T,G,d", [(2100, 1, 2048), (1100, 2, 2047), (1090, 1, 4104), (1030, 1, 8192), (530, 1, 9001), (520, 1, 16384)], ids=str)
def test_gated_rows_in_several_turns(T, G, d, first, shared, dtype):
    b = gate_batch(T=T, G=G, d=d, first=first, shared=shared, dtype=dtype)
    near(gate_run(b), gate_plain(b), gate_plain(b, size=True), T * G)


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "mixed", "f32"])
@pytest.mark.parametrize("T,d", [(2100, 2048), (2077, 2043), (1090, 4104), (1030, 8192), (1025, 5001), (530, 9001), (520, 16384)], ids=str)
def test_residual_rows_in_several_turns(T, d, types):
    b = res_batch(T=T, d=d, dtype=types[0], res=types[1])
    near(res_run(b), res_plain(b), res_plain(b, size=True), T)
