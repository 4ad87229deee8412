"""The selective scan on the GPU against its recurrence in 64 bits, token by token.

Tolerances.  Every result is a sum of products, so its error is bounded by the same sum over absolute
values, which the recurrence gives for absolute inputs ("size" below).  fp32: a result is formed by at most 64 + 128
additions in a chunk, with operands held to 24 bits, exponentials to 2^-22, and a handful of roundings
for each chunk that a state goes through: (256 + 16 chunks) 2^-24 size.  bf16: two operands of 16 bits in
a product, 2 * 2^-17 size more, and the rounding at the end, 2^-8 of the value.  The decay's gradient is a
difference of sums over its chunk: its size is that of the whole chunk.
"""
import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ the recurrence
def softplus(v):
    return torch.where(v > 30, v, torch.log1p(torch.exp(v.clamp_max(30))))


def recurrence(x, dt, A, B, C, D, S, dy, dS, size):
    """One sequence in 64 bits, x, dy [t, h, p], dt [t, h], B, C [t, h, n], S, dS [h, n, p]: results and gradients.
    size: the same sums over absolute values."""
    if size:
        x, B, C, D, S, dy, dS = (v.abs() for v in (x, B, C, D, S, dy, dS))
    T = len(x)
    a = torch.exp((dt * A).clamp_min(-150.0))
    y, saved = torch.empty_like(x), [S]
    for t in range(T):
        S = S * a[t, :, None, None] + (dt[t, :, None] * B[t])[..., None] * x[t, :, None]
        y[t] = (S * C[t, ..., None]).sum(1) + D[:, None] * x[t]
        saved.append(S)
    g = {k: torch.empty_like(v) for k, v in dict(dx=x, ddt=dt, dB=B, dC=C, dg=dt).items()}
    for t in reversed(range(T)):
        g["dC"][t] = (saved[t + 1] * dy[t, :, None]).sum(2)
        dS = dS + C[t, ..., None] * dy[t, :, None]
        u = (dS * B[t, ..., None]).sum(1)
        g["dx"][t] = dt[t, :, None] * u + D[:, None] * dy[t]
        g["ddt"][t] = (u * x[t]).sum(1)
        g["dB"][t] = dt[t, :, None] * (dS * x[t, :, None]).sum(2)
        g["dg"][t] = a[t] * (dS * saved[t]).sum((1, 2))
        dS = dS * a[t, :, None, None]
    return dict(y=y, S=S, dS0=dS, dyx=(dy * x).sum(2), **g)


def plain(b, size=False):
    c = b["case"]
    H, share, skip = c["H"], c["H"] // c["G"], c["skip"]
    w = lambda v: v.to(F64)  # noqa: E731
    zero = torch.zeros(H, dtype=F64, device=DEV)
    A, D, bias = w(b["A"]), zero if b["D"] is None else w(b["D"]), zero if b["bias"] is None else w(b["bias"])
    raw = w(b["dt"]) + bias
    dt = softplus(raw) if c["softplus"] else raw
    slope = torch.sigmoid(raw) if c["softplus"] else torch.ones_like(raw)
    x, dy = w(b["x"]), w(b["dy"])
    B, C = (w(b[k]).repeat_interleave(share, 1) for k in ("B", "C"))
    parts, at = [], skip
    for s, n in enumerate(c["lens"]):
        S0 = torch.zeros_like(b["dS"][s], dtype=F64) if b["S0"] is None else w(b["S0"][s])
        sl = slice(at, at + n)
        r = recurrence(x[sl], dt[sl], A, B[sl], C[sl], D, S0, dy[sl], w(b["dS"][s]) if b["use_dS"] else torch.zeros_like(S0), size)
        if size:  # a chunk's whole
            for i in range(0, n, 64):
                r["dg"][i:i + 64] = r["dg"][i:i + 64].sum(0)
        parts.append(r)
        at += n
    out = {k: torch.cat([p[k] for p in parts]) for k in ("y", "dx", "ddt", "dB", "dC", "dg", "dyx")}
    out.update({k: torch.stack([p[k] for p in parts]) for k in ("S", "dS0")})
    live = slice(skip, at)
    out["ddt"] = (out["ddt"] + (A.abs() if size else A) * out["dg"]) * slope[live]
    out["dA"], out["dbias"], out["dD"] = (out.pop("dg") * dt[live]).sum(0), out["ddt"].sum(0), out.pop("dyx").sum(0)
    for k in ("dB", "dC"):
        out[k] = out[k].view(at - skip, c["G"], share, c["N"]).sum(2)
    return out


def batch(lens=(70,), H=2, G=1, P=64, N=128, dtype=BF, start=True, softplus=True, skip=0, extra=0, seed=0, D=True, bias=True, rate=(1.0, 16.0), dS=True,
          step=(0.001, 0.1)):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    T = sum(lens) + skip + extra
    rand = lambda *s: torch.rand(*s, generator=gen, device=DEV)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    wide = [H * P, G * N, G * N]
    x, B, C = torch.nn.functional.silu(randn(T, sum(wide))).to(dtype).split(wide, 1)
    dt = step[0] * (step[1] / step[0]) ** rand(H)
    raw = 0.5 * randn(T, H) if softplus else dt * (0.5 + rand(T, H))
    return dict(case=dict(lens=list(lens), H=H, G=G, P=P, N=N, skip=skip, softplus=softplus), x=x.view(T, H, P), B=B.view(T, G, N), C=C.view(T, G, N), dt=raw.to(dtype),
                A=-(rate[0] + (rate[1] - rate[0]) * rand(H)), D=randn(H) if D else None,
                bias=(dt + torch.log(-torch.expm1(-dt)) if softplus else 0.1 * dt) if bias else None,
                S0=0.3 * randn(len(lens), H, N, P) if start else None, dy=randn(T, H, P).to(dtype), dS=0.3 * randn(len(lens), H, N, P), use_dS=dS,
                cu=torch.tensor([skip] + [skip + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device=DEV))


def gradients(b):
    c, dt = b["case"], b["x"].dtype
    T = b["x"].shape[0]
    wide = [c["H"] * c["P"], c["G"] * c["N"], c["G"] * c["N"]]
    gx, gB, gC = torch.full((T, sum(wide)), 7.0, dtype=dt, device=DEV).split(wide, 1)
    h = lambda: torch.full((c["H"],), 7.0, device=DEV)  # noqa: E731
    return dict(dx=gx.view(T, c["H"], c["P"]), ddt=torch.full((T, c["H"]), 7.0, dtype=dt, device=DEV), dA=h(), dB=gB.view(T, c["G"], c["N"]),
                dC=gC.view(T, c["G"], c["N"]), dD=h(), dbias=h(), dS0=torch.full_like(b["dS"], 7.0))


def make(b, y_dtype=None, train=True):
    c = b["case"]
    return Q.SelectiveScan(len(c["lens"]), b["x"].shape[0], c["H"], c["P"], c["N"], c["G"], softplus=c["softplus"], dtype=b["x"].dtype, y_dtype=y_dtype, train=train)


def run(b, y_dtype=None, train=True, layer=None, stream=None, out=None):
    c = b["case"]
    layer = layer or make(b, y_dtype, train)
    if out is None:
        out = dict(y=torch.full((b["x"].shape[0], c["H"], c["P"]), 7.0, dtype=y_dtype or b["x"].dtype, device=DEV), S=torch.full_like(b["dS"], 7.0))
        if train:
            out.update(gradients(b))
    inputs = [b[k] for k in ("x", "dt", "A", "B", "C", "cu")]
    call = layer.forward(*inputs, out["y"], D=b["D"], dt_bias=b["bias"], S0=b["S0"], S_out=out["S"], stream=stream)
    if train:
        layer.backward(*inputs, b["dy"], *(out[k] for k in ("dx", "ddt", "dA", "dB", "dC")), D=b["D"], dt_bias=b["bias"], dD=out["dD"],
                       ddt_bias=out["dbias"], S0=b["S0"], dS_out=b["dS"] if b["use_dS"] else None, dS0=out["dS0"], call=call, stream=stream)
    return out


def check(b, out):
    c = b["case"]
    want, size = plain(b), plain(b, size=True)
    live = slice(c["skip"], c["skip"] + sum(c["lens"]))
    chunks = max(c["lens"]) // 64 + 1
    for k, got in out.items():
        if k in ("y", "dx", "ddt", "dB", "dC"):  # tokens that no sequence has are not written
            assert (got[:live.start] == 7).all() and (got[live.stop:] == 7).all(), k
            got = got[live]
        if not want[k].numel():
            continue
        assert torch.isfinite(got).all(), k
        bound = (256 + 16 * chunks) * 2.0 ** -24 * size[k] + 1e-30
        if b["x"].dtype == BF and k not in ("S", "dS0") and not (k == "y" and got.dtype == F32):
            bound = bound + 2.0 ** -16 * size[k]
        if got.dtype == BF:
            bound = bound + 2.0 ** -8 * want[k].abs()
        over = ((got.to(F64) - want[k]).abs() / bound).max()
        assert over <= 1, (k, float(over))


CASES = [dict(lens=(1,)), dict(lens=(2,), N=64), dict(lens=(63,), start=False), dict(lens=(64,)), dict(lens=(65,), P=128), dict(lens=(130,), H=4, G=2),
         dict(lens=(0, 5, 64, 0, 1, 200, 0), H=3), dict(lens=(17, 300), H=2, P=128, N=64), dict(lens=(700,), H=2), dict(lens=(31, 257, 520), H=4, G=4, start=False),
         dict(lens=(90, 33), H=6, G=2, skip=5, extra=9), dict(lens=(129,), H=1, P=128, D=False, bias=False), dict(lens=(100,), H=2, softplus=False, dS=False)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join("%s%s" % kv for kv in c.items()).replace(" ", ""))
def test_forward_and_gradients(case, dtype):
    b = batch(dtype=dtype, **case)
    check(b, run(b))


@pytest.mark.parametrize("case", [dict(lens=(200, 31)), dict(lens=(600,), P=128)], ids=str)
def test_fp32_output_of_bf16_inputs(case):
    b = batch(**case)
    check(b, run(b, y_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rate,step", [((50.0, 400.0), (0.05, 1.0)), ((0.0, 0.001), (0.001, 0.1)), ((1e4, 1e5), (0.5, 2.0))], ids=["strong", "weak", "resets"])
def test_decays(rate, step, dtype):
    b = batch(lens=(150, 300), H=3, rate=rate, step=step, dtype=dtype)
    check(b, run(b))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_resets_among_weak_decays(dtype):
    """A token that forgets everything between tokens that forget nothing: differences of large sums."""
    b = batch(lens=(200,), H=2, softplus=False, bias=False, rate=(0.01, 0.02), dtype=dtype)
    b["dt"][50] = 2e5
    b["dt"][64] = 3e5
    b["x"][50] *= 1e-5
    b["x"][64] *= 1e-5
    check(b, run(b))


def test_forward_alone_and_states_in_place():
    b = batch(lens=(40, 700), H=2)
    want = run(b, train=False)
    S = b["S0"].clone()
    y = torch.empty_like(want["y"])
    make(b, train=False).forward(*(b[k] for k in ("x", "dt", "A", "B", "C", "cu")), y, D=b["D"], dt_bias=b["bias"], S0=S, S_out=S)
    assert torch.equal(y, want["y"]) and torch.equal(S, want["S"])


def test_long_sequence_in_two_calls():
    """A sequence read in two calls, the second from the first one's state, equals one call to fp32's accuracy."""
    b = batch(lens=(1000,), H=2, dtype=F32)
    whole = run(b, train=False)
    layer, S, ys = make(b, train=False), b["S0"], []
    for lo, hi in ((0, 333), (333, 1000)):
        y, out = torch.empty(hi - lo, 2, 64, device=DEV), torch.empty_like(b["S0"])
        layer.forward(*(b[k][lo:hi] for k in ("x", "dt")), b["A"], b["B"][lo:hi], b["C"][lo:hi], torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV), y,
                      D=b["D"], dt_bias=b["bias"], S0=S, S_out=out)
        S = out
        ys.append(y)
    size = plain(b, size=True)
    for got, k in ((torch.cat(ys), "y"), (S, "S")):
        assert ((got - whole[k]).abs() <= 2 * (256 + 16 * 16) * 2.0 ** -24 * size[k] + 1e-30).all()


def test_equal_inputs_give_equal_bits():
    b = batch(lens=(90, 500, 3), H=8, G=2)
    first, again = run(b), run(b)
    for k in first:
        assert torch.equal(first[k], again[k]), k


def test_many_short_sequences_and_many_heads():
    b = batch(lens=[1 + i % 5 for i in range(300)], H=2, N=64, dtype=F32)
    check(b, run(b))
    b = batch(lens=(70,), H=40, N=64)
    check(b, run(b))


def test_long_sequences_in_long_segments():
    """Many chunks on many heads: segments of 512 tokens, sequences that end inside one."""
    for lens in ((9000,), (513, 4100, 1, 511)):
        b = batch(lens=lens, H=16, N=64, dtype=F32)
        check(b, run(b, train=False))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [dict(H=10), dict(H=9, P=128), dict(H=34, G=2)], ids=["ten", "halves", "groups"])
def test_gradients_of_many_heads_in_one_workgroup(case, dtype):
    """1024 chunks and more leave a workgroup all heads of a group: 10, 18 and 17 parts of heads, of which it takes eight at once,
    in whole chunks and in chunks of a few tokens."""
    b = batch(lens=[130, 64, 0, 90] + [1 + i % 2 for i in range(1030)], N=64, dtype=dtype, **case)
    check(b, run(b))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gradients_in_long_segments(dtype):
    """130 heads make segments of 512 tokens: three of one sequence, one of another."""
    b = batch(lens=(1030, 70), H=130, N=64, dtype=dtype)
    check(b, run(b))


def test_more_sequences_than_one_search_tells_apart():
    """4200 sequences: the search for a chunk's sequence goes through two steps of 64 lanes.  A token's results do not depend on how
    many sequences there are, so they equal to the bit those of the same sequences in calls of 600, which the tests above hold to
    the recurrence."""
    lens = [i % 3 for i in range(4200)]
    b = batch(lens=lens, H=1, N=64)
    whole, at = run(b), 0
    for s in range(0, 4200, 600):
        n = sum(lens[s:s + 600])
        part = dict(b, case=dict(b["case"], lens=lens[s:s + 600]), cu=(b["cu"][s:s + 601] - at).contiguous(),
                    **{k: b[k][at:at + n].contiguous() for k in ("x", "dt", "B", "C", "dy")}, **{k: b[k][s:s + 600].clone() for k in ("S0", "dS")})
        out = run(part)
        for k, v in out.items():
            if k in ("S", "dS0"):
                assert torch.equal(v, whole[k][s:s + 600]), (s, k)
            elif k in ("y", "dx", "ddt", "dB", "dC"):
                assert torch.equal(v, whole[k][at:at + n]), (s, k)
        at += n


def test_steps_of_time_as_a_part_of_a_projection():
    b = batch(lens=(70, 30), H=3)
    want = run(b)
    wide = torch.full((100, 11), float("nan"), dtype=BF, device=DEV)
    wide[:, 4:7] = b["dt"]
    grad = torch.full((100, 9), 7.0, dtype=BF, device=DEV)
    out = dict(y=torch.empty_like(want["y"]), S=torch.empty_like(want["S"]), **gradients(b))
    out["ddt"] = grad[:, 1:4]
    run(dict(b, dt=wide[:, 4:7]), out=out)
    for k in want:
        assert torch.equal(out[k], want[k]), k
    assert (grad[:, 0] == 7).all() and (grad[:, 4:] == 7).all()


def test_infinite_inputs_stay_in_their_group_and_sequence():
    b = batch(lens=(150, 80), H=4, G=2)
    clean = run(b, train=False)
    b["B"][100, 1, 5] = float("inf")
    out = run(b, train=False)
    assert not torch.isfinite(out["y"][100:150, 2:]).all()
    assert torch.equal(out["y"][:150, :2], clean["y"][:150, :2]) and torch.equal(out["y"][:64], clean["y"][:64])
    assert torch.equal(out["y"][150:], clean["y"][150:]) and torch.equal(out["S"][1], clean["S"][1])


def test_nan_of_a_time_step_reaches_later_tokens_alone():
    for dtype in (BF, F32):
        b = batch(lens=(150, 80), H=4, G=2, dtype=dtype)
        clean = run(b, train=False)
        b["dt"][100, 1] = float("nan")
        out = run(b, train=False)
        assert torch.isnan(out["y"][100:150, 1]).all() and torch.isnan(out["S"][0, 1]).all()
        out["y"][100:150, 1], out["S"][0, 1] = clean["y"][100:150, 1], clean["S"][0, 1]
        assert torch.equal(out["y"], clean["y"]) and torch.equal(out["S"], clean["S"])


def test_gradients_of_states_in_place():
    for lens in ((70, 3), (900, 300)):
        b = batch(lens=lens, H=2, N=64)
        want = run(b)
        out = dict(y=torch.empty_like(want["y"]), S=torch.empty_like(want["S"]), **gradients(b))
        b["dS"] = out["dS0"] = b["dS"].clone()
        run(b, out=out)
        for k in want:
            assert torch.equal(out[k], want[k]), (lens, k)


def test_empty_batches_leave_zeros_for_the_parameters():
    for lens in ((), (0, 0)):
        b = batch(lens=lens, H=3, N=64)
        out = run(b)
        assert all((out[k] == 0).all() for k in ("dA", "dD", "dbias")), lens
        if lens:
            assert torch.equal(out["S"], b["S0"]) and torch.equal(out["dS0"], b["dS"])


def test_debug_mode_refuses_lists(monkeypatch):
    b = batch(lens=(20, 30), H=2, N=64)
    monkeypatch.setenv("SQ_DEBUG", "1")
    run(b)
    b["cu"][1] = 60
    with pytest.raises(Q.SQError, match="cu"):
        run(b, train=False)
    pool, y = torch.zeros(4, 2, 64, 64, device=DEV), torch.empty(3, 2, 64, dtype=BF, device=DEV)
    args = [b[k][:3] for k in ("x", "dt")] + [b["A"]] + [b[k][:3] for k in ("B", "C")] + [y]
    slots = lambda *s: torch.tensor(s, dtype=torch.int32, device=DEV)  # noqa: E731
    Q.scan_step(pool, slots(-1, 2, -1), *args)
    with pytest.raises(Q.SQError, match="repeated"):
        Q.scan_step(pool, slots(1, 2, 1), *args)
    x = torch.zeros(3, 16, dtype=BF, device=DEV)
    conv = [torch.zeros(4, 3, 16, dtype=BF, device=DEV), x, torch.zeros(16, 4, device=DEV), torch.empty_like(x)]
    Q.conv_step(conv[0], slots(9, 2, -1), *conv[1:])
    with pytest.raises(Q.SQError, match="repeated"):
        Q.conv_step(conv[0], slots(2, 0, 2), *conv[1:])


def test_gradients_against_differences():
    """The gradient of a weighted sum of y and S along a random direction, by central differences in 64 bits."""
    b = batch(lens=(37, 5), H=2, dtype=F32)
    out = run(b)
    gen = torch.Generator(device=DEV).manual_seed(5)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", bias="dbias", S0="dS0")

    def loss(at):
        c = dict(b, **{k: v for k, v in at.items()})
        r = plain(c)
        return (r["y"] * b["dy"].to(F64)).sum() + (r["S"] * b["dS"].to(F64)).sum()

    for k, g in names.items():
        d = torch.randn(b[k].shape, generator=gen, device=DEV, dtype=F64)
        h = 1e-6
        diff = (loss({k: b[k].to(F64) + h * d}) - loss({k: b[k].to(F64) - h * d})) / (2 * h)
        got = (out[g].to(F64) * d).sum()
        # differences: h^2 / 6 of the third derivative and 2^-52 / h of the loss; gradients: 2^-15 of each term
        assert abs(got - diff) <= 1e-4 * (out[g].to(F64) * d).abs().sum() + 1e-6 * abs(diff), (k, float(got), float(diff))


def test_nan_stays_in_its_head_and_sequence():
    b = batch(lens=(100, 80), H=3)
    b["dt"][30, 1] = float("nan")
    out = run(b, train=False)
    y = out["y"]
    assert torch.isnan(y[30:100, 1]).all() and torch.isnan(out["S"][0, 1]).all()
    b["dt"][30, 1] = 0.0
    clean = run(b, train=False)
    for h in (0, 2):
        assert torch.equal(y[:, h], clean["y"][:, h])
    assert torch.equal(y[100:], clean["y"][100:]) and torch.equal(out["S"][1], clean["S"][1])


def test_tokens_of_no_sequence_are_not_read():
    b = batch(lens=(70, 61), H=2, skip=6, extra=70)
    clean = run(b)
    for k in ("x", "dt", "B", "C", "dy"):
        b[k][:6] = float("nan")
        b[k][6 + 131:] = float("nan")
    out = run(b)
    for k in clean:
        assert torch.equal(out[k], clean[k]), k


def test_graph_replays():
    """A training step captured and replayed on new inputs, the layer's own eager work between the replays."""
    b = batch(lens=(90, 300), H=2)
    layer, eager = make(b), make(b)
    out = run(b, layer=layer)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, layer=layer, out=out)
    for seed in range(1, 5):
        new = batch(lens=(90, 300), H=2, seed=seed)
        for k in ("x", "dt", "A", "B", "C", "D", "bias", "S0", "dy", "dS"):
            b[k].copy_(new[k])
        graph.replay()
        want = run(new, layer=eager)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (seed, k)


def test_another_stream():
    b = batch(lens=(300,), H=2)
    want = run(b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out = run(b)
    s.synchronize()
    for k in want:
        assert torch.equal(out[k], want[k]), k


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("dtype,y_dtype", [(BF, BF), (F32, F32), (BF, F32)], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("n,H,G,P,N", [(1, 1, 1, 64, 64), (5, 4, 2, 64, 128), (3, 2, 1, 128, 64), (7, 3, 3, 128, 128)], ids=str)
def test_step(n, H, G, P, N, dtype, y_dtype):
    b = batch(lens=(1,) * n, H=H, G=G, P=P, N=N, dtype=dtype)
    pool = 0.3 * torch.randn(n + 3, H, N, P, device=DEV)
    before = pool.clone()
    slot = torch.randperm(n + 3, device=DEV)[:n].to(torch.int32)
    b["S0"] = pool[slot.long()].clone()
    y = torch.empty(n, H, P, dtype=y_dtype, device=DEV)
    Q.scan_step(pool, slot, b["x"], b["dt"], b["A"], b["B"], b["C"], y, D=b["D"], dt_bias=b["bias"])
    check(dict(b, dy=torch.zeros_like(b["dy"])), dict(y=y, S=pool[slot.long()]))
    rest = torch.ones(n + 3, dtype=torch.bool, device=DEV)
    rest[slot.long()] = False
    assert torch.equal(pool[rest], before[rest])


def test_step_leaves_out_requests_without_a_slot():
    b = batch(lens=(1,) * 4, H=2, N=64)
    pool = torch.randn(3, 2, 64, 64, device=DEV)
    whole, y = pool.clone(), torch.full((4, 2, 64), 7.0, dtype=BF, device=DEV)
    args = (b["x"], b["dt"], b["A"], b["B"], b["C"], y)
    Q.scan_step(pool, torch.tensor([-1, 2, 3, 0], dtype=torch.int32, device=DEV), *args)
    assert (y[0] == 7).all() and (y[2] == 7).all() and (y[1] != 7).any() and (y[3] != 7).any()
    assert torch.equal(pool[1], whole[1]) and not torch.equal(pool[2], whole[2]) and not torch.equal(pool[0], whole[0])


def test_steps_follow_the_scan():
    """A prompt by the scan, then tokens one by one, against the whole sequence at once."""
    b = batch(lens=(75,), H=2, G=1, dtype=F32)
    whole, size = plain(b), plain(b, size=True)
    y, S = torch.empty(70, 2, 64, device=DEV), torch.empty(1, 2, 128, 64, device=DEV)
    make(b, train=False).forward(b["x"][:70], b["dt"][:70], b["A"], b["B"][:70], b["C"][:70], torch.tensor([0, 70], dtype=torch.int32, device=DEV), y, D=b["D"],
                                 dt_bias=b["bias"], S0=b["S0"], S_out=S)
    slot = torch.zeros(1, dtype=torch.int32, device=DEV)
    for t in range(70, 75):
        out = torch.empty(1, 2, 64, device=DEV)
        Q.scan_step(S, slot, *(b[k][t:t + 1] for k in ("x", "dt")), b["A"], b["B"][t:t + 1], b["C"][t:t + 1], out, D=b["D"], dt_bias=b["bias"])
        assert ((out[0] - whole["y"][t]).abs() <= 512 * 2.0 ** -24 * size["y"][t] + 1e-30).all()
    assert ((S[0] - whole["S"][0]).abs() <= 512 * 2.0 ** -24 * size["S"][0] + 1e-30).all()
