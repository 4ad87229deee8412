"""The sequence and window calls on the GPU against the recurrence in 64 bits, token by token.

Tolerances.  fp32 results: a few hundred fp32 operations of relative error 2^-24 on the way to
each, none of which amplifies (gates and keys have norm at most 1), and operands split to 24
bits: 1e-5 of the root mean square, relative 2-norm.  bf16 results: the rounding at the end,
at most 2^-8 of the value, over an intermediate good to 2^-16 of the root mean square
times the number of terms that come together (under 2^6): 2^-8 |x| + 2^-10 rms each.  Both with an absolute 1e-30: what lies below
fp32's range comes out as 0.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------ the recurrence
def recurrence(q, k, v, beta, g, S):
    """One sequence in 64 bits: q, k, v, g [t, h, .], beta [t, h], S [h, d, d]."""
    y = torch.zeros_like(v)
    for t in range(v.shape[0]):
        S = torch.exp(g[t])[:, :, None] * S
        u = beta[t][:, None] * (v[t] - torch.einsum("hij,hi->hj", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        y[t] = torch.einsum("hij,hi->hj", S, q[t])
    return y, S


def wide(x, share=1):
    x = x.detach().to("cpu", F64)
    return x.repeat_interleave(share, 1) if share > 1 else x


def plain(b, leaves=False):
    """Every sequence of a batch; leaves: the inputs as 64-bit leaves that take gradients."""
    c = b["case"]
    share = c["H"] // c["Hk"]
    x = {n: b[n].detach().to("cpu", F64).requires_grad_(leaves) for n in ("q", "k", "v", "beta", "g")}
    S0 = torch.zeros(len(c["lens"]), c["H"], c["d"], c["d"], dtype=F64) if b["S0"] is None else b["S0"].detach().to("cpu", F64)
    S0.requires_grad_(leaves)
    g = x["g"] if c["gate"] == "kda" else x["g"][..., None]
    # the floor that the library puts under log-gates; exp(-150) is as good as 0
    g = g.clamp_min(-150.0)
    ys, Ss, at = [], [], c.get("skip", 0)
    for s, n in enumerate(c["lens"]):
        sl = slice(at, at + n)
        y, S = recurrence(x["q"][sl].repeat_interleave(share, 1), x["k"][sl].repeat_interleave(share, 1), x["v"][sl], x["beta"][sl], g[sl], S0[s])
        ys.append(y), Ss.append(S)
        at += n
    return torch.cat(ys) if ys else None, torch.stack(Ss), x, S0


def near(got, want, what):
    """got (bf16 or fp32) against want (64 bits), by the tolerances at the top of this file."""
    g, w = got.detach().to("cpu", F64), want.detach()
    assert torch.isfinite(g).all(), what
    if w.numel() == 0:
        return
    rms = w.square().mean().sqrt()
    if got.dtype == F32:
        assert (g - w).norm() <= 1e-5 * w.norm() + 1e-30, (what, float((g - w).norm() / w.norm()))
    else:
        over = (g - w).abs() - (2.0 ** -8 * w.abs() + 2.0 ** -10 * rms + 1e-30)
        assert over.max() <= 0, (what, float(over.max() / rms))


def batch(gate="gdn", lens=(70,), H=2, Hk=None, d=128, dtype=BF, start=True, gates=(0.001, 0.5), skip=0, extra=0, seed=0, beta=None):
    Hk = Hk or H
    gen = torch.Generator(device=DEV).manual_seed(seed)
    t = sum(lens) + skip + extra
    rand = lambda *s: torch.rand(*s, generator=gen, device=DEV)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    unit = lambda *s: torch.nn.functional.normalize(randn(*s), dim=-1)  # noqa: E731
    gshape = (t, H) if gate == "gdn" else (t, H, d)
    b = dict(case=dict(gate=gate, lens=list(lens), H=H, Hk=Hk, d=d, skip=skip),
             q=unit(t, Hk, d).to(dtype), k=unit(t, Hk, d).to(dtype), v=randn(t, H, d).to(dtype),
             beta=(torch.sigmoid(randn(t, H)) if beta is None else torch.full((t, H), beta, device=DEV)).to(dtype),
             g=(-(gates[0] + (gates[1] - gates[0]) * rand(*gshape))).to(dtype),
             S0=0.3 * randn(len(lens), H, d, d) if start else None,
             cu=torch.tensor([skip] + [skip + sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device=DEV),
             dy=randn(t, H, d).to(dtype), dS=0.3 * randn(len(lens), H, d, d))
    return b


def run(b, y_dtype=None, train=False, layer=None, dS=True, stream=None):
    c = b["case"]
    t, dt = b["v"].shape[0], b["v"].dtype
    layer = layer or Q.ChunkedDelta(len(c["lens"]), t, c["H"], c["d"], c["gate"], c["Hk"], dt, y_dtype, train=train)
    out = dict(y=torch.full((t, c["H"], c["d"]), 7.0, dtype=y_dtype or dt, device=DEV), S=torch.full((len(c["lens"]), c["H"], c["d"], c["d"]), 7.0, device=DEV))
    layer.forward(b["q"], b["k"], b["v"], b["beta"], b["g"], b["cu"], out["y"], S0=b["S0"], S_out=out["S"], stream=stream)
    if train:
        for n in ("q", "k", "v", "beta", "g"):
            out["d" + n] = torch.full(b[n].shape, 7.0, dtype=dt, device=DEV)
        out["dS0"] = torch.full_like(out["S"], 7.0)
        layer.backward(b["q"], b["k"], b["v"], b["beta"], b["g"], b["cu"], b["dy"], *(out["d" + n] for n in ("q", "k", "v", "beta", "g")),
                       S0=b["S0"], dS_out=b["dS"] if dS else None, dS0=out["dS0"], stream=stream)
    return out


def check(b, out, train=False, dS=True):
    c = b["case"]
    y, S, x, S0 = plain(b, leaves=train)
    live = slice(c["skip"], c["skip"] + sum(c["lens"]))
    if y is not None:
        near(out["y"][live], y, "y")
    near(out["S"], S, "S")
    # tokens that no sequence has are not written
    for n in ["y"] + (["dq", "dk", "dv", "dbeta", "dg"] if train else []):
        assert (out[n][:live.start] == 7).all() and (out[n][live.stop:] == 7).all(), n
    if train:
        loss = (S * b["dS"].to("cpu", F64)).sum() if dS else 0.0 * S.sum()
        if y is not None:
            loss = loss + (y * b["dy"][live].to("cpu", F64)).sum()
        names = ["q", "k", "v", "beta", "g"]
        grads = torch.autograd.grad(loss, [x[n] for n in names] + [S0], allow_unused=True)
        for n, gr in zip(names, grads):
            if gr is not None:
                near(out["d" + n][live], gr[live], "d" + n)
        near(out["dS0"], grads[-1] if grads[-1] is not None else torch.zeros_like(S0), "dS0")


# ------------------------------------------------------------------ whole sequences
LENS = [(1,), (2,), (63,), (64,), (65,), (200,), (0, 1, 0), (16, 17, 15, 0, 48, 129), (1, 1, 1, 1)]


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(gate, lens):
    for dtype, d in ((BF, 128), (F32, 64)):
        b = batch(gate, lens, H=3, Hk=1, d=d, dtype=dtype, seed=len(lens))
        check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("d,dtype", [(128, BF), (128, F32), (64, BF), (64, F32)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (6, 2)])
def test_types_and_heads(gate, d, dtype, H, Hk):
    b = batch(gate, (90, 37), H=H, Hk=Hk, d=d, dtype=dtype, seed=H)
    check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_no_start_no_end_gradient(gate):
    b = batch(gate, (80, 5), start=False, seed=3)
    check(b, run(b, train=True, dS=False), train=True, dS=False)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("low,high", [(0.0, 0.0), (1.0, 3.0), (4.0, 9.0), (20.0, 60.0), (140.0, 200.0)])
def test_strong_gates(gate, low, high):
    """From no forgetting at all to everything forgotten at each token: sums of log-gates that
    would overflow or cancel if decays were formed from exponentials of positive sums."""
    for dtype in (BF, F32):
        b = batch(gate, (100,), H=2, d=64 if dtype == F32 else 128, dtype=dtype, gates=(low, high), seed=5)
        check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_resets_among_weak_gates(gate):
    """Log-gates of minus infinity (a document's end) at a few tokens, some channels only for KDA,
    weak ones elsewhere: what follows a reset keeps its accuracy."""
    b = batch(gate, (150,), H=2, dtype=F32, gates=(0.001, 0.3), seed=6)
    for t in (3, 15, 16, 63, 64, 80, 149):
        b["g"][t] = -math.inf
    if gate == "kda":
        b["g"][40, :, ::3] = -math.inf
        b["g"][41, :, 1::3] = -80.0
    out = run(b)
    check(b, out)


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_beta_at_its_ends(beta):
    """A beta of 0 writes nothing but has a gradient."""
    b = batch("gdn", (70,), beta=beta, dtype=F32, seed=7)
    check(b, run(b, train=True), train=True)


def test_repeated_keys():
    """The same key at every token: the pairs' matrix is as far from the identity as it gets."""
    b = batch("gdn", (128,), dtype=F32, gates=(0.0, 0.01), beta=1.0, seed=8)
    b["k"][:] = b["k"][0]
    check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("y_dtype", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_y_type(dtype, y_dtype):
    for gate in ("gdn", "kda"):
        b = batch(gate, (100,), dtype=dtype, seed=9)
        out = run(b, y_dtype=y_dtype)
        assert out["y"].dtype == y_dtype
        check(b, out)


def test_tokens_outside_the_sequences():
    b = batch("kda", (30, 70), skip=5, extra=9, H=2, Hk=1, seed=10)
    check(b, run(b, train=True), train=True)


def test_parts_of_one_projection():
    """q, k and v as column ranges of one wider tensor, other columns between them."""
    for dtype in (BF, F32):
        b = batch("gdn", (100, 20), H=4, Hk=2, d=64, dtype=dtype, seed=11)
        dense = run(b, train=True)
        t = b["q"].shape[0]
        wide_t = torch.full((t, 2 * 128 + 256 + 3 * 16), math.nan, dtype=dtype, device=DEV)
        at = 0
        for n, heads in (("q", 2), ("k", 2), ("v", 4)):
            part = wide_t[:, at:at + heads * 64].view(t, heads, 64)
            part.copy_(b[n])
            b[n] = part
            at += heads * 64 + 16
        strided = run(b, train=True)
        for n in dense:
            assert torch.equal(dense[n], strided[n]), n


def test_in_place_states():
    b = batch("gdn", (70, 0, 3), seed=12)
    want = run(b, train=True)
    state = b["S0"].clone()
    c = b["case"]
    layer = Q.ChunkedDelta(3, 73, c["H"], c["d"], "gdn", train=True)
    y = torch.empty_like(want["y"])
    layer.forward(b["q"], b["k"], b["v"], b["beta"], b["g"], b["cu"], y, S0=state, S_out=state)
    assert torch.equal(state, want["S"]) and torch.equal(y, want["y"])
    grad = b["dS"].clone()
    outs = [torch.empty_like(want["d" + n]) for n in ("q", "k", "v", "beta", "g")]
    layer.backward(b["q"], b["k"], b["v"], b["beta"], b["g"], b["cu"], b["dy"], *outs, dS_out=grad, dS0=grad)
    assert torch.equal(grad, want["dS0"])


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_parts_of_a_prompt(gate):
    """A prompt in two calls, resumed from its state, against one call."""
    b = batch(gate, (190,), H=2, dtype=F32, seed=13)
    whole = run(b)
    layer = Q.ChunkedDelta(1, 190, 2, 128, gate, dtype=F32)
    state, y = b["S0"].clone(), torch.empty_like(whole["y"])
    for lo, hi in ((0, 77), (77, 190)):
        part = [b[n][lo:hi] for n in ("q", "k", "v", "beta", "g")]
        layer.forward(*part, torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV), y[lo:hi], S0=state, S_out=state)
    assert (state - whole["S"]).norm() <= 1e-5 * whole["S"].norm()
    assert (y - whole["y"]).norm() <= 1e-5 * whole["y"].norm()


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_gradient_against_differences(gate):
    """Directional derivatives of the 64-bit loss by central differences, step 1e-6: their error
    is about 1e-9 of the loss; the fp32 gradients' is 1e-5 of their norm."""
    b = batch(gate, (75,), H=2, Hk=1, d=64, dtype=F32, seed=14)
    out = run(b, train=True)
    names = ["q", "k", "v", "beta", "g"]
    gen = torch.Generator().manual_seed(1)

    def loss(shift):
        moved = dict(b, **{n: b[n].to("cpu", F64) + shift * way[n] for n in names}, S0=b["S0"].to("cpu", F64) + shift * way["S0"])
        y, S, _, _ = plain(moved)
        return ((y * b["dy"].to("cpu", F64)).sum() + (S * b["dS"].to("cpu", F64)).sum()).item()

    for one in names + ["S0"]:
        way = {n: torch.randn(b[n].shape, generator=gen, dtype=F64) * (n == one) for n in names + ["S0"]}
        h = 1e-6
        diff = (loss(h) - loss(-h)) / (2 * h)
        grad = out["d" + one].to("cpu", F64)
        assert abs(diff - (grad * way[one]).sum().item()) <= 1e-5 * grad.norm().item() * way[one].norm().item(), one


def test_same_inputs_same_bits_and_other_streams():
    for gate in ("gdn", "kda"):
        b = batch(gate, (300, 111), H=6, Hk=2, seed=15)
        first = run(b, train=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            second = run(b, train=True)
        torch.cuda.current_stream().wait_stream(side)
        third = run(b, train=True, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
        for n in first:
            assert torch.equal(first[n], second[n]) and torch.equal(first[n], third[n]), n


def test_workspace_serves_smaller_batches():
    layer = Q.ChunkedDelta(4, 500, 2, 128, "kda", train=True)
    layer.work.fill_(255), layer.save.fill_(255)   # NaN patterns: nothing is read before it is written
    for lens in ((400, 100), (3,), (60, 0, 61, 62), (500,)):
        b = batch("kda", lens, seed=sum(lens))
        check(b, run(b, train=True, layer=layer), train=True)
    with pytest.raises(Q.SQError) as e:
        run(batch("kda", (2000,)), layer=layer)
    assert e.value.status == Q.SQ_ENOMEM


def test_debug_mode_checks_the_list(monkeypatch):
    monkeypatch.setenv("SQ_DEBUG", "1")
    b = batch("gdn", (10, 20))
    run(b)
    for bad in ([0, 12, 11], [-1, 10, 30], [0, 10, 31]):
        b["cu"] = torch.tensor(bad, dtype=torch.int32, device=DEV)
        with pytest.raises(Q.SQError) as e:
            run(b)
        assert e.value.status == Q.SQ_EINVAL and "cu[" in e.value.text


def test_python_refusals():
    b = batch("gdn", (10,), H=2)
    layer = Q.ChunkedDelta(1, 10, 2, 128)
    y = torch.empty_like(b["v"])
    args = [b[n] for n in ("q", "k", "v", "beta", "g", "cu")] + [y]

    def call(i, x):
        layer.forward(*args[:i], x, *args[i + 1:])
    with pytest.raises(ValueError):
        call(0, b["q"].float())
    with pytest.raises(ValueError):
        call(1, b["k"][:, :1])
    with pytest.raises(ValueError):
        call(2, b["v"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(TypeError):
        call(3, b["beta"].float())
    with pytest.raises(ValueError):
        call(4, b["g"][:5])
    with pytest.raises(TypeError):
        call(5, b["cu"].long())
    with pytest.raises(ValueError):
        call(2, b["v"].cpu())
    with pytest.raises(ValueError):
        layer.backward(*args, *args[:5])
    with pytest.raises(TypeError):
        Q.ChunkedDelta(1, 10, 2, 128, dtype=torch.float16)


def test_in_a_hip_graph():
    b = batch("gdn", (100, 40), H=4, Hk=2, seed=16)
    layer = Q.ChunkedDelta(2, 140, 4, 128, "gdn", 2, train=True)
    outs = run(b, train=True, layer=layer)   # warm up, and the results' buffers
    names = ("q", "k", "v", "beta", "g")

    def step():
        layer.forward(*(b[n] for n in names), b["cu"], outs["y"], S0=b["S0"], S_out=outs["S"])
        layer.backward(*(b[n] for n in names), b["cu"], b["dy"], *(outs["d" + n] for n in names), dS_out=b["dS"], dS0=outs["dS0"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        fresh = batch("gdn", (100, 40), H=4, Hk=2, seed=100 + i)
        for n in names + ("S0", "dy", "dS"):
            b[n].copy_(fresh[n])
        want = run(b, train=True)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(want[n], outs[n]), (i, n)


# ------------------------------------------------------------------ windows
def window_batch(gate, n, m, H, Hk, d, dtype, bits, lens=None, gates=(0.001, 0.5), row_bits=None, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=gen, device=DEV)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    unit = lambda *s: torch.nn.functional.normalize(randn(*s), dim=-1)  # noqa: E731
    slots = n + 3
    slot = torch.randperm(slots, generator=gen, device=DEV)[:n].to(torch.int32)
    b = dict(gate=gate, n=n, m=m, H=H, Hk=Hk, d=d, slot=slot, q=unit(n, m, Hk, d).to(dtype), k=unit(n, m, Hk, d).to(dtype), v=randn(n, m, H, d).to(dtype),
             beta=torch.sigmoid(randn(n, m, H)).to(dtype), g=(-(gates[0] + (gates[1] - gates[0]) * rand(*((n, m, H) if gate == "gdn" else (n, m, H, d))))).to(dtype),
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV))
    if bits == 32:
        b["state"] = 0.3 * randn(slots, H, d, d)
        b["start"] = b["state"][slot.long()]
    else:
        b["pool"] = Q.StatePool(slots, H, d, bits, gate, row_bits=row_bits)
        b["pool"].buf.fill_(0x5A)
        b["pool"].quant_state(slot, 0.3 * randn(n, H, d, d))
        b["start"] = b["pool"].dequant_state(slot)
    return b


def window(b, y=True, S=True, y_dtype=None):
    n, m, H, d = b["n"], b["m"], b["H"], b["d"]
    out_y = torch.full((n, m, H, d), 7.0, dtype=y_dtype or b["v"].dtype, device=DEV) if y else None
    out_S = torch.full((n, H, d, d), 7.0, device=DEV) if S else None
    args = (b["slot"], b["q"] if y else None, b["k"], b["v"], b["beta"], b["g"], out_y, out_S, b["lens"])
    if "state" in b:
        Q.f32_window_update(b["state"], *args, gate=b["gate"])
    else:
        b["pool"].window_update(*args)
    return out_y, out_S


def check_window(b, out_y, out_S):
    share = b["H"] // b["Hk"]
    lens = [b["m"]] * b["n"] if b["lens"] is None else [min(max(x, 0), b["m"]) for x in b["lens"].tolist()]
    g = wide(b["g"] if b["gate"] == "kda" else b["g"][..., None]).clamp_min(-150.0)
    q, k = (wide(b[x]).repeat_interleave(share, 2) for x in ("q", "k"))
    v, beta, start = wide(b["v"]), wide(b["beta"]), wide(b["start"])
    ys, Ss = torch.zeros(v.shape, dtype=F64), []
    for i, n in enumerate(lens):
        y, S = recurrence(q[i, :n], k[i, :n], v[i, :n], beta[i, :n], g[i, :n], start[i])
        ys[i, :n] = y
        Ss.append(S)
        if out_y is not None:
            assert (out_y[i, n:] == 0).all()
    if out_y is not None:
        near(out_y, ys, "y")
    if out_S is not None:
        near(out_S, torch.stack(Ss), "S")


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("m", [1, 2, 5, 15, 16])
@pytest.mark.parametrize("bits", ["packed", 32])
def test_window(gate, m, bits):
    for d, dtype in ((128, BF), (64, F32)):
        b = window_batch(gate, 3, m, 4, 2, d, dtype, [4, 6, 8, 16] if bits == "packed" else 32, seed=m)
        before = b["state"].clone() if bits == 32 else b["pool"].buf.clone()
        check_window(b, *window(b))
        assert torch.equal(before, b["state"] if bits == 32 else b["pool"].buf)   # only read


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("bits", ["packed", 32])
def test_window_lengths(gate, bits):
    """Requests of none, some and all of their tokens; counts outside [0, length] are held to it."""
    b = window_batch(gate, 6, 5, 3, 1, 128, BF, [6, 8, 4] if bits == "packed" else 32, lens=[0, 1, 5, 3, -2, 9], seed=20)
    y, S = window(b)
    check_window(b, y, S)
    assert torch.equal(S[0], b["start"][0]) and torch.equal(S[4], b["start"][4])
    y2, none = window(b, S=False)
    none2, S2 = window(b, y=False)
    assert torch.equal(y, y2) and torch.equal(S, S2) and none is None and none2 is None


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("low,high", [(0.0, 0.0), (3.0, 9.0), (20.0, 60.0), (140.0, 300.0)])
def test_window_strong_gates(gate, low, high):
    for dtype in (BF, F32):
        b = window_batch(gate, 2, 16, 2, 2, 128, dtype, 32, gates=(low, high), seed=21)
        check_window(b, *window(b))


@pytest.mark.parametrize("d,dtype", [(128, BF), (128, F32), (64, BF), (64, F32)])
def test_window_types(d, dtype):
    for y_dtype in (BF, F32):
        for gate in ("gdn", "kda"):
            b = window_batch(gate, 2, 7, 4, 4, d, dtype, [6, 16, 8, 4], seed=22)
            check_window(b, *window(b, y_dtype=y_dtype))


@pytest.mark.parametrize("d", [64, 128])
def test_window_per_row_widths(d):
    grain = 16 if d == 64 else 8
    rows = [[4] * grain + [6] * (2 * grain) + [8] * (d - 3 * grain), [4] * d, [6] * (d - grain) + [8] * grain]
    b = window_batch("kda", 3, 6, 3, 3, d, BF, [0, 0, 0], row_bits=rows, seed=23)
    check_window(b, *window(b))


def test_window_of_one_is_the_step():
    """One token: y and S' of the split decode step, whose arithmetic differs in rounding only."""
    b = window_batch("gdn", 4, 1, 3, 3, 128, F32, [6, 4, 8], seed=24)
    y, S = window(b)
    y1, S1 = torch.empty(4, 3, 128, device=DEV), torch.empty_like(S)
    b["pool"].decode_update(b["slot"], *(b[n].reshape(4, *b[n].shape[2:]) for n in ("q", "k", "v", "beta", "g")), y1, S1)
    assert (y.view_as(y1) - y1).norm() <= 1e-5 * y1.norm() and (S - S1).norm() <= 1e-5 * S1.norm()


def test_window_kept_in_the_pool():
    """The speculative step's end: S_out stored by quant_state reads back as its quantization."""
    b = window_batch("kda", 5, 4, 3, 3, 64, BF, [6, 8, 16], lens=[2, 0, 4, 1, 3], seed=25)
    _, S = window(b, y=False)
    other = Q.StatePool(5, 3, 64, [6, 8, 16], "kda")
    ident = torch.arange(5, dtype=torch.int32, device=DEV)
    other.quant_state(ident, S)
    b["pool"].quant_state(b["slot"], S)
    assert torch.equal(other.dequant_state(ident), b["pool"].dequant_state(b["slot"]))


def test_window_debug_slots(monkeypatch):
    monkeypatch.setenv("SQ_DEBUG", "1")
    b = window_batch("gdn", 3, 2, 2, 2, 64, BF, [6, 6])
    window(b)
    b["slot"][1] = b["slot"][0]
    with pytest.raises(Q.SQError) as e:
        window(b)
    assert e.value.status == Q.SQ_EINVAL


def test_window_offsets_past_32_bits():
    """A slot whose record begins past 2^31 (and 2^32) bytes."""
    H, d, slots = 64, 128, 5200
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB of device memory")
    pool = Q.StatePool(slots, H, d, [6] * H)
    assert pool.slot_stride * (slots - 1) > 1 << 32
    gen = torch.Generator(device=DEV).manual_seed(2)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    slot = torch.tensor([slots - 1, 0, slots // 2], dtype=torch.int32, device=DEV)
    pool.quant_state(slot, 0.3 * randn(3, H, d, d))
    unit = torch.nn.functional.normalize(randn(3, 2, H, d), dim=-1).to(BF)
    b = dict(gate="gdn", n=3, m=2, H=H, Hk=H, d=d, slot=slot, q=unit, k=unit.flip(1).contiguous(), v=randn(3, 2, H, d).to(BF), beta=torch.sigmoid(randn(3, 2, H)).to(BF),
             g=-torch.rand(3, 2, H, generator=gen, device=DEV).to(BF), lens=None, pool=pool, start=pool.dequant_state(slot))
    check_window(b, *window(b))
