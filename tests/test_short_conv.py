"""The short convolution on the GPU against its formula in 64 bits.

Tolerances.  p is a sum of at most five products in fp32, and SiLU adds an exponential and a reciprocal (2^-21):
16 * 2^-24 of the sum of absolute values for p, 2^-20 for what goes through SiLU (its slope is at most 1.1, the slope's
own at most 1).  Gradients of the inputs are sums of at most four such products.  dweight and dbias sum them
over the tokens, a lane up to 32 blocks of 32 and then tens of partial sums: 2^-20 + 1200 * 2^-24 of the sum of absolute
values at most.  bf16 results: 2^-8 of the value more.
"""
import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def batch(lens=(70,), C=64, W=4, dtype=BF, act="silu", bias=True, start=True, skip=0, extra=0, wide=0, seed=0, dS=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    T, n = sum(lens) + skip + extra, len(lens)
    return dict(case=dict(lens=list(lens), C=C, W=W, act=act, skip=skip), x=randn(T, C + wide).to(dtype)[:, :C], weight=0.5 * randn(C, W),
                bias=0.3 * randn(C) if bias else None, S0=randn(n, W - 1, C).to(dtype) if start else None, dy=randn(T, C).to(dtype),
                dS=randn(n, W - 1, C).to(dtype) if dS else None,
                cu=torch.tensor([skip] + [skip + sum(lens[:i + 1]) for i in range(n)], dtype=torch.int32, device=DEV))


def plain(b, size=False):
    """Results and gradients; size: the sums over absolute values."""
    c, W, C = b["case"], b["case"]["W"], b["case"]["C"]
    w = lambda v: v.to(F64).abs() if size else v.to(F64)  # noqa: E731
    weight, bias = w(b["weight"]), 0.0 if b["bias"] is None else w(b["bias"])
    out = dict(y=[], S=[], dx=[], dS0=[])
    dw, db, at = torch.zeros(C, W, dtype=F64, device=DEV), torch.zeros(C, dtype=F64, device=DEV), c["skip"]
    for s, n in enumerate(c["lens"]):
        rows = torch.cat([torch.zeros(W - 1, C, dtype=F64, device=DEV) if b["S0"] is None else w(b["S0"][s]), w(b["x"][at:at + n])])
        p = sum(rows[j:j + n] * weight[:, j] for j in range(W)) + bias
        sig = torch.sigmoid(p)
        silu = c["act"] == "silu"
        out["y"].append(p if size or not silu else p * sig)
        out["S"].append(rows[n:])
        # the slope: at most 1.1, and off by as much as p is
        dp = w(b["dy"][at:at + n]) * ((1.1 + p if size else sig * (1 + p * (1 - sig))) if silu else 1.0)
        d = torch.zeros_like(rows)
        if b["dS"] is not None:
            d[n:] += w(b["dS"][s])
        for j in range(W):
            d[j:j + n] += dp * weight[:, j]
            dw[:, j] += (dp * rows[j:j + n]).sum(0)
        db += dp.sum(0)
        out["dx"].append(d[W - 1:])
        out["dS0"].append(d[:W - 1])
        at += n
    return dict(y=torch.cat(out["y"]), dx=torch.cat(out["dx"]), S=torch.stack(out["S"]), dS0=torch.stack(out["dS0"]), dweight=dw, dbias=db)


def run(b, layer=None, stream=None, train=True, out=None):
    c, dt, T, n = b["case"], b["x"].dtype, b["x"].shape[0], len(b["case"]["lens"])
    layer = layer or Q.ShortConv(n, T, c["C"], c["W"], act=c["act"], dtype=dt, train=train)
    full = lambda *s, dtype=dt: torch.full(s, 7.0, dtype=dtype, device=DEV)  # noqa: E731
    if out is None:
        out = dict(y=full(T, c["C"]), S=full(n, c["W"] - 1, c["C"]))
        if train:
            out.update(dx=full(T, c["C"]), dweight=full(c["C"], c["W"], dtype=F32), dbias=full(c["C"], dtype=F32), dS0=full(n, c["W"] - 1, c["C"]))
    layer.forward(b["x"], b["weight"], b["cu"], out["y"], bias=b["bias"], S0=b["S0"], S_out=out["S"], stream=stream)
    if train:
        layer.backward(b["x"], b["weight"], b["cu"], b["dy"], out["dx"], out["dweight"], bias=b["bias"], dbias=out["dbias"], S0=b["S0"], dS_out=b["dS"],
                       dS0=out["dS0"], stream=stream)
    return out


def check(b, out):
    c = b["case"]
    want, size = plain(b), plain(b, size=True)
    live = slice(c["skip"], c["skip"] + sum(c["lens"]))
    for k, got in out.items():
        if k in ("y", "dx"):
            assert (got[:live.start] == 7).all() and (got[live.stop:] == 7).all(), k
            got = got[live]
        if k == "S":
            assert torch.equal(got.to(F64), want[k])  # copies
            continue
        if not want[k].numel():
            continue
        bound = (2.0 ** -20 + (1200 * 2.0 ** -24 if k in ("dweight", "dbias") else 0.0)) * size[k] + 1e-30
        if got.dtype == BF:
            bound = bound + 2.0 ** -8 * want[k].abs()
        over = ((got.to(F64) - want[k]).abs() / bound).max()
        assert over <= 1, (k, float(over))


CASES = [dict(lens=(1,), C=1), dict(lens=(2,), C=8, W=2), dict(lens=(3,), C=9, W=3), dict(lens=(0, 1, 2, 3, 4, 0), C=40), dict(lens=(64,), C=512),
         dict(lens=(129, 1, 33), C=520, W=3), dict(lens=(300,), C=1001), dict(lens=(127, 128, 129), C=24, start=False), dict(lens=(70, 5), C=48, wide=16),
         dict(lens=(70, 5), C=48, wide=3), dict(lens=(90,), C=72, skip=7, extra=40), dict(lens=(65,), C=16, act=None, bias=False, dS=False),
         dict(lens=(5000, 1), C=16), dict(lens=(31, 32), C=2000, W=2)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join("%s%s" % kv for kv in c.items()).replace(" ", ""))
def test_forward_and_gradients(case, dtype):
    b = batch(dtype=dtype, **case)
    check(b, run(b))


def test_many_short_sequences():
    b = batch(lens=[i % 6 for i in range(700)], C=24)
    check(b, run(b))


def test_unaligned_tensors():
    """Tensors that begin in the middle of 16 bytes are read by the element."""
    b = batch(lens=(40,), C=32)
    want = run(b, train=False)["y"]
    buf = torch.zeros(40 * 32 + 1, dtype=BF, device=DEV)[1:].view(40, 32)
    buf.copy_(b["x"])
    assert torch.equal(run(dict(b, x=buf), train=False)["y"], want)


def test_large_and_infinite_inputs():
    b = batch(lens=(20,), C=16, dtype=F32, bias=False, start=False)
    b["weight"].fill_(1.0)
    b["x"][5] = 1e30
    b["x"][12] = -1e30
    out = run(b)
    assert torch.isfinite(out["y"]).all() and torch.isfinite(out["dx"]).all()
    assert (out["y"][5] == 1e30).all() and (out["y"][12:16].abs() < 1e-5).all()


def test_equal_inputs_give_equal_bits():
    b = batch(lens=(900, 33, 2000), C=600)
    first, again = run(b), run(b)
    for k in first:
        assert torch.equal(first[k], again[k]), k


def test_tokens_of_no_sequence_are_not_read():
    b = batch(lens=(70, 61), C=40, skip=6, extra=70)
    clean = run(b)
    for k in ("x", "dy"):
        b[k][:6] = float("nan")
        b[k][6 + 131:] = float("nan")
    out = run(b)
    for k in clean:
        assert torch.equal(out[k], clean[k]), k


def test_graph_replays():
    b = batch(lens=(90, 300), C=64)
    layer, eager = (Q.ShortConv(2, 390, 64, 4, train=True) for _ in range(2))
    out = run(b, layer=layer)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, layer=layer, out=out)
    for seed in range(1, 5):
        new = batch(lens=(90, 300), C=64, seed=seed)
        for k in ("x", "weight", "bias", "S0", "dy", "dS"):
            b[k].copy_(new[k])
        graph.replay()
        want = run(new, layer=eager)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (seed, k)


def test_activation_far_from_zero():
    """SiLU and its slope relative to themselves: one tap of 1, so that p is the input.  Tolerances as derived for the gated norm's
    gates: 2^-20 of SiLU, 2^-19 of its slope's terms."""
    b = batch(lens=(501,), C=64, dtype=F32, bias=False, start=False, dS=False)
    b["x"].copy_(torch.linspace(-80, 80, 501 * 64, device=DEV).view(501, 64))
    b["dy"].fill_(1.0)
    b["weight"].zero_()
    b["weight"][:, 3] = 1.0
    out, v = run(b), b["x"].to(F64)
    s, rest = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
    off = float(((out["y"].to(F64) - v * s).abs() / (v * s).abs().clamp_min(1e-300)).max())
    assert off <= 2.0 ** -20, off
    off = float(((out["dx"].to(F64) - s * (1 + v * rest)).abs() / (s * (1 + v.abs() * rest))).max())
    assert off <= 2.0 ** -19, off


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,C,W,act,wide", [(1, 1, 2, "silu", 0), (5, 64, 4, "silu", 8), (130, 40, 3, None, 0), (3, 1001, 4, "silu", 1)], ids=str)
def test_step(n, C, W, act, wide, dtype):
    b = batch(lens=(1,) * n, C=C, W=W, act=act, wide=wide, dtype=dtype)
    pool = torch.randn(n + 3, W - 1, C, device=DEV).to(dtype)
    before = pool.clone()
    slot = torch.randperm(n + 3, device=DEV)[:n].to(torch.int32)
    b["S0"] = pool[slot.long()].clone()
    y = torch.empty(n, C, dtype=dtype, device=DEV)
    Q.conv_step(pool, slot, b["x"], b["weight"], y, bias=b["bias"], act=act)
    check(b, dict(y=y, S=pool[slot.long()]))
    rest = torch.ones(n + 3, dtype=torch.bool, device=DEV)
    rest[slot.long()] = False
    assert torch.equal(pool[rest], before[rest])


def test_step_leaves_out_requests_without_a_slot():
    b = batch(lens=(1,) * 4, C=16)
    pool = torch.randn(3, 3, 16, device=DEV).to(BF)
    whole, y = pool.clone(), torch.full((4, 16), 7.0, dtype=BF, device=DEV)
    Q.conv_step(pool, torch.tensor([-1, 2, 3, 0], dtype=torch.int32, device=DEV), b["x"], b["weight"], y)
    assert (y[0] == 7).all() and (y[2] == 7).all() and (y[1] != 7).any() and (y[3] != 7).any()
    assert torch.equal(pool[1], whole[1]) and torch.equal(pool[2, 2], b["x"][1]) and torch.equal(pool[0, :2], whole[0, 1:])


def test_steps_follow_the_convolution():
    b = batch(lens=(30,), C=48)
    whole = run(b, train=False)
    y, S = torch.empty(20, 48, dtype=BF, device=DEV), torch.empty(1, 3, 48, dtype=BF, device=DEV)
    Q.ShortConv(1, 20, 48, 4).forward(b["x"][:20], b["weight"], torch.tensor([0, 20], dtype=torch.int32, device=DEV), y, bias=b["bias"], S0=b["S0"], S_out=S)
    slot = torch.zeros(1, dtype=torch.int32, device=DEV)
    for t in range(20, 30):
        out = torch.empty(1, 48, dtype=BF, device=DEV)
        Q.conv_step(S, slot, b["x"][t:t + 1], b["weight"], out, bias=b["bias"])
        assert torch.equal(out[0], whole["y"][t])
    assert torch.equal(S, whole["S"])


def test_empty_batches_leave_zeros_for_the_parameters():
    for lens in ((), (0, 0)):
        b = batch(lens=lens, C=72, dtype=F32)
        out = run(b)
        assert (out["dweight"] == 0).all() and (out["dbias"] == 0).all(), lens
        if lens:
            assert torch.equal(out["S"], b["S0"]) and torch.equal(out["dS0"], b["dS"])


# ------------------------------------------------------------------ many blocks
# 8192 channels are 32 tiles, of which the gradients have 128 workgroups each, 16384 channels 64 tiles of 64: more blocks
# of 128 tokens than that, and a workgroup walks over several.
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [dict(lens=[i % 6 for i in range(300)], C=8192, W=2), dict(lens=[1 + i % 5 for i in range(300)], C=8190, W=3),
                                  dict(lens=[i % 6 for i in range(200)], C=8192), dict(lens=[130, 3, 257, 40] * 9, C=16384)],
                         ids=["three-w2", "three-odd", "two", "long"])
def test_a_workgroup_takes_several_blocks(case, dtype):
    b = batch(dtype=dtype, **case)
    check(b, run(b))


def test_one_object_for_its_largest_batch_and_for_smaller_ones():
    """Batches of 131 slots in two turns, and smaller ones of up to 128 in one: more blocks, in the same workspace."""
    layer = Q.ShortConv(129, 400, 8192, 4, train=True)
    for n in (129, 125, 60, 1):
        b = batch(lens=[1 + i % 5 for i in range(n)], C=8192, seed=n)
        check(b, run(b, layer=layer))


def test_more_sequences_than_one_search_tells_apart():
    """4200 sequences: the search for a block's sequence goes through two steps of 64 lanes."""
    b = batch(lens=[i % 3 for i in range(4200)], C=24)
    check(b, run(b))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,C,W", [(1100, 41, 4), (2100, 2056, 3), (2103, 2056, 2)], ids=str)
def test_step_with_several_requests_to_a_lane(n, C, W, dtype):
    """Two requests to a lane, and eight, the last lanes' fewer; some without a slot."""
    b = batch(lens=(1,) * n, C=C, W=W, dtype=dtype, wide=7)
    pool = torch.randn(n + 3, W - 1, C, device=DEV).to(dtype)
    before = pool.clone()
    slot = torch.randperm(n + 3, device=DEV)[:n].to(torch.int32)
    b["S0"] = pool[slot.long()].clone()
    out = slot.clone()
    out[::97] = -1
    y = torch.full((n, C), 7.0, dtype=dtype, device=DEV)
    Q.conv_step(pool, out, b["x"], b["weight"], y, bias=b["bias"])
    left = out < 0
    assert (y[left] == 7).all() and torch.equal(pool[slot[left].long()], before[slot[left].long()])
    keep = ~left
    c = dict(b, case=dict(b["case"], lens=[1] * int(keep.sum())), x=b["x"][keep], dy=b["dy"][keep], S0=b["S0"][keep], dS=b["dS"][keep])
    check(c, dict(y=y[keep], S=pool[slot[keep].long()]))
