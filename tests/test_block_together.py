"""The short convolution, the scan or the delta rule, and the norms one after another, as a layer runs them.

Tolerances.  Everything is in fp32: a chain of some ten operators and projections, each good to 2^-20 of the sum of absolute
values of its terms, of which there are at most a few hundred of either sign: 10 * 2^-20 * sqrt(400), 2e-4 of the root mean square
(relative 2-norm) for results and gradients."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

pytestmark = pytest.mark.gpu
F32, F64 = torch.float32, torch.float64
DEV = "cuda"


def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "state_space_block.py")
    spec = importlib.util.spec_from_file_location("state_space_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rms(x):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def silu(x):
    return x * torch.sigmoid(x)


def convolve(x, taps, bias):
    rows = torch.cat([torch.zeros(taps.shape[1] - 1, x.shape[1], dtype=x.dtype, device=x.device), x])
    return silu(sum(rows[j:j + len(x)] * taps[:, j] for j in range(taps.shape[1])) + bias)


def plain_logits(m, w, seqs):
    """The example's model in 64 bits, sequence by sequence and token by token."""
    out = []
    for s in seqs:
        r = w["embed"][s.to(DEV)]
        z, xbc, dt = (rms(r) * w["first"] @ w["into"]).split([m.INNER, m.CHANNELS, m.H], 1)
        x, B, C = convolve(xbc, w["taps"], w["taps_bias"]).split(m.PARTS, 1)
        x, B, C = x.unflatten(1, (m.H, m.P)), *(v.unflatten(1, (m.G, m.N)).repeat_interleave(m.H // m.G, 1) for v in (B, C))
        dt = torch.nn.functional.softplus(dt + w["dt_bias"])
        S, ys = torch.zeros(m.H, m.N, m.P, dtype=F64, device=DEV), []
        for t in range(len(s)):
            S = S * torch.exp(dt[t] * w["A"])[:, None, None] + (dt[t, :, None] * B[t])[..., None] * x[t, :, None]
            ys.append((S * C[t, ..., None]).sum(1) + w["D"][:, None] * x[t])
        y = rms(torch.stack(ys).flatten(1) * silu(z)) * w["gate"][0]
        r = r + w["scale"] * rms(y @ w["out"]) * w["post"]
        out.append(rms(r) * w["last"] @ w["head"])
    return torch.cat(out)


def near(got, want, what):
    assert (got.to(F64) - want).norm() <= 2e-4 * want.norm() + 1e-12, (what, float((got.to(F64) - want).norm() / want.norm()))


def test_a_state_space_block_and_its_gradients():
    m = example()
    model = m.Model(seed=3)
    seqs = [s for s in m.batch(torch.Generator().manual_seed(4), 3, 80)] + [torch.tensor([7])]
    tokens, cu = m.flat(seqs)
    logits = model.logits(model.layers(4, len(tokens)), tokens, cu)
    up = torch.randn(logits.shape, generator=torch.Generator(DEV).manual_seed(5), device=DEV)
    logits.backward(up)
    w = {k: v.detach().to(F64).requires_grad_() for k, v in model.w.items()}
    want = plain_logits(m, w, seqs)
    near(logits.detach(), want.detach(), "logits")
    grads = torch.autograd.grad(want, list(w.values()), up.to(F64))
    for (k, v), g in zip(model.w.items(), grads):
        near(v.grad, g, k)


def test_the_example_runs_and_its_steps_follow_the_whole():
    m = example()
    got = m.main(steps=3, count=6)
    assert all(torch.isfinite(torch.tensor(got["losses"]))) and got["tokens"].shape == (8, 6)
    # the same tokens read at once give the logits that the steps gave
    model, seqs = got["model"], [torch.cat([p, t.cpu()]) for p, t in zip(got["prompts"], got["tokens"])]
    tokens, cu = m.flat(seqs)
    with torch.no_grad():
        whole = model.logits(model.layers(len(seqs), len(tokens)), tokens, cu)
    for i, p in enumerate(got["prompts"]):
        near(got["seen"][i], whole[int(cu[i]) + len(p) - 1:int(cu[i + 1]) - 1].to(F64), i)


def test_a_delta_layer_and_its_gradients():
    """Projection, convolution, delta rule with q, k and v as parts of the convolution's output, gated norm of the heads."""
    gen = torch.Generator(DEV).manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    lens, H, Hk, d = [37, 70], 2, 1, 64
    T, parts = sum(lens), [Hk * d, Hk * d, H * d]
    C = sum(parts)
    cu = torch.tensor([0, 37, 107], dtype=torch.int32, device=DEV)
    w = dict(x=randn(T, C), taps=0.5 * randn(C, 3), bias=0.1 * randn(C), beta=torch.sigmoid(randn(T, H)), g=-0.1 * torch.rand(T, H, generator=gen, device=DEV),
             z=randn(T, H, d), norm=1 + 0.1 * randn(d))
    conv, layer = Q.ShortConv(2, T, C, 3, dtype=F32, train=True), Q.ChunkedDelta(2, T, H, d, n_key_heads=Hk, dtype=F32, train=True)
    norm = Q.GatedNorm(H, d, act="sigmoid", dtype=F32, train=True)
    heads = [Hk, Hk, H]
    cut = lambda t: [p.unflatten(1, (h, d)) for p, h in zip(t.split(parts, 1), heads)]  # noqa: E731
    qkv, y, out = torch.empty(T, C, device=DEV), torch.empty(T, H, d, device=DEV), torch.empty(T, H, d, device=DEV)
    conv.forward(w["x"], w["taps"], cu, qkv, bias=w["bias"])
    qkv *= 0.3  # keys of a norm about 1
    layer.forward(*cut(qkv), w["beta"], w["g"], cu, y)
    norm.forward(y, w["z"], w["norm"], out)
    up = randn(T, H, d)
    new = torch.empty_like
    dy, dz, dnorm, grads = new(y), new(y), new(w["norm"]), [torch.empty(T, h, d, device=DEV) for h in heads]
    norm.backward(y, w["z"], w["norm"], up, dy, dz, dnorm)
    dbeta, dg = new(w["beta"]), new(w["g"])
    layer.backward(*cut(qkv), w["beta"], w["g"], cu, dy, *grads, dbeta, dg)
    dqkv = 0.3 * torch.cat([v.flatten(1) for v in grads], 1)
    dx, dtaps, dbias = new(w["x"]), new(w["taps"]), new(w["bias"])
    conv.backward(w["x"], w["taps"], cu, dqkv, dx, dtaps, bias=w["bias"], dbias=dbias)

    leaf = {k: v.to(F64).requires_grad_() for k, v in w.items()}
    ys = []
    for a, b in ((0, 37), (37, 107)):
        q, k, v = cut(0.3 * convolve(leaf["x"][a:b], leaf["taps"], leaf["bias"]))
        q, k = (t.repeat_interleave(H // Hk, 1) for t in (q, k))
        S = torch.zeros(H, d, d, dtype=F64, device=DEV)
        for t in range(b - a):
            S = S * torch.exp(leaf["g"][a + t])[:, None, None]
            S = S + k[t][..., None] * (leaf["beta"][a + t][:, None] * (v[t] - (S * k[t][..., None]).sum(1)))[:, None]
            ys.append((S * q[t][..., None]).sum(1))
    want = rms(torch.stack(ys)) * leaf["norm"] * torch.sigmoid(leaf["z"])
    near(out, want.detach(), "out")
    for (k, got), g in zip(dict(x=dx, taps=dtaps, bias=dbias, beta=dbeta, g=dg, z=dz, norm=dnorm).items(), torch.autograd.grad(want, list(leaf.values()), up.to(F64))):
        near(got, g, k)
