"""What stands around a recurrent layer: the short causal convolution, the selective state-space scan, and the norms.

Four operators, each in its plain form and as the library's calls:

* ``conv``:  a depthwise causal convolution of a few taps with SiLU over ragged sequences, its gradients, and its
  step on a pool of the last inputs;
* ``scan``:  the state-space recurrence S_t = e^{dt A} S_{t-1} + dt B x^T, y = S_t^T C + D x with dt = softplus(raw + bias),
  its gradients, and its step on a pool of states;
* ``gate``:  the norm after a layer, with its gate: rms(x) w act(z) or rms(x act(z)) w;
* ``residual``: the norms around a block: r' = r + scale rms(o) w_post, h = rms(r') w.

A case's ``do`` says which pass is meant: ``forward``, ``train`` (forward and every gradient) or ``step`` (one token a request).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a prefill batch of a serving engine: q, k and v of 48 heads on 16 key heads, prompts of every length in one call
        dict(name="conv_prefill_ragged", op="conv", do="forward", n=12, tokens=12001, channels=10240, width=4, dtype="bf16", bias=False, start=False),
        # a training step's layer: a packed batch of 32 heads on 16 key heads
        dict(name="conv_train", op="conv", do="train", n=4, tokens=8192, channels=8192, width=4, dtype="bf16", bias=True, start=False),
        # a decode step at full load: two tokens and three rows of state a request
        dict(name="conv_step_many", op="conv", do="step", n=512, channels=10240, width=4, dtype="bf16", bias=True),
        # one short prompt of a chat turn: all launches and little work
        dict(name="scan_one_prompt", op="scan", do="forward", n=1, tokens=200, heads=64, groups=1, d_head=64, d_state=128, dtype="bf16", start=False),
        # the next part of one long prompt, resumed from its state: a long sequential axis
        dict(name="scan_prefill_long", op="scan", do="forward", n=1, tokens=8192, heads=64, groups=8, d_head=64, d_state=128, dtype="bf16", start=True),
        # a training step's layer: packed documents of unlike lengths, one B and C for all heads
        dict(name="scan_train", op="scan", do="train", n=4, tokens=8192, heads=32, groups=1, d_head=64, d_state=128, dtype="bf16", start=False),
        # a small model trained in full precision, states carried in
        dict(name="scan_train_f32_small", op="scan", do="train", n=5, tokens=701, heads=8, groups=2, d_head=64, d_state=64, dtype="f32", start=True),
        # a decode step at full load: every request's states read and written
        dict(name="scan_step_many", op="scan", do="step", n=512, heads=64, groups=8, d_head=64, d_state=128, dtype="bf16"),
        # the gated norm behind a delta-rule layer in training: rows of one head
        dict(name="gate_train_heads", op="gate", do="train", tokens=8192, groups=32, d=128, first=False, shared=True, dtype="bf16"),
        # the gated norm behind a state-space layer in decoding: the gate before the norm, a few wide rows
        dict(name="gate_step_wide", op="gate", do="forward", tokens=8, groups=1, d=4096, first=True, shared=False, dtype="bf16"),
        # between two blocks of a model in training: norm after the one, scaled sum, norm before the next, an fp32 residual
        dict(name="residual_train", op="residual", do="train", tokens=8192, d=4096, post=True, scale=True, dtype="bf16", res="f32"),
        # the same in decoding without the norm after: a few rows of an odd number of tokens
        dict(name="residual_step", op="residual", do="forward", tokens=33, d=5120, post=False, scale=False, dtype="bf16", res="bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op, dtype = rng.choice(["conv", "scan", "gate", "residual"]), rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        do = rng.choice(["forward", "train", "step"])
        c = dict(op=op, do=do, n=_log(rng, 1, 16 if do != "step" else 512), channels=8 * _log(rng, 4, 1000) + rng.choice([0, 0, 0, 1, 4]),
                 width=rng.choice([2, 3, 4, 4]), dtype=dtype, bias=rng.random() < 0.5)
        if do != "step":
            c.update(tokens=max(c["n"], _log(rng, 1, 8192 if do == "forward" else 4000)), start=rng.random() < 0.5)
        return c
    if op == "scan":
        do, groups = rng.choice(["forward", "train", "step"]), rng.choice([1, 1, 2, 4, 8])
        c = dict(op=op, do=do, n=_log(rng, 1, 16 if do != "step" else 300), heads=groups * rng.choice([1, 2, 3, 4]), groups=groups,
                 d_head=rng.choice([64, 64, 128]), d_state=rng.choice([64, 128, 128]), dtype=dtype)
        if do != "step":
            c.update(tokens=max(c["n"], _log(rng, 1, 8192 if do == "forward" else 3000)), start=rng.random() < 0.5)
        return c
    tokens = _log(rng, 1, 6000)
    if op == "gate":
        groups = rng.choice([1, 2, 4, 8, 16, 32])
        return dict(op=op, do=rng.choice(["forward", "train"]), tokens=tokens, groups=groups, d=_log(rng, 16, 4096 // groups) if rng.random() < 0.5 else
                    rng.choice([64, 128]), first=rng.random() < 0.5, shared=rng.random() < 0.5, dtype=dtype)
    return dict(op=op, do=rng.choice(["forward", "train"]), tokens=tokens, d=8 * _log(rng, 8, 700) + rng.choice([0, 0, 0, 1, 4]), post=rng.random() < 0.5,
                scale=rng.random() < 0.5, dtype=dtype, res=rng.choice(["f32", dtype]))


# ------------------------------------------------------------------ inputs
def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEV)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _lengths(gen, n, tokens):
    """n lengths of at least 1 that add up to `tokens`, spread over a factor of about 30."""
    w = torch.exp(3.4 * torch.rand(n, generator=gen, device=DEV).double()).cpu()
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * (tokens - n) + 0.5).long()
    cut[-1] = tokens - n
    return (torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)) + 1).tolist()


def _sequences(case, gen):
    """Where the sequences of a batch begin: for the kernels and, token by token, for the plain forms."""
    lens = _lengths(gen, case["n"], case["tokens"])
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    seq = torch.repeat_interleave(torch.arange(case["n"], device=DEV), torch.tensor(lens, device=DEV))
    return dict(lens=lens, cu=cu, seq=seq, pos=torch.arange(case["tokens"], device=DEV) - cu.long()[seq],
                at=torch.cat([i * max(lens) + torch.arange(m) for i, m in enumerate(lens)]).to(DEV))


def _slots(case, gen):
    slots = case["n"] + case["n"] // 4 + 1
    return slots, torch.randperm(slots, generator=gen, device=DEV)[:case["n"]].to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    make = {"conv": _prepare_conv, "scan": _prepare_scan, "gate": _prepare_gate, "residual": _prepare_residual}
    return dict(case=case, **make[case["op"]](case, gen))


def _prepare_conv(case, gen):
    n, c, w, dt = case["n"], case["channels"], case["width"], TYPES[case["dtype"]]
    rows = n if case["do"] == "step" else case["tokens"]
    # the convolved channels are a part of one projection's output, as a layer has them
    wide = torch.empty(rows, c + 8 * (c // 16), dtype=dt, device=DEV)
    x = wide[:, :c]
    x.copy_(_randn(gen, rows, c))
    s = dict(x=x, weight=(2 * _rand(gen, c, w) - 1) / w ** 0.5, bias=0.2 * _randn(gen, c) if case["bias"] else None, y=torch.empty(rows, c, dtype=dt, device=DEV))
    if case["do"] == "step":
        slots, s["slot"] = _slots(case, gen)
        s["pool"] = _randn(gen, slots, w - 1, c).to(dt)
        return s
    s.update(_sequences(case, gen))
    s["S0"] = _randn(gen, n, w - 1, c).to(dt) if case["start"] else None
    s["S"] = torch.empty(n, w - 1, c, dtype=dt, device=DEV)
    if case["do"] == "train":
        s["dy"], s["dS"] = _randn(gen, rows, c).to(dt), _randn(gen, n, w - 1, c).to(dt)
        s["grads"] = [torch.empty(rows, c, dtype=dt, device=DEV), torch.empty(c, w, device=DEV), torch.empty(c, device=DEV) if case["bias"] else None,
                      torch.empty(n, w - 1, c, dtype=dt, device=DEV) if case["start"] else None]
    if own:  # the layer's handle, with its workspace
        import quantized_gated_delta_amd as Q
        s["layer"] = Q.ShortConv(n, rows, c, w, act="silu", dtype=dt, train=case["do"] == "train")
    return s


def _prepare_scan(case, gen):
    n, h, g, p, ns, dt = case["n"], case["heads"], case["groups"], case["d_head"], case["d_state"], TYPES[case["dtype"]]
    rows = n if case["do"] == "step" else case["tokens"]
    # x, B and C are parts of the convolution's output
    parts = [h * p, g * ns, g * ns]
    x, b, c = torch.nn.functional.silu(_randn(gen, rows, sum(parts))).to(dt).split(parts, 1)
    s = dict(x=x.view(rows, h, p), B=b.view(rows, g, ns), C=c.view(rows, g, ns), dt=(0.5 * _randn(gen, rows, h)).to(dt), A=-(1 + 15 * _rand(gen, h)),
             D=1 + 0.2 * _randn(gen, h), y=torch.empty(rows, h, p, dtype=dt, device=DEV))
    step = torch.exp(math.log(0.001) + math.log(100.0) * _rand(gen, h))  # steps of 0.001 to 0.1
    s["bias"] = step + torch.log(-torch.expm1(-step))
    if case["do"] == "step":
        slots, s["slot"] = _slots(case, gen)
        s["pool"] = 0.3 * _randn(gen, slots, h, ns, p)
        return s
    s.update(_sequences(case, gen))
    s["S0"] = 0.3 * _randn(gen, n, h, ns, p) if case["start"] else None
    s["S"] = torch.empty(n, h, ns, p, device=DEV)
    if case["do"] == "train":
        s["dy"], s["dS"] = _randn(gen, rows, h, p).to(dt), 0.3 * _randn(gen, n, h, ns, p)
        gx, gb, gc = torch.empty(rows, sum(parts), dtype=dt, device=DEV).split(parts, 1)
        s["grads"] = dict(dx=gx.view(rows, h, p), ddt=torch.empty(rows, h, dtype=dt, device=DEV), dA=torch.empty(h, device=DEV), dB=gb.view(rows, g, ns),
                          dC=gc.view(rows, g, ns), dD=torch.empty(h, device=DEV), ddt_bias=torch.empty(h, device=DEV),
                          dS0=torch.empty(n, h, ns, p, device=DEV) if case["start"] else None)
    if own:  # the layer's handle, with its workspaces
        import quantized_gated_delta_amd as Q
        s["layer"] = Q.SelectiveScan(n, rows, h, p, ns, n_groups=g, dtype=dt, train=case["do"] == "train")
    return s


def _prepare_gate(case, gen):
    t, g, d, dt = case["tokens"], case["groups"], case["d"], TYPES[case["dtype"]]
    # the gate is a part of one projection's output
    z = torch.empty(t, g * d + 8 * g, dtype=dt, device=DEV)[:, 8 * g:].view(t, g, d)
    z.copy_(_randn(gen, t, g, d))
    s = dict(x=(0.5 * _randn(gen, t, g, d)).to(dt), z=z, weight=1 + 0.1 * _randn(gen, *([d] if case["shared"] else [g, d])), y=torch.empty(t, g, d, dtype=dt, device=DEV))
    if case["do"] == "train":
        s["dy"] = _randn(gen, t, g, d).to(dt)
        s["grads"] = [torch.empty(t, g, d, dtype=dt, device=DEV), torch.empty(t, g, d, dtype=dt, device=DEV), torch.empty_like(s["weight"])]
    if own:  # the norm's handle, with its workspace
        import quantized_gated_delta_amd as Q
        s["layer"] = Q.GatedNorm(g, d, act="silu", gate_first=case["first"], shared_weight=case["shared"], eps=EPS, dtype=dt, train=case["do"] == "train")
    return s


def _prepare_residual(case, gen):
    t, d, dt, rt = case["tokens"], case["d"], TYPES[case["dtype"]], TYPES[case["res"]]
    s = dict(o=_randn(gen, t, d).to(dt), r=(2 * _randn(gen, t, d)).to(rt), weight=1 + 0.1 * _randn(gen, d), post=1 + 0.1 * _randn(gen, d) if case["post"] else None,
             scale=0.5 + 0.1 * _randn(gen, d) if case["scale"] else None, out=torch.empty(t, d, dtype=rt, device=DEV), h=torch.empty(t, d, dtype=dt, device=DEV))
    if case["do"] == "train":
        s["dh"], s["dout"] = _randn(gen, t, d).to(dt), (0.5 * _randn(gen, t, d)).to(rt)
        s["grads"] = dict(do=torch.empty(t, d, dtype=dt, device=DEV), dr=torch.empty(t, d, dtype=rt, device=DEV), dweight=torch.empty(d, device=DEV),
                          dpost=torch.empty(d, device=DEV) if case["post"] else None, dscale=torch.empty(d, device=DEV) if case["scale"] else None)
    if own:  # the norm's handle, with its workspace
        import quantized_gated_delta_amd as Q
        s["layer"] = Q.ResidualNorm(d, eps=EPS, dtype=dt, res_dtype=rt, train=case["do"] == "train")
    return s


# ------------------------------------------------------------------ plain forms
def _silu(p):
    return p / (1 + torch.exp(-p))


def _conv(x, weight, bias, S0, s):
    """x [t, c], S0 [n, w - 1, c]: y, and the last w - 1 inputs of each sequence."""
    w, seq, pos = weight.shape[1], s["seq"], s["pos"]
    p = x * weight[:, w - 1]
    for k in range(1, w):  # the token k before
        ahead = torch.cat([torch.zeros_like(x[:k]), x[:-k] if k < len(x) else x[:0]])[:len(x)]
        before = S0[seq, (w - 1 - k + pos).clamp_max(w - 2)]
        p = p + torch.where((pos >= k)[:, None], ahead, before) * weight[:, w - 1 - k]
    if bias is not None:
        p = p + bias
    lens, last = torch.diff(s["cu"].long()), s["cu"].long()[1:]
    back = torch.arange(w - 1, device=x.device)
    at = lens[:, None] - (w - 1) + back  # row of the sequence, negative: of S0
    own_rows = x[(last[:, None] - (w - 1) + back).clamp_min(0)]
    S = torch.where((at >= 0)[..., None], own_rows, S0.gather(1, (at + w - 1).clamp(0, w - 2)[..., None].expand(-1, -1, x.shape[1])))
    return _silu(p), S


def _plain_conv(s):
    case, f = s["case"], torch.float32
    dt = TYPES[case["dtype"]]
    if case["do"] == "step":
        slot, x = s["slot"].long(), s["x"].to(f)
        rows = torch.cat([s["pool"][slot].to(f), x[:, None]], 1)
        p = (rows * s["weight"].t()).sum(1)
        if case["bias"]:
            p = p + s["bias"]
        s["pool"][slot] = rows[:, 1:].to(dt)
        return {"y": _silu(p).to(dt), "pool": s["pool"]}
    S0 = s["S0"] if s["S0"] is not None else torch.zeros_like(s["S"])
    if case["do"] == "forward":
        y, S = _conv(s["x"].to(f), s["weight"], s["bias"], S0.to(f), s)
        return {"y": y.to(dt), "S": S.to(dt)}
    leaf = {k: v.detach().to(f).requires_grad_() for k, v in dict(x=s["x"], weight=s["weight"], bias=s["bias"], S0=s["S0"]).items() if v is not None}
    y, S = _conv(leaf["x"], leaf["weight"], leaf.get("bias"), leaf.get("S0", S0.to(f)), s)
    grads = torch.autograd.grad([y, S], list(leaf.values()), [s["dy"].to(f), s["dS"].to(f)])
    return {"y": y.detach().to(dt), "S": S.detach().to(dt), **{"d" + k: v.to(dt if k in ("x", "S0") else f) for k, v in zip(leaf, grads)}}


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(x.clamp_max(20))))


def _chunked(x, dt, A, B, C, S, c):
    """x [n, t, h, p], dt [n, t, h], B, C [n, t, g, s], S [n, h, s, p], all fp32: y without D x and the final state, c tokens at a time."""
    n, t, h, p = x.shape
    share, pad = h // B.shape[2], -t % c
    if pad:  # tokens of no time: they leave the state as it is
        x, B, C = (torch.nn.functional.pad(v, (0, 0, 0, 0, 0, pad)) for v in (x, B, C))
        dt = torch.nn.functional.pad(dt, (0, 0, 0, pad))
    cut = lambda v: v.reshape(n, -1, c, v.shape[2], v.shape[3]).permute(1, 0, 3, 2, 4).contiguous()  # noqa: E731
    x, B, C = cut(x), cut(B), cut(C)
    dt = dt.reshape(n, -1, c, h).permute(1, 0, 3, 2)  # [chunks, n, h, c]
    G = (dt.double() * A.double()[:, None]).cumsum(-1)
    low = torch.ones(c, c, device=x.device, dtype=torch.bool).tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).float())
    pair = (C @ B.transpose(-1, -2)).repeat_interleave(share, 2) * decay * dt[..., None, :]
    into, out_of, fade = torch.exp(G.float()), torch.exp((G[..., -1:] - G).float()) * dt, torch.exp(G[..., -1].float())
    added = (B.repeat_interleave(share, 2) * out_of[..., None]).transpose(-1, -2) @ x
    y = pair @ x
    reads = C.repeat_interleave(share, 2) * into[..., None]
    ys = []
    for i in range(len(x)):
        ys.append(y[i] + reads[i] @ S)
        S = fade[i][..., None, None] * S + added[i]
    return torch.stack(ys).permute(1, 0, 3, 2, 4).reshape(n, t + pad, h, p)[:, :t], S


def _padded(x, s, wide):
    """Tokens [t, ...] in a batch padded with zeros, [n, longest, ...]."""
    n, longest = len(s["lens"]), max(s["lens"])
    return torch.zeros(n * longest, *x.shape[1:], device=x.device, dtype=wide).index_copy(0, s["at"], x.to(wide)).view(n, longest, *x.shape[1:])


def _scan(x, dt, A, B, C, D, bias, S0, s):
    f = torch.float32
    step = _softplus(dt.to(f) + bias)
    y, S = _chunked(_padded(x, s, f), _padded(step, s, f), A, _padded(B, s, f), _padded(C, s, f), S0, 64)
    return y.flatten(0, 1).index_select(0, s["at"]) + D[:, None] * x.to(f), S


def _plain_scan(s):
    case, f = s["case"], torch.float32
    to, share = TYPES[case["dtype"]], case["heads"] // case["groups"]
    if case["do"] == "step":
        slot, x = s["slot"].long(), s["x"].to(f)
        dt = _softplus(s["dt"].to(f) + s["bias"])
        B, C = (s[k].to(f).repeat_interleave(share, 1) for k in ("B", "C"))
        S = s["pool"][slot] * torch.exp(dt * s["A"])[..., None, None] + (dt[..., None] * B)[..., None] * x[:, :, None]
        s["pool"][slot] = S
        return {"y": ((S * C[..., None]).sum(2) + s["D"][:, None] * x).to(to), "pool": s["pool"]}
    S0 = s["S0"] if s["S0"] is not None else torch.zeros_like(s["S"])
    names = ["x", "dt", "A", "B", "C", "D", "bias"]
    if case["do"] == "forward":
        y, S = _scan(*(s[k] for k in names), S0, s)
        return {"y": y.to(to), "S": S}
    leaf = {k: s[k].detach().to(f).requires_grad_() for k in names + (["S0"] if s["S0"] is not None else [])}
    y, S = _scan(*(leaf[k] for k in names), leaf.get("S0", S0), s)
    grads = torch.autograd.grad([y, S], list(leaf.values()), [s["dy"].to(f), s["dS"]])
    return {"y": y.detach().to(to), "S": S.detach(), **{"d" + k: v.to(to if k in ("x", "dt", "B", "C") else f) for k, v in zip(leaf, grads)}}


def _rms(x):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _gate(x, z, weight, first):
    return _rms(x * _silu(z)) * weight if first else _rms(x) * weight * _silu(z)


def _plain_gate(s):
    case, f = s["case"], torch.float32
    to = TYPES[case["dtype"]]
    if case["do"] == "forward":
        return {"y": _gate(s["x"].to(f), s["z"].to(f), s["weight"], case["first"]).to(to)}
    leaf = {k: s[k].detach().to(f).requires_grad_() for k in ("x", "z", "weight")}
    y = _gate(*leaf.values(), case["first"])
    dx, dz, dw = torch.autograd.grad(y, list(leaf.values()), s["dy"].to(f))
    return {"y": y.detach().to(to), "dx": dx.to(to), "dz": dz.to(to), "dweight": dw}


def _residual(o, r, weight, post, scale):
    a = o if post is None else _rms(o) * post
    out = r + (a if scale is None else scale * a)
    return out, _rms(out) * weight


def _plain_residual(s):
    case, f = s["case"], torch.float32
    to, rt = TYPES[case["dtype"]], TYPES[case["res"]]
    if case["do"] == "forward":
        out, h = _residual(s["o"].to(f), s["r"].to(f), s["weight"], s["post"], s["scale"])
        return {"out": out.to(rt), "h": h.to(to)}
    leaf = {k: s[k].detach().to(f).requires_grad_() for k in ("o", "r", "weight", "post", "scale") if s[k] is not None}
    out, h = _residual(*(leaf.get(k) for k in ("o", "r", "weight", "post", "scale")))
    grads = torch.autograd.grad([out, h], list(leaf.values()), [s["dout"].to(f), s["dh"].to(f)])
    return {"out": out.detach().to(rt), "h": h.detach().to(to), **{"d" + k: v.to({"o": to, "r": rt}.get(k, f)) for k, v in zip(leaf, grads)}}


# ------------------------------------------------------------------ the library's calls
def _own_conv(s):
    case = s["case"]
    if case["do"] == "step":
        import quantized_gated_delta_amd as Q
        Q.conv_step(s["pool"], s["slot"], s["x"], s["weight"], s["y"], bias=s["bias"], act="silu")
        return {"y": s["y"], "pool": s["pool"]}
    s["layer"].forward(s["x"], s["weight"], s["cu"], s["y"], bias=s["bias"], S0=s["S0"], S_out=s["S"])
    if case["do"] == "forward":
        return {"y": s["y"], "S": s["S"]}
    dx, dw, db, dS0 = s["grads"]
    s["layer"].backward(s["x"], s["weight"], s["cu"], s["dy"], dx, dw, bias=s["bias"], dbias=db, S0=s["S0"], dS_out=s["dS"], dS0=dS0)
    return {"y": s["y"], "S": s["S"], "dx": dx, "dweight": dw, **({"dbias": db} if db is not None else {}), **({"dS0": dS0} if dS0 is not None else {})}


def _own_scan(s):
    case = s["case"]
    if case["do"] == "step":
        import quantized_gated_delta_amd as Q
        Q.scan_step(s["pool"], s["slot"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["y"], D=s["D"], dt_bias=s["bias"])
        return {"y": s["y"], "pool": s["pool"]}
    inputs = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"])
    s["layer"].forward(*inputs, s["y"], D=s["D"], dt_bias=s["bias"], S0=s["S0"], S_out=s["S"])
    if case["do"] == "forward":
        return {"y": s["y"], "S": s["S"]}
    g = s["grads"]
    s["layer"].backward(*inputs, s["dy"], g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], D=s["D"], dt_bias=s["bias"], dD=g["dD"], ddt_bias=g["ddt_bias"],
                        S0=s["S0"], dS_out=s["dS"], dS0=g["dS0"])
    return {"y": s["y"], "S": s["S"], "dbias": g["ddt_bias"], **{k: v for k, v in g.items() if v is not None and k != "ddt_bias"}}


def _own_gate(s):
    s["layer"].forward(s["x"], s["z"], s["weight"], s["y"])
    if s["case"]["do"] == "forward":
        return {"y": s["y"]}
    dx, dz, dw = s["grads"]
    s["layer"].backward(s["x"], s["z"], s["weight"], s["dy"], dx, dz, dw)
    return {"y": s["y"], "dx": dx, "dz": dz, "dweight": dw}


def _own_residual(s):
    s["layer"].forward(s["o"], s["r"], s["out"], weight=s["weight"], h=s["h"], post_weight=s["post"], scale=s["scale"])
    if s["case"]["do"] == "forward":
        return {"out": s["out"], "h": s["h"]}
    g = s["grads"]
    s["layer"].backward(s["o"], s["r"], s["dh"], s["dout"], g["do"], g["dr"], weight=s["weight"], dweight=g["dweight"], post_weight=s["post"],
                        dpost_weight=g["dpost"], scale=s["scale"], dscale=g["dscale"])
    return {"out": s["out"], "h": s["h"], **{k: v for k, v in g.items() if v is not None}}


def run(state):
    call = {"conv": (_plain_conv, _own_conv), "scan": (_plain_scan, _own_scan), "gate": (_plain_gate, _own_gate), "residual": (_plain_residual, _own_residual)}
    return call[state["case"]["op"]][bool(own)](state)


# ------------------------------------------------------------------ work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["do"] == "train"
    if case["op"] == "conv":
        n, c, w = case["n"], case["channels"], case["width"]
        if case["do"] == "step":
            return {"bytes": n * c * e * 2 * w + 4 * c * w, "flops": n * c * (2 * w + 4)}
        t = case["tokens"]
        state = n * (w - 1) * c * e
        return {"bytes": t * c * e * (5 if train else 2) + state * ((4 if case["start"] else 2) if train else 1 + case["start"]) + 4 * c * w * (3 if train else 1),
                "flops": t * c * (2 * w + 4) * (4 if train else 1)}
    if case["op"] == "scan":
        n, h, g, p, ns = (case[k] for k in ("n", "heads", "groups", "d_head", "d_state"))
        states = 4 * n * h * ns * p
        t = n if case["do"] == "step" else case["tokens"]
        # a token: x, dt, B and C in, y out; the state's update and its reading, 5 operations for each entry
        tokens, flops = t * e * (2 * h * p + h + 2 * g * ns), 5.0 * t * h * ns * p
        if case["do"] == "step":
            return {"bytes": tokens + 2 * states, "flops": flops}
        if not train:
            return {"bytes": tokens + states * (1 + case["start"]), "flops": flops}
        back = t * e * (3 * h * p + 2 * h + 4 * g * ns)
        return {"bytes": tokens + back + states * (2 + 3 * case["start"]), "flops": 3 * flops}
    if case["op"] == "gate":
        rows = case["tokens"] * case["groups"] * case["d"]
        return {"bytes": rows * e * (8 if train else 3), "flops": rows * (30 if train else 10)}
    rows, er = case["tokens"] * case["d"], 2 if case["res"] == "bf16" else 4
    return {"bytes": rows * ((4 * e + 5 * er) if train else 2 * e + 2 * er), "flops": rows * (25 if train else 8)}


# ------------------------------------------------------------------ exact
def _sig(x):
    return torch.sigmoid(x)


def _exact_conv(case, s):
    f, w = torch.float64, case["width"]
    weight, bias = s["weight"].to(f), s["bias"].to(f) if s["bias"] is not None else 0.0
    if case["do"] == "step":
        slot, pool = s["slot"].long(), s["pool"].clone()
        rows = torch.cat([s["pool"][slot], s["x"][:, None]], 1)
        pool[slot] = rows[:, 1:]
        p = torch.einsum("nwc,cw->nc", rows.to(f), weight) + bias
        return {"y": p * _sig(p), "pool": pool.to(f)}
    cu = s["cu"].tolist()
    ys, Ss, dxs, dS0s, dw, db = [], [], [], [], torch.zeros_like(weight), torch.zeros_like(weight[:, 0])
    for i in range(case["n"]):
        head = s["S0"][i].to(f) if s["S0"] is not None else torch.zeros(w - 1, case["channels"], dtype=f, device=DEV)
        rows = torch.cat([head, s["x"][cu[i]:cu[i + 1]].to(f)])
        m = len(rows) - w + 1
        p = sum(rows[j:j + m] * weight[:, j] for j in range(w)) + bias
        ys.append(p * _sig(p))
        Ss.append(rows[m:])
        if case["do"] == "train":
            dp = s["dy"][cu[i]:cu[i + 1]].to(f) * _sig(p) * (1 + p * (1 - _sig(p)))
            drows = torch.zeros_like(rows)
            drows[m:] += s["dS"][i].to(f)
            for j in range(w):
                drows[j:j + m] += dp * weight[:, j]
                dw[:, j] += (dp * rows[j:j + m]).sum(0)
            db += dp.sum(0)
            dxs.append(drows[w - 1:])
            dS0s.append(drows[:w - 1])
    out = {"y": torch.cat(ys), "S": torch.stack(Ss)}
    if case["do"] == "train":
        out.update(dx=torch.cat(dxs), dweight=dw, **({"dbias": db} if case["bias"] else {}), **({"dS0": torch.stack(dS0s)} if case["start"] else {}))
    return out


def _exact_scan(case, s):
    f, share = torch.float64, case["heads"] // case["groups"]
    A, D, bias = (s[k].to(f) for k in ("A", "D", "bias"))
    if case["do"] == "step":
        slot, pool, x = s["slot"].long(), s["pool"].to(f), s["x"].to(f)
        dt = torch.nn.functional.softplus(s["dt"].to(f) + bias, threshold=40)
        B, C = (s[k].to(f).repeat_interleave(share, 1) for k in ("B", "C"))
        S = pool[slot] * torch.exp(dt * A)[..., None, None] + torch.einsum("nh,nhs,nhp->nhsp", dt, B, x)
        pool[slot] = S
        return {"y": torch.einsum("nhsp,nhs->nhp", S, C) + D[:, None] * x, "pool": pool}
    n, longest = case["n"], max(s["lens"])
    train = case["do"] == "train"
    S = s["S0"].to(f) if s["S0"] is not None else torch.zeros_like(s["S"]).to(f)
    if train and longest * S.numel() * 8 > 100e9:
        return None
    raw = s["dt"].to(f) + bias
    step = _padded(torch.nn.functional.softplus(raw, threshold=40), s, f)  # 0 behind a sequence's end
    x, B, C = _padded(s["x"], s, f), *(_padded(s[k], s, f).repeat_interleave(share, 2) for k in ("B", "C"))
    a = torch.exp(step * A)
    y, saved = torch.empty_like(x), torch.empty(longest + 1 if train else 1, *S.shape, dtype=f, device=DEV)
    saved[0] = S
    for t in range(longest):
        S = S * a[:, t, :, None, None] + (step[:, t, :, None] * B[:, t])[..., None] * x[:, t, :, None]
        y[:, t] = (S * C[:, t, ..., None]).sum(2)
        if train:
            saved[t + 1] = S
    back = lambda v: v.flatten(0, 1).index_select(0, s["at"])  # noqa: E731
    out = {"y": back(y + D[:, None] * x), "S": S}
    if not train:
        return out
    dy, dS = _padded(s["dy"], s, f), s["dS"].to(f)
    dx, dB, dC, dg, ds = torch.empty_like(x), torch.empty_like(B), torch.empty_like(C), torch.empty_like(step), torch.empty_like(step)
    for t in reversed(range(longest)):
        dC[:, t] = (saved[t + 1] * dy[:, t, :, None]).sum(3)
        dS = dS + C[:, t, ..., None] * dy[:, t, :, None]
        u = (dS * B[:, t, ..., None]).sum(2)
        dx[:, t] = step[:, t, :, None] * u
        ds[:, t] = (u * x[:, t]).sum(2)
        dB[:, t] = step[:, t, :, None] * (dS * x[:, t, :, None]).sum(3)
        dg[:, t] = a[:, t] * (dS * saved[t]).sum((2, 3))
        dS = dS * a[:, t, :, None, None]
    group = lambda v: back(v).view(case["tokens"], case["groups"], share, -1).sum(2)  # noqa: E731
    draw_ = back(ds + A * dg) * _sig(raw)
    out.update(dx=back(dx + D[:, None] * dy), ddt=draw_, dA=(back(dg) * back(step)).sum(0), dB=group(dB), dC=group(dC),
               dD=(s["dy"].to(f) * s["x"].to(f)).sum((0, 2)), dbias=draw_.sum(0))
    if case["start"]:
        out["dS0"] = dS
    return out


def _rms_back(n, rstd, dn):
    """The gradient through n = x rstd."""
    return rstd * (dn - n * (dn * n).mean(-1, keepdim=True))


def _exact_gate(case, s):
    f = torch.float64
    x, z, w = (s[k].to(f) for k in ("x", "z", "weight"))
    act, slope = z * _sig(z), _sig(z) * (1 + z * (1 - _sig(z)))
    u = x * act if case["first"] else x
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    n = u * rstd
    y = n * w if case["first"] else n * w * act
    if case["do"] == "forward":
        return {"y": y}
    dy = s["dy"].to(f)
    over = (0,) if not case["shared"] else (0, 1)
    if case["first"]:
        du = _rms_back(n, rstd, dy * w)
        return {"y": y, "dx": du * act, "dz": du * x * slope, "dweight": (dy * n).sum(over)}
    return {"y": y, "dx": _rms_back(n, rstd, dy * w * act), "dz": dy * n * w * slope, "dweight": (dy * n * act).sum(over)}


def _exact_residual(case, s):
    f = torch.float64
    o, r, w = (s[k].to(f) for k in ("o", "r", "weight"))
    scale = s["scale"].to(f) if s["scale"] is not None else torch.ones_like(w)
    ro = torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
    a = o * ro * s["post"].to(f) if case["post"] else o
    out = r + scale * a
    rn = torch.rsqrt(out.square().mean(-1, keepdim=True) + EPS)
    n = out * rn
    got = {"out": out, "h": n * w}
    if case["do"] == "forward":
        return got
    dh = s["dh"].to(f)
    total = s["dout"].to(f) + _rms_back(n, rn, dh * w)
    da = total * scale
    got.update(do=_rms_back(o * ro, ro, da * s["post"].to(f)) if case["post"] else da, dr=total, dweight=(dh * n).sum(0))
    if case["post"]:
        got["dpost"] = (da * o * ro).sum(0)
    if case["scale"]:
        got["dscale"] = (total * a).sum(0)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "gate": _exact_gate, "residual": _exact_residual}[case["op"]](case, s)
