"""The gated Delta rule over whole sequences and over windows of drafted tokens, and the check of drafted tokens.

Four operators, each in its plain form and as the library's call:

* ``prefill``: y and the final state of ragged sequences (chunked form);
* ``train``:   the same with every gradient;
* ``window``:  the recurrent form over a few tokens per request, on the packed state pool or an fp32 one;
* ``verify``:  how many drafted tokens stand against the target's probabilities, and the token after them.

A state S (d x d) follows S_t = (I - beta k k^T) diag(exp g) S_{t-1} + beta k v^T and is read as y_t = S_t^T q.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt of a chat turn: all launches and little work
        dict(name="prefill_one_prompt", op="prefill", gate="gdn", n=1, tokens=200, heads=48, key_heads=16, d=128, dtype="bf16", start=False),
        # a prefill batch of a serving engine: prompts of every length in one call, three value heads to a key head
        dict(name="prefill_gdn_ragged", op="prefill", gate="gdn", n=12, tokens=12001, heads=48, key_heads=16, d=128, dtype="bf16", start=False),
        # the next part of one long prompt, resumed from its state: few heads' worth of parallel work, a long sequential axis
        dict(name="prefill_kda_long", op="prefill", gate="kda", n=1, tokens=8192, heads=32, key_heads=32, d=128, dtype="bf16", start=True),
        # a training step's layer: a packed batch in bf16
        dict(name="train_gdn", op="train", gate="gdn", n=4, tokens=8192, heads=32, key_heads=16, d=128, dtype="bf16", start=False),
        # the same with a gate per key channel, packed documents of unlike lengths, states carried in
        dict(name="train_kda", op="train", gate="kda", n=3, tokens=4001, heads=32, key_heads=32, d=128, dtype="bf16", start=True),
        # a small model trained in full precision
        dict(name="train_f32_small", op="train", gate="gdn", n=5, tokens=701, heads=8, key_heads=8, d=64, dtype="f32", start=True),
        # drafted tokens of a few requests read against their packed states: a serving engine at low load
        dict(name="window_few_requests", op="window", gate="gdn", n=8, length=4, heads=48, key_heads=48, d=128, bits="6", dtype="bf16", ragged=False, keep=False),
        # the same at full load
        dict(name="window_many_requests", op="window", gate="gdn", n=512, length=5, heads=48, key_heads=48, d=128, bits="6", dtype="bf16", ragged=False, keep=False),
        # the accepted tokens, another number for each request (none for some), brought into the states: 4, 6 and 8 bits by head
        dict(name="window_accepted_kda", op="window", gate="kda", n=128, length=4, heads=32, key_heads=32, d=128, bits="4,6,8", dtype="bf16", ragged=True, keep=True),
        # greedy decoding of one request
        dict(name="verify_greedy_one", op="verify", n=1, length=4, vocab=32000, dtype="bf16", draft=False, temperature=0.0, ragged=False),
        # sampled decoding, the draft model's own probabilities known
        dict(name="verify_sampled", op="verify", n=64, length=4, vocab=131072, dtype="bf16", draft=True, temperature=0.8, ragged=False),
        # drafts looked up in the prompt (no probabilities of their own), an odd vocabulary, fp32 logits, unlike numbers of drafts
        dict(name="verify_lookup_f32", op="verify", n=256, length=3, vocab=50001, dtype="f32", draft=False, temperature=1.0, ragged=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prefill", "train", "window", "verify"])
    gate, dtype, d = rng.choice(["gdn", "kda"]), rng.choice(["bf16", "bf16", "f32"]), rng.choice([128, 128, 64])
    if op in ("prefill", "train"):
        key_heads = rng.choice([1, 2, 4, 8, 16])
        heads = key_heads * rng.choice([1, 1, 2, 3])
        n = _log(rng, 1, 16)
        tokens = max(n, _log(rng, 1, 8192 if op == "prefill" else 4000))
        return dict(op=op, gate=gate, n=n, tokens=tokens, heads=heads, key_heads=key_heads, d=d, dtype=dtype, start=rng.random() < 0.5)
    if op == "window":
        key_heads = rng.choice([1, 2, 4, 8, 16])
        heads = key_heads * rng.choice([1, 1, 2, 3])
        return dict(op=op, gate=gate, n=_log(rng, 1, 300), length=rng.randint(1, 16), heads=heads, key_heads=key_heads, d=d,
                    bits=rng.choice(["6", "8", "4", "4,6,8", "6,16", "32"]), dtype=dtype, ragged=rng.random() < 0.5, keep=rng.random() < 0.5)
    return dict(op=op, n=_log(rng, 1, 100), length=rng.randint(1, 8), vocab=_log(rng, 500, 70000), dtype=dtype, draft=rng.random() < 0.5,
                temperature=rng.choice([0.0, 0.7, 1.0, 1.3]), ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEV)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _unit(gen, *shape):
    return torch.nn.functional.normalize(_randn(gen, *shape), dim=-1)


def _gates(gen, case, *lead):
    """Log-gates of tokens: a rate for each head or channel, as in a layer's parameters, that each token scales."""
    per = (case["heads"],) if case["gate"] == "gdn" else (case["heads"], case["d"])
    rate = 0.001 + 0.499 * _rand(gen, *per)
    return -rate * (0.5 + _rand(gen, *lead, *per))


def _lengths(gen, n, tokens):
    """n lengths of at least 1 that add up to `tokens`, spread over a factor of about 30."""
    w = torch.exp(3.4 * torch.rand(n, generator=gen, device=DEV).double()).cpu()
    cut = torch.floor(torch.cumsum(w, 0) / w.sum() * (tokens - n) + 0.5).long()
    cut[-1] = tokens - n
    return (torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long)) + 1).tolist()


def _bits(case):
    each = [int(b) for b in case["bits"].split(",")]
    return [each[h % len(each)] for h in range(case["heads"])]


def _record(gen, n, bits, d):
    """Packed records of one head, [n, bytes]: codes, row scales, column scales; 16 bits: the state as binary16."""
    if bits == 16:
        return (0.5 * _randn(gen, n, d * d)).half().view(torch.uint8)
    top = 2 ** (bits - 1) - 1
    code = torch.round((0.35 * top * _randn(gen, n, d, d)).clamp(-top, top)).to(torch.int32) & (2 ** bits - 1)
    if bits == 8:
        raw = code.to(torch.uint8)
    elif bits == 4:
        c = code.view(n, d, d // 2, 2)
        raw = (c[..., 0] | c[..., 1] << 4).to(torch.uint8)
    else:
        c = code.view(n, d, d // 4, 4)
        w = c[..., 0] | c[..., 1] << 6 | c[..., 2] << 12 | c[..., 3] << 18
        raw = torch.stack([w & 255, w >> 8 & 255, w >> 16 & 255], -1).to(torch.uint8)
    r = (0.5 + _rand(gen, n, d)) / top
    c = 0.5 + _rand(gen, n, d)
    return torch.cat([raw.reshape(n, -1), r.view(torch.uint8), c.view(torch.uint8)], 1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    make = {"prefill": _prepare_sequences, "train": _prepare_sequences, "window": _prepare_window, "verify": _prepare_verify}
    return dict(case=case, **make[case["op"]](case, gen))


def _prepare_sequences(case, gen):
    n, t, h, hk, d, dt = case["n"], case["tokens"], case["heads"], case["key_heads"], case["d"], TYPES[case["dtype"]]
    lens = _lengths(gen, n, t)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    # q, k and v are parts of one projection's output, as a layer has them
    qkv = torch.empty(t, (2 * hk + h) * d, dtype=dt, device=DEV)
    q, k, v = (x.view(t, -1, d) for x in qkv.split([hk * d, hk * d, h * d], 1))
    q.copy_(_unit(gen, t, hk, d))
    k.copy_(_unit(gen, t, hk, d))
    v.copy_(_randn(gen, t, h, d))
    s = dict(lens=lens, cu=cu, q=q, k=k, v=v, beta=torch.sigmoid(_randn(gen, t, h)).to(dt), g=_gates(gen, case, t).to(dt),
             S0=0.3 * _randn(gen, n, h, d, d) if case["start"] else None)
    # where each token stands in a batch padded to the longest sequence
    s["at"] = torch.cat([i * max(lens) + torch.arange(m) for i, m in enumerate(lens)]).to(DEV)
    s["y"], s["S"] = torch.empty(t, h, d, dtype=dt, device=DEV), torch.empty(n, h, d, d, device=DEV)
    if case["op"] == "train":
        s["dy"], s["dS"] = _randn(gen, t, h, d).to(dt), 0.3 * _randn(gen, n, h, d, d)
        s["grads"] = [torch.empty(x.shape, dtype=dt, device=DEV) for x in (q, k, v, s["beta"], s["g"])]
        s["grads"].append(torch.empty_like(s["S0"]) if case["start"] else None)
    if own:  # the workspaces that a program keeps beside its model
        import quantized_gated_delta_amd as Q
        s["layer"] = Q.ChunkedDelta(n, t, h, d, case["gate"], n_key_heads=hk, dtype=dt, train=case["op"] == "train")
    return s


def _prepare_window(case, gen):
    n, m, h, hk, d, dt = case["n"], case["length"], case["heads"], case["key_heads"], case["d"], TYPES[case["dtype"]]
    slots = n + n // 4 + 1
    s = dict(q=_unit(gen, n, m, hk, d).to(dt), k=_unit(gen, n, m, hk, d).to(dt), v=_randn(gen, n, m, h, d).to(dt),
             beta=torch.sigmoid(_randn(gen, n, m, h)).to(dt), g=_gates(gen, case, n, m).to(dt))
    s["slot"] = torch.randperm(slots, generator=gen, device=DEV)[:n].to(torch.int32)
    s["lens"] = torch.randint(0, m + 1, (n,), generator=gen, device=DEV, dtype=torch.int32) if case["ragged"] else None
    s["y"] = torch.empty(n, m, h, d, dtype=dt, device=DEV)
    s["S"] = torch.empty(n, h, d, d, device=DEV) if case["keep"] else None
    if case["bits"] == "32":
        s["pool"] = 0.3 * _randn(gen, slots, h, d, d)
        return s
    s["pool"] = torch.cat([_record(gen, slots, b, d) for b in _bits(case)], 1)
    if own:  # the pool's handle
        import quantized_gated_delta_amd as Q
        s["handle"] = Q.StatePool(slots, h, d, _bits(case), case["gate"])
        s["handle"].buf.copy_(s["pool"].view(-1))
    return s


def _prepare_verify(case, gen):
    n, m, v, dt = case["n"], case["length"], case["vocab"], TYPES[case["dtype"]]
    target = (3 * _randn(gen, n, m + 1, v)).to(dt)
    target[:, :, v // 7:v // 7 + 5] = -math.inf  # tokens that a grammar or a user forbids
    draft = (target[:, :m].float() + 0.7 * _randn(gen, n, m, v)).to(dt)
    # the tokens that the draft proposes: drawn from it, or its best one
    noise = 0.0 if not case["temperature"] else -torch.log(-torch.log(_rand(gen, n, m, v).clamp(1e-7, 1 - 1e-7))) * case["temperature"]
    tokens = (draft.float() + noise).argmax(-1).to(torch.int32)
    s = dict(target=target, draft=draft if case["draft"] else None, tokens=tokens, u=_rand(gen, n, m), e=-torch.log1p(-_rand(gen, n, v)).clamp_max(80.0).add_(1e-10))
    s["lens"] = torch.randint(0, m + 1, (n,), generator=gen, device=DEV, dtype=torch.int32) if case["ragged"] else None
    s["accepted"], s["next"] = (torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2))
    if own:  # its workspace
        import quantized_gated_delta_amd as Q
        s["checker"] = Q.DraftVerifier(n, m, v)
    return s


# ------------------------------------------------------------------ plain forms
def _inverse(a):
    """(I + a)^-1 of strictly lower triangular a: the product of (I + (-a)^(2^i))."""
    c = a.shape[-1]
    eye = torch.eye(c, device=a.device, dtype=a.dtype)
    power, inv, reach = -a, eye - a, 2
    while reach < c:
        power = power @ power
        inv = inv + inv @ power
        reach *= 2
    return inv


def _chunked(q, k, v, beta, g, S, c):
    """q, k, v, g [n, t, h, d], beta [n, t, h], S [n, h, d, d], all fp32: y [n, t, h, d] and the final state, c tokens at a time.
    g has a last axis of 1 where a head has one gate."""
    n, t, h, d = v.shape
    pad = -t % c
    if pad:  # tokens that leave the state as it is
        q, k, v, g = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)) for x in (q, k, v, g))
        beta = torch.nn.functional.pad(beta, (0, 0, 0, pad))
    q, k, v, g = (x.view(n, -1, c, h, x.shape[-1]).permute(1, 0, 3, 2, 4).contiguous() for x in (q, k, v, g))  # [chunks, n, h, c, .]
    beta = beta.view(n, -1, c, h).permute(1, 0, 3, 2)[..., None]
    G = g.cumsum(-2)
    low = torch.ones(c, c, device=q.device, dtype=torch.bool).tril()
    if g.shape[-1] == 1:
        decay = torch.exp((G - G.transpose(-1, -2)).masked_fill(~low, -math.inf))
        kk, qk = (k @ k.transpose(-1, -2)) * decay, (q @ k.transpose(-1, -2)) * decay
    else:
        kd = torch.exp((G[..., :, None, :] - G[..., None, :, :]).masked_fill(~low[:, :, None], -math.inf)) * k[..., None, :, :]
        kk, qk = (kd @ k[..., None]).squeeze(-1), (kd @ q[..., None]).squeeze(-1)
    T = _inverse(beta * kk.tril(-1)) * beta.transpose(-1, -2)
    k_in, q_in, k_out = k * torch.exp(G), q * torch.exp(G), k * torch.exp(G[..., -1:, :] - G)
    fade = torch.exp(G[..., -1, :])[..., None]
    w, u0 = T @ k_in, T @ v
    ys = []
    for i in range(len(v)):
        u = u0[i] - w[i] @ S
        ys.append(q_in[i] @ S + qk[i] @ u)
        S = fade[i] * S + k_out[i].transpose(-1, -2) @ u
    y = torch.stack(ys).permute(1, 0, 3, 2, 4).reshape(n, t + pad, h, d)
    return y[:, :t], S


def _padded(x, s, wide):
    """Tokens [t, ...] in a batch padded with zeros, [n, longest, ...]."""
    n, longest = len(s["lens"]), max(s["lens"])
    return torch.zeros(n * longest, *x.shape[1:], device=x.device, dtype=wide).index_copy(0, s["at"], x.to(wide)).view(n, longest, *x.shape[1:])


def _plain_sequences(s, q, k, v, beta, g, S0):
    case, share = s["case"], s["case"]["heads"] // s["case"]["key_heads"]
    f = torch.float32
    q, k = (_padded(x, s, f).repeat_interleave(share, 2) for x in (q, k))
    v, beta, g = (_padded(x, s, f) for x in (v, beta, g))
    if S0 is None:
        S0 = torch.zeros_like(s["S"])
    y, S = _chunked(q, k, v, beta, g if case["gate"] == "kda" else g[..., None], S0, 16 if case["gate"] == "kda" else 64)
    return y.flatten(0, 1).index_select(0, s["at"]).to(TYPES[case["dtype"]]), S


def _plain_prefill(s):
    y, S = _plain_sequences(s, *(s[x] for x in ("q", "k", "v", "beta", "g", "S0")))
    return {"y": y, "S": S}


def _plain_train(s):
    names = ["q", "k", "v", "beta", "g"] + (["S0"] if s["S0"] is not None else [])
    leaf = {x: s[x].detach().requires_grad_() for x in names}
    y, S = _plain_sequences(s, *(leaf.get(x) for x in ("q", "k", "v", "beta", "g", "S0")))
    grads = torch.autograd.grad([y, S], list(leaf.values()), [s["dy"], s["dS"]])
    return {"y": y.detach(), "S": S.detach(), **{"d" + x: gr for x, gr in zip(names, grads)}}


def _unpack(rec, bits, d, wide):
    """The states that records [n, bytes] of one head stand for."""
    n = rec.shape[0]
    if bits == 16:
        return rec.contiguous().view(torch.float16).to(wide).view(n, d, d)
    size = d * d * bits // 8
    raw, scales = rec[:, :size], rec[:, size:].contiguous().view(torch.float32).to(wide)
    if bits == 8:
        code = raw.contiguous().view(torch.int8).to(torch.int32)
    elif bits == 4:
        code = torch.stack([raw & 15, raw >> 4], -1).to(torch.int32)
    else:
        b = raw.reshape(n, -1, 3).to(torch.int32)
        w = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16
        code = torch.stack([w & 63, w >> 6 & 63, w >> 12 & 63, w >> 18], -1)
    code = code.view(n, d, d)
    code = torch.where(code >= 2 ** (bits - 1), code - 2 ** bits, code).to(wide)
    return code * scales[:, :d, None] * scales[:, None, d:]


def _pool_states(s, wide):
    case, slot = s["case"], s["slot"].long()
    if case["bits"] == "32":
        return s["pool"][slot].to(wide)
    d, bits, rec = case["d"], _bits(case), s["pool"][slot]
    size = [2 * d * d if b == 16 else d * d * b // 8 + 8 * d for b in bits]
    parts = rec.split(size, 1)
    S = torch.empty(len(slot), len(bits), d, d, device=DEV, dtype=wide)
    for b in sorted(set(bits)):  # all heads of one width at once
        heads = [h for h in range(len(bits)) if bits[h] == b]
        S[:, heads] = _unpack(torch.stack([parts[h] for h in heads], 1).flatten(0, 1), b, d, wide).view(len(slot), -1, d, d)
    return S


def _window_inputs(s, wide):
    """The inputs with the tokens past a request's length made to leave its state as it is and to read nothing."""
    case, share = s["case"], s["case"]["heads"] // s["case"]["key_heads"]
    q, k, v, beta, g = (s[x].to(wide) for x in ("q", "k", "v", "beta", "g"))
    q, k = q.repeat_interleave(share, 2), k.repeat_interleave(share, 2)
    if s["lens"] is not None:
        live = torch.arange(case["length"], device=DEV) < s["lens"][:, None]
        q, k, v, g, beta = (torch.where(live.view(*live.shape, *[1] * (x.dim() - 2)), x, 0) for x in (q, k, v, g, beta))
    return q, k, v, beta, g if case["gate"] == "kda" else g[..., None]


def _plain_window(s):
    y, S = _chunked(*_window_inputs(s, torch.float32), _pool_states(s, torch.float32), s["case"]["length"])
    y = y.to(TYPES[s["case"]["dtype"]])
    return {"y": y, "S": S} if s["case"]["keep"] else {"y": y}


def _plain_verify(s):
    case, (n, m, v) = s["case"], (s["case"]["n"], s["case"]["length"], s["case"]["vocab"])
    tokens, target, each = s["tokens"].long(), s["target"].float(), torch.arange(n, device=DEV)
    lens = torch.full((n,), m, device=DEV) if s["lens"] is None else s["lens"].long()
    if not case["temperature"]:
        best = target.argmax(-1)
        right = best[:, :m] == tokens
    else:
        p = torch.exp((target - target.amax(-1, keepdim=True)) / case["temperature"])
        p = p / p.sum(-1, keepdim=True)
        if s["draft"] is None:
            q = torch.zeros(n, m, v, device=DEV).scatter_(2, tokens[..., None], 1.0)
        else:
            q = s["draft"].float()
            q = torch.exp((q - q.amax(-1, keepdim=True)) / case["temperature"])
            q = q / q.sum(-1, keepdim=True)
        right = s["u"] * q.gather(2, tokens[..., None]).squeeze(-1) < p[:, :m].gather(2, tokens[..., None]).squeeze(-1)
    right &= torch.arange(m, device=DEV) < lens[:, None]
    accepted = right.long().cumprod(1).sum(1)
    if not case["temperature"]:
        after = best[each, accepted]
    else:
        q = torch.where((accepted < lens)[:, None], q[each, accepted.clamp_max(m - 1)], 0)
        rest = (p[each, accepted] - q).clamp_min(0)
        rest = torch.where((rest > 0).any(1, keepdim=True), rest, p[each, accepted])
        after = (rest / s["e"]).argmax(-1)
    return {"accepted": accepted.to(torch.int32), "next": after.to(torch.int32)}


# ------------------------------------------------------------------ the library's calls
def _own_prefill(s):
    s["layer"].forward(s["q"], s["k"], s["v"], s["beta"], s["g"], s["cu"], s["y"], S0=s["S0"], S_out=s["S"])
    return {"y": s["y"], "S": s["S"]}


def _own_train(s):
    dq, dk, dv, dbeta, dg, dS0 = s["grads"]
    s["layer"].forward(s["q"], s["k"], s["v"], s["beta"], s["g"], s["cu"], s["y"], S0=s["S0"], S_out=s["S"])
    s["layer"].backward(s["q"], s["k"], s["v"], s["beta"], s["g"], s["cu"], s["dy"], dq, dk, dv, dbeta, dg, S0=s["S0"], dS_out=s["dS"], dS0=dS0)
    return {"y": s["y"], "S": s["S"], "dq": dq, "dk": dk, "dv": dv, "dbeta": dbeta, "dg": dg, **({} if dS0 is None else {"dS0": dS0})}


def _own_window(s):
    if s["case"]["bits"] == "32":
        import quantized_gated_delta_amd as Q
        Q.f32_window_update(s["pool"], s["slot"], s["q"], s["k"], s["v"], s["beta"], s["g"], y=s["y"], S_out=s["S"], lens=s["lens"], gate=s["case"]["gate"])
    else:
        s["handle"].window_update(s["slot"], s["q"], s["k"], s["v"], s["beta"], s["g"], y=s["y"], S_out=s["S"], lens=s["lens"])
    return {"y": s["y"], "S": s["S"]} if s["case"]["keep"] else {"y": s["y"]}


def _own_verify(s):
    s["checker"].verify(s["target"], s["tokens"], s["accepted"], s["next"], draft=s["draft"], accept_u=s["u"], sample_e=s["e"], lens=s["lens"],
                        temperature=s["case"]["temperature"])
    return {"accepted": s["accepted"], "next": s["next"]}


def run(state):
    call = {"prefill": (_plain_prefill, _own_prefill), "train": (_plain_train, _own_train),
            "window": (_plain_window, _own_window), "verify": (_plain_verify, _own_verify)}[state["case"]["op"]]
    return call[bool(own)](state)


# ------------------------------------------------------------------ work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "verify":
        n, m, v = case["n"], case["length"], case["vocab"]
        if not case["temperature"]:
            return {"bytes": n * (m + 1) * v * e, "flops": n * (m + 1) * v}
        rows = m + 1 + (m if case["draft"] else 0)
        return {"bytes": n * (rows * v * e + 4 * v), "flops": n * v * (4 * rows + 3)}
    h, hk, d = case["heads"], case["key_heads"], case["d"]
    t = case["tokens"] if case["op"] != "window" else case["n"] * case["length"]
    # a token: q and k of the key heads, v, beta, g in, y out; the update and its reading, 7 operations for each entry of a state
    tokens = t * e * (2 * hk * d + 2 * h * d + h + h * (d if case["gate"] == "kda" else 1))
    flops, states = 7.0 * t * h * d * d, 4 * case["n"] * h * d * d
    if case["op"] == "prefill":
        return {"bytes": tokens + states * (1 + case["start"]), "flops": flops}
    if case["op"] == "train":
        # forwards, and backwards: the inputs and y's gradient in, a gradient for each input out
        back = t * e * (4 * hk * d + 3 * h * d + 2 * h + 2 * h * (d if case["gate"] == "kda" else 1))
        return {"bytes": tokens + back + states * (2 + 3 * case["start"]), "flops": 3 * flops}
    pool = states if case["bits"] == "32" else case["n"] * sum(2 * d * d if b == 16 else d * d * b // 8 + 8 * d for b in _bits(case))
    return {"bytes": tokens + pool + (states if case["keep"] else 0), "flops": flops}


# ------------------------------------------------------------------ exact
def _steps(q, k, v, beta, a, S, saved=None):
    """The recurrence token by token, everything in 64 bits: q, k, v, a [n, t, h, .]; `saved` gets each state before its token."""
    y = torch.empty_like(v)
    for t in range(v.shape[1]):
        if saved is not None:
            saved[t] = S
        S = S * a[:, t, :, :, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.sum(S * k[:, t, :, :, None], 2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        y[:, t] = torch.sum(S * q[:, t, :, :, None], 2)
    return y, S


def _steps_back(q, k, v, beta, a, saved, S_last, dy, dS):
    """The adjoint of _steps: gradients of q, k, v, beta, log a (each [n, t, h, .]) and of the first state."""
    dq, dk, dv, db, dg = (torch.empty_like(x) for x in (q, k, v, beta, a))
    S = S_last
    for t in reversed(range(v.shape[1])):
        kt, bt, at, before = k[:, t], beta[:, t, :, None], a[:, t, :, :, None], saved[t]
        faded = before * at
        e = v[:, t] - torch.sum(faded * kt[..., None], 2)
        dq[:, t] = torch.sum(S * dy[:, t, :, None], 3)
        dS = dS + q[:, t, :, :, None] * dy[:, t, :, None]
        du = torch.sum(dS * kt[..., None], 2)
        dv[:, t] = bt * du
        db[:, t] = torch.sum(du * e, 2)
        dk[:, t] = torch.sum(dS * (bt * e)[:, :, None], 3) - torch.sum(faded * (bt * du)[:, :, None], 3)
        dS = (dS - kt[..., None] * (bt * du)[:, :, None]) * at
        whole = torch.sum(dS * before, 3)
        dg[:, t] = whole if a.shape[-1] > 1 else torch.sum(whole, 2, keepdim=True)
        S = before
    return dq, dk, dv, db, dg, dS


def exact(case, seed):
    if case["op"] == "verify":
        return None
    s, f = prepare(case, seed), torch.float64
    if case["op"] == "window":
        q, k, v, beta, g = _window_inputs(s, f)
        y, S = _steps(q, k, v, beta, torch.exp(g), _pool_states(s, f))
        return {"y": y, "S": S} if case["keep"] else {"y": y}
    share, longest = case["heads"] // case["key_heads"], max(s["lens"])
    q, k = (_padded(s[x], s, f).repeat_interleave(share, 2) for x in ("q", "k"))
    v, beta, g = (_padded(s[x], s, f) for x in ("v", "beta", "g"))
    a = torch.exp(g if case["gate"] == "kda" else g[..., None])
    S0 = torch.zeros_like(s["S"]).to(f) if s["S0"] is None else s["S0"].to(f)
    if case["op"] == "train" and longest * S0.numel() * 8 > 120e9:
        return None
    back = lambda x: x.flatten(0, 1).index_select(0, s["at"])  # noqa: E731
    saved = torch.empty(longest, *S0.shape, dtype=f, device=DEV) if case["op"] == "train" else None
    y, S = _steps(q, k, v, beta, a, S0, saved)
    out = {"y": back(y), "S": S}
    if case["op"] == "prefill":
        return out
    dq, dk, dv, db, dg, dS0 = _steps_back(q, k, v, beta, a, saved, S, _padded(s["dy"], s, f), s["dS"].to(f))
    shared = lambda x: back(x).view(case["tokens"], case["key_heads"], share, case["d"]).sum(2)  # noqa: E731
    out.update(dq=shared(dq), dk=shared(dk), dv=back(dv), dbeta=back(db), dg=back(dg if case["gate"] == "kda" else dg[..., 0]))
    if case["start"]:
        out["dS0"] = dS0
    return out
