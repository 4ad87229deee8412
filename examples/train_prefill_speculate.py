"""One gated-Delta layer from training to speculative decoding, on one GPU.

    python examples/train_prefill_speculate.py

1. A language model of one layer (embedding, gated Delta rule with the token before as the key, output
   matrix) is trained on ragged batches of sequences that repeat a hidden word: ``ChunkedDelta``
   forward and backward behind a ``torch.autograd.Function``.
2. Prompts of different lengths are read in one call, and their final states stored in a packed pool
   (``quant_state``).
3. Tokens are generated several at a time: m tokens are looked up in the text so far, one ``window_update``
   reads all of them against the pool, ``DraftVerifier`` says how many stand and what comes next, a second
   ``window_update`` gives the states after those, and ``quant_state`` stores them, one requantization
   for the whole window.

``generate`` returns the tokens and the part of the drafted ones that stood.  On an fp32 pool, greedy
speculative decoding gives the tokens that one window per token gives.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import quantized_gated_delta_amd as Q  # noqa: E402

VOCAB, WIDTH, H, HK, D = 64, 128, 4, 2, 64


class Delta(torch.autograd.Function):
    """y of the sequences that cu marks off, with gradients; `layer` is a ChunkedDelta(train=True), which
    holds the saved states of one forward call: a second one before the first one's backward needs a layer of its own."""

    @staticmethod
    def forward(ctx, layer, cu, q, k, v, beta, g):
        y = torch.empty_like(v)
        call = layer.forward(q, k, v, beta, g, cu, y)
        ctx.layer, ctx.cu, ctx.call = layer, cu, call
        ctx.save_for_backward(q, k, v, beta, g)
        return y

    @staticmethod
    def backward(ctx, dy):
        inputs = ctx.saved_tensors
        grads = [torch.empty_like(x) for x in inputs]
        ctx.layer.backward(*inputs, ctx.cu, dy.contiguous(), *grads, call=ctx.call)
        return (None, None, *grads)


class Model:
    def __init__(self, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        shapes = dict(embed=(VOCAB + 1, WIDTH), q=(WIDTH, HK * D), k=(WIDTH, HK * D), v=(WIDTH, H * D), beta=(WIDTH, H),
                      g=(WIDTH, H), out=(H * D, VOCAB))
        self.w = {}
        for name, (rows, cols) in shapes.items():
            scale = 1.0 if name == "embed" else rows ** -0.5
            self.w[name] = (scale * torch.randn(rows, cols, generator=gen)).to(device).requires_grad_()

    def inputs(self, tokens, before):
        """q, k, v, beta, g of tokens of any shape and the tokens before them (VOCAB: none)."""
        x = self.w["embed"][tokens]
        part = {n: (self.w["embed"][before] if n == "k" else x) @ self.w[n] for n in ("q", "k", "v", "beta", "g")}
        q, k = (torch.nn.functional.normalize(part[n].unflatten(-1, (HK, D)), dim=-1) for n in ("q", "k"))
        gate = torch.nn.functional.logsigmoid(part["g"] + 4.0)  # mostly kept
        return q, k, part["v"].unflatten(-1, (H, D)), torch.sigmoid(part["beta"]), gate

    def logits(self, y):
        return y.flatten(-2) @ self.w["out"]


def flat(seqs):
    """The tokens of all sequences, those before them, and where each sequence begins and ends."""
    start = torch.tensor([VOCAB])
    cu = torch.tensor([0] + [len(s) for s in seqs]).cumsum(0).to(torch.int32)
    return torch.cat(seqs).cuda(), torch.cat([torch.cat([start, s[:-1]]) for s in seqs]).cuda(), cu.cuda()


def batch(gen, n, longest):
    """n sequences, each a word of 6 tokens repeated."""
    seqs = []
    for _ in range(n):
        word = torch.randperm(VOCAB, generator=gen)[:6]
        seqs.append(word.repeat(longest // 6 + 2)[:int(torch.randint(longest // 2, longest + 2, (1,), generator=gen))])
    return seqs


def train(model, steps=150, n=16, longest=90, seed=1):
    gen = torch.Generator().manual_seed(seed)
    layer = Q.ChunkedDelta(n, n * longest, H, D, n_key_heads=HK, dtype=torch.float32, train=True)
    opt = torch.optim.Adam(model.w.values(), lr=5e-3)
    losses = []
    for _ in range(steps):
        seqs = batch(gen, n, longest)
        tokens, before, cu = flat([s[:-1] for s in seqs])
        y = Delta.apply(layer, cu, *(x.contiguous() for x in model.inputs(tokens, before)))
        loss = torch.nn.functional.cross_entropy(model.logits(y), torch.cat([s[1:] for s in seqs]).cuda())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def prefill(model, prompts):
    """The states after each prompt and the (greedy) token that follows it."""
    tokens, before, cu = flat(prompts)
    layer = Q.ChunkedDelta(len(prompts), len(tokens), H, D, n_key_heads=HK, dtype=torch.float32)
    q, k, v, beta, g = model.inputs(tokens, before)
    y, S = torch.empty_like(v), torch.empty(len(prompts), H, D, D, device="cuda")
    layer.forward(q, k, v, beta, g, cu, y, S_out=S)
    return S, model.logits(y[cu[1:].long() - 1]).argmax(-1)


class Packed:
    """The states of n requests in a packed pool."""

    def __init__(self, S, bits=8):
        n = S.shape[0]
        self.pool, self.slot = Q.StatePool(n, H, D, [bits] * H), torch.arange(n, dtype=torch.int32, device="cuda")
        self.store(S)

    def store(self, S):
        self.pool.quant_state(self.slot, S)

    def window(self, *inputs, **out):
        self.pool.window_update(self.slot, *inputs, **out)


class Full:
    """The same in fp32."""

    def __init__(self, S):
        self.S, self.slot = S.clone(), torch.arange(S.shape[0], dtype=torch.int32, device="cuda")

    def store(self, S):
        self.S.copy_(S)

    def window(self, *inputs, **out):
        Q.f32_window_update(self.S, self.slot, *inputs, **out)


def look_up(text, m):
    """What followed the last token of `text` when it was there before; else that token again."""
    for i in range(len(text) - 2, -1, -1):
        if text[i] == text[-1]:
            return (text[i + 1:i + 1 + m] * m)[:m]
    return [text[-1]] * m


@torch.no_grad()
def generate(model, states, prompts, first, count, m, temperature=0.0, seed=2):
    """`count` tokens for each request from its `first` on, m drafted at a time (0: none)."""
    n, gen = first.numel(), torch.Generator("cuda").manual_seed(seed)
    check = Q.DraftVerifier(n, max(m, 1), VOCAB)
    S = torch.empty(n, H, D, D, device="cuda")
    accepted, after = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    lens = torch.full((n,), m, dtype=torch.int32, device="cuda")
    texts = [p.tolist() + [t] for p, t in zip(prompts, first.tolist())]  # the last token is in no state yet
    drafted = stood = 0
    while min(len(t) - len(p) for t, p in zip(texts, prompts)) <= count:
        rows = torch.tensor([t[-2:] + look_up(t, max(m, 1)) for t in texts], device="cuda")
        inputs = [x.contiguous() for x in model.inputs(rows[:, 1:], rows[:, :-1])]
        y = torch.empty_like(inputs[2])
        states.window(*inputs, y=y)
        u = torch.rand(n, max(m, 1), device="cuda", generator=gen)
        e = torch.empty(n, VOCAB, device="cuda").exponential_(generator=gen)
        check.verify(model.logits(y).contiguous(), rows[:, 2:].to(torch.int32).contiguous(), accepted, after,
                     accept_u=u, sample_e=e, lens=lens, temperature=temperature)
        states.window(*inputs, S_out=S, lens=accepted + 1)
        states.store(S)
        for text, row, a, t in zip(texts, rows.tolist(), accepted.tolist(), after.tolist()):
            text += row[2:2 + a] + [t]
            drafted, stood = drafted + m, stood + a
    return [t[len(p):len(p) + count] for t, p in zip(texts, prompts)], stood / max(drafted, 1)


def main(steps=150, count=48, m=4):
    model = Model()
    losses = train(model, steps)
    print("loss %.3f -> %.3f" % (losses[0], losses[-1]))
    prompts = [s[:-1] for s in batch(torch.Generator().manual_seed(9), 8, 60)]
    S, first = prefill(model, prompts)
    one, _ = generate(model, Full(S), prompts, first, count, 0)
    several, rate = generate(model, Full(S), prompts, first, count, m)
    packed, packed_rate = generate(model, Packed(S), prompts, first, count, m)
    sampled, sampled_rate = generate(model, Packed(S), prompts, first, count, m, temperature=0.8)
    right = sum(t == p[(len(p) + i) % 6].item() for o, p in zip(packed, prompts) for i, t in enumerate(o)) / (count * len(prompts))
    print("fp32 states: %d drafted tokens at a time give the tokens of one at a time: %s (accepted %.0f %%)" % (m, one == several, 100 * rate))
    print("8-bit states: %.0f %% of the tokens continue the word (accepted %.0f %%; sampled, %.0f %%)" % (
        100 * right, 100 * packed_rate, 100 * sampled_rate))
    return dict(losses=losses, one=one, several=several, packed=packed, sampled=sampled, right=right, rates=(rate, packed_rate, sampled_rate))


if __name__ == "__main__":
    main()
