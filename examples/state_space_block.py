"""One state-space block from training to decoding, on one GPU.

    python examples/state_space_block.py

1. A language model of one block is trained on ragged batches: residual norm, input projection, ``ShortConv``,
   ``SelectiveScan``, ``GatedNorm``, output projection, residual norm, output matrix.  Each operator is behind a
   ``torch.autograd.Function``; x, B and C stay parts of the convolution's output, and their gradients parts of
   one tensor.
2. Prompts of different lengths are read in one call; the convolution's last inputs and the scan's states go
   into pools.
3. Tokens are generated one by one: ``conv_step`` and ``scan_step`` on the pools, the norms as in training.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import quantized_gated_delta_amd as Q  # noqa: E402

VOCAB, WIDTH, H, P, G, N, TAPS = 48, 96, 4, 64, 2, 64, 4
INNER, PARTS = H * P, [H * P, G * N, G * N]
CHANNELS = sum(PARTS)


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, layer, cu, x, weight, bias, S_out):
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        layer.forward(x, weight, cu, y, bias=bias, S_out=S_out)
        ctx.layer, ctx.cu = layer, cu
        ctx.save_for_backward(x, weight, bias)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        dx, dw, db = torch.empty(x.shape, dtype=x.dtype, device=x.device), torch.empty_like(weight), torch.empty_like(bias)
        ctx.layer.backward(x, weight, ctx.cu, dy.contiguous(), dx, dw, bias=bias, dbias=db)
        return None, None, dx, dw, db, None


def parts(xbc):
    """x, B and C as parts of one tensor."""
    x, b, c = xbc.split(PARTS, 1)
    return x.unflatten(1, (H, P)), b.unflatten(1, (G, N)), c.unflatten(1, (G, N))


class Scan(torch.autograd.Function):
    """`layer` is a SelectiveScan(train=True), which holds the saved states of one forward call."""

    @staticmethod
    def forward(ctx, layer, cu, xbc, dt, A, D, bias, S_out):
        x, b, c = parts(xbc)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        ctx.call = layer.forward(x, dt, A, b, c, cu, y, D=D, dt_bias=bias, S_out=S_out)
        ctx.layer, ctx.cu = layer, cu
        ctx.save_for_backward(xbc, dt, A, D, bias)
        return y

    @staticmethod
    def backward(ctx, dy):
        xbc, dt, A, D, bias = ctx.saved_tensors
        x, b, c = parts(xbc)
        grad, ddt = torch.empty_like(xbc), torch.empty(dt.shape, dtype=dt.dtype, device=dt.device)
        dx, db, dc = parts(grad)
        dA, dD, dbias = torch.empty_like(A), torch.empty_like(D), torch.empty_like(bias)
        ctx.layer.backward(x, dt, A, b, c, ctx.cu, dy.contiguous(), dx, ddt, dA, db, dc, D=D, dt_bias=bias, dD=dD, ddt_bias=dbias, call=ctx.call)
        return None, None, grad, ddt, dA, dD, dbias, None


class Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, layer, x, z, weight):
        y = torch.empty_like(x)
        layer.forward(x, z, weight, y)
        ctx.layer = layer
        ctx.save_for_backward(x, z, weight)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, weight = ctx.saved_tensors
        dx, dz, dw = torch.empty_like(x), torch.empty(z.shape, dtype=z.dtype, device=z.device), torch.empty_like(weight)
        ctx.layer.backward(x, z, weight, dy.contiguous(), dx, dz, dw)
        return None, dx, dz, dw


class Residual(torch.autograd.Function):
    """r + scale * rms(o) * post and its norm; without r, post and scale: o and its norm."""

    @staticmethod
    def forward(ctx, layer, o, r, weight, post, scale):
        r_out, h = torch.empty_like(o), torch.empty_like(o)
        layer.forward(o, r, r_out, weight=weight, h=h, post_weight=post, scale=scale)
        ctx.layer = layer
        ctx.save_for_backward(o, r, weight, post, scale)
        return r_out, h

    @staticmethod
    def backward(ctx, dr_out, dh):
        o, r, weight, post, scale = ctx.saved_tensors
        new = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
        do, dr, dw, dpost, dscale = (new(t) for t in (o, r, weight, post, scale))
        ctx.layer.backward(o, r, dh.contiguous(), dr_out.contiguous(), do, dr, weight=weight, dweight=dw, post_weight=post, dpost_weight=dpost, scale=scale,
                           dscale=dscale)
        return None, do, dr, dw, dpost, dscale


class Model:
    def __init__(self, seed=0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        w = dict(embed=randn(VOCAB, WIDTH), into=randn(WIDTH, INNER + CHANNELS + H) / WIDTH ** 0.5, taps=0.5 * randn(CHANNELS, TAPS), taps_bias=torch.zeros(CHANNELS),
                 A=-(1 + 3 * torch.rand(H, generator=gen)), D=torch.ones(H), dt_bias=torch.full((H,), -2.0), gate=torch.ones(1, INNER),
                 out=randn(INNER, WIDTH) / INNER ** 0.5, first=torch.ones(WIDTH), post=torch.ones(WIDTH), scale=torch.full((WIDTH,), 0.5), last=torch.ones(WIDTH),
                 head=randn(WIDTH, VOCAB) / WIDTH ** 0.5)
        self.w = {k: v.to(device).requires_grad_() for k, v in w.items()}
        kinds = dict(dtype=torch.float32, train=True)
        self.gate = Q.GatedNorm(1, INNER, gate_first=True, shared_weight=False, **kinds)
        self.norm = Q.ResidualNorm(WIDTH, **kinds)

    def layers(self, n_seq, n_tokens):
        """A convolution and a scan with workspaces for batches of up to these sizes."""
        return (Q.ShortConv(n_seq, n_tokens, CHANNELS, TAPS, dtype=torch.float32, train=True),
                Q.SelectiveScan(n_seq, n_tokens, H, P, N, G, dtype=torch.float32, train=True))

    def project(self, h):
        return (h @ self.w["into"]).split([INNER, CHANNELS, H], 1)

    def finish(self, y, z, r):
        """Logits from the scan's output, its gate, and the residual."""
        w = self.w
        y = Gate.apply(self.gate, y.reshape(-1, 1, INNER), z.unflatten(1, (1, INNER)), w["gate"]).flatten(1)
        return Residual.apply(self.norm, y @ w["out"], r, w["last"], w["post"], w["scale"])[1] @ w["head"]

    def logits(self, layers, tokens, cu, S_conv=None, S_scan=None):
        """Of every token of the sequences; S_conv, S_scan: where their final states go."""
        w, (conv, scan) = self.w, layers
        r, h = Residual.apply(self.norm, w["embed"][tokens], None, w["first"], None, None)
        z, xbc, dt = self.project(h)
        xbc = Conv.apply(conv, cu, xbc, w["taps"], w["taps_bias"], S_conv)
        y = Scan.apply(scan, cu, xbc, dt, w["A"], w["D"], w["dt_bias"], S_scan)
        return self.finish(y, z, r)

    @torch.no_grad()
    def step(self, tokens, slot, conv_pool, scan_pool):
        """Logits after one more token of each request, whose states are on its slot of the pools."""
        w, n = self.w, len(tokens)
        r, h = Residual.apply(self.norm, w["embed"][tokens], None, w["first"], None, None)
        z, xbc, dt = self.project(h)
        out, y = torch.empty(n, CHANNELS, device="cuda"), torch.empty(n, H, P, device="cuda")
        Q.conv_step(conv_pool, slot, xbc, w["taps"], out, bias=w["taps_bias"])
        x, b, c = parts(out)
        Q.scan_step(scan_pool, slot, x, dt, w["A"], b, c, y, D=w["D"], dt_bias=w["dt_bias"])
        return self.finish(y, z, r)


def flat(seqs):
    """The tokens of all sequences, and where each one begins and ends."""
    cu = torch.tensor([0] + [len(s) for s in seqs]).cumsum(0).to(torch.int32)
    return torch.cat(seqs).cuda(), cu.cuda()


def batch(gen, n, longest):
    """n sequences, each a word of 3 tokens repeated."""
    seqs = []
    for _ in range(n):
        word = torch.randperm(VOCAB, generator=gen)[:3]
        seqs.append(word.repeat(longest // 3 + 2)[:int(torch.randint(longest // 2, longest + 2, (1,), generator=gen))])
    return seqs


def train(model, steps=200, n=16, longest=70, seed=1):
    gen = torch.Generator().manual_seed(seed)
    layers = model.layers(n, n * longest)
    opt = torch.optim.Adam(model.w.values(), lr=5e-3)
    losses = []
    for _ in range(steps):
        seqs = batch(gen, n, longest)
        tokens, cu = flat([s[:-1] for s in seqs])
        loss = torch.nn.functional.cross_entropy(model.logits(layers, tokens, cu), torch.cat([s[1:] for s in seqs]).cuda())
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def generate(model, prompts, count):
    """`count` greedy tokens for each prompt, and the logits that each came from."""
    n = len(prompts)
    tokens, cu = flat(prompts)
    conv_pool, scan_pool = torch.empty(n, TAPS - 1, CHANNELS, device="cuda"), torch.empty(n, H, N, P, device="cuda")
    logits = model.logits(model.layers(n, len(tokens)), tokens, cu, conv_pool, scan_pool)[cu[1:].long() - 1]
    slot, out, seen = torch.arange(n, dtype=torch.int32, device="cuda"), [], []
    for _ in range(count):
        seen.append(logits)
        out.append(logits.argmax(-1))
        logits = model.step(out[-1], slot, conv_pool, scan_pool)
    return torch.stack(out, 1), torch.stack(seen, 1)


def main(steps=200, count=24):
    model = Model()
    losses = train(model, steps)
    print("loss %.3f -> %.3f" % (losses[0], losses[-1]))
    prompts = [s[:-1] for s in batch(torch.Generator().manual_seed(9), 8, 60)]
    tokens, seen = generate(model, prompts, count)
    right = sum(t == p[(len(p) + i) % 3].item() for o, p in zip(tokens.tolist(), prompts) for i, t in enumerate(o)) / tokens.numel()
    print("%.0f %% of the generated tokens continue the word" % (100 * right))
    return dict(model=model, losses=losses, prompts=prompts, tokens=tokens, seen=seen)


if __name__ == "__main__":
    main()
