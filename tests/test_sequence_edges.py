"""The sequence and window calls where their kernels take another way: gates of unlike strength,
large batches, keys that resemble each other.  Oracle and tolerances as in test_sequence.py.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q
from tests.test_sequence import BF, DEV, F32, batch, check, check_window, near, recurrence, run, window, window_batch

pytestmark = pytest.mark.gpu


def strong_blocks(b, low=20.0, high=60.0):
    """Every other block of 16 tokens under gates that no block's common reference can hold."""
    g = b["g"]
    weak = (torch.arange(g.shape[0], device=DEV) // 16 % 2 == 0).view(-1, *[1] * (g.dim() - 1))
    strong = -(low + (high - low) * torch.rand(g.shape, generator=torch.Generator(DEV).manual_seed(1), device=DEV))
    b["g"] = torch.where(weak, g, strong.to(g.dtype))
    return b


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, F32), (128, F32)])
def test_strong_gates_on_shared_key_heads(gate, d, dtype):
    """Three heads one after another in a workgroup, each with blocks of both kinds; equal bits every time."""
    b = strong_blocks(batch(gate, (130, 64, 75), H=6, Hk=2, d=d, dtype=dtype, gates=(0.001, 0.3), seed=30))
    first = run(b, train=True)
    check(b, first, train=True)
    for _ in range(5):
        again = run(b, train=True)
        for n in first:
            assert torch.equal(first[n], again[n]), n


def alike(shape, cosine, seed):
    """Unit keys, any two of them at about this cosine (1: one key at every token)."""
    gen = torch.Generator(DEV).manual_seed(seed)
    randn = lambda *s: torch.nn.functional.normalize(torch.randn(*s, generator=gen, device=DEV), dim=-1)  # noqa: E731
    return torch.nn.functional.normalize(cosine ** 0.5 * randn(*shape[:-3], 1, *shape[-2:]) + (1 - cosine) ** 0.5 * randn(*shape), dim=-1)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("m", [5, 9, 12, 16])
@pytest.mark.parametrize("cosine,beta", [(0.9, 0.9), (0.99, 0.9), (0.99, 0.99), (1.0, 1.0)])
def test_window_of_similar_keys(gate, m, cosine, beta):
    """Drafts that repeat tokens: the pairs' matrix is far from the identity, its powers grow and cancel."""
    for bits in (32, [4, 6, 8, 16]):
        b = window_batch(gate, 3, m, 4, 2, 128, F32, bits, gates=(0.0, 0.01), seed=31)
        b["k"] = alike(b["k"].shape, cosine, 32)
        b["beta"].fill_(beta)
        check_window(b, *window(b))


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("cosine,beta", [(0.99, 0.99), (1.0, 1.0)])
def test_sequence_of_similar_keys(gate, cosine, beta):
    b = batch(gate, (130, 40), H=2, d=64, dtype=F32, gates=(0.0, 0.01), beta=beta, seed=33)
    b["k"] = alike(b["k"].shape, cosine, 34)
    check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("reset", [-math.inf, -100.0, -50.0])
@pytest.mark.parametrize("at", [(0,), (3, 10), (0, 1, 2, 3, 12, 13, 14, 15)], ids=str)
def test_window_resets_among_weak_gates(gate, reset, at):
    """Gates that forget everything before and after weak ones: what lies between them keeps its accuracy."""
    for bits in (32, [6, 4]):
        b = window_batch(gate, 3, 16, 2, 1, 128, F32, bits, gates=(0.001, 0.1), seed=35)
        b["g"][:, list(at)] = reset
        check_window(b, *window(b))


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, F32)])
def test_gates_above_one_after_a_reset(gate, d, dtype):
    """The log-gates of a block dip to -95 and come back to -50: the sum at the block's end does not show it."""
    b = batch(gate, (70,), H=2, Hk=1, d=d, dtype=dtype, gates=(0.0, 0.1), seed=37)
    b["g"][19], b["g"][20], b["beta"][19] = -95.0, 45.0, 0.0
    check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, F32)])
def test_window_gates_above_one_after_a_reset(gate, d, dtype):
    b = window_batch(gate, 2, 16, 2, 1, d, dtype, 32, gates=(0.0, 0.1), seed=36)
    b["g"][:, 3], b["g"][:, 4], b["beta"][:, 3] = -95.0, 45.0, 0.0
    check_window(b, *window(b))


def test_speculative_step():
    """The step as the header describes it: a window of the last sampled token and m drafts for y, the draft check, the
    same window with lens = accepted + 1 into the state.  Against one token at a time in 64 bits."""
    n, m, H, d, V = 6, 4, 2, 64, 50
    gen = torch.Generator(DEV).manual_seed(38)
    table = {x: torch.randn(V, H * d, generator=gen, device=DEV) for x in "qkv"}
    table.update(beta=torch.rand(V, H, generator=gen, device=DEV), g=-torch.rand(V, H, generator=gen, device=DEV))
    for x in "qk":
        table[x] = torch.nn.functional.normalize(table[x].view(V, H, d), dim=-1).view(V, H * d)
    out = torch.randn(H * d, V, generator=gen, device=DEV)
    S0 = 0.3 * torch.randn(n, H, d, d, generator=gen, device=DEV)
    last = torch.randint(0, V, (n,), generator=gen, device=DEV)

    def step(tok, S):  # one token of one request in 64 bits: the best next token and the state
        row = {x: table[x][tok].to("cpu", torch.float64) for x in table}
        y, S = recurrence(*(row[x].view(1, H, d) for x in "qkv"), row["beta"].view(1, H), row["g"].view(1, H, 1), S)
        return int((y.flatten() @ out.to("cpu", torch.float64)).argmax()), S

    # drafts: request i's first i tokens are the best ones, the rest are not
    drafts, states, best = torch.zeros(n, m, dtype=torch.long, device=DEV), [], []
    for i in range(n):
        tok, S, trail = int(last[i]), S0[i].to("cpu", torch.float64), []
        for j in range(m + 1):
            tok, S = step(tok, S)
            trail.append((tok, S))
            if j < m:
                drafts[i, j] = tok if j < i else (tok + 1) % V
                if j >= i:
                    break
        states.append(trail[-1][1]), best.append(trail[-1][0])
    window_tokens = torch.cat([last[:, None], drafts], 1)
    q, k, v = (table[x][window_tokens].view(n, m + 1, H, d) for x in "qkv")
    beta, g = (table[x][window_tokens] for x in ("beta", "g"))
    pool, slot = S0.clone(), torch.arange(n, dtype=torch.int32, device=DEV)
    y, S = torch.empty_like(v), torch.empty_like(S0)
    accepted, after = (torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2))
    Q.f32_window_update(pool, slot, q, k, v, beta, g, y=y)
    Q.DraftVerifier(n, m, V).verify((y.flatten(-2) @ out).contiguous(), drafts.to(torch.int32), accepted, after, temperature=0.0)
    Q.f32_window_update(pool, slot, None, k, v, beta, g, S_out=S, lens=accepted + 1)
    assert accepted.tolist() == [min(i, m) for i in range(n)] and after.tolist() == best
    near(S, torch.stack(states), "S")


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("d,dtype", [(128, BF), (64, F32)])
def test_a_gate_of_nan_is_seen(gate, d, dtype):
    """A log-gate that is not a number leaves none in its head's results from its token on, as in the decode step, and
    none of it in any other head or sequence."""
    b = batch(gate, (100, 90), H=4, Hk=2, d=d, dtype=dtype, seed=39)
    clean = run(b, train=True)
    b["g"][(130, 2) if gate == "gdn" else (130, 2, 7)] = math.nan
    out = run(b, train=True)
    assert out["y"][130:, 2].isnan().all() and out["S"][1, 2].isnan().all()
    for n in ("dv", "dbeta", "dg"):
        assert out[n][130, 2].isnan().any(), n
        others = [0, 1, 3]
        assert torch.equal(out[n][:, others], clean[n][:, others]) and torch.equal(out[n][:100], clean[n][:100]), n
    for n in ("dq", "dk"):
        assert out[n][130, 1].isnan().any() and torch.equal(out[n][:, 0], clean[n][:, 0]) and torch.equal(out[n][:100], clean[n][:100]), n
    assert torch.equal(out["S"][0], clean["S"][0]) and torch.equal(out["y"][:100], clean["y"][:100])

    b = window_batch(gate, 2, 7, 4, 2, d, dtype, [4, 6, 8, 16], seed=40)
    clean = window(b)
    b["g"][(1, 3, 2) if gate == "gdn" else (1, 3, 2, 7)] = math.nan
    y, S = window(b)
    assert y[1, 3:, 2].isnan().all() and S[1, 2].isnan().all()
    y[1, :, 2], S[1, 2] = clean[0][1, :, 2], clean[1][1, 2]
    assert torch.equal(y, clean[0]) and torch.equal(S, clean[1])


def ragged(n, seed, longest=40):
    """Lengths of n sequences: empty ones, short ones, a few of more than one chunk."""
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, longest, (n,), generator=gen).tolist()
    lens[n // 3], lens[n // 2], lens[-1], lens[0] = 130, 65, 64, 0
    return tuple(lens)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("d,dtype", [(128, BF), (128, F32), (64, BF), (64, F32)])
def test_batches_of_many_heads_and_sequences(gate, d, dtype):
    """From 2048 slices of 16 columns on the forward scan takes 32 to a workgroup; an odd number of (sequence, head) pairs."""
    H, n = 5, (2048 * 16 // d + 4) // 5
    n += n % 2 == 0
    assert n * H * d // 16 >= 2048
    b = batch(gate, ragged(n, 41, 24), H=H, Hk=1, d=d, dtype=dtype, seed=42)
    check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_pairs_y_of_the_other_type(gate, dtype):
    b = batch(gate, ragged(53, 43, 24), H=5, Hk=5, dtype=dtype, start=False, gates=(0.0, 9.0), seed=44)
    check(b, run(b, y_dtype=F32 if dtype == BF else BF))


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("n", [64, 65, 129])
def test_many_sequences(gate, n):
    """The chunks' sequences are found 64 at a time: one round of probes, two."""
    b = batch(gate, ragged(n, n, 24), H=1, d=64, dtype=F32, skip=3, extra=2, seed=45)
    check(b, run(b, train=True), train=True)


@pytest.mark.parametrize("gate", ["gdn", "kda"])
def test_thousands_of_sequences(gate):
    """Three rounds of probes.  Forward against 64 bits, gradients against those of 60 sequences at a time, which the
    tests above hold to 64 bits: each within 1e-5 of their norm of them, so 2e-5 of each other."""
    n = 4200
    b = batch(gate, ragged(n, n, 2), H=1, d=64, dtype=F32, seed=45)
    out = run(b, train=True)
    check(b, out)
    parts = {x: [] for x in ("dq", "dk", "dv", "dbeta", "dg", "dS0")}
    for lo in range(0, n, 60):
        t0, t1 = int(b["cu"][lo]), int(b["cu"][lo + 60])
        part = {x: b[x][t0:t1].clone() for x in ("q", "k", "v", "beta", "g", "dy")}
        part.update({x: b[x][lo:lo + 60].clone() for x in ("S0", "dS")}, cu=b["cu"][lo:lo + 61] - t0, case=dict(b["case"], lens=b["case"]["lens"][lo:lo + 60]))
        got = run(part, train=True)
        for x in parts:
            parts[x].append(got[x])
    for x in parts:
        want = torch.cat(parts[x])
        assert (out[x] - want).norm() <= 2e-5 * want.norm(), x


@pytest.mark.parametrize("gate", ["gdn", "kda"])
@pytest.mark.parametrize("low,high", [(3.0, 9.0), (20.0, 60.0), (140.0, 300.0)])
def test_window_strong_gates_on_a_packed_pool(gate, low, high):
    for d, dtype in ((128, BF), (64, F32)):
        b = window_batch(gate, 4, 16, 4, 2, d, dtype, [4, 6, 8, 16], lens=[16, 9, 1, 0], gates=(low, high), seed=46)
        check_window(b, *window(b))
