"""sq_verify_draft on the GPU against the definition in 64 bits.

Tokens have to be equal, except where the 64-bit values themselves leave the choice open by less
than the fp32 arithmetic's error: 1e-5 relative, for a comparison u q < p or between the two
best scores r / e (r is a difference: 1e-5 of p).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
EDGE = 1e-5


def softmax(x, temperature):
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    m = x.max(-1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(np.isneginf(m), 0.0, np.exp((x - m) / temperature))
    z = e.sum(-1, keepdims=True)
    return np.divide(e, z, out=np.zeros_like(e), where=z > 0)


def plain(target, tokens, draft, u, e, lens, temperature):
    """accepted, next, and for each whether the choice is closer than EDGE."""
    n, m = tokens.shape
    V = target.shape[-1]
    accepted, after, open_ = np.zeros(n, int), np.zeros(n, int), np.zeros(n, bool)
    for b in range(n):
        L = m if lens is None else min(max(int(lens[b]), 0), m)
        if not temperature:
            clean = np.where(np.isnan(target[b]), -np.inf, np.minimum(target[b], np.finfo(np.float32).max))
            best = [int(r.argmax()) if r.max() > -np.inf else -1 for r in clean]
            a = 0
            while a < L and best[a] == tokens[b, a]:
                a += 1
            accepted[b], after[b] = a, best[a]
            continue
        p = softmax(target[b], temperature)
        q = softmax(draft[b], temperature) if draft is not None else None
        a = 0
        while a < L:
            x = tokens[b, a]
            if not 0 <= x < V:
                break
            px, qx = p[a, x], 1.0 if q is None else q[a, x]
            left = float(u[b, a]) * qx
            if left != px and abs(left - px) <= EDGE * max(left, px):
                open_[b] = True
            if not left < px:
                break
            a += 1
        r, scale = p[a].copy(), p[a].copy()
        if a < L:
            if q is not None:
                r = r - q[a]
                scale = np.maximum(p[a], q[a])
            elif 0 <= tokens[b, a] < V:
                r[tokens[b, a]] -= 1
        doubt = EDGE * scale
        r = np.maximum(r, 0)
        if not (r > 0).any():
            r = p[a]
        score = r / e[b]
        accepted[b] = a
        after[b] = int(score.argmax()) if (r > 0).any() else -1
        if (r > 0).any():
            top = after[b]
            hi, rest = score + doubt / e[b], score[top] - doubt[top] / e[b][top]
            hi[top] = -1
            open_[b] |= bool((hi >= rest).any())
    return accepted, after, open_


def call(target, tokens, draft=None, u=None, e=None, lens=None, temperature=1.0, checker=None):
    n, m = tokens.shape
    checker = checker or Q.DraftVerifier(n, m, target.shape[-1])
    accepted, after = (torch.full((n,), 77, dtype=torch.int32, device=DEV) for _ in range(2))
    checker.verify(target, tokens, accepted, after, draft=draft, accept_u=u, sample_e=e, lens=lens, temperature=temperature)
    return accepted, after


def make(n, m, V, dtype=torch.bfloat16, draft=True, seed=0, spread=3.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    target = (spread * randn(n, m + 1, V)).to(dtype)
    d = (target[:, :m].float() + 0.7 * randn(n, m, V)).to(dtype)
    noise = -torch.log(-torch.log(torch.rand(n, m, V, generator=gen, device=DEV).clamp(1e-7, 1 - 1e-7)))
    tokens = (d.float() + noise).argmax(-1).to(torch.int32)
    u = torch.rand(n, m, generator=gen, device=DEV)
    e = -torch.log1p(-torch.rand(n, V, generator=gen, device=DEV)) + 1e-9
    return dict(target=target, tokens=tokens, draft=d if draft else None, u=u, e=e)


def check(x, lens=None, temperature=1.0, checker=None, most_open=0.2):
    got = call(lens=lens, temperature=temperature, checker=checker, **x)
    host = {k: None if v is None else v.float().cpu().numpy().astype(np.float64) if v.is_floating_point() else v.cpu().numpy() for k, v in x.items()}
    a, t, open_ = plain(host["target"], host["tokens"], host["draft"], host["u"], host["e"], None if lens is None else lens.cpu().numpy(), temperature)
    sure = ~open_
    assert open_.mean() <= most_open
    assert np.array_equal(got[0].cpu().numpy()[sure], a[sure]) and np.array_equal(got[1].cpu().numpy()[sure], t[sure])
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temperature", [0.0, 0.3, 1.0, 2.5])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 255, 2048, 2049, 4097, 50001])
def test_vocabularies(dtype, temperature, V):
    """Odd sizes put the rows at every alignment; the longest is split over workgroups."""
    for draft in (True, False):
        check(make(3, 2, V, dtype, draft, seed=V), temperature=temperature)


@pytest.mark.parametrize("m", [1, 3, 8, 32])
@pytest.mark.parametrize("draft", [True, False])
def test_drafts(m, draft):
    n = 9
    lens = torch.arange(n, dtype=torch.int32, device=DEV) * (m + 2) // (n - 1) - 1   # -1 .. m + 1
    check(make(n, m, 3001, draft=draft, seed=m), lens=lens)
    check(make(n, m, 3001, draft=draft, seed=m + 50), lens=lens, temperature=0.0)


def test_many_requests():
    check(make(300, 4, 1000, seed=1))


def test_parts_of_a_request_are_all_seen():
    """Many workgroups to each request, many requests: the token is the best of all the parts, every time.  Scores
    nearer to each other than 1e-3 (some 1e-6 in fp32, a hundredfold where p - q nearly vanishes) are left open."""
    n, V = 64, 100003
    for seed in range(40):
        x = make(n, 1, V, torch.bfloat16, seed=seed + 100)
        accepted, after = call(**x)
        p, q = (torch.softmax(x[k].double(), -1) for k in ("target", "draft"))
        each = torch.arange(n, device=DEV)
        a = accepted.long()
        rest = (p[each, a] - torch.where((a == 0)[:, None], q[:, 0], 0)).clamp_min(0) / x["e"].double()
        top = rest.topk(2, -1)
        sure = top.values[:, 1] < (1 - 1e-3) * top.values[:, 0]
        assert sure.sum() > n / 2
        assert torch.equal(after.long()[sure], top.indices[sure, 0]), seed


def test_noise_below_zero_takes_a_token_out():
    """Whether the draft gave the token more than the target or less."""
    for draft in (True, False):
        for V in (100, 50001):
            x = make(8, 2, V, draft=draft, seed=V + draft)
            x["u"].fill_(2.0)   # nothing stands unless p > 2 q
            accepted, before = check(x)
            x["e"][:, 1::2] = -1e-10
            accepted, after = check(x)
            assert (after >= 0).all() and (after % 2 == 0).all()


def test_equal_distributions_accept_all():
    x = make(20, 4, 500, seed=2)
    x["draft"] = x["target"][:, :4].contiguous()
    accepted, _ = check(x)
    assert (accepted == 4).all()


def test_ties_go_to_the_lower_token():
    V = 9000
    target = torch.zeros(2, 2, V, device=DEV)
    target[0, 0, 5000] = target[0, 0, 17] = 4.0
    target[1, 0, 8999] = 1.0
    tokens = torch.tensor([[17], [8999]], dtype=torch.int32, device=DEV)
    accepted, after = call(target, tokens, temperature=0.0)
    assert accepted.tolist() == [1, 1] and after.tolist() == [0, 0]
    # sampled: equal scores everywhere but at the rejected token 0
    same = torch.zeros(1, 2, V, device=DEV)
    accepted, after = call(same, torch.zeros(1, 1, dtype=torch.int32, device=DEV), u=torch.full((1, 1), 0.9, device=DEV), e=torch.ones(1, V, device=DEV))
    assert accepted.tolist() == [0] and after.tolist() == [1]


def test_masked_rows():
    """Minus infinity and NaN take a token out; a row without any token left accepts nothing and gives -1; a row of the
    type's lowest value is a uniform one."""
    for dtype in (torch.bfloat16, torch.float32):
        V = 4100
        x = make(5, 2, V, dtype, seed=3)
        x["target"][0, 0] = -math.inf
        x["target"][1, 0, :] = -math.inf
        x["target"][1, 0, 77] = 1.0
        x["tokens"][1, 0] = 77
        x["target"][2, 0, 1::2] = math.nan
        x["target"][3] = torch.finfo(dtype).min
        x["target"][4, 0, 1234] = math.inf
        x["tokens"][4, 0] = 1234
        x["draft"][4, 0] = -math.inf   # a draft row without probabilities: u * 0 < p stands
        accepted, after = check(x)
        assert accepted[0] == 0 and after[0] == -1 and accepted[1] >= 1 and accepted[4] >= 1
        accepted, after = check(x, temperature=0.0)
        assert accepted[0] == 0 and after[0] == -1 and accepted[1] >= 1 and accepted[4] >= 1


def test_tokens_outside_the_vocabulary():
    for temperature in (0.0, 1.0):
        for draft in (True, False):
            x = make(3, 2, 600, draft=draft, seed=4)
            x["tokens"][0, 0], x["tokens"][1, 0], x["tokens"][2, 0] = -1, 600, 2 ** 31 - 1
            accepted, after = call(temperature=temperature, **x)
            assert (accepted == 0).all() and ((after >= 0) & (after < 600)).all()


def test_nothing_left_of_the_target():
    """p = q, and the draft proposes a token of probability 0: it is rejected, r is 0 everywhere, and
    the token comes from p."""
    V = 5000
    t = torch.full((1, 2, V), -math.inf, device=DEV)
    t[:, :, 3000:3004] = 0.0
    e = torch.ones(1, V, device=DEV)
    e[0, 3002] = 0.5
    accepted, after = call(t, torch.tensor([[5]], dtype=torch.int32, device=DEV), draft=t[:, :1].contiguous(), u=torch.full((1, 1), 0.5, device=DEV), e=e)
    assert accepted.tolist() == [0] and after.tolist() == [3002]


@pytest.mark.parametrize("V", [9, 1000, 70000])
def test_nothing_left_in_any_number_of_parts(V):
    """As above, with the vocabulary in one part and in many."""
    t = torch.full((2, 2, V), -math.inf, device=DEV)
    t[:, :, V // 2:V // 2 + 3] = 0.0
    e = torch.ones(2, V, device=DEV)
    e[0, V // 2 + 1] = e[1, V // 2 + 2] = 0.5
    tokens = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    accepted, after = call(t, tokens, draft=t[:, :1].contiguous(), u=torch.full((2, 1), 0.5, device=DEV), e=e)
    assert accepted.tolist() == [0, 0] and after.tolist() == [V // 2 + 1, V // 2 + 2]


def test_padded_rows():
    """Logits as a part of a wider, padded output layer."""
    x = make(4, 3, 1001, seed=5)
    dense = call(**x)
    wide_t = torch.full((4, 4, 1040), math.nan, dtype=x["target"].dtype, device=DEV)
    wide_d = torch.full((4, 3, 1003), math.nan, dtype=x["target"].dtype, device=DEV)
    wide_t[:, :, :1001], wide_d[:, :, :1001] = x["target"], x["draft"]
    x["target"], x["draft"] = wide_t[:, :, :1001], wide_d[:, :, :1001]
    padded = call(**x)
    assert all(torch.equal(a, b) for a, b in zip(dense, padded))


def test_draws_from_the_target():
    """Over many seeds the first token (accepted, or drawn after a rejection) has the target's distribution
    whatever the draft's: 40000 draws, each frequency within 5 standard deviations."""
    V, n = 6, 20000
    gen = torch.Generator(device=DEV).manual_seed(6)
    target = torch.tensor([0.5, -1.0, 2.0, 0.0, -math.inf, 1.0], device=DEV)
    draft = torch.tensor([1.5, 1.0, -1.0, 0.3, 0.5, -0.5], device=DEV)
    p, q = torch.softmax(target, 0).cpu().double(), torch.softmax(draft, 0)
    count = torch.zeros(V, dtype=torch.float64)
    for _ in range(2):
        tokens = torch.multinomial(q, n, replacement=True, generator=gen).view(n, 1).to(torch.int32)
        u = torch.rand(n, 1, generator=gen, device=DEV)
        e = -torch.log1p(-torch.rand(n, V, generator=gen, device=DEV)) + 1e-9
        accepted, after = call(target.expand(n, 2, V).contiguous(), tokens, draft=draft.expand(n, 1, V).contiguous(), u=u, e=e)
        first = torch.where(accepted > 0, tokens[:, 0], after).long()
        count += torch.bincount(first, minlength=V).cpu().double()
    total = 2 * n
    assert (((count / total) - p).abs() <= 5 * (p * (1 - p) / total).sqrt() + 1e-12).all(), (count / total, p)


def test_same_bits_other_stream_and_graph():
    x = make(8, 4, 40000, seed=7)
    checker = Q.DraftVerifier(8, 4, 40000)
    first = call(checker=checker, **x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = call(**x)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    accepted, after = (torch.empty(8, dtype=torch.int32, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        checker.verify(x["target"], x["tokens"], accepted, after, draft=x["draft"], accept_u=x["u"], sample_e=x["e"])
    for i in range(4):
        fresh = make(8, 4, 40000, seed=70 + i)
        for k in x:
            x[k].copy_(fresh[k])
        want = call(**x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(accepted, want[0]) and torch.equal(after, want[1]), i


def test_python_refusals():
    x = make(2, 3, 100)
    checker = Q.DraftVerifier(2, 3, 100)
    out = [torch.empty(2, dtype=torch.int32, device=DEV) for _ in range(2)]
    ok = dict(draft=x["draft"], accept_u=x["u"], sample_e=x["e"])
    with pytest.raises(TypeError):
        checker.verify(x["target"].half(), x["tokens"], *out, **ok)
    with pytest.raises(ValueError):
        checker.verify(x["target"][:, :, :50], x["tokens"], *out, **ok)
    with pytest.raises(ValueError):
        checker.verify(x["target"], x["tokens"], *out, **dict(ok, draft=x["draft"].float()))
    with pytest.raises(TypeError):
        checker.verify(x["target"], x["tokens"].long(), *out, **ok)
    with pytest.raises(TypeError):
        checker.verify(x["target"], x["tokens"], *out, **dict(ok, accept_u=None))
    with pytest.raises(ValueError):
        checker.verify(x["target"], x["tokens"], *out, **dict(ok, sample_e=x["e"][:1]))
    with pytest.raises(Q.SQError):   # a larger batch than the workspace
        y = make(40, 3, 100)
        call(checker=checker, **y)
