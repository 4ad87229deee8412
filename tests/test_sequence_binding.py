"""What the Python classes of the sequence and draft-check calls refuse before anything is
enqueued.  The tensors lie in host memory and say that they are on the device, so no GPU is needed."""
import pytest

torch = pytest.importorskip("torch")

import quantized_gated_delta_amd as Q

BF = torch.bfloat16


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def device(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def sequence(n=100, heads=4, key_heads=2, d=128):
    x = dict(q=device(n, key_heads, d), k=device(n, key_heads, d), v=device(n, heads, d), beta=device(n, heads), g=device(n, heads),
             cu=torch.tensor([0, n], dtype=torch.int32).as_subclass(OnDevice), y=device(n, heads, d))
    return Q.ChunkedDelta(1, n, heads, d, n_key_heads=key_heads, device="cpu", train=True), x


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_one_token_expanded_to_all(name):
    """Storage for one token behind a shape of many: the kernels would read past it."""
    layer, x = sequence()
    x[name] = x[name][:1].expand(100, -1, -1)
    assert x[name].stride(0) == 0
    with pytest.raises(ValueError, match=name):
        layer.forward(*x.values(), stream=0)
    y = x.pop("y")
    grads = [torch.empty(x[n].shape, dtype=BF).as_subclass(OnDevice) for n in ("q", "k", "v", "beta", "g")]
    with pytest.raises(ValueError, match=name):
        layer.backward(*x.values(), y, *grads, stream=0)


def test_tokens_that_overlap():
    layer, x = sequence()
    x["v"] = device(100 * 4 * 128).as_strided((100, 4, 128), (128, 128, 1))
    with pytest.raises(ValueError, match="v"):
        layer.forward(*x.values(), stream=0)


@pytest.mark.parametrize("shape", [(1, 1, 1000), (4, 1, 1000), (1, 3, 1000)], ids=str)
@pytest.mark.parametrize("which", ["target", "draft"])
def test_one_row_of_logits_expanded(shape, which):
    checker = Q.DraftVerifier(4, 2, 1000, device="cpu")
    target, draft = device(4, 3, 1000), device(4, 2, 1000)
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    if which == "target":
        target = device(*shape).expand(4, 3, 1000)
    else:
        draft = device(shape[0], min(shape[1], 2), 1000).expand(4, 2, 1000)
    with pytest.raises(ValueError, match=which):
        checker.verify(target, device(4, 2, **i32), device(4, **i32), device(4, **i32), draft=draft, accept_u=device(4, 2, **f32),
                       sample_e=device(4, 1000, **f32), stream=0)


@pytest.mark.parametrize("n,m", [(1, 1), (1, 2), (5, 1)])
def test_one_row_expanded_over_one_axis(n, m):
    """Where only one axis has more than one row, its stride is the rows'."""
    checker = Q.DraftVerifier(n, m, 64, device="cpu")
    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    with pytest.raises(ValueError, match="target"):
        checker.verify(device(1, 1, 64).expand(n, m + 1, 64), device(n, m, **i32), device(n, **i32), device(n, **i32),
                       accept_u=device(n, m, **f32), sample_e=device(n, 64, **f32), stream=0)


@pytest.mark.parametrize("temperature", [3e-39, 3.5e-39, 4.2e-39])
def test_temperature_whose_scale_overflows(temperature):
    """1 / T is still finite, log2(e) / T, which the kernels scale by, is not."""
    from tests.test_sequence_abi import refused, verify
    refused(Q.SQ_EINVAL, "temperature", verify, temperature=temperature)


def test_header_says_which_tokens_a_speculative_step_keeps():
    """A window holds the last sampled token and the drafts after it: of those that stand one more is kept than drafts."""
    from quantized_gated_delta_amd import sq
    text = " ".join(open(sq.HEADER).read().replace("\n *", " ").split())
    assert "lens = accepted + 1" in text and "length m + 1" in text
    assert "lens = the accepted tokens" not in text


def gradients(x):
    return [torch.empty(x[n].shape, dtype=BF).as_subclass(OnDevice) for n in ("q", "k", "v", "beta", "g")]


def test_backward_belongs_to_the_last_forward(monkeypatch):
    """What backward reads is the last forward call's; an earlier one's is refused by its number, a batch of other
    sizes by those."""
    from quantized_gated_delta_amd import sq
    backs = []
    monkeypatch.setattr(sq, "sq_chunk_forward", lambda *a, **k: None)
    monkeypatch.setattr(sq, "sq_chunk_backward", lambda *a, **k: backs.append(a))
    layer, x = sequence()
    y = x["y"]
    inputs = [x[n] for n in ("q", "k", "v", "beta", "g", "cu")]

    def back(inputs=inputs, y=y, **kw):
        layer.backward(*inputs, y, *gradients(x), **kw)
    with pytest.raises(RuntimeError, match="forward"):
        back()
    first = layer.forward(*inputs, y)
    back(call=first)
    back()
    second = layer.forward(*inputs, y)
    assert second != first
    with pytest.raises(RuntimeError, match="forward"):
        back(call=first)
    back(call=second)
    back(call=second)   # as often as wanted
    assert len(backs) == 4
    layer.forward(*(t[:60] for t in inputs[:5]), inputs[5], y[:60])   # another batch
    with pytest.raises(RuntimeError, match="forward"):
        back()


def test_a_refused_forward_leaves_what_the_last_one_saved(monkeypatch):
    from quantized_gated_delta_amd import sq
    monkeypatch.setattr(sq, "sq_chunk_forward", lambda *a, **k: None)
    monkeypatch.setattr(sq, "sq_chunk_backward", lambda *a, **k: None)
    layer, x = sequence()
    inputs = [x[n] for n in ("q", "k", "v", "beta", "g", "cu")]
    call = layer.forward(*inputs, x["y"])
    with pytest.raises(ValueError):
        layer.forward(*inputs, x["y"][:50])
    layer.backward(*inputs, x["y"], *gradients(x), call=call)


OUT_OF_MEMORY = """
import os, resource, sys
sys.path.insert(0, %r)
os.environ["SQ_DEBUG"] = "1"
import quantized_gated_delta_amd as Q
from tests.test_sequence_abi import P, BIG
Q.lib()
n = 1 << 27   # 512 MB of host memory for the list's copy
d = Q.seq_desc(n, 0, 1, 64, Q.SQ_GATE_GDN, Q.SQ_BF16, Q.SQ_BF16)
pool = Q.sq_pool_create(n, 1, 64, 64, [4], Q.SQ_GATE_GDN, P, Q.sq_pool_bytes(n, 1, 64, 64, [4], Q.SQ_GATE_GDN))
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + (256 << 20), resource.RLIM_INFINITY))
for call in (lambda: Q.sq_chunk_forward(d, P, P, P, P, P, P, None, P, P, None, P, save_bytes=0, work_bytes=BIG, stream=0),
             lambda: Q.sq_check_slots(pool, P, n, 0)):
    try:
        call()
        print("no error")
    except Q.SQError as e:
        print("ENOMEM" if e.status == Q.SQ_ENOMEM else e)
"""


def test_debug_checks_without_host_memory():
    """The copies that the debug checks take of a list may find no memory: an error, not an exception through C."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", OUT_OF_MEMORY % root], capture_output=True, text=True, timeout=100, cwd=root)
    assert out.returncode == 0 and out.stdout.split() == ["ENOMEM", "ENOMEM"], (out.returncode, out.stdout, out.stderr[-500:])


def test_outputs_of_the_draft_check_apart_from_its_lists():
    """accepted is written while other workgroups still read lens and tokens: the same memory is refused."""
    from tests.test_sequence_abi import P, refused, verify
    apart = dict(tokens=P, lens=P + 4096, accepted=P + 8192, next_token=P + 12288)
    for change in (dict(accepted=P + 4096), dict(accepted=P), dict(next_token=P + 4096 + 8), dict(next_token=P + 8192 + 8), dict(accepted=P + 4096 - 4),
                   dict(next_token=P + 44)):
        refused(Q.SQ_EINVAL, "overlap", verify, **dict(apart, **change))
