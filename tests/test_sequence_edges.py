"""The sequence and window calls where their kernels take another way: gates of unlike strength,
large batches, keys that resemble each other.  Oracle and tolerances as in test_sequence.py.
"""
import pytest

torch = pytest.importorskip("torch")

from tests.test_sequence import BF, DEV, F32, batch, check, run

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
