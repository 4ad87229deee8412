"""The example's autograd function does not take another call's saved states for its own."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_two_forwards_before_a_backward():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "train_prefill_speculate.py")
    spec = importlib.util.spec_from_file_location("train_prefill_speculate", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Model()
    layer = example.Q.ChunkedDelta(4, 400, example.H, example.D, n_key_heads=example.HK, dtype=torch.float32, train=True)

    def forward(seed):
        tokens, before, cu = example.flat(example.batch(torch.Generator().manual_seed(seed), 4, 40))
        return example.Delta.apply(layer, cu, *(x.contiguous() for x in model.inputs(tokens, before))).square().mean()
    first, second = forward(1), forward(1)
    second.backward()   # the last forward's: fine
    with pytest.raises(RuntimeError, match="forward"):
        first.backward()
