"""The example runs, and its parts agree with each other."""
import importlib.util
import os

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_train_prefill_speculate():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "train_prefill_speculate.py")
    spec = importlib.util.spec_from_file_location("train_prefill_speculate", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main()
    assert got["losses"][-1] < 0.5 * got["losses"][0]       # the gradients lead downhill
    assert got["one"] == got["several"]                     # drafts change nothing but the number of calls
    assert all(len(o) == 48 and all(0 <= t < example.VOCAB for t in o) for o in got["packed"] + got["sampled"])
    assert got["right"] > 0.8                               # the states survive the pool
