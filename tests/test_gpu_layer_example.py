"""The layer operators together with the state update, as a model calls them
(examples/decode_step.py), against the same step in plain torch from the same codes.

The two differ by bf16 roundings of the projections and of y (2^-8 each, 2 layers x 3 of
them) and by the E4M3 codes that such a difference moves (2^-4 of a value): logits of
standard deviation near 1 differ by a few percent, their log probabilities by less than 0.3."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_step():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for args in (["--layers", "2"], ["--layers", "2", "--batch", "1", "--drafts", "1"], ["--layers", "1", "--batch", "50"]):
        print("[gpu] decode step", args, flush=True)
        assert m.main(args + ["--check"]) < 0.3
