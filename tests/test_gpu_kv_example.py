"""The example that runs projections, cache, attention and page pool together."""
import importlib.util
import os

import pytest

from gpu_helpers import torch_cuda

pytestmark = pytest.mark.gpu


def test_cached_attention_example():
    torch_cuda()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "cached_attention.py")
    spec = importlib.util.spec_from_file_location("cached_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # a code is within 2^-4 of its value, 3.6 % of it in the mean square of a
    # uniform mantissa or less; two layers add attention outputs with about
    # that error to hidden states of their own size
    assert m.main() < 0.05


def test_example_reads_shared_tokens_once():
    """The continuations are so many that attention takes what they share apart; errors as above."""
    torch_cuda()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "cached_attention.py")
    spec = importlib.util.spec_from_file_location("cached_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    worst, apart = m.continuations(m.Layers())
    assert apart and worst < 0.05
