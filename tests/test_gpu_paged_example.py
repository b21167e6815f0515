"""examples/paged_speculation.py: speculative decoding over a paged, forked and compacted cache emits
exactly the tokens of decoding one at a time."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_speculation.py")


@pytest.mark.parametrize("seed,K", [(7, 15), (8, 20), (9, 3)])
def test_speculation_over_pages_is_greedy(w4v_mod, gpu, seed, K):
    spec = importlib.util.spec_from_file_location("paged_speculation", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got, want, steps = example.main(seed=seed, count=30, K=K)
    assert got == want and steps <= 30
