"""The cache calls and verification together, as examples/kv_round.py runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_rounds():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "kv_round.py")
    spec = importlib.util.spec_from_file_location("kv_round", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rounds, gamma = 12, 4
    history, kv_len, kept, margin = example.run(batch=5, gamma=gamma, prompt=70, rounds=rounds)
    for tokens, n in zip(history, kv_len):
        assert n == len(tokens) - 1  # all but the newest token are in the cache
    assert 1.0 <= kept <= gamma + 1
    # A logit sums 512 terms of size ~1/sqrt(512) times bf16 attention results (off by
    # 2^-9 of values below about 3, one in 512 each): below 0.01 together, and as much
    # again between the draft positions' winner and its neighbour.
    assert margin <= 0.02, margin
