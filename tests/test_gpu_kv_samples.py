"""Page plans, norms and rotation, shared prefixes, sinks and verification together, as examples/kv_samples.py runs
them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


# A margin is the difference of two logits' errors, each a sum of 512 terms of the output projection (standard deviation
# 1 / sqrt(512)) times the error of a state.  bf16: an attention result of up to 4 is rounded in the calls and again in
# the check, which differ by a step (2^-7 at 4) where a sum lies next to a border; if all did, a logit would be off by
# 2^-7 in standard deviation at each of two layers, so 0.06 is nearly four of a difference's.  fp32: results differ
# by 2^-18 of scores up to 12 at most, so by 2^-14 of values.
@pytest.mark.parametrize("dtype,most", [(torch.bfloat16, 0.06), (torch.float32, 1e-3)])
@pytest.mark.parametrize("samples,prompt,page", [(4, 150, 16), (1, 40, 32)])
def test_samples(dtype, most, samples, prompt, page):
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "kv_samples.py")
    spec = importlib.util.spec_from_file_location("kv_samples", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    gamma = 4
    history, kv_len, kept, margin, free, pages = example.run(prompts=3, samples=samples, gamma=gamma, prompt=prompt, rounds=8,
                                                             page=page, dtype=dtype)
    for tokens, n in zip(history, kv_len):
        assert n == len(tokens) - 1  # all but the newest token are in the cache
    assert 1.0 <= kept <= gamma + 1
    assert margin <= most, margin
    assert free == pages  # every page came back
