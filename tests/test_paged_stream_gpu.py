"""The example's speculated stream, token for token: every token is the target's
choice after the tokens before it."""
import importlib.util
import os

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.build()
    spec = importlib.util.spec_from_file_location("paged_decoding", os.path.join(ROOT, "examples", "paged_decoding.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("prompt,k", [([11, 222, 3333, 44, 5], 5), ([7], 3), (list(range(100, 133)), 8)])
def test_every_token_of_a_greedy_stream_is_the_targets_choice(m, prompt, k):
    """The target alone, fed the speculated tokens one at a time, would have chosen
    each of them.  Logits of the same prefix differ by the bf16 roundings of
    library products over 1 or K + 1 rows, an ulp or two of the logits (steps of
    2^-7 of the largest): within four such steps of the largest a choice is a tie.
    A wrong page, position or rollback shows as a token the target ranks far
    below that."""
    new = 64
    out, rate = m.decode(prompt, new, k, greedy=True)
    assert len(out) == new and 1.0 <= rate <= k + 1
    model = m.TinyDecoder()
    cache, feed, ties = model.cache(model.layers), list(prompt), 0
    for i, token in enumerate(out):
        z = model.forward(cache, 0, feed, model.layers)[-1].float()
        top = float(z.max())
        assert float(z[token]) >= top - 4 * 2.0 ** -7 * abs(top), (i, token, int(z.argmax()))
        ties += int(z.argmax()) != token
        feed = [token]
    assert ties <= new // 8, ties
