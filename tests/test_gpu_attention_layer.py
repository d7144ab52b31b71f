"""GPU: the example's attention layer, end to end.

Token by token and as one prompt the cache holds the same tokens, but a page
that fills in several calls may encode its earlier tokens twice (their scale
grew), so keys and values differ by one more E4M3 rounding in places: half a step,
2^-4 of a value at most and far less in the mean; an attention output averages
many of them.  The output projection quantizes both again.  Their relative
difference stays below the E4M3 rounding itself, 2^-4.
"""
import importlib.util
import os

import pytest

from tests.gpu_common import announce

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")


@pytest.mark.parametrize("requests,prompt,tokens", [(3, 200, 5), (1, 1, 3)])
def test_decoding_agrees_with_the_prompt(requests, prompt, tokens):
    spec = importlib.util.spec_from_file_location("attention_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    announce(f"attention layer: {requests} requests, prompt {prompt}, {tokens} tokens")
    assert m.run(requests, prompt, tokens, hidden=512, verbose=False) <= 2.0 ** -4
