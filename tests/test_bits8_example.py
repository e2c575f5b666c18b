"""The 8-bit decode example: its operators together, as a program runs them."""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "bits8_decode.py")


def load():
    spec = importlib.util.spec_from_file_location("bits8_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
@pytest.mark.parametrize("requests,prompt,steps,layers,hidden,q_heads,kv_heads,dim", [
    (5, 90, 6, 2, 512, 8, 2, 64), (3, 200, 20, 1, 1024, 8, 8, 128), (9, 40, 3, 3, 512, 6, 2, 256)])
def test_decode_example(requests, prompt, steps, layers, hidden, q_heads, kv_heads, dim):
    """Against plain attention over the cache's rows as ple_kv8_read gives them.  Codes of four significant bits at scales of
    powers of two are exact in bf16, so keys and values are the same on both sides.  A score's sums differ by the roundings
    of fp32 and the weights are rounded to fp16 (2^-11 each): 2^-10 of the largest value with both, and the output's own
    rounding to bf16, half a step of at most 2^-8 of it."""
    error, ms = load().main(requests, prompt, steps, layers, hidden, q_heads, kv_heads, dim)
    assert error <= 2 ** -8 + 2 ** -9, error
    assert ms > 0
