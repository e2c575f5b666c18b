"""The 4-bit decode example: its operators together, as a program runs them."""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp4_decode.py")


def load():
    spec = importlib.util.spec_from_file_location("fp4_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
@pytest.mark.parametrize("requests,prompt,steps,hidden,q_heads,kv_heads,dim", [
    (5, 90, 6, 512, 8, 2, 64), (3, 200, 4, 1024, 8, 8, 128), (9, 40, 3, 512, 6, 2, 256)])
def test_decode_example(requests, prompt, steps, hidden, q_heads, kv_heads, dim):
    """Against plain attention over the cache's rows as ple_kv4_read gives them.  Those are rounded to bf16 (half a step
    2^-9 of the value, which 2^-8 bounds): a key's rounding moves a score s by up to 2^-8 |q||k| scale, a value's the
    output by 2^-8 of the largest value, and the output itself is rounded to bf16.  Queries and keys have unit variance,
    so |q||k| scale is about sqrt(dim) <= 16 and the bound is 2 * 16 * 2^-8 + 2 * 2^-8 of the largest value; roundings
    of independent signs stay well below it."""
    error, ms = load().main(requests, prompt, steps, hidden, q_heads, kv_heads, dim)
    assert error <= (2 * dim ** 0.5 + 2) * 2 ** -8, error
    assert ms > 0
