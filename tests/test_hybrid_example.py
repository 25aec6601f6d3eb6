"""examples/hybrid_decode.py: the paged attention layers and the KDA layers served together."""
from __future__ import annotations

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
def test_steps_agree_with_one_prompt(dtype):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import hybrid_decode as E
    finally:
        sys.path.pop(0)
    # Both ways round each of the 4 layers' outputs and sums to bfloat16 (half a step is 2^-8 of the value),
    # in another order: at most 3 roundings a layer on either side apart.  An E4M3 cache can put a key
    # or value that differs in its last bfloat16 bit into the next code (half a step 2^-4), in 2 layers.
    limit = 4 * 3 * 2 * 2.0 ** -8 + (2 * 2.0 ** -4 if dtype != torch.bfloat16 else 0.0)
    assert E.serve(E.Hybrid(cache_dtype=dtype)) <= limit
