"""The example layer: projection, append, attention and output product together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "attention_layer.py")

# Standard normal values in 8 bits are off by max / 127 / sqrt(12), max about
# 4.2: 0.95 %.  The projection adds two such errors (1.35 %), the cache a third
# (1.65 % of keys and values).  Scores of unit variance are then off by
# sqrt(1.35^2 + 1.65^2) = 2.1 % of 1, so are the probabilities, and the output by
# sqrt(2.1^2 + 1.65^2) = 2.7 %, the roundings to 16 bits (0.2 % each) aside.
LIMIT = 1.5 * 0.027


@pytest.mark.parametrize("hidden,heads,kv_heads,page,dtype", [
    (1024, 8, 2, 64, torch.bfloat16), (1024, 16, 16, 16, torch.float16), (2048, 16, 2, 128, torch.float16)])
def test_layer_over_prompts_and_tokens(hidden, heads, kv_heads, page, dtype):
    print("layer", hidden, heads, kv_heads, page, dtype, flush=True)
    spec = importlib.util.spec_from_file_location("attention_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    prompts, steps = m.run(hidden, heads, kv_heads, page=page, dtype=dtype)
    print("errors", prompts, steps, flush=True)
    assert prompts <= LIMIT and steps <= LIMIT
