"""The example layer: trained for a few steps, then prompts and single tokens."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "linear_attention_layer.py")


def _example():
    spec = importlib.util.spec_from_file_location("linear_attention_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_trains_and_serves(dtype):
    """The loss falls, and what is served token by token is what the whole
    sequences give.  Served and whole, every token goes through the same roundings: in
    bf16 those of q, k and v (2^-9 of each, which the projection's different
    summation order may flip), of o and of y, so 6 half-units of the largest
    value, 6 * 2^-8; in fp32 sums of `dim` = 128 terms three deep, 3 * 128 *
    2^-24 doubled for both sides.  The recurrence mixes up to 100 tokens of
    random sign whose flips are independent; twice the bound covers them."""
    m = _example()
    torch.manual_seed(0)
    layer = m.LinearAttentionLayer(128, 4, 2, 32, 512, "cuda:0", dtype)
    losses = m.train(layer, 8, 2, 100)
    print(losses, flush=True)
    assert losses[-1] < 0.9 * losses[0]
    worst, size = m.serve(layer, [70, 1, 33], 5)
    bound = 12 * 2.0 ** -8 if dtype is torch.bfloat16 else 12 * 128 * 2.0 ** -24
    print(worst, size, flush=True)
    assert worst <= bound * size
