"""The example block: its gradients against central differences of its own loss, its training, and
decoding against the whole sequence."""
import os
import sys

import pytest
import torch

from parity import case

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_trains_and_decodes(gpu_lib):
    import matrix_memory_block as ex
    case("example block")
    first, last, far = ex.main(width=128, heads=4, batch=4, steps=48, iterations=30, verbose=False)
    assert last < first
    # float32 operands both ways: the recurrence's bar of 1e-5 for each, over the largest value
    assert far < 1e-4


def test_gradient_of_the_residual_stream(gpu_lib):
    """d loss / dx along a direction. Rounding h to bfloat16 makes the loss a staircase whose steps, 2^-9 of
    each of many values at random, a wide difference averages out: 0.5% of the slope is left a wide margin."""
    import matrix_memory_block as ex
    case("example block gradient")
    block = ex.Block(128, 2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, c, u = (torch.randn((2, 40, 128), generator=gen, device="cuda") for _ in range(3))

    def loss(t):
        return float((block.forward(x + t * u)[0].double() * c.double()).sum())
    _, _, saved = block.forward(x)
    dx = block.backward(c, saved)[0]
    slope = float((dx.double() * u.double()).sum())
    eps = 0.02
    want = (loss(eps) - loss(-eps)) / (2 * eps)
    assert abs(slope - want) < 0.02 * float(dx.double().norm() * u.double().norm() / (2 * 40 * 128) ** 0.5)
