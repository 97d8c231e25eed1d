"""GPU parity of the gated delta layer's operators in the forms that large calls take, and of the bits of bf16 results."""
import pytest
import torch

import test_state_space_gpu as base

pytestmark = pytest.mark.gpu
mc = base.mc
DEV = base.DEV


def rounded_between(got, lower, upper):
    """Whether bf16 values are what a number from `lower` to `upper` (64 bits, element by element) rounds to."""
    return bool(((got.double() >= lower.to(torch.bfloat16).double()) & (got.double() <= upper.to(torch.bfloat16).double())).all())


@pytest.mark.parametrize("size", [(64, 32, 64), (16, 48, 100), (128, 64, 200), (200, 32, 130)], ids=lambda s: "-".join(map(str, s)))
def test_bf16_outputs_are_fp32_sums_rounded_once(mc, size):
    """With bf16 operands y is the fp32 call's on the same numbers, rounded.  Both sum the same products, all of them
    positive here but for the small corrections, in fp32; their orders may differ, by no more than the 16 roundings that a
    sum of 64 products in 16 x 16 x 32 instructions, its parts and the scale go through: 2^-20 of y."""
    P, V, L = size
    gen = torch.Generator().manual_seed(11)
    one = lambda *s: 0.5 + torch.rand(s, generator=gen) / 2  # noqa: E731
    q, k, v = one(2, 2 * P, L), one(2, 2 * P, L) / (8 * P) ** 0.5, one(2, 4 * V, L)
    g, beta = -0.1 * torch.rand(2, 4, L, generator=gen), 0.25 * one(2, 4, L)
    low = [x.to(DEV, torch.bfloat16) for x in (q, k, v)]
    g, beta = g.to(DEV), beta.to(DEV)
    y = mc.gated_delta_fwd(*low, g, beta, key_heads=2)
    want = mc.gated_delta_fwd(*(x.float() for x in low), g, beta, key_heads=2).double()
    assert bool((want > 0).all())
    rounded = rounded_between(y, want * (1 - 2.0 ** -20), want * (1 + 2.0 ** -20))
    assert rounded
