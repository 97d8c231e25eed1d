"""GPU parity of the gated delta layer's operators in the forms that large calls take, and of the bits of bf16 results."""
import pytest
import torch

import delta_reference as ref
import test_norm_f8_gpu as layer
import test_state_space_gpu as base

pytestmark = pytest.mark.gpu
mc = base.mc
DEV, TDT = base.DEV, base.TDT


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


# ------------------------------------------------------------------ channel-major layer norm: 2, 4 and 8 time lanes

#             B  L     C    time lanes forward and backward; ends inside the last tile of each
LANES = {(4, 1003, 40): (1, 2), (8, 1003, 40): (2, 4), (8, 1701, 70): (4, 8), (16, 1701, 33): (8, 8), (4, 1003, 1100): (1, 2),
         (8, 1701, 300): (4, 8)}


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("size", LANES, ids=lambda s: "-".join(map(str, s)))
def test_layer_norm_over_time_lanes(mc, size, ragged, dt):
    B, L, C = size
    code = mc.BF16 if dt == "bf16" else mc.F32
    form = [mc.layer_norm_describe(*size, dtype=code, channel_major=True, backward=b).split() for b in (False, True)]
    assert [f[:2] for f in form] == [["algo=norm_rows", f"lanes={n}"] for n in LANES[size]]
    (x, cx), (dy, cdy), w, b, n, want = layer.norm_case(B, L, C, dt, True, ragged, True)
    (y, cy), (dx, cdx) = base.out_view((B, C, L), dt), base.out_view((B, C, L), dt)
    stats = mc.layer_norm_stats(x, channel_major=True)
    stats.fill_(float("nan"))
    kw = dict(channel_major=True, lengths=n[1])
    mc.layer_norm_fwd(x, w, b, y=y, stats=stats, **kw)
    _, dw, db = mc.layer_norm_bwd(x, dy, stats, w, b, dx=dx, **kw)
    layer.agree("y", y.transpose(1, 2), *want["y"], ref.HALF[dt])
    layer.agree("dx", dx.transpose(1, 2), *want["dx"], ref.HALF[dt])
    layer.agree("dw", dw, *want["dw"])
    layer.agree("db", db, *want["db"])
    # several tiles to a work-group
    ws = torch.full((3 * 8 * C + 64,), 0xff, dtype=torch.uint8, device=DEV)
    dx2, dw, db = mc.layer_norm_bwd(x, dy, stats, w, b, workspace=ws[:3 * 8 * C], **kw)
    assert torch.equal(dx2, dx) and bool((ws[3 * 8 * C:] == 0xff).all())
    layer.agree("dw of three work-groups", dw, *want["dw"])
    layer.agree("db of three work-groups", db, *want["db"])
    for check in (cx, cdy, cy, cdx):
        check()
