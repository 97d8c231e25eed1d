"""Every form of the state-space kernels against the plain 64-bit forms.  Which form a size takes is a rule
with measured costs, so each case first asks the library which one it is, and fails if the rule has moved
on: then the case needs another size, or the form has gone.
"""
import pytest

import test_state_space_gpu as base

pytestmark = pytest.mark.gpu
mc = base.mc

#         B  D     L     N  G    gate   softplus ragged state skip       forward form, backward text
SCANS = [((2, 3, 900, 5, 1, True, True, True, True, True), "64x16 segments=1", "segments=8 carry_segments=1"),
         ((3, 4, 2040, 3, 1, True, True, True, True, True), "64x16 segments=1", "carry_segments=1"),
         ((1, 64, 3100, 2, 1, True, True, False, True, True), "64x16 segments=4", "segments=25 carry_segments=4"),
         ((2, 300, 500, 4, 1, False, True, True, True, True), "64x8 segments=1", "segments=4"),
         ((2, 2000, 1100, 2, 1, True, True, True, True, True), "64x8 segments=1", "segments=1"),
         ((2, 4100, 129, 3, 1, True, True, False, True, True), "16x8 segments=1", "segments=1"),
         ((5, 4000, 258, 2, 2, True, True, True, True, True), "16x8 segments=1", "segments=1"),
         ((2, 3, 40, 5, 1, True, True, True, True, True), "16x8shared segments=1", "segments=1"),
         ((5, 8, 300, 33, 1, True, True, True, True, True), "16x8shared segments=1", "beside=3"),
         # blocks of 16 states one after the other, over time segments side by side
         ((1, 130, 300, 33, 130, True, True, False, True, True), "segments=1", "segments=3 carry_segments=1 beside=1")]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case,fwd,bwd", SCANS, ids=lambda c: "-".join(map(str, c)) if isinstance(c, tuple) else "")
def test_scan_form(mc, case, fwd, bwd, dt):
    code = 1 if dt == "bf16" else 0
    assert fwd in mc.selective_scan_fwd_describe(*case[:5], dtype=code)
    assert bwd in mc.selective_scan_bwd_describe(*case[:5], dtype=code)
    base.test_scan(mc, case, dt)


#             B  L     O     K           kernel
PRODUCTS = [((1, 15, 70, 384), "algo=i8_few tokens=16"),
            ((2, 16, 70, 384), "algo=i8_few tokens=32"),
            ((7, 9, 70, 1152), "algo=i8_few tokens=64"),
            ((1, 1111, 1777, 1024), "tile=64 stages=4 splits=1"),
            ((3, 301, 700, 256), "tile=64 stages=4 splits=1"),
            ((2, 33, 200, 16512), "tile=64 stages=4 splits=8"),
            ((3, 500, 1600, 128), "tile=128 stages=2 splits=1"),
            ((1, 1500, 1600, 256), "tile=128 stages=2 splits=1"),
            ((3, 500, 1601, 384), "tile=128 stages=2 splits=1"),
            ((3, 500, 1601, 1024), "tile=128 stages=2 splits=1"),
            ((1, 1500, 1601, 4096), "tile=128 stages=4 splits=1"),
            ((3, 500, 1600, 4224), "tile=128 stages=4 splits=1"),
            ((1, 3003, 3100, 128), "tile=256 stages=2 splits=1"),
            ((3, 1001, 3100, 256), "tile=256 stages=2 splits=1"),
            ((3, 1001, 3100, 384), "tile=256 stages=2 splits=1"),
            ((1, 3003, 3101, 1024), "tile=256 stages=2 splits=1"),
            ((7, 429, 3101, 1152), "tile=256 stages=2 splits=1")]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case,kernel", PRODUCTS, ids=lambda c: "-".join(map(str, c)) if isinstance(c, tuple) else "")
def test_product_form(mc, case, kernel, out):
    B, L, O, K = case
    assert kernel in mc.matmul_i8_describe(B * L, O, K)
    base.test_integer_product(mc, case, out)


def test_product_streams_its_output(mc):
    """The 256 tile that writes past the caches (bf16 outputs of 128 MB), several stages deep."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randint(-127, 128, (8195, 640), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (8203, 640), generator=gen, device="cuda", dtype=torch.int8)
    s, ws = torch.rand(8195, device="cuda"), torch.rand(8203, device="cuda")
    assert "tile=256" in mc.matmul_i8_describe(8195, 8203, 640)
    y = mc.matmul_i8(q, s, w, ws, out_dtype=torch.bfloat16)
    ycm = mc.matmul_i8(q, s, w, ws, out_dtype=torch.bfloat16, length=1639)
    for i in range(0, 8195, 1639):
        # sums below 2^24 are exact in fp32, in any order
        want = (q[i:i + 1639].float() @ w.float().t() * s[i:i + 1639, None] * ws).bfloat16()
        assert torch.equal(y[i:i + 1639], want) and torch.equal(ycm[i // 1639], want.t()), i
