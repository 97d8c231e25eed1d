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


#           B  D   L     N   G  gate  softplus ragged state skip        limits, slice (sequences x groups x channels x steps)
SLICES = [((3, 40, 300, 5, 2, True, True, True, True, True),
           [(0, "1x1x16x128"), (20000, "1x1x20x128"), (50000, "2x2x20x128"), (100000, "3x2x20x128"), (10 ** 9, "3x2x20x300")]),
          ((2, 50, 700, 40, 1, True, True, True, True, True),
           [(0, "beside=1 slice=1x1x16x128"), (300000, "beside=3 slice=1x1x32x128"), (1000000, "beside=3 slice=2x1x50x128")]),
          ((1, 20, 5000, 3, 1, False, True, True, False, True),
           [(30000, "segments=4 carry_segments=1 beside=1 slice=1x1x20x512"),
            (200000, "segments=20 carry_segments=3 beside=1 slice=1x1x20x2560")]),
          ((2, 8, 6000, 20, 1, True, False, True, True, False),
           [(200000, "beside=2 slice=2x1x8x256"), (800000, "segments=8 carry_segments=1 beside=2 slice=2x1x8x1024")])]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case,limits", SLICES, ids=lambda c: "-".join(map(str, c)) if isinstance(c, tuple) else "")
def test_backward_scan_in_slices(mc, case, limits, dt):
    """The same gradients from whatever workspace the caller has, none of it past the workspace's end."""
    import torch
    B, D, L, N, G, gate, sp, ragged, state, skip = case
    h, d, nh, n = base.scan_data(case, dt)
    want = base.scan_reference(h, nh, sp)
    v = {k: base.view(base.poison(d[k], nh))[0] for k in ("x", "delta", "dy", "z") if k in d}
    Bm, Cm = (base.poison(d[k], nh) for k in ("Bm", "Cm"))
    common = dict(D=d.get("D"), z=v.get("z"), delta_bias=d.get("bias"), softplus=sp, lengths=n)
    states = mc.selective_scan_states(v["x"], d["A"])
    mc.selective_scan_fwd(v["x"], v["delta"], d["A"], Bm, Cm, initial_state=d.get("h0"), states=states, **common)
    code = 1 if dt == "bf16" else 0
    for limit, text in limits:
        size = mc.selective_scan_bwd_workspace(*case[:5], dtype=code, limit=limit)
        assert text in mc.selective_scan_bwd_describe(*case[:5], dtype=code, workspace_bytes=size)
        buf = torch.full((size + 4096,), 0xa5, dtype=torch.uint8, device=base.DEV)
        outs = {k: base.out_view((B, D, L), dt) for k in ("dx", "ddelta") + (("dz",) if gate else ())}
        for repeat in range(2):                                 # what a call leaves in the workspace does not matter
            dh0 = torch.full((B, D, N), float("nan"), device=base.DEV)
            r = mc.selective_scan_bwd(v["x"], v["delta"], d["A"], Bm, Cm, v["dy"], states, d_final_state=d.get("dfs"),
                                      d_initial_state=dh0, workspace=buf[:size], **{k: o[0] for k, o in outs.items()}, **common)
            for name in ("dx", "ddelta", "dz", "dA", "dB", "dC", "dD", "ddelta_bias"):
                if r[name] is not None:
                    base.agree(name, r[name], want[name], dt if name in outs else "f32", (case, limit))
            base.agree("dh0", dh0, want["dh0"], "f32", (case, limit))
            for _, check in outs.values():
                check()
        assert bool((buf[size:] == 0xa5).all())
    with pytest.raises(ValueError):
        mc.selective_scan_bwd(v["x"], v["delta"], d["A"], Bm, Cm, v["dy"], states, workspace=buf[:1000], **common)
