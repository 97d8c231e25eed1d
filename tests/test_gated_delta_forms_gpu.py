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


@pytest.mark.parametrize("size", [(64, 32, 64), (128, 64, 128), (200, 32, 64)], ids=lambda s: "-".join(map(str, s)))
def test_errors_have_either_sign(mc, size):
    """fp32 operands are three planes of eight bits, and of their products those below 2^-24 are left out.  With planes cut
    towards zero that is 2 x 2^-9 x 2^-17 = 2^-25 of every product on average, always of its sign, and a state's value is a
    sum of products of what came from two more: all positive here, so the errors' average would be 2^-25 more than once.
    Rounded to nearest, what is left out averages 0."""
    P, V, L = size
    gen = torch.Generator().manual_seed(31)
    one = lambda *s: 0.5 + torch.rand(s, generator=gen) / 2  # noqa: E731
    q, k, v = one(2, 2 * P, L), one(2, 2 * P, L) / (64 * P) ** 0.5, one(2, 4 * V, L)
    g, beta = -0.1 * torch.rand(2, 4, L, generator=gen), 0.25 * one(2, 4, L)
    s = torch.empty(2, 4, P, V, device=DEV)
    mc.gated_delta_fwd(*(t.to(DEV) for t in (q, k, v, g, beta)), key_heads=2, final_state=s)
    want = ref.rule(*(t.double() for t in (q, k, v, g, beta)), 2)[1]
    mean = float(((s.double().cpu() - want) / want).mean())
    print(f"  mean error {mean:.2e}", flush=True)
    assert abs(mean) <= 2.0 ** -25


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


# ------------------------------------------------------------------ 8-bit float products: every tile

#            T     C     O      kernel; ends inside the tiles, one block of k, odd and even numbers of blocks
PRODUCTS = [((1500, 100, 1601), "tile=128 stages=2 splits=1"),
            ((1500, 300, 1600), "tile=128 stages=2 splits=1"),
            ((1500, 8200, 1601), "tile=128 stages=2 splits=3"),
            ((3003, 100, 3100), "tile=256 stages=2 splits=1"),
            ((3003, 250, 3101), "tile=256 stages=2 splits=1"),
            ((3003, 300, 3100), "tile=256 stages=2 splits=1"),
            ((3100, 1100, 3003), "tile=256 stages=2 splits=1")]


# What a bf16 output may be off by before it is rounded, of the sum of its products' magnitudes: the 8-bit matrix instruction
# adds eight products at a time and drops what lies below 2^-13 of the largest, 7 x 2^-13 of that at most.
DROPPED = 2.0 ** -10


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("size,kernel", PRODUCTS, ids=lambda s: "-".join(map(str, s)) if isinstance(s, tuple) else "")
def test_product_tiles(mc, size, kernel, out):
    """Against the 64-bit product, with either order of y; and the bits of the small tiles, which add each output's products
    in the same order, for some hundred tokens at a time."""
    T, C, O = size
    f = base.Data(2, "f32")
    x, w = layer.f8_inputs(f, T, C, "f32"), torch.randn(O, C, generator=f.gen) * C ** -0.5
    b = torch.randn(O, generator=f.gen)
    q, s, wq, ws = *mc.quantize_f8(x.to(DEV)), *mc.quantize_f8(w.to(DEV))
    K = q.shape[1]
    assert kernel in mc.matmul_f8_describe(T, O, K)
    e, we = s.view(torch.uint8).cpu().t().int() - 127, ws.view(torch.uint8).cpu().t().int() - 127
    want, size_of = ref.product(q.float().cpu(), e, wq.float().cpu(), we)
    bound = (K / 16 + 8) * ref.U * size_of + 2 * ref.U * (size_of + b.abs().double())
    if out == "bf16":
        bound = bound + DROPPED * size_of
    kw = dict(out_dtype=TDT[out])
    y = mc.matmul_f8(q, s, wq, ws, b.to(DEV), **kw)
    layer.agree("y", y, want + b.double(), bound, ref.HALF[out])
    for L in {T, max(d for d in range(1, 33) if T % d == 0)}:
        z = torch.full((T // L, O, L), float("nan"), dtype=TDT[out], device=DEV)
        mc.matmul_f8(q, s, wq, ws, b.to(DEV), length=L, y=z)
        assert torch.equal(z.transpose(1, 2).reshape(T, O), y), L
    whole = mc.matmul_f8(q, s, wq, ws, b.to(DEV), workspace=torch.empty(0, dtype=torch.uint8, device=DEV), **kw)
    layer.agree("without splits", whole, want + b.double(), bound, ref.HALF[out])
    for t in range(0, T, 150):
        n = min(t + 150, T)
        if n - t <= 64:
            continue                                   # the kernel of few tokens adds in an order of its own
        assert "tile=64" in mc.matmul_f8_describe(n - t, O, K)
        part = mc.matmul_f8(q[t:n].contiguous(), s[:, t:n].contiguous(), wq, ws, b.to(DEV),
                            workspace=torch.empty(0, dtype=torch.uint8, device=DEV), **kw)
        assert torch.equal(part, whole[t:n]), t


@pytest.mark.parametrize("size", [(1, 64, 64), (3, 130, 70), (16, 1000, 333), (17, 700, 1500), (33, 2000, 90), (64, 4096, 200)],
                         ids=lambda s: "-".join(map(str, s)))
def test_bf16_products_of_few_tokens_are_fp32_sums_rounded_once(mc, size):
    """Few tokens wait for their loads, not for their products: the same sums for both types."""
    T, C, O = size
    f = base.Data(14, "f32")
    x, w, b = layer.f8_inputs(f, T, C, "f32"), torch.randn(O, C, generator=f.gen), torch.randn(O, generator=f.gen)
    args = (*mc.quantize_f8(x.to(DEV)), *mc.quantize_f8(w.to(DEV)), b.to(DEV))
    assert "algo=f8_few" in mc.matmul_f8_describe(T, O, args[0].shape[1])
    y = mc.matmul_f8(*args)
    assert torch.equal(mc.matmul_f8(*args, out_dtype=torch.bfloat16), y.to(torch.bfloat16))


def test_product_past_the_caches(mc):
    """A bf16 output of 128 MB, which is written past the caches: 50 of its rows, and both orders of all of it."""
    T, C, O, L = 8200, 250, 8200, 41
    assert T * O * 2 >= 128 << 20 and "tile=256" in mc.matmul_f8_describe(T, O, 256)
    f = base.Data(12, "f32")
    x, w = torch.randn(T, C, generator=f.gen), torch.randn(O, C, generator=f.gen)
    q, s, wq, ws = *mc.quantize_f8(x.to(DEV)), *mc.quantize_f8(w.to(DEV))
    y = mc.matmul_f8(q, s, wq, ws, out_dtype=torch.bfloat16)
    rows = torch.cat([torch.arange(20), torch.randint(T, (10,), generator=f.gen), torch.arange(T - 20, T)])
    e, we = s.view(torch.uint8).cpu().t().int() - 127, ws.view(torch.uint8).cpu().t().int() - 127
    want, size_of = ref.product(q.float().cpu()[rows], e[rows], wq.float().cpu(), we)
    layer.agree("rows", y[rows.to(DEV)], want, (256 / 16 + 8) * ref.U * size_of + DROPPED * size_of, ref.HALF["bf16"])
    z = torch.full((T // L, O, L), float("nan"), dtype=torch.bfloat16, device=DEV)
    mc.matmul_f8(q, s, wq, ws, length=L, y=z)
    assert torch.equal(z.transpose(1, 2).reshape(T, O), y)


@pytest.mark.parametrize("T", [5, 40, 100])
def test_product_of_numbers_of_all_sizes(mc, T):
    """Products from 2^-18 to 2^17 side by side: what is dropped stays within DROPPED.  All are positive here, so
    that it adds up."""
    gen = torch.Generator().manual_seed(13)
    C, O = 640, 90
    x, w = (torch.exp2(-9 + 17.5 * torch.rand(n, C, generator=gen)) for n in (T, O))
    x[0], w[0] = 2.0 ** -6, 1.0                        # one large product among eight, the others just below what it keeps
    x[0, 3::8] = 256.0
    x[1], w[1] = 0.0625, 448.0                         # in blocks of k that turn against each other
    x[1, ::64] = 448.0
    q, wq = (t.to(DEV).to(torch.float8_e4m3fn) for t in (x, w))
    one, wone = (torch.full((C // 128, n), 127, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu) for n in (T, O))
    want, size_of = ref.product(q.float().cpu(), torch.zeros(T, C // 128, dtype=torch.int32), wq.float().cpu(),
                                torch.zeros(O, C // 128, dtype=torch.int32))
    sums = (C / 16 + 8) * ref.U * size_of
    layer.agree("bf16", mc.matmul_f8(q, one, wq, wone, out_dtype=torch.bfloat16), want, sums + DROPPED * size_of, ref.HALF["bf16"])
    layer.agree("fp32", mc.matmul_f8(q, one, wq, wone), want, sums, ref.HALF["f32"])
