"""GPU parity of layer norm and of the block-scaled 8-bit products against plain 64-bit forms (delta_reference.py),
element by element, with the bounds derived there.
"""
import numpy as np
import pytest
import torch

import delta_reference as ref
import test_state_space_gpu as base

pytestmark = pytest.mark.gpu
mc = base.mc
DEV, TDT = base.DEV, base.TDT
INF = float("inf")


def agree(name, got, want, bound, half=0.0):
    got = got.double().cpu()
    assert got.shape == want.shape
    worst = float(((got - want).abs() / (bound + half * want.abs() + 1e-37)).nan_to_num(INF, INF, INF).max())
    print(f"  {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, (name, worst)


# ------------------------------------------------------------------ layer norm

#         B  L    C
NORM = [(1, 1, 1), (2, 3, 5), (3, 70, 100), (1, 65, 512), (5, 9, 513), (2, 7, 1001), (1, 130, 1025), (3, 5, 2048),
        (1, 17, 2049), (2, 3, 4100), (1, 5, 8192), (2, 3, 8200), (1, 2, 20000), (1, 600, 40), (2, 300, 2000)]


def norm_case(B, L, C, dt, major, ragged, params, seed=1):
    f = base.Data(seed, dt)
    size = torch.exp(0.5 * torch.randn(C, generator=f.gen))
    shift = 3 * torch.randn(B, L, 1, generator=f.gen)
    x = (torch.randn(B, L, C, generator=f.gen) * size + shift).to(TDT[dt])
    dy = torch.randn(B, L, C, generator=f.gen).to(TDT[dt])
    w, b = (f.make(C, shift=1.0, scale=0.3, dtype=torch.float32), f.make(C, dtype=torch.float32)) if params else ((None,) * 2,) * 2
    n = f.lengths(B, L) if ragged else (None, None)
    want = ref.layer_norm(x.double(), None if w[0] is None else torch.from_numpy(w[0]),
                          None if b[0] is None else torch.from_numpy(b[0]), 1e-5, n[0], dy.double())

    def place(t):
        t = t.to(DEV)
        if n[0] is not None:
            t = base.poison(t.transpose(1, 2).contiguous(), n[0]).transpose(1, 2)
        return base.view((t.transpose(1, 2) if major else t).contiguous())
    return place(x), place(dy), w[1], b[1], n, want


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("major", [False, True], ids=["tokens", "channels"])
@pytest.mark.parametrize("ragged,params", [(False, True), (True, False), (True, True)])
@pytest.mark.parametrize("size", NORM, ids=lambda s: "-".join(map(str, s)))
def test_layer_norm(mc, size, ragged, params, major, dt):
    B, L, C = size
    (x, cx), (dy, cdy), w, b, n, want = norm_case(B, L, C, dt, major, ragged, params)
    shape = (B, C, L) if major else (B, L, C)
    (y, cy), (dx, cdx) = base.out_view(shape, dt), base.out_view(shape, dt)
    stats = mc.layer_norm_stats(x, channel_major=major)
    stats.fill_(float("nan"))
    mc.layer_norm_fwd(x, w, b, channel_major=major, lengths=n[1], y=y, stats=stats)
    _, dw, db = mc.layer_norm_bwd(x, dy, stats, w, b, channel_major=major, lengths=n[1], dx=dx)
    back = (lambda t: t.transpose(1, 2)) if major else (lambda t: t)
    agree("y", back(y), *want["y"], ref.HALF[dt])
    valid = torch.ones(B, L, dtype=torch.bool) if n[0] is None else torch.arange(L) < torch.as_tensor(np.clip(n[0], 0, L))[:, None]
    for i, name in enumerate(("mean", "rstd")):
        value, bound = (t[..., 0][valid] for t in want[name])
        if value.numel():
            agree(name, stats.view(2, B, L)[i].cpu()[valid], value, bound)
    agree("dx", back(dx), *want["dx"], ref.HALF[dt])
    assert (dw is None) == (w is None) and (db is None) == (b is None)
    if params:
        agree("dw", dw, *want["dw"])
        agree("db", db, *want["db"])
    for check in (cx, cdy, cy, cdx):
        check()
    # tokens alone, without a batch
    if B == 1 and n[0] is None:
        assert torch.equal(mc.layer_norm_fwd(x[0], w, b, channel_major=major), y[0])


@pytest.mark.parametrize("major", [False, True], ids=["tokens", "channels"])
@pytest.mark.parametrize("size", [(3, 300, 70), (2, 200, 1500), (2, 40, 9000)], ids=lambda s: "-".join(map(str, s)))
def test_layer_norm_under_a_small_workspace(mc, size, major):
    """One row of partial sums, or a few: the same dx, and dw and db within their bounds."""
    B, L, C = size
    (x, _), (dy, _), w, b, n, want = norm_case(B, L, C, "f32", major, True, True, 2)
    stats = mc.layer_norm_stats(x, channel_major=major)
    mc.layer_norm_fwd(x, w, b, channel_major=major, lengths=n[1], stats=stats)
    kw = dict(channel_major=major, lengths=n[1])
    dx = mc.layer_norm_bwd(x, dy, stats, w, b, **kw)[0]
    for rows in (1, 3):
        ws = torch.full((rows * 8 * C + 64,), 0xff, dtype=torch.uint8, device=DEV)
        dx2, dw, db = mc.layer_norm_bwd(x, dy, stats, w, b, workspace=ws[:rows * 8 * C], **kw)
        assert torch.equal(dx, dx2) and bool((ws[rows * 8 * C:] == 0xff).all())
        agree("dw", dw, *want["dw"])
        agree("db", db, *want["db"])


def test_layer_norm_far_from_zero(mc):
    """A mean of 10^4 standard deviations, and tokens of one value: no cancellation, no division by zero."""
    gen = torch.Generator().manual_seed(3)
    x = (torch.randn(4, 1, 300, generator=gen) + 10000.0).float()
    x[2:] = 5.0
    want = ref.layer_norm(x.double(), None, None, 1e-5, None)
    for major in (False, True):
        t = (x.transpose(1, 2) if major else x).contiguous().to(DEV)
        y = mc.layer_norm_fwd(t, channel_major=major)
        agree("y", y.transpose(1, 2) if major else y, *want["y"], ref.HALF["f32"])
        assert not y[2:].any()


def test_layer_norm_repeats_streams_and_graphs(mc):
    for major in (False, True):
        (x, _), (dy, _), w, b, n, _ = norm_case(3, 90, 700, "bf16", major, True, True, 4)
        stats = mc.layer_norm_stats(x, channel_major=major)
        kw = dict(channel_major=major, lengths=n[1])

        def work():
            y = mc.layer_norm_fwd(x, w, b, stats=stats, **kw)
            return (y,) + mc.layer_norm_bwd(x, dy, stats, w, b, **kw)
        first = [t.clone() for t in work()]
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            second = work()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, second))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = work()
        for _ in range(3):
            dy.mul_(-0.5)
            w.mul_(1.25)
            graph.replay()
            got = [t.clone() for t in held]
            want = [t.clone() for t in work()]
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))


# ------------------------------------------------------------------ 8-bit floating point

def f8_inputs(f, T, C, dt):
    """Tokens and blocks of very different sizes, zeros, borders of the 8-bit format."""
    x = torch.randn(T, C, generator=f.gen) * torch.exp(3 * torch.randn(T, 1, generator=f.gen))
    x[:, ::7] *= 30
    if T > 2:
        x[1] = 0.0
        x[2, :min(C, 128)] = 0.0
        x[2, 0] = 448.0 * 2.0 ** -9
    if C > 3:
        x[0, 1], x[0, 3] = 2.0 ** -120, -0.0
    return x.to(TDT[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("major", [False, True], ids=["tokens", "channels"])
@pytest.mark.parametrize("size", [(1, 1, 1), (2, 5, 3), (3, 70, 128), (1, 64, 130), (4, 33, 500), (2, 130, 1030)],
                         ids=lambda s: "-".join(map(str, s)))
def test_quantiser(mc, size, major, dt):
    """Every bit of q and its powers, from views too; a block with an infinity or NaN becomes NaN."""
    B, L, C = size
    x = f8_inputs(base.Data(1, dt), B * L, C, dt)
    want_q, want_e, _ = ref.quantize(x.float())
    t = x.view(B, L, C).to(DEV)
    t, check = base.view((t.transpose(1, 2) if major else t).contiguous())
    q, scale = mc.quantize_f8(t, channel_major=major)
    assert q.dtype == torch.float8_e4m3fn and scale.dtype == torch.float8_e8m0fnu
    assert q.shape == (B * L, want_q.shape[1]) and scale.shape == (want_q.shape[1] // 128, B * L)
    assert torch.equal(q.float().cpu(), want_q)
    assert torch.equal(scale.view(torch.uint8).cpu().t().int(), (want_e + 127).int())
    check()
    if B * L < 4:
        return
    x[3, C - 1] = INF
    x[1, 0] = float("nan")
    _, _, bad = ref.quantize(x.float())
    t = x.view(B, L, C).to(DEV)
    q, scale = mc.quantize_f8((t.transpose(1, 2) if major else t).contiguous(), channel_major=major)
    value = q.float().view(B * L, -1, 128) * scale.float().t()[..., None]
    assert torch.equal(value.isnan().cpu(), bad[..., None].expand(-1, -1, 128))


#       T    C     O     few tokens, tiles of 64, 128, 256, splits of k, ends inside every tile
F8 = [(1, 64, 64), (3, 130, 70), (16, 1000, 333), (17, 128, 129), (40, 257, 1000), (64, 4096, 200), (65, 500, 90),
      (200, 128, 300), (333, 700, 1500), (130, 8192, 140), (1100, 300, 1030), (2100, 260, 2200), (66, 20000, 65)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("size", F8, ids=lambda s: "-".join(map(str, s)))
def test_product(mc, size, bias, out):
    """Against the 64-bit product of the quantised operands.  fp32: sums of 16 products at a time, exact or off by a few U
    of their magnitudes, C / 16 sums after each other.  bf16: the 8-bit matrix instruction keeps 13 bits or more below the
    largest of the 64 products that it adds, each product 2^-13 at most of that, and the output has half a step."""
    T, C, O = size
    f = base.Data(2, "f32")
    x, w = f8_inputs(f, T, C, "f32"), torch.randn(O, C, generator=f.gen) * C ** -0.5
    q, s = mc.quantize_f8(x.to(DEV))
    wq, ws = mc.quantize_f8(w.to(DEV))
    b = torch.randn(O, generator=f.gen) if bias else None
    e, we = s.view(torch.uint8).cpu().t().int() - 127, ws.view(torch.uint8).cpu().t().int() - 127
    want, size_of = ref.product(q.float().cpu(), e, wq.float().cpu(), we)
    bound = (q.shape[1] / 16 + 8) * ref.U * size_of
    if out == "bf16":
        bound = bound + 2.0 ** -13 * size_of
    if bias:
        want = want + b.double()
        bound = bound + 2 * ref.U * (size_of + b.abs().double())
    args = (q, s, wq, ws, None if b is None else b.to(DEV))
    y = mc.matmul_f8(*args, out_dtype=TDT[out])
    print(mc.matmul_f8_describe(T, O, q.shape[1]))
    agree("y", y, want, bound, ref.HALF[out])
    # a matrix of the output's own; channel-major in batches; without a workspace no splits
    for L in {T, max(d for d in range(1, 33) if T % d == 0)}:
        z = torch.full((T // L, O, L), float("nan"), dtype=TDT[out], device=DEV)
        assert mc.matmul_f8(*args, length=L, y=z) is z
        assert torch.equal(z.transpose(1, 2).reshape(T, O), y), L
    none = mc.matmul_f8(*args, out_dtype=TDT[out], workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    agree("without splits", none, want, bound, ref.HALF[out])


def test_product_keeps_fp32(mc):
    """Terms of 2^14 that cancel beside terms of 1: an fp32 output holds the small ones' sum to 2^-9."""
    T, C, O = 70, 256, 80
    x = torch.ones(T, C)
    x[:, 0], x[:, 1] = 128.0, 128.0
    w = torch.ones(O, C)
    w[:, 0], w[:, 1] = 128.0, -128.0
    q, s, wq, ws = *mc.quantize_f8(x.to(DEV)), *mc.quantize_f8(w.to(DEV))
    y = mc.matmul_f8(q, s, wq, ws)
    assert float((y - 254.0).abs().max()) <= 2.0 ** -9


@pytest.mark.parametrize("T", [5, 200])
def test_bad_blocks_stay_in_their_rows(mc, T):
    f = base.Data(4, "f32")
    x, w = torch.randn(T, 300, generator=f.gen), torch.randn(90, 300, generator=f.gen)
    wq, ws = mc.quantize_f8(w.to(DEV))
    for out in (torch.float32, torch.bfloat16):
        clean = mc.matmul_f8(*mc.quantize_f8(x.to(DEV)), wq, ws, out_dtype=out)
        z = x.clone()
        z[2, 7], z[4, 299] = INF, float("nan")
        y = mc.matmul_f8(*mc.quantize_f8(z.to(DEV)), wq, ws, out_dtype=out)
        rest = [t for t in range(T) if t not in (2, 4)]
        assert torch.equal(y[rest], clean[rest]) and bool(y[[2, 4]].isnan().all())


def test_weight_gradient_through_turned_blocks(mc):
    """A training step of y = x w^T: dx = dy w and dw = dy^T x with blocks along what each sums over."""
    f = base.Data(5, "f32")
    T, C, O = 150, 200, 170
    x, w, dy = (torch.randn(*s, generator=f.gen).to(DEV) for s in ((T, C), (O, C), (T, O)))
    dx = mc.matmul_f8(*mc.quantize_f8(dy), *mc.quantize_f8(w[None], channel_major=True))
    dw = mc.matmul_f8(*mc.quantize_f8(dy[None], channel_major=True), *mc.quantize_f8(x[None], channel_major=True))
    # each 8-bit operand is off by half a step, 2^-4 of the value at most
    for got, a, b in ((dx, dy, w), (dw, dy.t(), x)):
        a, b = a.double().cpu(), b.double().cpu()
        assert got.shape == (a @ b).shape
        assert bool(((got.double().cpu() - a @ b).abs() <= 2 * 2.0 ** -4 * 1.04 * (a.abs() @ b.abs())).all())


def test_f8_repeats_streams_and_graphs(mc):
    f = base.Data(6, "bf16")
    x, w = f.make(3, 60, 700)[1], f.make(500, 700)[1]

    def work():
        return mc.matmul_f8(*mc.quantize_f8(x), *mc.quantize_f8(w), out_dtype=torch.bfloat16, length=60)
    first = work()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = work()
    torch.cuda.synchronize()
    assert torch.equal(first, second)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for _ in range(3):
        x.mul_(-1.5)
        graph.replay()
        got, want = held.clone(), work()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
