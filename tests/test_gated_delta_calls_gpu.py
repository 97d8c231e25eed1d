"""Calls of the gated delta layer's operators that the documentation allows and the other tests do not make: a scale of the
caller's, operands and outputs far from each other, scales that say NaN.
"""
import functools

import pytest
import torch

import delta_reference as ref
import test_gated_delta_gpu as rule
import test_state_space_gpu as base

pytestmark = pytest.mark.gpu
mc = base.mc
DEV, TDT = base.DEV, base.TDT


class Scaled(rule.Case):
    SCALE = -0.7

    def kw(self):
        return dict(super().kw(), scale=self.SCALE)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("l2norm", [False, True])
def test_a_scale_of_the_callers(mc, monkeypatch, l2norm, dt):
    """Both passes and the step with queries scaled by -0.7 instead of P^-0.5."""
    monkeypatch.setattr(ref, "rule", functools.partial(ref.rule, scale=Scaled.SCALE))
    c = Scaled(2, 2, 4, 48, 40, 101, dt, 21, l2norm, True, True)
    rule.compare(c, rule.run(mc, c))
    one = {k: v[..., 0].contiguous() for k, v in c.dev.items()}
    alone = dict(key_heads=2, l2norm=l2norm, scale=Scaled.SCALE)
    s = c.s0[1].clone()
    y = mc.gated_delta_step(*(one[k] for k in ("q", "k", "v", "g", "beta")), s, **alone)
    want, ws = ref.rule(*(c.host[k][..., :1] for k in ("q", "k", "v", "g", "beta")), 2, l2norm=l2norm,
                        state=torch.from_numpy(c.s0[0]).double())
    rows = [b for b in range(2) if c.lengths[0][b] > 0]          # the first step of the others is poisoned
    a = (3 * 48 + 16) * ref.U
    rule.agree("y of a step", y[rows], want[rows, :, 0], a, ref.HALF[dt])
    rule.agree("its state", s[rows], ws[rows], a, ref.HALF["f32"])


def far(shape, like):
    """A view of two parts 2^31 elements and more apart, with the values of `like`."""
    step = (1 << 31) + 64
    stride = like[0].stride()
    t = torch.as_strided(torch.empty(step + like[0].numel(), dtype=like.dtype, device=DEV), shape, (step, *stride))
    t.copy_(like)
    return t


@pytest.mark.parametrize("major", [False, True], ids=["tokens", "channels"])
def test_norm_and_quantiser_far_apart(mc, major):
    """Sequences whose offsets pass 2^31 elements and 2^32 bytes: the bits of neighbouring ones."""
    gen = torch.Generator().manual_seed(22)
    shape = (2, 300, 70) if major else (2, 70, 300)
    x, dy = (torch.randn(shape, generator=gen).to(DEV, torch.bfloat16) for _ in range(2))
    w, b = torch.randn(300, generator=gen).to(DEV), torch.randn(300, generator=gen).to(DEV)
    kw = dict(channel_major=major)
    stats = mc.layer_norm_stats(x, **kw)
    near = (mc.layer_norm_fwd(x, w, b, stats=stats, **kw), *mc.layer_norm_bwd(x, dy, stats, w, b, **kw), *mc.quantize_f8(x, **kw))
    fx, fdy, y, dx = (far(shape, t) for t in (x, dy, x, x))
    stats.fill_(float("nan"))
    mc.layer_norm_fwd(fx, w, b, y=y, stats=stats, **kw)
    _, dw, db = mc.layer_norm_bwd(fx, fdy, stats, w, b, dx=dx, **kw)
    for got, want in zip((y, dx, dw, db, *mc.quantize_f8(fx, **kw)), near):
        assert torch.equal(got.float(), want.float())


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product_of_operands_past_4_gb(mc, out):
    """The last of 40000 tokens of 131072 channels: the bits of a product of their own."""
    T, K, O = 40000, 131072, 40
    gen = torch.Generator(device=DEV).manual_seed(23)
    q = torch.randint(0, 0x70, (T, K), dtype=torch.uint8, device=DEV, generator=gen).view(torch.float8_e4m3fn)
    wq = torch.randint(0, 0x70, (O, K), dtype=torch.uint8, device=DEV, generator=gen).view(torch.float8_e4m3fn)
    s = torch.randint(120, 130, (K // 128, T), dtype=torch.uint8, device=DEV, generator=gen).view(torch.float8_e8m0fnu)
    ws = torch.randint(120, 130, (K // 128, O), dtype=torch.uint8, device=DEV, generator=gen).view(torch.float8_e8m0fnu)
    kw = dict(out_dtype=TDT[out], workspace=torch.empty(0, dtype=torch.uint8, device=DEV))      # no splits
    y = mc.matmul_f8(q, s, wq, ws, **kw)
    last = s.view(torch.uint8)[:, -150:].contiguous().view(torch.float8_e8m0fnu)
    assert "tile=64" in mc.matmul_f8_describe(150, O, K)
    assert torch.equal(y[-150:], mc.matmul_f8(q[-150:].contiguous(), last, wq, ws, **kw))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 40, 80, 300])
def test_scales_that_say_nan_and_the_outermost_powers(mc, T, out):
    """A scale of 255 makes the token, or the channel, NaN, whatever its numbers; 2^-127 and 2^127 meet as 1."""
    K, O = 256, 80
    f8 = lambda t: t.view(torch.float8_e8m0fnu)  # noqa: E731
    q, wq = (torch.ones(n, K, device=DEV).to(torch.float8_e4m3fn) for n in (T, O))
    s, ws = (torch.full((K // 128, n), 127, dtype=torch.uint8, device=DEV) for n in (T, O))
    q[3] = 0.0
    s[1, 2] = s[0, 3] = ws[0, 7] = 255
    y = mc.matmul_f8(q, f8(s), wq, f8(ws), out_dtype=TDT[out])
    bad = torch.zeros(T, O, dtype=torch.bool, device=DEV)
    bad[2:4] = True
    bad[:, 7] = True
    assert torch.equal(y.isnan(), bad) and bool((y[~bad] == 256.0).all())
    q[3] = 1.0
    s.fill_(0)
    ws.fill_(254)
    assert bool((mc.matmul_f8(q, f8(s), wq, f8(ws), out_dtype=TDT[out]) == 256.0).all())
