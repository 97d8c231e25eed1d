"""Gated delta rule, layer norm and block-scaled 8-bit products without a GPU: every refusal of the C ABI (fake device
addresses that are never dereferenced), the binding's checks, workspace sizes, and the plain forms' gradients
against differences.
"""
import ctypes

import pytest
import torch

import convolution_implicit_gemm_nchw_amd as mc
import delta_reference as ref
import test_state_space_cpu as base

OK, E_NULL, E_DIM, E_DT, E_ALIAS, E_ALIGN, E_WS, E_BIG = (base.OK, base.E_NULL, base.E_DIM, base.E_DT, base.E_ALIAS,
                                                          base.E_ALIGN, base.E_WS, base.E_BIG)
SIZE_MAX = (1 << 64) - 1
at = base.at


def rows(i, D, L=40):
    return mc._Rows(at(i), D * L, L)


def delta_args(**kw):
    d = mc._GatedDelta(B=2, Hk=2, Hv=4, P=8, V=6, L=40, l2norm=1, scale=0.5, q=rows(0, 16), k=rows(1, 16), v=rows(2, 24),
                       g=rows(3, 4), beta=rows(4, 4), initial_state=at(5), lengths=at(6), y=rows(7, 24), final_state=at(8),
                       states=at(9), dy=rows(10, 24), d_final_state=at(11), dq=rows(12, 16), dk=rows(13, 16),
                       dv=rows(14, 24), dg=at(15), dbeta=at(16), d_initial_state=at(17))
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def dfwd(dtype=0, ws=at(30), wb=1 << 24, **kw):
    return mc.lib().gated_delta_fwd(ctypes.byref(delta_args(**kw)), dtype, ws, wb, None)


def dbwd(dtype=0, ws=at(30), wb=1 << 24, **kw):
    return mc.lib().gated_delta_bwd(ctypes.byref(delta_args(**kw)), dtype, ws, wb, None)


def test_delta_refusals():
    lib = mc.lib()
    assert lib.gated_delta_fwd(None, 0, None, 0, None) == E_NULL
    assert lib.gated_delta_bwd(None, 0, None, 0, None) == E_NULL
    assert lib.gated_delta_step(None, 0, None, 1, None, None, None) == E_NULL
    none = mc._Rows(None, 0, 0)
    for call in (dfwd, dbwd):
        for bad in ({"B": 0}, {"Hk": 0}, {"Hv": -1}, {"Hv": 3}, {"Hk": 8}, {"P": 0}, {"P": 257}, {"V": 0}, {"V": 513},
                    {"L": 0}, {"L": (1 << 30) + 1}, {"Hv": 65538}, {"k": mc._Rows(at(1), 640, -40)}):
            assert call(**bad) == E_DIM, bad
        assert call(dtype=2) == E_DT
        assert call(B=1 << 29) == E_BIG
        assert call(v=mc._Rows(at(2), 1 << 50, 40)) == E_BIG
        for name in ("q", "k", "v", "g", "beta"):
            assert call(**{name: none}) == E_NULL, name
        assert call(g=mc._Rows(at(3) + 2, 160, 40)) == E_ALIGN
        assert call(dtype=1, q=mc._Rows(at(0) + 1, 640, 40)) == E_ALIGN
        assert call(dtype=1, beta=mc._Rows(at(4) + 2, 160, 40)) == E_ALIGN      # fp32 beside bf16
        assert call(states=at(9) + 4) == E_ALIGN
        assert call(ws=at(30) + 8) == E_ALIGN
        assert call(ws=None, wb=0) == E_NULL
        assert call(wb=4096) == E_WS
    assert dfwd(y=none) == E_NULL
    assert dfwd(y=rows(2, 24)) == E_ALIAS
    assert dfwd(y=mc._Rows(at(7), 960, 39)) == E_DIM                            # rows of y overlap
    assert dfwd(final_state=at(5)) == E_ALIAS                                   # states are not updated in place
    assert dfwd(states=at(0)) == E_ALIAS
    assert dfwd(states=at(30) + 4096) == E_ALIAS                                # on the workspace
    for name in ("dy", "dq", "dk", "dv"):
        assert dbwd(**{name: none}) == E_NULL, name
    for name in ("dg", "dbeta", "states"):
        assert dbwd(**{name: None}) == E_NULL, name
    assert dbwd(dq=rows(10, 16)) == E_ALIAS
    assert dbwd(dk=rows(12, 16)) == E_ALIAS
    assert dbwd(dg=at(16)) == E_ALIAS
    assert dbwd(d_initial_state=at(11)) == E_ALIAS

    def step(slots=2, state=at(20), out=at(21), slot_of=None, **kw):
        kw = {**dict(L=1, q=rows(0, 16, 1), k=rows(1, 16, 1), v=rows(2, 24, 1), g=rows(3, 4, 1), beta=rows(4, 4, 1),
                     y=rows(7, 24, 1)), **kw}
        return lib.gated_delta_step(ctypes.byref(delta_args(**kw)), kw.pop("dtype", 0), state, slots, slot_of, out, None)
    assert step(L=2) == E_DIM and step(slots=0) == E_DIM and step(slots=3) == E_DIM
    assert step(state=None) == E_NULL and step(out=None) == E_NULL
    assert step(out=at(20) + 64) == E_ALIAS                                     # shifted on its own input
    assert step(out=at(0)) == E_ALIAS
    assert step(y=rows(2, 24, 1)) == E_ALIAS


def tokens(i, B=2, L=40, C=24, major=False):
    return mc._Tokens(at(i), L * C, 1 if major else C, L if major else 1)


def norm_args(major=False, **kw):
    n = mc._LayerNorm(B=2, L=40, C=24, eps=1e-5, x=tokens(0, major=major), weight=at(1), bias=at(2), lengths=at(3),
                      y=tokens(4, major=major), stats=at(5), dy=tokens(6, major=major), dx=tokens(7, major=major), dw=at(8),
                      db=at(9))
    for k, v in kw.items():
        setattr(n, k, v)
    return n


def nfwd(dtype=0, **kw):
    return mc.lib().layer_norm_fwd(ctypes.byref(norm_args(**kw)), dtype, None)


def nbwd(dtype=0, ws=at(30), wb=1 << 20, **kw):
    return mc.lib().layer_norm_bwd(ctypes.byref(norm_args(**kw)), dtype, ws, wb, None)


@pytest.mark.parametrize("major", [False, True])
def test_layer_norm_refusals(major):
    lib = mc.lib()
    assert lib.layer_norm_fwd(None, 0, None) == E_NULL and lib.layer_norm_bwd(None, 0, None, 0, None) == E_NULL
    for call in (nfwd, nbwd):
        for bad in ({"B": 0}, {"L": 0}, {"C": 0}, {"C": (1 << 20) + 1}, {"x": mc._Tokens(at(0), 960, 24, 2)},
                    {"x": mc._Tokens(at(0), -960, 1 if major else 24, 40 if major else 1)},
                    {"x": tokens(0, major=not major)}):
            assert call(major=major, **bad) == E_DIM, bad
        assert call(major=major, dtype=3) == E_DT
        assert call(major=major, B=1 << 20, L=1 << 20) == E_BIG
        assert call(major=major, x=mc._Tokens(None, 0, 24, 1)) != OK
        assert call(major=major, weight=at(1) + 2) == E_ALIGN
    assert nfwd(major=major, y=tokens(0, major=major)) == E_ALIAS               # in place
    assert nfwd(major=major, stats=at(4)) == E_ALIAS
    assert nbwd(major=major, stats=None) == E_NULL
    assert nbwd(major=major, dx=tokens(6, major=major)) == E_ALIAS
    assert nbwd(major=major, dw=at(9)) == E_ALIAS
    assert nbwd(major=major, ws=None, wb=0) == E_NULL
    assert nbwd(major=major, wb=24 * 8 - 1) == E_WS
    assert nbwd(major=major, db=at(30)) == E_ALIAS
    for eps in (-1e-5, float("nan"), float("inf")):
        assert nfwd(major=major, eps=eps) == E_DIM


def test_f8_refusals():
    lib = mc.lib()
    q = [2, 40, 24, 0, at(0), 960, 24, 1, at(1), at(2), None]

    def quant(**kw):
        a = list(q)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.quantize_f8(*a)
    assert quant(_0=0) == E_DIM and quant(_1=0) == E_DIM and quant(_2=0) == E_DIM and quant(_2=131073) == E_DIM
    assert quant(_3=2) == E_DT
    assert quant(_6=24, _7=2) == E_DIM and quant(_5=-960) == E_DIM
    assert quant(_0=1 << 20, _1=1 << 20) == E_BIG
    assert quant(_4=None) == E_NULL and quant(_8=None) == E_NULL and quant(_9=None) == E_NULL
    assert quant(_4=at(0) + 2) == E_ALIGN and quant(_8=at(1) + 8) == E_ALIGN
    assert quant(_8=at(0)) == E_ALIAS and quant(_9=at(1) + 128) == E_ALIAS
    m = [2, 40, 24, 256, at(0), at(1), at(2), at(3), at(4), 0, 0, at(5), None, 0, None]

    def product(**kw):
        a = list(m)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return lib.matmul_f8(*a)
    assert product(_0=0) == E_DIM and product(_2=0) == E_DIM and product(_3=0) == E_DIM and product(_3=200) == E_DIM
    assert product(_3=131072 + 128) == E_DIM
    assert product(_10=2) == E_DT
    assert product(_0=1 << 20, _1=1 << 11) == E_BIG
    for i in (4, 5, 6, 7, 11):
        assert product(**{f"_{i}": None}) == E_NULL, i
    assert product(_4=at(0) + 4) == E_ALIGN and product(_6=at(2) + 1) == E_ALIGN and product(_8=at(4) + 1) == E_ALIGN
    assert product(_11=at(0)) == E_ALIAS and product(_11=at(1) - 4) == E_ALIAS
    assert product(_12=None, _13=64) == E_NULL


def test_binding_refusals():
    """What the Python functions refuse before any GPU call: types, shapes, strides, devices."""
    z = torch.zeros
    q, v, g = z(2, 16, 40), z(2, 24, 40), z(2, 4, 40)

    def bad(fn, *a, **k):
        with pytest.raises((ValueError, RuntimeError, TypeError)):
            fn(*a, **k)
    for fn in (lambda **k: mc.gated_delta_fwd(**{**dict(q=q, k=q, v=v, g=g, beta=g, key_heads=2), **k}),):
        bad(fn)                                                        # not on a GPU
        bad(fn, key_heads=3)
        bad(fn, k=z(2, 16, 41))
        bad(fn, v=z(2, 25, 40))
        bad(fn, g=z(2, 4, 40, dtype=torch.bfloat16))
        bad(fn, q=z(2, 16, 40, dtype=torch.float16))
        bad(fn, lengths=z(2))
        bad(fn, initial_state=z(2, 4, 8, 7))
    bad(mc.gated_delta_step, z(2, 16), z(2, 16), z(2, 24), z(2, 4), z(2, 4), z(2, 4, 8, 6), key_heads=2)
    bad(mc.layer_norm_fwd, z(3, 8))
    bad(mc.layer_norm_fwd, z(3, 8, dtype=torch.float64))
    bad(mc.layer_norm_bwd, z(3, 8), z(3, 8), z(2, 3))
    bad(mc.quantize_f8, z(3, 8))
    bad(mc.matmul_f8, z(3, 128, dtype=torch.int8), z(1, 3), z(3, 128, dtype=torch.int8), z(1, 3))
    bad(mc.matmul_f8, z(3, 128), z(1, 3), z(3, 128), z(1, 3), out_dtype=torch.float16)


# ------------------------------------------------------------------ workspaces

SIZES = [(1, 1, 1, 1, 1, 1), (2, 2, 4, 64, 64, 999), (8, 16, 32, 128, 128, 8192), (1, 4, 4, 256, 512, 100000),
         (1 << 15, 1, 2, 16, 16, 3), (1, 1, 48, 100, 30, 1 << 22), (3, 1, 3, 250, 17, 130)]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_delta_under_any_limit(size, dt, backward):
    """The size under a limit is within it, or the least there is; a call given that much uses that much."""
    least = mc.gated_delta_workspace(*size, dtype=dt, backward=backward, limit=0)
    before = 0
    for limit in [0, least - 1, least] + [10 ** k for k in range(4, 10)] + [SIZE_MAX]:
        w = mc.gated_delta_workspace(*size, dtype=dt, backward=backward, limit=limit)
        assert w == least or least < w <= min(limit, mc.MAX_WORKSPACE_BYTES)
        assert before <= w
        before = w
        assert mc.gated_delta_describe(*size, dtype=dt, backward=backward, workspace_bytes=w).endswith(f" ws={w}")
    with pytest.raises(ValueError):
        mc.gated_delta_describe(*size, dtype=dt, backward=backward, workspace_bytes=least - 1)


def test_other_workspaces_under_any_limit():
    need, lib = ctypes.c_size_t(0), mc.lib()
    for shape in ((1, 1, 1), (4, 2048, 1000), (2, 77, 9000), (1, 3, 1 << 20)):
        n = mc._LayerNorm(B=shape[0], L=shape[1], C=shape[2], x=mc._Tokens(at(0), 0, shape[2], 1),
                          dy=mc._Tokens(at(1), 0, shape[2], 1), dx=mc._Tokens(at(2), 0, shape[2], 1))
        before = 0
        for limit in (0, 1000, 10 ** 6, 10 ** 9, SIZE_MAX):
            assert lib.layer_norm_bwd_workspace_size(ctypes.byref(n), 0, limit, ctypes.byref(need)) == OK
            assert need.value == 8 * shape[2] or need.value <= limit
            assert before <= need.value
            before = need.value
    for shape in ((1, 1, 1, 128), (1, 100, 70, 8192), (4, 2048, 8192, 4096)):
        for limit in (0, 1000, 10 ** 6, 10 ** 9, SIZE_MAX):
            assert lib.matmul_f8_workspace_size(*shape, limit, ctypes.byref(need)) == OK
            assert need.value <= min(limit, mc.MAX_WORKSPACE_BYTES)


# ------------------------------------------------------------------ the plain forms

@pytest.mark.parametrize("l2norm", [False, True])
def test_rule_gradients_against_differences(l2norm):
    """Central differences in a random direction: of third order in the step 1e-4, so off by about 1e-8."""
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    B, Hk, Hv, P, V, L = 2, 2, 4, 3, 5, 7
    x = [r(B, Hk * P, L) * 0.5, r(B, Hk * P, L) * 0.5, r(B, Hv * V, L), -r(B, Hv, L).abs(), torch.sigmoid(r(B, Hv, L)),
         r(B, Hv, P, V)]
    d = [r(*t.shape) for t in x]
    wy, ws = r(B, Hv * V, L), r(B, Hv, P, V)

    def loss(*a):
        y, s = ref.rule(*a[:5], Hk, l2norm=l2norm, state=a[5], lengths=torch.tensor([L, 3]))
        return (y * wy).sum() + (s * ws).sum()
    leaves = [t.clone().requires_grad_() for t in x]
    loss(*leaves).backward()
    got = sum((t.grad * e).sum() for t, e in zip(leaves, d))
    h = 1e-4
    want = (loss(*(t + h * e for t, e in zip(x, d))) - loss(*(t - h * e for t, e in zip(x, d)))) / (2 * h)
    assert abs(got - want) <= 1e-6 * abs(want) + 1e-6


def test_norm_gradients_against_differences():
    gen = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b, dy = r(2, 5, 9) + 1, r(9), r(9), r(2, 5, 9)
    n = torch.tensor([5, 2])
    g = ref.layer_norm(x, w, b, 1e-5, n, dy)
    dirs = [r(2, 5, 9), r(9), r(9)]
    got = sum((g[k][0] * d).sum() for k, d in zip(("dx", "dw", "db"), dirs))
    h = 1e-5
    f = lambda s: (ref.layer_norm(*(t + s * h * d for t, d in zip((x, w, b), dirs)), 1e-5, n)["y"][0] * dy).sum()  # noqa: E731
    assert abs(got - (f(1) - f(-1)) / (2 * h)) <= 1e-6 * (1 + abs(got))


def test_quantiser_reference():
    """Borders of the plain quantiser: powers that fit exactly, just above, the least and zero."""
    x = torch.zeros(6, 130)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 448.0, 448.0000305, 1.75, 2.0 ** -149
    x[4, 129], x[5, 3] = 7.0, float("inf")
    q, e, bad = ref.quantize(x)
    assert e[:, 0].tolist()[:5] == [0, 1, -8, -127, -127] and e[4, 1] == -6
    assert bad.tolist() == [[False, False]] * 5 + [[True, False]]
    assert q[0, 0] == 448 and q[2, 0] == 448 and q[4, 129] == 448
