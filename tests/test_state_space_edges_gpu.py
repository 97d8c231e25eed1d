"""State-space operators where a multiplication by zero does not clear what it meets: states, parameters and
steps that hold infinities or NaN next to the padding of a ragged batch, and decays that leave fp32.
"""
import pytest
import torch

import test_state_space_gpu as base

pytestmark = pytest.mark.gpu
mc = base.mc
DEV, TDT = base.DEV, base.TDT
INF = float("inf")

#         B  D     L     N  the forward pass takes        lengths
SHAPES = [(2, 3, 900, 5, "64x16 segments=1", [897, 450]),
          (2, 300, 500, 4, "64x8 segments=1", [1, 403]),
          (2, 4100, 129, 3, "16x8 segments=1", [128, 30]),
          (2, 3, 300, 17, "16x8shared segments=1", [3, 290]),
          (1, 64, 3100, 2, "64x16 segments=4", [1029])]


def inputs(B, D, L, N, dt, seed=0):
    f = base.Data(seed, dt)
    d = {k: f.make(B, D, L)[1] for k in ("x", "delta", "z", "dy")}
    d["B"], d["C"] = f.make(B, 1, N, L)[1], f.make(B, 1, N, L)[1]
    d["A"] = torch.full((D, N), -0.01, device=DEV)
    d["D"] = f.make(D, dtype=torch.float32)[1]
    d["h0"] = f.make(B, D, N, dtype=torch.float32)[1]
    d["dfs"] = f.make(B, D, N, dtype=torch.float32)[1]
    return d


def forward_backward(mc, d, n, gate):
    B, D, L = d["x"].shape
    common = dict(D=d["D"], z=d["z"] if gate else None, softplus=True, lengths=n)
    r = {"fs": torch.full_like(d["h0"], 7.0), "dh0": torch.full_like(d["h0"], 7.0)}
    states = mc.selective_scan_states(d["x"], d["A"])
    r["y"] = mc.selective_scan_fwd(d["x"], d["delta"], d["A"], d["B"], d["C"], initial_state=d["h0"],
                                   final_state=r["fs"], states=states, **common)
    r.update(mc.selective_scan_bwd(d["x"], d["delta"], d["A"], d["B"], d["C"], d["dy"], states,
                                   d_final_state=d["dfs"], d_initial_state=r["dh0"], **common))
    return r


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("B,D,L,N,form,lengths", SHAPES)
def test_padding_is_zero_whatever_a_row_holds(mc, B, D, L, N, form, lengths, gate, dt):
    """A state of infinity, an infinite gradient of the final state and a NaN parameter stay in their rows
    and out of the padding."""
    assert form in mc.selective_scan_fwd_describe(B, D, L, N)
    d = inputs(B, D, L, N, dt)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    clean = forward_backward(mc, d, n, gate)
    d["h0"][0, 1] = INF
    d["dfs"][B - 1, 0] = -INF
    d["D"][2] = float("nan")
    r = forward_backward(mc, d, n, gate)
    assert bool((r["fs"][0, 1] == INF).all())
    others = [c for c in range(D) if c not in (0, 1, 2)]
    for name in ("y", "dx", "ddelta") + (("dz",) if gate else ()):
        for b, m in enumerate(lengths):
            assert not r[name][b, :, m:].any() and bool(r[name][b, :, m:].isfinite().all()), (name, b)
        assert torch.equal(r[name][:, others], clean[name][:, others]), name
    for name in ("dB", "dC"):
        for b, m in enumerate(lengths):
            assert not r[name][b, :, :, m:].any() and bool(r[name][b, :, :, m:].isfinite().all()), (name, b)
    assert torch.equal(r["dA"][others], clean["dA"][others])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L,N,form,lengths", SHAPES)
def test_decay_past_fp32(mc, B, D, L, N, form, lengths, dt):
    """A so negative that A log2(e) is no fp32 number: every decay is 0, as for -1e30, and a step past the
    end leaves the state as it is."""
    d = inputs(B, D, L, N, dt, seed=1)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    d["A"].fill_(-1e30)
    want = forward_backward(mc, d, n, True)
    assert bool(want["fs"].isfinite().all())
    for a in (-3e38, -INF):
        d["A"].fill_(a)
        got = forward_backward(mc, d, n, True)
        for k in want:
            assert want[k] is None or torch.equal(got[k], want[k]), (a, k)


@pytest.mark.parametrize("N", [3, 16])
def test_step_of_size_zero(mc, N):
    """softplus(-200) is 0 in fp32: the state stays, whatever finite decay it has."""
    f = base.Data(2, "f32")
    x, Bm, state = f.make(2, 5)[1], f.make(2, 1, N)[1], f.make(2, 5, N)[1]
    delta, out = torch.full_like(x, -200.0), torch.empty(2, 5, N, device=DEV)
    for a in (-1.0, -1e30, -3e38):
        mc.selective_scan_step(x, delta, torch.full((5, N), a, device=DEV), Bm, Bm, state, softplus=True, state_out=out)
        assert torch.equal(out, state), a


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_convolution_gradients_keep_an_infinity_in_its_tap(mc, dt):
    """Without an activation dw[k] = sum_t dy[t] x[t-K+1+k]: an infinity at the last step reaches the last
    tap alone, whatever the length leaves of an eight-step tile."""
    K, D = 4, 3
    for L, n in ((13, None), (16, None), (24, 13), (700, 509)):
        f = base.Data(L, dt)
        x, dy, w = f.make(2, D, L)[1], f.make(2, D, L)[1], f.make(D, K)[1]
        h0 = f.make(2, D, K - 1)[1]
        lengths = None if n is None else torch.tensor([n, n], dtype=torch.int32, device=DEV)
        call = dict(lengths=lengths, initial_state=h0, bias=torch.zeros(D, device=DEV))
        clean = mc.causal_conv1d_bwd(x, w, dy, **call)
        x[1, 1, (n or L) - 1] = INF
        dy[1, 1, (n or L) - 1] = 1.0
        dx, dw, db = mc.causal_conv1d_bwd(x, w, dy, **call)
        assert float(dw[1, K - 1]) == INF and bool(dw[1, :K - 1].isfinite().all()), (L, n, dw[1])
        assert bool(dx.isfinite().all()) and bool(db.isfinite().all())
        assert torch.equal(dw[[0, 2]], clean[1][[0, 2]])
    # one valid step: of the state before it only the taps that reach it
    x, dy, w, h0 = (base.Data(9, dt).make(*s)[1] for s in ((1, D, 20), (1, D, 20), (D, K), (1, D, K - 1)))
    h0[0, 1, K - 2] = INF
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    _, dw, _ = mc.causal_conv1d_bwd(x, w, dy, lengths=one, initial_state=h0)
    finite = dw[1].isfinite().tolist()
    assert finite == [True, True, False, True], dw[1]


def test_slices_of_one_buffer(mc):
    """Operands and outputs that lie in one buffer without sharing an element: slices along time, every
    other channel, batches inside channels.  One element more is refused."""
    B, D, L, N = 2, 5, 24, 3
    f = base.Data(4, "f32")
    x, dl, w = f.make(B, D, L)[1], f.make(B, D, L)[1], f.make(D, 4)[1]
    want = mc.causal_conv1d_fwd(x, w, silu=True)
    time = torch.zeros(B, D, 2 * L, device=DEV)
    inner = torch.zeros(D, 2, B, L, device=DEV).permute(2, 1, 0, 3)
    for xs, ys in ((time[:, :, :L], time[:, :, L:]), (time[:, :, L:], time[:, :, :L]),
                   (torch.zeros(B, 2 * D, L, device=DEV)[:, i::2] for i in (0, 1)), (inner[:, 0], inner[:, 1])):
        xs.copy_(x)
        mc.causal_conv1d_fwd(xs, w, silu=True, y=ys)
        assert torch.equal(ys, want) and torch.equal(xs, x)
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(time[:, :, :L], w, y=time[:, :, L - 1:2 * L - 1])
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(inner[:, 0], w, y=inner[:, 0])
    # the three gradients of a scan next to each other, row by row
    A, Bm, Cm = -torch.rand(D, N, device=DEV), f.make(B, 1, N, L)[1], f.make(B, 1, N, L)[1]
    states = mc.selective_scan_states(x, A)
    mc.selective_scan_fwd(x, dl, A, Bm, Cm, z=x, softplus=True, states=states)
    r = mc.selective_scan_bwd(x, dl, A, Bm, Cm, x, states, z=x, softplus=True)
    out = torch.zeros(B, D, 3, L, device=DEV)
    mc.selective_scan_bwd(x, dl, A, Bm, Cm, x, states, z=x, softplus=True, dx=out[:, :, 0], ddelta=out[:, :, 1],
                          dz=out[:, :, 2])
    for i, k in enumerate(("dx", "ddelta", "dz")):
        assert torch.equal(out[:, :, i], r[k]), k
    # one step: every other value of a buffer
    pairs, state = torch.zeros(B, 2 * D, device=DEV), f.make(B, D, 3)[1]
    y = mc.causal_conv1d_step(x[..., 0], state.clone(), w)
    pairs[:, ::2] = x[..., 0]
    mc.causal_conv1d_step(pairs[:, ::2], state, w, y=pairs[:, 1::2])
    assert torch.equal(pairs[:, 1::2], y)
