"""GPU parity of the state-space operators against plain 64-bit forms (ssm_reference.py), element by
element, with the bounds derived there.  Activations are views into larger buffers whose other elements
must stay untouched; outputs are pre-filled with NaN, so an unwritten element fails; what lies past a
sequence's length is poisoned with NaN and infinities.
"""
import numpy as np
import pytest
import torch

import ssm_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def mc():
    import convolution_implicit_gemm_nchw_amd as m
    return m


def _say(*a):
    print(*a, flush=True)


class Data:
    """Seeded inputs of one element type: host values (already rounded to it, in 64 bits) and device copies."""

    def __init__(self, seed, dt):
        self.gen, self.dt = torch.Generator().manual_seed(seed), dt

    def make(self, *shape, scale=1.0, shift=0.0, dtype=None):
        t = (torch.randn(shape, generator=self.gen) * scale + shift).to(dtype or TDT[self.dt])
        return t.double().numpy(), t.to(DEV)

    def lengths(self, B, L):
        n = torch.randint(0, L + 1, (B,), generator=self.gen, dtype=torch.int32)
        special = torch.tensor([L, 0, 1, L + 5, -3], dtype=torch.int32)   # full, empty, one, clamped twice
        n[:min(B, 5)] = special[:B]
        return n.numpy(), n.to(DEV)


def view(t, lead=3, tail=5):
    """t's values as a view [B, D, L] inside a larger buffer filled with 7s, and a check of the rest."""
    B, D, L = t.shape
    buf = torch.full((B, D + 2, lead + L + tail), 7.0, dtype=t.dtype, device=t.device)
    v = buf[:, 1:D + 1, lead:lead + L]
    v.copy_(t)

    def untouched():
        rest = buf.clone()
        rest[:, 1:D + 1, lead:lead + L] = 7.0
        assert bool((rest == 7.0).all())
    return v, untouched


def out_view(shape, dt):
    return view(torch.full(shape, float("nan"), dtype=TDT[dt], device=DEV))


def poison(t, lengths):
    """NaN and infinities past each sequence's length (last axis time)."""
    if lengths is None:
        return t
    L = t.shape[-1]
    past = torch.arange(L) >= torch.as_tensor(np.clip(lengths, 0, L))[:, None]
    past = past.view(past.shape[0], *([1] * (t.dim() - 2)), L).to(t.device).expand_as(t)
    bad = torch.full_like(t, float("nan"))
    bad[..., ::3] = float("inf")
    return torch.where(past, bad, t)


def agree(name, got, pair, kind, case):
    worst = ref.within(got.double().cpu().numpy(), *pair, kind)
    _say(f"{case} {name}: {worst:.3f} of the bound")
    assert worst <= 1.0, (name, worst)


# ------------------------------------------------------------------ causal convolution

#            B  D   L     K  silu  bias  ragged state
CONV = [(1, 1, 1, 4, True, True, False, False),
        (2, 5, 1, 1, False, False, False, False),
        (6, 3, 7, 4, True, True, True, True),
        (2, 9, 8, 2, True, False, False, True),
        (3, 4, 9, 8, True, True, True, True),
        (5, 7, 65, 3, False, True, True, True),
        (2, 3, 523, 4, True, True, False, False),
        (6, 2, 2051, 5, True, True, True, False),
        (1, 3, 4100, 7, True, True, False, True),
        (40, 2, 600, 6, True, True, False, True)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", CONV, ids=lambda c: "-".join(map(str, c)))
def test_convolution(mc, case, dt):
    B, D, L, K, act, has_bias, ragged, state = case
    f = Data(B * 1000 + L + K, dt)
    (xh, x), (wh, w), (dyh, dy) = f.make(B, D, L), f.make(D, K, scale=K ** -0.5), f.make(B, D, L)
    bh, bias = f.make(D, scale=0.3, dtype=torch.float32) if has_bias else (None, None)
    hh, h0 = f.make(B, D, K - 1) if state else (None, None)
    gh, dfs = f.make(B, D, K - 1) if state else (None, None)
    nh, n = f.lengths(B, L) if ragged else (None, None)
    (xv, _), (dyv, _) = view(poison(x, nh)), view(poison(dy, nh))
    want = ref.conv(xh, wh, bh, act, hh, nh, dyh, gh)
    (y, rest), fs = out_view((B, D, L), dt), torch.full((B, D, K - 1), float("nan"), dtype=TDT[dt], device=DEV)
    mc.causal_conv1d_fwd(xv, w, bias=bias, silu=act, initial_state=h0, lengths=n, y=y, final_state=fs)
    agree("y", y, want["y"], dt, case)
    assert np.array_equal(fs.double().cpu().numpy(), want["fs"][0])
    rest()
    (dx, rest), dh0 = out_view((B, D, L), dt), torch.full((B, D, K - 1), float("nan"), dtype=TDT[dt], device=DEV)
    first = None
    for workspace in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        ws = {} if workspace is None else {"workspace": torch.empty(16, dtype=torch.uint8, device=DEV)}
        _, dw, db = mc.causal_conv1d_bwd(xv, w, dyv, bias=bias, silu=act, initial_state=h0, lengths=n, d_final_state=dfs,
                                         dx=dx, d_initial_state=dh0, **ws)
        agree("dx", dx, want["dx"], dt, case)
        agree("dw", dw, want["dw"], "f32", case)
        agree("dh0", dh0, want["dh0"], dt, case)
        assert (db is None) == (bias is None)
        if db is not None:
            agree("db", db, want["db"], "f32", case)
        rest()
        if first is None:
            first = (dw.clone(), dx.clone())
    again = mc.causal_conv1d_bwd(xv, w, dyv, bias=bias, silu=act, initial_state=h0, lengths=n, d_final_state=dfs)
    assert torch.equal(again[1], first[0]) and torch.equal(again[0], first[1])     # bitwise repeatable


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 4, 8])
def test_convolution_step_continues_the_prompt(mc, dt, K):
    """Prompt, then tokens one by one: the same values as the whole sequence at once."""
    B, D, L, more = 3, 37, 5, 6
    f = Data(K, dt)
    (xh, x), (wh, w), (bh, bias) = f.make(B, D, L + more), f.make(D, K), f.make(D, dtype=torch.float32)
    want = ref.conv(xh, wh, bh, True)
    state = torch.full((B, D, K - 1), float("nan"), dtype=TDT[dt], device=DEV)
    mc.causal_conv1d_fwd(x[:, :, :L], w, bias=bias, silu=True, final_state=state)
    # a pool of states in another order, one unused row
    pool = torch.full((B + 2, D, K - 1), 5.0, dtype=TDT[dt], device=DEV)
    slots = torch.tensor([4, 0, 3, -1, 9], dtype=torch.int32, device=DEV)
    pool[slots[:B].long()] = state
    for t in range(L, L + more):
        col = (want["y"][0][:, :, t], want["y"][1][:, :, t])
        y = mc.causal_conv1d_step(x[:, :, t], state, w, bias=bias, silu=True)
        agree("y", y, col, dt, (K, t))
        xt = torch.cat([x[:, :, t], torch.full((2, D), float("nan"), dtype=TDT[dt], device=DEV)])
        yp = mc.causal_conv1d_step(xt, pool, w, bias=bias, silu=True, slots=slots)
        assert torch.equal(yp[:B], y) and not yp[B:].any()
    assert torch.equal(pool[slots[:B].long()], state)
    assert bool((pool[[1, 2]] == 5.0).all())
    assert np.array_equal(state.double().cpu().numpy(), xh[:, :, L + more - K + 1:])


# ------------------------------------------------------------------ selective scan

#        B  D   L     N   G  gate   softplus ragged state skip
SCAN = [(1, 1, 1, 1, 1, False, False, False, False, False),
        (2, 6, 1, 16, 2, True, True, False, True, True),
        (6, 4, 7, 5, 1, True, True, True, True, True),
        (2, 3, 8, 16, 3, False, True, False, False, True),
        (3, 18, 130, 16, 1, True, True, True, True, True),
        (5, 20, 511, 8, 2, True, True, True, False, False),
        (1, 5, 513, 16, 1, True, False, False, True, True),
        (2, 2, 1100, 17, 1, True, True, False, True, True),
        (6, 2, 1030, 33, 2, True, True, True, True, True),
        (1, 33, 70, 64, 1, False, True, False, True, True),
        (1, 2, 2600, 3, 1, True, True, False, True, True),
        (2, 3, 4400, 5, 1, True, True, True, True, True),          # few rows: the time axis split
        (3, 17, 3200, 16, 1, False, True, True, True, True),
        (2, 2110, 129, 5, 1, True, True, False, True, True),       # many rows: four per wave, several chunks
        (3, 1500, 260, 3, 2, True, True, True, True, True)]


def scan_data(case, dt):
    B, D, L, N, G, gate, sp, ragged, state, skip = case
    f = Data(D * 1000 + L + N, dt)
    h, d = {}, {}

    def put(name, *shape, **kw):
        h[name], d[name] = f.make(*shape, **kw)
    put("x", B, D, L)
    # steps of about 0.05 to 1, so that memories of all lengths occur
    put("delta", B, D, L, scale=0.8, shift=-1.0 if sp else 0.0)
    if not sp:
        h["delta"], d["delta"] = np.abs(h["delta"]) * 0.25, d["delta"].abs() * 0.25
    put("Bm", B, G, N, L)
    put("Cm", B, G, N, L)
    put("dy", B, D, L)
    if gate:
        put("z", B, D, L)
    put("A", D, N, dtype=torch.float32)
    h["A"], d["A"] = -np.exp(h["A"]).astype(np.float32).astype(np.float64), None
    d["A"] = torch.from_numpy(h["A"]).float().to(DEV)
    if skip:
        put("D", D, dtype=torch.float32)
    if sp:
        put("bias", D, dtype=torch.float32, scale=0.5)
    if state:
        put("h0", B, D, N, dtype=torch.float32)
        put("dfs", B, D, N, dtype=torch.float32)
    nh, n = f.lengths(B, L) if ragged else (None, None)
    return h, d, nh, n


def scan_reference(h, nh, sp):
    return ref.scan(h["x"], h["delta"], h["A"], h["Bm"], h["Cm"], h.get("D"), h.get("z"), h.get("bias"), sp,
                    h.get("h0"), nh, h["dy"], h.get("dfs"))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", SCAN, ids=lambda c: "-".join(map(str, c)))
def test_scan(mc, case, dt):
    B, D, L, N, G, gate, sp, ragged, state, skip = case
    h, d, nh, n = scan_data(case, dt)
    want = scan_reference(h, nh, sp)
    v = {k: view(poison(d[k], nh))[0] for k in ("x", "delta", "dy", "z") if k in d}
    # B and C as slices of one buffer with channels before and after
    bc = torch.cat([poison(d[k], nh).reshape(B, G * N, L) for k in ("Bm", "Cm")] + [d["x"][:, :1]], 1)
    Bm, Cm = bc[:, :G * N].unflatten(1, (G, N)), bc[:, G * N:2 * G * N].unflatten(1, (G, N))
    (y, rest), fs = out_view((B, D, L), dt), torch.full((B, D, N), float("nan"), device=DEV)
    states = mc.selective_scan_states(v["x"], d["A"])
    common = dict(D=d.get("D"), z=v.get("z"), delta_bias=d.get("bias"), softplus=sp, lengths=n)
    mc.selective_scan_fwd(v["x"], v["delta"], d["A"], Bm, Cm, initial_state=d.get("h0"), y=y, final_state=fs,
                          states=states, **common)
    agree("y", y, want["y"], dt, case)
    agree("fs", fs, want["fs"], "f32", case)
    rest()
    # without a workspace the time axis stays whole
    none = torch.empty(1, dtype=torch.uint8, device=DEV)
    states2, fs2 = torch.full_like(states, float("nan")), torch.full_like(fs, float("nan"))
    y2 = mc.selective_scan_fwd(v["x"], v["delta"], d["A"], Bm, Cm, initial_state=d.get("h0"), final_state=fs2,
                               states=states2, workspace=none, **common)
    agree("y whole", y2, want["y"], dt, case)
    agree("fs whole", fs2, want["fs"], "f32", case)
    assert bool(states.isfinite().all()) and bool(states2.isfinite().all())
    dh0 = torch.full((B, D, N), float("nan"), device=DEV)
    outs = {k: out_view((B, D, L), dt) for k in ("dx", "ddelta") + (("dz",) if gate else ())}
    args = (v["x"], v["delta"], d["A"], Bm, Cm, v["dy"], states)
    r = mc.selective_scan_bwd(*args, d_final_state=d.get("dfs"), d_initial_state=dh0,
                              **{k: o[0] for k, o in outs.items()}, **common)
    for name in ("dx", "ddelta", "dz", "dA", "dB", "dC", "dD", "ddelta_bias"):
        if r[name] is None:
            assert (name, {"dz": gate, "dD": skip, "ddelta_bias": sp}[name]) == (name, False)
            continue
        agree(name, r[name], want[name], dt if name in outs else "f32", case)
    agree("dh0", dh0, want["dh0"], "f32", case)
    for _, check in outs.values():
        check()
    again = mc.selective_scan_bwd(*args, d_final_state=d.get("dfs"), **common)
    for name, t in r.items():
        assert t is None or torch.equal(t, again[name]), name      # bitwise repeatable


# more than 16 states where the channels alone fill the card: one block of 16 after the other
# (few channels, in SCAN, take them side by side)
BLOCKS = [(5, 848, 9, 33, 1, True, True, True, True, True),
          (3, 1400, 131, 17, 1, False, True, True, False, True),
          (9, 470, 2, 64, 1, True, False, False, True, False),
          (1, 40, 1, 50, 2, True, True, False, True, True)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", BLOCKS, ids=lambda c: "-".join(map(str, c)))
def test_scan_of_many_states(mc, case, dt):
    test_scan(mc, case, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("N,G", [(1, 1), (5, 2), (16, 1), (64, 2)])
def test_scan_step_continues_the_prompt(mc, dt, N, G):
    B, D, L, more = 3, 34, 9, 4
    case = (B, D, L + more, N, G, True, True, False, True, True)
    h, d, _, _ = scan_data(case, dt)
    want = scan_reference(h, None, True)
    common = dict(D=d["D"], delta_bias=d["bias"], softplus=True)
    state = torch.full((B, D, N), float("nan"), device=DEV)
    mc.selective_scan_fwd(d["x"][..., :L], d["delta"][..., :L], d["A"], d["Bm"][..., :L], d["Cm"][..., :L],
                          z=d["z"][..., :L], initial_state=d["h0"], final_state=state, **common)
    pool = torch.full((B + 2, D, N), 5.0, device=DEV)
    slots = torch.tensor([4, 0, 3, -1, 9], dtype=torch.int32, device=DEV)
    pool[slots[:B].long()] = state
    pad = lambda t: torch.cat([t, torch.full((2,) + t.shape[1:], float("nan"), dtype=t.dtype, device=DEV)])  # noqa: E731
    for t in range(L, L + more):
        # slices along time: channels are L + more apart
        at = [d[k][..., t] for k in ("x", "delta", "Bm", "Cm", "z")]
        old = state.clone()
        out = torch.full_like(state, float("nan"))
        y = mc.selective_scan_step(at[0], at[1], d["A"], at[2], at[3], state, z=at[4], state_out=out, **common)
        assert torch.equal(state, old)
        y2 = mc.selective_scan_step(at[0], at[1], d["A"], at[2], at[3], state, z=at[4], **common)
        assert torch.equal(y, y2) and torch.equal(out, state)
        agree("y", y, tuple(q[..., t] for q in want["y"]), dt, (N, G, t))
        p = [pad(a) for a in at]
        yp = mc.selective_scan_step(p[0], p[1], d["A"], p[2], p[3], pool, z=p[4], slots=slots, **common)
        assert torch.equal(yp[:B], y) and not yp[B:].any()
    agree("state", state, want["fs"], "f32", (N, G))
    assert torch.equal(pool[slots[:B].long()], state) and bool((pool[[1, 2]] == 5.0).all())


def test_scan_values_at_the_ends(mc):
    """Step sizes from 0 to overflow, exponents that underflow, gates at +-90: finite where the definition
    is, and a NaN or infinity reaches its own row from its own step on only."""
    B, D, L, N = 1, 3, 40, 4
    x = torch.ones(B, D, L, device=DEV)
    delta = torch.linspace(-120, 60, L, device=DEV).repeat(B, D, 1).contiguous()
    z = torch.linspace(-90, 90, L, device=DEV).repeat(B, D, 1).contiguous()
    A = -torch.tensor([[1e-6, 1.0, 50.0, 3e4]] * D, device=DEV)
    Bm = torch.ones(B, 1, N, L, device=DEV)
    h = [t.double().cpu().numpy() for t in (x, delta, A, Bm, Bm)]
    want = ref.scan(*h, z=z.double().cpu().numpy())
    y = mc.selective_scan_fwd(x, delta, A, Bm, Bm, z=z, softplus=True)
    agree("y", y, want["y"], "f32", "ends")
    x[0, 1, 17], x[0, 2, 33] = float("nan"), float("inf")
    y2 = mc.selective_scan_fwd(x, delta, A, Bm, Bm, z=z, softplus=True)
    assert torch.equal(y2[0, 0], y[0, 0]) and torch.equal(y2[0, 1, :17], y[0, 1, :17])
    assert torch.equal(y2[0, 2, :33], y[0, 2, :33])
    assert bool(y2[0, 1, 17:].isnan().all()) and not bool(y2[0, 2, 33:].isfinite().any())


# ------------------------------------------------------------------ 8-bit products

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 3, 127, 128, 129, 1000, 2000, 4096, 5000, 9000])
def test_quantisation(mc, dt, C):
    f = Data(C, dt)
    T = 37
    xh, x = f.make(T, C)
    x[3] = 0
    x[5] *= 1e-30
    x[6, C // 2] = float("nan")
    x[7, C - 1] = float("-inf")
    # every multiple of half a step: 127 is the largest value, so the quotient is exact
    ties = torch.arange(-127, 128, dtype=torch.float32) / 2
    x[8] = 0
    x[8, :min(C, 255)] = ties[:min(C, 255)].to(x.dtype)
    x[8, 0] = 127.0
    if dt == "f32":
        x[9] *= 1e-41 if C > 1 else 1.0                          # below the normal numbers
    xh = x.double().cpu().numpy()
    q, s = mc.quantize_tokens(x)
    wq, ws = ref.quantize(xh)
    pad = -(-C // 128) * 128
    assert q.shape == (T, pad) and not q[:, C:].any()
    assert np.array_equal(q[:, :C].cpu().numpy(), wq)
    # one division, rounded once (a subnormal scale by an absolute half step)
    np.testing.assert_allclose(s.cpu().numpy().astype(np.float64), ws, rtol=2.0 ** -23, atol=2e-45, equal_nan=True)
    # channel-major and strided rows give the same bits
    for L, B in ((T, 1), (1, T)):
        xc = x.view(B, L, C).transpose(1, 2).contiguous()
        big = torch.full((B, C + 3, L + 5), 9.0, dtype=x.dtype, device=DEV)
        big[:, 1:C + 1, 2:L + 2] = xc
        q2, s2 = mc.quantize_tokens(big[:, 1:C + 1, 2:L + 2], channel_major=True)
        assert torch.equal(q2, q) and torch.equal(s2.isnan(), s.isnan())
        assert torch.equal(s2.nan_to_num(), s.nan_to_num())
    wide = torch.full((T, C + 7), 9.0, dtype=x.dtype, device=DEV)
    wide[:, 3:C + 3] = x
    q3, _ = mc.quantize_tokens(wide[:, 3:C + 3])
    assert torch.equal(q3, q)


#       B  L    O     K(padded)
I8 = [(1, 1, 1, 128), (1, 3, 17, 128), (2, 1, 64, 256), (1, 16, 128, 1024), (3, 5, 257, 640), (1, 33, 1000, 384),
      (2, 65, 130, 256), (1, 256, 512, 512), (3, 100, 300, 128), (1, 530, 515, 896), (7, 1, 4096, 4096),
      (1, 24, 40, 131072), (1, 130, 8200, 128), (1, 2050, 33, 256), (2, 50, 70, 8192), (1, 66, 200, 16512)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("case", I8, ids=lambda c: "-".join(map(str, c)))
def test_integer_product(mc, case, out):
    """The integer sum is exact, so the result is the definition's fp32 roundings, bit for bit."""
    B, L, O, K = case
    T = B * L
    gen = torch.Generator().manual_seed(T + O + K)
    q = torch.randint(-127, 128, (T, K), generator=gen, dtype=torch.int8)
    w = torch.randint(-127, 128, (O, K), generator=gen, dtype=torch.int8)
    q[0] = 127
    w[0] = -128                        # the largest sum: 127 * 128 * 131072 < 2^31
    qs, ws = torch.rand(T, generator=gen) * 0.1, torch.rand(O, generator=gen) * 0.1
    bias = torch.randn(O, generator=gen)
    total = torch.zeros(T, O, dtype=torch.float64)
    for k in range(0, K, 8192):
        total += q[:, k:k + 8192].double() @ w[:, k:k + 8192].double().t()
    assert float(total.abs().max()) < 2 ** 31
    plain = total.float() * qs[:, None] * ws
    d = [t.to(DEV) for t in (q, qs, w, ws, bias)]
    for b in (None, bias):
        want = (plain if b is None else plain + b).to(TDT[out])
        for cm in (False, True):
            shape = (B, O, L) if cm else (T, O)
            expect = want.view(B, L, O).transpose(1, 2).contiguous() if cm else want
            for ws_bytes in (None, 16):
                y = torch.full(shape, float("nan"), dtype=TDT[out], device=DEV)
                work = {} if ws_bytes is None else {"workspace": torch.empty(16, dtype=torch.uint8, device=DEV)}
                mc.matmul_i8(d[0], d[1], d[2], d[3], bias=None if b is None else d[4], length=L if cm else None, y=y, **work)
                # the bias may be added in one rounding with the scale
                got, ex = y.cpu().double(), expect.double()
                step = (2.0 ** -23 if out == "f32" else 2.0 ** -7) * ex.abs() + (0 if b is None else 2.0 ** -23) * plain.abs().double().max()
                assert bool(((got - ex).abs() <= (0 if b is None else step)).all()), (case, cm, ws_bytes)


def test_integer_product_of_a_token_with_nan(mc):
    x = torch.ones(4, 128, device=DEV)
    x[2, 5] = float("inf")
    q, s = mc.quantize_tokens(x)
    w = torch.ones(20, 128, dtype=torch.int8, device=DEV)
    y = mc.matmul_i8(q, s, w, torch.ones(20, device=DEV))
    assert bool(y[2].isnan().all()) and bool(y[[0, 1, 3]].isfinite().all())


# ------------------------------------------------------------------ streams, graphs, far offsets

def test_other_stream_and_graph_replays(mc):
    """A layer's step recorded into a graph and replayed between eager calls gives the eager results."""
    B, D, L, N = 2, 40, 70, 16
    f = Data(11, "bf16")
    x, dl, z, dy = (f.make(B, D, L)[1] for _ in range(4))
    Bm, Cm = (f.make(B, 1, N, L)[1] for _ in range(2))
    w, bias = f.make(D, 4)[1], f.make(D, dtype=torch.float32)[1]
    A = -torch.rand(D, N, device=DEV) - 0.1
    wq, ws = mc.quantize_tokens(f.make(D, D)[1])

    def layer():
        u = mc.causal_conv1d_fwd(x, w, bias=bias, silu=True)
        states = mc.selective_scan_states(u, A)
        y = mc.selective_scan_fwd(u, dl, A, Bm, Cm, z=z, softplus=True, states=states)
        g = mc.selective_scan_bwd(u, dl, A, Bm, Cm, dy, states, z=z, softplus=True)
        dx, dw, db = mc.causal_conv1d_bwd(x, w, g["dx"], bias=bias, silu=True)
        q, s = mc.quantize_tokens(y, channel_major=True)
        return [y, dx, dw, db, g["dA"], g["dB"], g["dC"], mc.matmul_i8(q, s, wq, ws)]
    eager = [t.clone() for t in layer()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer()
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    explicit = mc.causal_conv1d_fwd(x, w, bias=bias, silu=True, stream=side)
    side.synchronize()
    assert torch.equal(explicit, mc.causal_conv1d_fwd(x, w, bias=bias, silu=True))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for i in range(4):
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, held):
            assert torch.equal(a, b), i
        x.mul_(1.25)                   # new inputs between the replays
        eager = [t.clone() for t in layer()]


def test_large_outputs(mc):
    """Outputs large enough to be written past the caches: bit for bit those of two halves that are not."""
    f = Data(9, "bf16")
    x = torch.randn(2, 1024, 32769, device=DEV).bfloat16()            # 128 MB and odd rows
    w, bias = f.make(1024, 4)[1], f.make(1024, dtype=torch.float32)[1]
    y = mc.causal_conv1d_fwd(x, w, bias=bias, silu=True)
    for i in range(2):
        assert torch.equal(y[i:i + 1], mc.causal_conv1d_fwd(x[i:i + 1], w, bias=bias, silu=True))
    B, D, N = 66, 4096, 16                                             # 17 MB of states
    x, dl, z = (torch.randn(B, D, device=DEV).bfloat16() for _ in range(3))
    Bm, Cm = (torch.randn(B, 1, N, device=DEV).bfloat16() for _ in range(2))
    A, state = -torch.rand(D, N, device=DEV), torch.randn(B, D, N, device=DEV)
    out = torch.empty_like(state)
    y = mc.selective_scan_step(x, dl, A, Bm, Cm, state, z=z, softplus=True, state_out=out)
    for i in (slice(0, 33), slice(33, 66)):
        part = state[i].clone()
        assert torch.equal(y[i], mc.selective_scan_step(x[i], dl[i], A, Bm[i], Cm[i], part, z=z[i], softplus=True))
        assert torch.equal(part, out[i])
    gen = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randint(-127, 128, (8195, 128), generator=gen, device=DEV, dtype=torch.int8)
    wq = torch.randint(-127, 128, (8203, 128), generator=gen, device=DEV, dtype=torch.int8)
    s, ws = torch.rand(8195, device=DEV), torch.rand(8203, device=DEV)
    y = mc.matmul_i8(q, s, wq, ws, out_dtype=torch.bfloat16)          # 134 MB
    for i in (slice(0, 4000), slice(4000, 8195)):
        assert torch.equal(y[i], mc.matmul_i8(q[i], s[i], wq, ws, out_dtype=torch.bfloat16))


def test_offsets_past_32_bits(mc):
    """Rows of one buffer more than 2^31 elements apart."""
    D, L, N = 3, 20, 4
    far = (1 << 31) + 24
    buf = torch.zeros(far + 4096, dtype=torch.bfloat16, device=DEV)
    f = Data(5, "bf16")
    xh, x = f.make(2, D, L)
    v = buf.as_strided((2, D, L), (far, L, 1), 8)
    v.copy_(x)
    out = buf.as_strided((2, D, L), (far, L, 1), 1024)
    w, bias = f.make(D, 4)[1], f.make(D, dtype=torch.float32)[1]
    mc.causal_conv1d_fwd(v, w, bias=bias, silu=True, y=out)
    assert torch.equal(out, mc.causal_conv1d_fwd(x, w, bias=bias, silu=True))
    A, Bm = -torch.rand(D, N, device=DEV), f.make(2, 1, N, L)[1]
    out.zero_()
    states = mc.selective_scan_states(x, A)
    mc.selective_scan_fwd(v, v, A, Bm, Bm, z=v, softplus=True, y=out, states=states)
    assert torch.equal(out, mc.selective_scan_fwd(x, x, A, Bm, Bm, z=x, softplus=True))
    a = mc.selective_scan_bwd(v, v, A, Bm, Bm, v, states, z=v, softplus=True, dx=out)
    b = mc.selective_scan_bwd(x, x, A, Bm, Bm, x, states, z=x, softplus=True)
    for k in b:
        assert b[k] is None or torch.equal(a[k], b[k]), k
    q, s = mc.quantize_tokens(v, channel_major=True)
    q2, s2 = mc.quantize_tokens(x, channel_major=True)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_binding_refusals_on_the_device(mc):
    x, w = torch.zeros(2, 6, 40, device=DEV), torch.zeros(6, 4, device=DEV)
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(x.transpose(1, 2), w)                     # wrong channel count
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(torch.zeros(2, 40, 6, device=DEV).transpose(1, 2), w)   # time not contiguous
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(x, w.bfloat16())
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(x.half(), w.half())
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(x, w, y=x)                                # in place
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(x, w, lengths=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        mc.causal_conv1d_fwd(x, torch.zeros(6, 9, device=DEV))
    A, Bm = torch.zeros(6, 4, device=DEV), torch.zeros(2, 1, 4, 40, device=DEV)
    with pytest.raises(ValueError):
        mc.selective_scan_fwd(x, x, A, Bm, Bm[..., :39])
    with pytest.raises(ValueError):
        mc.selective_scan_fwd(x, x, torch.zeros(6, 65, device=DEV), torch.zeros(2, 1, 65, 40, device=DEV),
                              torch.zeros(2, 1, 65, 40, device=DEV))
    with pytest.raises(ValueError):
        mc.selective_scan_bwd(x, x, A, Bm, Bm, x, torch.zeros(3, device=DEV))
    with pytest.raises(ValueError):
        mc.selective_scan_step(x[..., 0], x[..., 0], A, Bm[..., 0], Bm[..., 0], torch.zeros(3, 6, 4, device=DEV))
    q = torch.zeros(4, 128, dtype=torch.int8, device=DEV)
    s = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError):
        mc.matmul_i8(q, s, q[:, :64].contiguous(), s)
    with pytest.raises(ValueError):
        mc.matmul_i8(q, s, q, s, length=3)
