"""GPU parity of the gated delta rule against the plain 64-bit form (delta_reference.py), element by element, with the
bounds derived there.  Activations are views into larger buffers whose other elements must stay untouched; outputs are
pre-filled with NaN; what lies past a sequence's length is poisoned with NaN and infinities.
"""
import pytest
import torch

import delta_reference as ref
import test_state_space_gpu as base

pytestmark = pytest.mark.gpu
mc = base.mc
DEV, TDT = base.DEV, base.TDT
INF = float("inf")

#         B  Hk Hv  P    V   L
SIZES = [(1, 1, 1, 1, 1, 1),
         (2, 1, 3, 5, 7, 3),
         (3, 2, 2, 64, 16, 63),
         (5, 2, 4, 33, 20, 64),
         (2, 1, 2, 65, 33, 65),
         (5, 1, 1, 128, 32, 130),
         (1, 3, 6, 96, 48, 200),
         (5, 1, 2, 129, 17, 70),
         (1, 1, 1, 256, 512, 66),
         (2, 2, 2, 200, 130, 129)]


class Case:
    """Seeded operands of one problem: host values in 64 bits (already rounded) and device views."""

    def __init__(self, B, Hk, Hv, P, V, L, dt, seed, l2norm, ragged, state):
        f = base.Data(seed, dt)
        self.size, self.dt, self.l2norm, self.Hk = (B, Hk, Hv, P, V, L), dt, l2norm, Hk
        self.host, self.dev, self.checks = {}, {}, []
        n = f.lengths(B, L) if ragged else (None, None)
        self.lengths = n
        # without normalisation inside, keys of about length one: the rule itself grows without bound otherwise
        for name, rows, scale in (("q", Hk * P, 1.0), ("k", Hk * P, 1.0 if l2norm else 0.9 * P ** -0.5), ("v", Hv * V, 1.0),
                                  ("dy", Hv * V, 1.0)):
            self.put(name, f.make(B, rows, L, scale=scale))
        decay = -torch.rand(B, Hv, L, generator=f.gen).exp2() * torch.rand(B, Hv, 1, generator=f.gen)
        beta = torch.sigmoid(torch.randn(B, Hv, L, generator=f.gen))
        beta[..., ::5] = 0.0                                     # what is not written, and what is written whole
        beta[..., 2::7] = 1.0
        decay[..., 4::9] = 0.0
        if L > 20:
            decay[:, 0, 11], decay[:, 0, 17] = -INF, -300.0      # forgets all
        self.put("g", (decay.double().numpy(), decay.to(DEV)))
        self.put("beta", (beta.double().numpy(), beta.to(DEV)))
        shape = (B, Hv, P, V)
        self.s0 = f.make(*shape, scale=0.3, dtype=torch.float32) if state else (None, None)
        self.ds = f.make(*shape, dtype=torch.float32) if state else (None, None)

    def put(self, name, pair):
        self.host[name] = torch.from_numpy(pair[0]).double()
        self.dev[name], check = base.view(base.poison(pair[1], self.lengths[0]))
        self.checks.append(check)

    def untouched(self):
        for c in self.checks:
            c()

    def kw(self):
        return dict(key_heads=self.Hk, l2norm=self.l2norm, lengths=self.lengths[1])

    def operands(self):
        return [self.dev[k] for k in ("q", "k", "v", "g", "beta")]

    def expect(self):
        """{name: value} in 64 bits."""
        leaves = {k: self.host[k].clone().requires_grad_() for k in ("q", "k", "v", "g", "beta")}
        s0 = None if self.s0[0] is None else torch.from_numpy(self.s0[0]).double().requires_grad_()
        seen = []
        y, s = ref.rule(*leaves.values(), self.Hk, l2norm=self.l2norm, state=s0, lengths=self.lengths[0], seen=seen)
        loss = (y * self.host["dy"]).sum()
        if s0 is not None:
            loss = loss + (s * torch.from_numpy(self.ds[0]).double()).sum()
        if loss.requires_grad:
            loss.backward()
        r = {"y": y.detach(), "s": s.detach()}
        for k, t in leaves.items():
            r["d" + k] = torch.zeros_like(t) if t.grad is None else t.grad
        if s0 is not None:
            r["ds0"] = s0.grad
        # through x / |x| a gradient d becomes (d - n (n d)) / |x|, a difference of terms of the size of d / |x|
        self.terms = {name: float((x.grad / size.detach()).abs().max()) for name, (x, size) in zip(("dq", "dk"), seen)
                      if x.grad is not None}
        return r


def run(mc, c, limit=None):
    """{name: tensor} of both passes; limit: the workspace's size, 0 the least."""
    B, Hk, Hv, P, V, L = c.size
    ws = [None, None]
    if limit is not None:
        for i in range(2):
            n = mc.gated_delta_workspace(*c.size, dtype=mc.BF16 if c.dt == "bf16" else mc.F32, backward=bool(i), limit=limit)
            ws[i] = torch.full((n + 64,), 0xff, dtype=torch.uint8, device=DEV)
            c.checks.append(lambda t=ws[i], n=n: None if bool((t[n:] == 0xff).all()) else pytest.fail("past the workspace"))
            ws[i] = ws[i][:n]
    r = {"s": torch.full((B, Hv, P, V), float("nan"), device=DEV)}
    r["y"], check = base.out_view((B, Hv * V, L), c.dt)
    c.checks.append(check)
    states = mc.gated_delta_states(c.dev["q"], c.dev["v"], c.dev["g"], key_heads=Hk)
    states.fill_(float("nan"))
    mc.gated_delta_fwd(*c.operands(), initial_state=c.s0[1], y=r["y"], final_state=r["s"], states=states, workspace=ws[0],
                       **c.kw())
    grads = {}
    for name, rows in (("dq", Hk * P), ("dk", Hk * P), ("dv", Hv * V)):
        grads[name], check = base.out_view((B, rows, L), c.dt)
        c.checks.append(check)
    if c.ds[1] is not None:
        r["ds0"] = torch.full_like(r["s"], float("nan"))
    r.update(mc.gated_delta_bwd(*c.operands(), c.dev["dy"], states, d_final_state=c.ds[1], d_initial_state=r.get("ds0"),
                                workspace=ws[1], **grads, **c.kw()))
    return r


def agree(name, got, want, absolute, relative, scale=0.0):
    got = got.double().cpu()
    assert got.shape == want.shape
    top = max(float(want.abs().max()), scale)
    bound = absolute * top + relative * want.abs() + 1e-37
    worst = float(((got - want).abs() / bound).nan_to_num(INF, INF, INF).max())
    print(f"  {name}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, (name, worst)


def compare(c, got):
    B, Hk, Hv, P, V, L = c.size
    want = c.expect()
    # d g is a difference of what flows in and out of the states: against the largest of those
    h = c.host
    flow = float((want["dq"] * h["q"]).view(B, Hk, P, L).sum(2).abs().max() + (want["dk"] * h["k"]).view(B, Hk, P, L).sum(2).abs().max())
    if c.s0[0] is not None:
        flow += float((torch.from_numpy(c.ds[0]).double() * want["s"]).sum((2, 3)).abs().max())
    for name, v in got.items():
        passes = 1 if name in ("y", "s") else 2
        stored = c.dt if name in ("y", "dq", "dk", "dv") else "f32"
        a, r = ref.rule_bound(P, L, stored if name == "y" else "f32", passes)
        agree(name, v, want[name], a, ref.HALF[stored], flow if name == "dg" else c.terms.get(name, 0.0))
        if c.lengths[0] is not None and name not in ("s", "ds0"):
            for b, n in enumerate(c.lengths[0]):
                assert not v[b, :, max(0, min(int(n), L)):].any(), (name, "padding")
    c.untouched()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("l2norm,ragged,state", [(True, True, True), (False, False, False), (True, False, False),
                                                 (False, True, True)])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(map(str, s)))
def test_passes(mc, size, l2norm, ragged, state, dt):
    c = Case(*size, dt, 1, l2norm, ragged, state)
    compare(c, run(mc, c))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(5, 1, 2, 40, 20, 300), (3, 2, 4, 130, 33, 150), (2, 1, 1, 128, 64, 260)],
                         ids=lambda s: "-".join(map(str, s)))
def test_slices_under_a_small_workspace(mc, size, dt):
    """The least workspace takes one sequence and chunk at a time, larger ones several: the same bits."""
    c = Case(*size, dt, 2, True, True, True)
    whole = run(mc, c)
    compare(c, whole)
    B, Hk, Hv, P, V, L = size
    code = mc.BF16 if dt == "bf16" else mc.F32
    most = mc.gated_delta_workspace(*size, dtype=code)
    forms = set()
    for limit in (0, most // 9, most // 3, most - 1):
        forms.add(mc.gated_delta_describe(*size, dtype=code, workspace_bytes=max(
            limit, mc.gated_delta_workspace(*size, dtype=code, limit=limit))).split()[1])
        part = run(mc, c, limit)
        for k in whole:
            assert torch.equal(part[k], whole[k]), (k, limit)
        c.untouched()
    assert len(forms) >= 2 and "slice=1x1" in forms


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("l2norm", [False, True])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1), (3, 2, 4, 5, 7), (4, 1, 2, 64, 64), (2, 2, 2, 100, 70), (3, 1, 3, 256, 512),
                                  (65, 4, 4, 128, 128)], ids=lambda s: "-".join(map(str, s)))
def test_step(mc, size, l2norm, dt):
    """One token: a step's states written elsewhere, in place, and in a pool with unused rows."""
    B, Hk, Hv, P, V = size
    f = base.Data(3, dt)
    host, dev = {}, {}
    for name, rows, scale in (("q", Hk * P, 1.0), ("k", Hk * P, 1.0 if l2norm else 0.9 * P ** -0.5), ("v", Hv * V, 1.0)):
        h, t = f.make(B, rows + 3, scale=scale)
        host[name], dev[name] = torch.from_numpy(h)[:, 2:-1].double(), t[:, 2:-1]
    g, beta = -torch.rand(B, Hv, generator=f.gen), torch.rand(B, Hv, generator=f.gen)
    g[0, 0] = -INF
    s0 = f.make(B, Hv, P, V, scale=0.3, dtype=torch.float32)
    want_y, want_s = ref.rule(*(host[k][..., None] for k in "qkv"), g.double()[..., None], beta.double()[..., None], Hk,
                              l2norm=l2norm, state=torch.from_numpy(s0[0]).double())
    args = [dev["q"], dev["k"], dev["v"], g.to(DEV), beta.to(DEV)]
    out = torch.full_like(s0[1], float("nan"))
    y = mc.gated_delta_step(*args, s0[1], key_heads=Hk, l2norm=l2norm, state_out=out)
    # sums of P terms, three times, none of them in 16 bits
    a = (3 * P + 16) * ref.U
    agree("y", y, want_y[..., 0], a, ref.HALF[dt])
    agree("state", out, want_s, a, ref.HALF["f32"])
    place = s0[1].clone()
    assert torch.equal(mc.gated_delta_step(*args, place, key_heads=Hk, l2norm=l2norm), y) and torch.equal(place, out)
    if B < 3:
        return
    pool = torch.full((B + 2, Hv, P, V), 7.0, device=DEV)
    slots = torch.arange(B, dtype=torch.int32) + 2
    slots[1] = -1
    slots[2] = B + 2
    for b in range(B):
        if 0 <= slots[b] < B + 2:
            pool[int(slots[b])] = s0[1][b]
    yp = mc.gated_delta_step(*args, pool, key_heads=Hk, l2norm=l2norm, slots=slots.to(DEV))
    used = [b for b in range(B) if b not in (1, 2)]
    assert not yp[[1, 2]].any() and torch.equal(yp[used], y[used])
    assert torch.equal(pool[slots[used].long().to(DEV)], out[used])
    rest = [s for s in range(B + 2) if s not in slots[used].tolist()]
    assert bool((pool[rest] == 7.0).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_prompt_then_steps(mc, dt):
    """A prompt in two parts and then token by token: the whole prompt's outputs and state."""
    size = (2, 2, 4, 48, 40, 101)
    c = Case(*size, dt, 4, True, False, True)
    B, Hk, Hv, P, V, L = size
    want = c.expect()
    ops, s, ys = c.operands(), c.s0[1], []
    for lo, hi in ((0, 70), (70, 97)):
        nxt = torch.empty_like(s)
        ys.append(mc.gated_delta_fwd(*(x[..., lo:hi] for x in ops), key_heads=Hk, l2norm=True, initial_state=s, final_state=nxt))
        s = nxt
    for t in range(97, L):
        ys.append(mc.gated_delta_step(*(x[..., t] for x in ops), s, key_heads=Hk, l2norm=True)[..., None])
    a, _ = ref.rule_bound(P, L, dt)
    a += (L - 97) * (3 * P + 16) * ref.U
    agree("y", torch.cat(ys, 2), want["y"], a, ref.HALF[dt])
    agree("state", s, want["s"], ref.rule_bound(P, L, "f32")[0] + (L - 97) * (3 * P + 16) * ref.U, ref.HALF["f32"])


def test_gradients_against_differences(mc):
    """The kernels' gradients, in a random direction, against central differences of the 64-bit forward pass: off by
    the kernels' bound on each part, and 1e-6 for the difference."""
    size = (2, 1, 2, 20, 18, 90)
    c = Case(*size, "f32", 5, True, False, True)
    c.host["g"] = c.host["g"].clamp(min=-3.0)
    c.dev["g"].copy_(c.host["g"].float())
    got = run(mc, c)
    gen = torch.Generator().manual_seed(9)
    names = ("q", "k", "v", "g", "beta")
    x = {k: c.host[k] for k in names}
    x["g"] = c.dev["g"].double().cpu()
    x["s0"] = torch.from_numpy(c.s0[0]).double()
    dirs = {k: torch.randn(v.shape, generator=gen, dtype=torch.float64) for k, v in x.items()}

    def loss(step):
        a = {k: v + step * dirs[k] for k, v in x.items()}
        y, s = ref.rule(*(a[k] for k in names), c.Hk, l2norm=True, state=a["s0"])
        return float((y * c.host["dy"]).sum() + (s * torch.from_numpy(c.ds[0]).double()).sum())
    h = 1e-5
    want = (loss(h) - loss(-h)) / (2 * h)
    have, room = 0.0, 1e-6 * abs(want)
    a, _ = ref.rule_bound(20, 90, "f32", 2)
    for k in x:
        d = got["d" + k].double().cpu()
        have += float((d * dirs[k]).sum())
        room += a * float(d.abs().max()) * float(dirs[k].norm()) * 4      # errors of either sign add up as lengths do
    print(have, want, room)
    assert abs(have - want) <= room


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_what_is_not_finite_stays(mc, dt):
    """NaN and infinities of one value channel, head or sequence leave the others' bits as they are."""
    size = (2, 2, 4, 40, 50, 100)
    c = Case(*size, dt, 6, True, True, True)
    c.lengths = (None, torch.tensor([100, 40], dtype=torch.int32, device=DEV))
    c.dev = {k: v.nan_to_num(0.0, 0.0, -5.0).contiguous() for k, v in c.dev.items()}
    c.checks = []
    clean = run(mc, c)
    c.dev["v"][0, 3, 20] = INF                                   # channel 3 of head 0
    c.s0[1][0, 2, :, 7] = float("nan")                           # channel 7 of head 2
    c.dev["q"][1, 45, 10] = float("nan")                         # the second key head of sequence 1: value heads 2 and 3
    r = run(mc, c)
    keep = [i for i in range(200) if i not in (3, 107)]
    assert torch.equal(r["y"][0, keep], clean["y"][0, keep])
    assert torch.equal(r["y"][1, :100], clean["y"][1, :100])
    assert torch.equal(r["s"][1], clean["s"][1])                 # no state depends on a query
    assert not bool(r["y"][0, 3, 20:].isfinite().any()) and not bool(r["y"][0, 107].isfinite().any())
    for k in ("y", "dq", "dk", "dv", "dg", "dbeta"):
        assert not r[k][1, :, 40:].any(), k
    for k in ("dq", "dk"):
        assert torch.equal(r[k][1, :40], clean[k][1, :40]), k


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_repeats_streams_and_graphs(mc, dt):
    """The same bits twice, on another stream, and from a graph replayed among eager work."""
    size = (3, 2, 4, 70, 40, 150)
    c = Case(*size, dt, 7, True, True, True)
    first, again = run(mc, c), run(mc, c)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        third = run(mc, c)
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], again[k]) and torch.equal(first[k], third[k]), k
    states = mc.gated_delta_states(c.dev["q"], c.dev["v"], c.dev["g"], key_heads=c.Hk)
    s, ds0 = torch.empty_like(c.s0[1]), torch.empty_like(c.s0[1])
    token = [x[..., 0] for x in c.operands()]

    def work():
        y = mc.gated_delta_fwd(*c.operands(), initial_state=c.s0[1], final_state=s, states=states, **c.kw())
        g = mc.gated_delta_bwd(*c.operands(), c.dev["dy"], states, d_final_state=c.ds[1], d_initial_state=ds0, **c.kw())
        t = mc.gated_delta_step(*token, c.s0[1], key_heads=c.Hk, l2norm=True, state_out=torch.empty_like(s))
        return {"y": y, "s": s, "ds0": ds0, **g, "t": t}
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(3):
        for x in ("v", "dy"):
            c.dev[x].mul_(-0.5)
        c.s0[1].mul_(0.5)
        graph.replay()
        got = {k: v.clone() for k, v in held.items()}
        want = {k: v.clone() for k, v in work().items()}
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k].nan_to_num(), want[k].nan_to_num()), (k, i)


def test_growing_decays(mc):
    """Log decays a little above zero: what the state holds grows, by e^0.03 a step here, and the errors with it."""
    size = (1, 1, 2, 32, 16, 70)
    c = Case(*size, "f32", 8, True, False, False)
    g = torch.full((1, 2, 70), 0.03)
    c.host["g"] = g.double()
    c.dev["g"].copy_(g)
    want, got = c.expect(), run(mc, c)
    a, _ = ref.rule_bound(32, 70, "f32", 2)
    for k in ("y", "s", "dq", "dk", "dv", "dbeta"):
        agree(k, got[k], want[k], a * 9, ref.HALF["f32"])        # e^(0.03 * 70) = 8.2


def test_far_offsets(mc):
    """Rows of a batch whose offsets pass 2^32 bytes and 2^31 elements."""
    B, P, V, L = 2, 16, 16, 70
    far = (1 << 31) + 64
    buf = torch.empty(far + (2 * P + V) * L, dtype=torch.bfloat16, device=DEV)
    qkv = torch.as_strided(buf, (B, 2 * P + V, L), (far, L, 1))
    gen = torch.Generator().manual_seed(10)
    x = torch.randn(B, 2 * P + V, L, generator=gen).to(torch.bfloat16)
    qkv.copy_(x)
    g, beta = -torch.rand(B, 1, L, generator=gen), torch.rand(B, 1, L, generator=gen)
    got = mc.gated_delta_fwd(qkv[:, :P], qkv[:, P:2 * P], qkv[:, 2 * P:], g.to(DEV), beta.to(DEV), l2norm=True)
    x = x.to(DEV)
    want = mc.gated_delta_fwd(x[:, :P], x[:, P:2 * P], x[:, 2 * P:], g.to(DEV), beta.to(DEV), l2norm=True)
    assert torch.equal(got, want)
