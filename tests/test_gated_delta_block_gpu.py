"""The gated delta block (gated_delta.py): prompts and tokens agree with each other and with the block computed in 64
bits, training gradients with automatic differentiation of the 64-bit form.

Tolerances, relative in the 2-norm.  Training: a bf16 rounding is off by at most 2^-8 of the value; the chains have at
most 12 of them in sequence (six forward, six backward), 0.047 in the worst case, so 2^-4.  Serving, of what the
block adds to h: an e4m3 value is off by half a step, 2^-4 of it at the most and 0.026 in the mean square; queries,
keys, values and gates each carry two such roundings, the output two more, ten independent ones in all: 0.082, so 2^-3.
That is a mean square over many values: a token whose queries and keys happen to be near orthogonal has a small y, larger
errors relative to it, and a normalised y all the same, so the norms are those of all tokens together.
"""
import pytest
import torch

import delta_reference as ref

pytestmark = pytest.mark.gpu

TOL, TOL_SERVING = 2.0 ** -4, 2.0 ** -3
NAMES = ("w_in", "w_out", "w_conv", "b_conv", "w_norm", "b_norm", "w_mix", "decay", "a0")


@pytest.fixture(scope="module")
def block():
    from convolution_implicit_gemm_nchw_amd.gated_delta import GatedDeltaBlock
    return GatedDeltaBlock(M=96, Hk=2, Hv=4, P=32, V=24, K=4, seed=3)


def norm(x, w, b=0.0):
    d = x - x.mean(1, keepdim=True)
    return d * torch.rsqrt((d * d).mean(1, keepdim=True) + 1e-5) * w[:, None] + (b if isinstance(b, float) else b[:, None])


def plain(p, h, parts, Hk):
    """The block in 64 bits on the CPU, h [B, M, L] -> [B, M, L]."""
    B, _, L = h.shape
    Hv, K, D = p["decay"].shape[0], p["w_conv"].shape[1], p["w_conv"].shape[0]
    xab = p["w_in"] @ norm(h, p["w_norm"], p["b_norm"])
    x, a, b = xab[:, :D], xab[:, D:D + Hv], xab[:, D + Hv:]
    full = torch.cat([x.new_zeros(B, D, K - 1), x], 2)
    u = torch.nn.functional.silu((full.unfold(2, K, 1) * p["w_conv"][:, None]).sum(3) + p["b_conv"][:, None])
    g = -torch.exp(p["decay"])[:, None] * torch.nn.functional.softplus(a + p["a0"][:, None])
    y, _ = ref.rule(*(t.contiguous() for t in u.split(parts, 1)), g, torch.sigmoid(b), Hk, l2norm=True)
    return h + p["w_out"] @ norm(y, p["w_mix"])


def params(b):
    return {n: getattr(b, n).double().cpu().requires_grad_() for n in NAMES}


def rel(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    return float((got - want).norm() / want.norm())


def test_training_gradients(block):
    gen = torch.Generator().manual_seed(0)
    h = torch.randn(3, 96, 70, generator=gen).to(torch.bfloat16)
    dout = torch.randn(3, 96, 70, generator=gen).to(torch.bfloat16)
    out, grads = block.train_step(h.cuda(), dout.cuda())
    p = params(block)
    hd = h.double().requires_grad_()
    want = plain(p, hd, block.parts, block.Hk)
    want.backward(dout.double())
    assert rel(out, want.detach()) < TOL
    assert sorted(grads) == sorted(NAMES + ("h",))
    for name, g in grads.items():
        w = hd.grad if name == "h" else p[name].grad
        e = rel(g, w)
        print(name, e, flush=True)
        assert g.shape == w.shape and e < TOL, (name, e)


def test_prompt_then_tokens(block):
    gen = torch.Generator().manual_seed(1)
    B, L, more = 3, 70, 5
    h = torch.randn(B, L + more, 96, generator=gen).to(torch.bfloat16).cuda()
    with torch.no_grad():
        want = plain(params(block), h.double().cpu().transpose(1, 2), block.parts, block.Hk).transpose(1, 2)
    want = want - h.double().cpu()
    lengths = torch.tensor([L, 0, 17], dtype=torch.int32, device="cuda")
    states = block.states(B)
    padded = h[:, :L].clone()
    for b, n in enumerate(lengths.tolist()):
        padded[b, n:] = float("nan")
    out = block.prompt(padded, states, lengths)
    for b, n in enumerate(lengths.tolist()):
        if n:
            e = rel(out[b, :n].double() - h[b, :n].double(), want[b, :n])
            print("prompt", b, e, flush=True)
            assert e < TOL_SERVING
    # the tokens that follow each prompt, one at a time, the states in a pool
    pool = [torch.zeros((B + 1,) + s.shape[1:], dtype=s.dtype, device="cuda") for s in states]
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    for p, s in zip(pool, states):
        p[slots.long()] = s
    have, truth = [], []
    for k in range(more):
        x = torch.stack([h[b, n + k] for b, n in enumerate(lengths.tolist())])
        y, y2 = block.token(x, states), block.token(x, pool, slots=slots)
        assert torch.equal(y, y2)
        for b, n in enumerate(lengths.tolist()):
            have.append(y[b].double() - x[b].double())
            truth.append(want[b, n + k])
            print("token", b, k, rel(have[-1], truth[-1]), flush=True)
    assert rel(torch.stack(have), torch.stack(truth)) < TOL_SERVING


def test_tokens_from_a_graph(block):
    """A captured token step, replayed: the eager steps' outputs and states."""
    gen = torch.Generator().manual_seed(2)
    hs = torch.randn(4, 3, 96, generator=gen).to(torch.bfloat16).cuda()
    eager, held = block.states(3), block.states(3)
    x = hs[0].clone()
    block.token(x, block.states(3))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.token(x, held)
    for s in held:
        s.zero_()
    for h in hs:
        x.copy_(h)
        graph.replay()
        want = block.token(h, eager)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip(held, eager))
