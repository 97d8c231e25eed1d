"""The state-space block (state_space.py): prompts and tokens agree with each other and with the block
computed in 64 bits, training gradients with automatic differentiation of the 64-bit form.

Tolerances, relative in the 2-norm.  Training: a bf16 rounding is off by at most 2^-8 of the value; the
chains have at most 8 of them in sequence, 2^-5 in the worst case.  Serving: a value held in 8 bits is
off by max / 440 rms (a uniform error over a step of max / 127), and the largest of 96 normal values is
about 2.5 times their size: 0.6 % for each of the four quantised operands of the two products, at most
doubled where x and z meet in the gated product: 4.8 % if all add up, so 2^-4.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TOL, TOL_SERVING = 2.0 ** -5, 2.0 ** -4


@pytest.fixture(scope="module")
def block():
    from convolution_implicit_gemm_nchw_amd.state_space import StateSpaceBlock
    return StateSpaceBlock(M=96, D=136, N=16, K=4, R=8, seed=3)


def plain(p, h):
    """The block in 64 bits on the CPU, h [B, M, L] -> [B, M, L]."""
    B, _, L = h.shape
    D, N, K = p["A"].shape[0], p["A"].shape[1], p["w_conv"].shape[1]
    xz = p["w_in"] @ h
    x, z = xz[:, :D], xz[:, D:]
    full = torch.cat([x.new_zeros(B, D, K - 1), x], 2)
    u = torch.nn.functional.silu((full.unfold(2, K, 1) * p["w_conv"][:, None]).sum(3) + p["b_conv"][:, None])
    dt = torch.nn.functional.softplus(p["w_dt"] @ (p["w_r"] @ u) + p["b_dt"][:, None])
    bc = p["w_bc"] @ u
    hs, ys = h.new_zeros(B, D, N), []
    for t in range(L):
        hs = torch.exp(dt[:, :, t, None] * p["A"]) * hs + (dt * u)[:, :, t, None] * bc[:, None, :N, t]
        ys.append((hs * bc[:, None, N:, t]).sum(2) + p["skip"] * u[:, :, t])
    return p["w_out"] @ (torch.stack(ys, 2) * torch.nn.functional.silu(z))


def params(b):
    names = ("w_in", "w_out", "w_conv", "b_conv", "w_r", "w_bc", "w_dt", "A", "skip", "b_dt")
    return {n: getattr(b, n).double().cpu().requires_grad_() for n in names}


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
    want = plain(p, hd)
    want.backward(dout.double())
    assert rel(out, want.detach()) < TOL
    for name, g in grads.items():
        w = hd.grad if name == "h" else p[name].grad
        e = rel(g, w)
        print(name, e, flush=True)
        assert g.shape == w.shape and e < TOL, (name, e)


def test_prompt_then_tokens(block):
    gen = torch.Generator().manual_seed(1)
    B, L, more = 3, 50, 5
    h = torch.randn(B, L + more, 96, generator=gen).to(torch.bfloat16).cuda()
    with torch.no_grad():
        want = plain(params(block), h.double().cpu().transpose(1, 2)).transpose(1, 2)
    lengths = torch.tensor([L, 0, 17], dtype=torch.int32, device="cuda")
    states = block.states(B)
    padded = h[:, :L].clone()
    for b, n in enumerate(lengths.tolist()):
        padded[b, n:] = float("nan")
    out = block.prompt(padded, states, lengths)
    for b, n in enumerate(lengths.tolist()):
        if n:
            e = rel(out[b, :n], want[b, :n])
            print("prompt", b, e, flush=True)
            assert e < TOL_SERVING
    # the tokens that follow each prompt, one at a time, the states in a pool
    pool = [torch.zeros((B + 1,) + s.shape[1:], dtype=s.dtype, device="cuda") for s in states]
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    for p, s in zip(pool, states):
        p[slots.long()] = s
    for k in range(more):
        x = torch.stack([h[b, n + k] for b, n in enumerate(lengths.tolist())])
        y, y2 = block.token(x, states), block.token(x, pool, slots=slots)
        assert torch.equal(y, y2)
        for b, n in enumerate(lengths.tolist()):
            e = rel(y[b], want[b, n + k])
            print("token", b, k, e, flush=True)
            assert e < TOL_SERVING
