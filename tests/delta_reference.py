"""Plain 64-bit forms of the gated delta rule, layer norm and the block-scaled 8-bit products (torch on the
CPU; the rule one time step after the other), and the tolerances of their tests.

U = 2^-24 is half a step of fp32, relative.  A sum of n terms, in any order, is off by at most n U of the sum
of their magnitudes.  A stored value is off by half a step of its type.
"""
import torch

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ gated delta rule

def rule(q, k, v, g, beta, Hk, scale=None, l2norm=False, state=None, lengths=None, seen=None):
    """(y [B, Hv V, L], final state [B, Hv, P, V]) in 64 bits; differentiable.  `seen`, a list, takes the normalised
    queries and keys and what they were divided by."""
    B, Hv, L = g.shape
    P, V, rep = q.shape[1] // Hk, v.shape[1] // Hv, Hv // Hk
    q, k = q.view(B, Hk, P, L), k.view(B, Hk, P, L)
    if l2norm:
        size = [torch.sqrt((x * x).sum(2, keepdim=True) + 1e-6) for x in (q, k)]
        q, k = q / size[0], k / size[1]
        if seen is not None:
            q.retain_grad()
            k.retain_grad()
            seen += [(q, size[0]), (k, size[1])]
    q, k = (x.repeat_interleave(rep, 1) for x in (q, k))
    q = q * (P ** -0.5 if scale is None else scale)
    v = v.view(B, Hv, V, L)
    S = torch.zeros(B, Hv, P, V, dtype=torch.float64) if state is None else state
    n = torch.full((B,), L) if lengths is None else torch.as_tensor(lengths).clamp(0, L)
    ys = []
    for t in range(L):
        on = (t < n).view(B, 1, 1, 1)
        old = torch.exp(g[:, :, t])[:, :, None, None] * S
        z = v[..., t] - (old * k[..., t, None]).sum(2)
        new = old + k[..., t, None] * (beta[:, :, t, None] * z)[:, :, None]
        S = torch.where(on, new, S)
        ys.append(torch.where(on[..., 0], (new * q[..., t, None]).sum(2), torch.zeros((), dtype=torch.float64)))
    return torch.stack(ys, 3).reshape(B, Hv * V, L), S


def rule_bound(P, L, dt, passes=1):
    """(absolute part, of the output's largest magnitude; relative part, of the value).

    A value's way leads through sums of P terms (the key with the state, the query with the state) and of 64
    (the inverse, the state's update, the scores), 2 P + 192 terms in all, and once more for a gradient, whose
    operands come from a forward pass.  With keys of length one at most, step sizes up to 2 and decays up to 1 no
    error grows on its way through the states (I - beta k k^T has no norm above 1), and the chunks' errors add up:
    as many as there are chunks, in the worst case.  Decays that grow a little are counted in by the caller.
    A bf16 result of the scores with the corrected values takes 16 bits of both (2^-15 of their product), a
    sum of 64 of them against the largest result: 8 where they add up as lengths do."""
    chunks = (L + 63) // 64
    absolute = passes * (2 * P + 192) * U * chunks
    if dt == "bf16":
        absolute += 8 * 2.0 ** -15
    return absolute, HALF[dt]


# ------------------------------------------------------------------ layer norm

def layer_norm(x, w, b, eps, lengths, dy=None):
    """{name: (value, bound)} of x [B, L, C] (tokens first): y, mean, rstd, and with dy also dx, dw, db, for fp32
    arithmetic before the output is stored.  No thread adds more than 48 + C / 128 terms one after the other."""
    B, L, C = x.shape
    n = 48 + C / 128
    keep = torch.ones(B, L, 1, dtype=torch.bool)
    if lengths is not None:
        keep = torch.arange(L)[None, :, None] < torch.as_tensor(lengths).clamp(0, L).view(B, 1, 1)
    x = torch.where(keep, x, torch.zeros((), dtype=torch.float64))
    w = torch.ones(C, dtype=torch.float64) if w is None else w
    b = torch.zeros(C, dtype=torch.float64) if b is None else b
    mean = x.mean(2, keepdim=True)
    d = x - mean
    var = (d * d).mean(2, keepdim=True)
    r = (var + eps).rsqrt()
    e_mean = (n + 3) * U * x.abs().mean(2, keepdim=True)
    # an error of the mean changes each difference by it, and the mean square by its square only: the
    # differences add to zero
    e_d = e_mean + U * d.abs()
    e_r = r * ((n + 8) * U + e_mean ** 2 * r * r)
    norm = d * r
    e_norm = e_d * r + d.abs() * e_r + U * norm.abs()
    y = norm * w + b
    out = {"y": (y * keep, (e_norm * w.abs() + 2 * U * ((norm * w).abs() + b.abs())) * keep),
           "mean": (mean, e_mean), "rstd": (r, e_r)}
    if dy is not None:
        dy = torch.where(keep, dy, torch.zeros((), dtype=torch.float64))
        h = dy * w
        s, t = h.mean(2, keepdim=True), (h * norm).mean(2, keepdim=True)
        e_s = (n + 3) * U * h.abs().mean(2, keepdim=True)
        e_t = (n + 4) * U * (h * norm).abs().mean(2, keepdim=True) + (h.abs() * e_norm).mean(2, keepdim=True)
        inner = h - s - norm * t
        e_inner = e_s + norm.abs() * e_t + e_norm * t.abs() + 4 * U * (h.abs() + s.abs() + (norm * t).abs())
        out["dx"] = (r * inner * keep, (r * e_inner + inner.abs() * e_r + U * (r * inner).abs()) * keep)
        count = B * L
        out["dw"] = ((dy * norm).sum((0, 1)), (count * U * (dy * norm).abs() + dy.abs() * e_norm).sum((0, 1)))
        out["db"] = (dy.sum((0, 1)), count * U * dy.abs().sum((0, 1)))
    return out


# ------------------------------------------------------------------ 8-bit floating point

def quantize(x):
    """(q as float32 values, exponent int [tokens, blocks], bad) of x [tokens, C] float32: the least 2^e, e >= -127, with
    max|x| <= 448 2^e in each block of 128, and x / 2^e rounded to nearest even."""
    T, C = x.shape
    pad = (-C) % 128
    x = torch.nn.functional.pad(x.double(), (0, pad)).view(T, -1, 128)
    m = x.abs().amax(2)
    bad = ~x.isfinite().all(2)
    m = torch.where(bad, torch.ones_like(m), m)
    frac, e = torch.frexp(m / 448.0)                 # m / 448 = frac 2^e, frac in [1/2, 1)
    e = torch.where(frac == 0.5, e - 1, e)           # the power itself
    e = torch.where(m == 0, torch.full_like(e, -127), e.clamp(min=-127))
    # m / 448 may round to a power that lies below it: 448 2^e is exact
    e = torch.where(m > 448.0 * torch.exp2(e.double()), e + 1, e)
    one = x * torch.exp2(-e.double())[..., None]
    q = one.float().to(torch.float8_e4m3fn).float()
    return q.view(T, -1), e, bad


def product(q, e, wq, we):
    """(sum, sum of magnitudes) [T, O] in 64 bits of the quantised operands."""
    a = q.double().view(q.shape[0], -1, 128) * torch.exp2(e.double())[..., None]
    w = wq.double().view(wq.shape[0], -1, 128) * torch.exp2(we.double())[..., None]
    a, w = a.view(q.shape[0], -1), w.view(wq.shape[0], -1)
    return a @ w.t(), a.abs() @ w.abs().t()
