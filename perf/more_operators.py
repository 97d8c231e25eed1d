"""Workloads of the gated delta layer's operators: the gated delta rule (prompts, training, single
tokens), layer normalisation, and products in 8-bit floating point with a scale for each block of 128,
each as a user's program calls it.

``run`` computes one pass: with ``own`` false from elementary torch operations, with ``own`` true
through this package's entry points.  ``exact`` gives the same outputs from the definitions in
64 bits.  Activations of the delta rule are [B, channels, L] (time fastest), as in the rest of the
package; layer norm and the products take tokens first or channels first.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
#
# Delta rule: B sequences, Hk heads of queries and keys of P channels, Hv heads of values of V
# channels (Hv / Hk of them share a key head), L steps.

def listed():
    return [
        # one long prompt: two value heads to a key head, keys normalised inside, final state kept
        {"name": "delta_prompt", "op": "delta_fwd", "dtype": "bf16", "B": 1, "Hk": 16, "Hv": 32, "P": 128, "V": 128,
         "L": 4096, "ragged": False},
        # ragged prompts (one empty, one of a single token) that continue from saved states, odd heads
        {"name": "delta_ragged", "op": "delta_fwd", "dtype": "f32", "B": 5, "Hk": 3, "Hv": 6, "P": 96, "V": 80,
         "L": 531, "ragged": True},
        # a training step: forward and backward
        {"name": "delta_train", "op": "delta_train", "dtype": "bf16", "B": 2, "Hk": 16, "Hv": 16, "P": 128, "V": 128,
         "L": 2048},
        # the same in fp32 with shared keys and sizes that divide by nothing
        {"name": "delta_train_odd", "op": "delta_train", "dtype": "f32", "B": 1, "Hk": 3, "Hv": 6, "P": 72, "V": 100,
         "L": 999},
        # one new token for each of many sequences: the states' bytes
        {"name": "delta_tokens", "op": "delta_step", "dtype": "bf16", "B": 64, "Hk": 16, "Hv": 32, "P": 128, "V": 128},
        # one new token of one sequence: latency
        {"name": "delta_token", "op": "delta_step", "dtype": "f32", "B": 1, "Hk": 8, "Hv": 8, "P": 64, "V": 64},
        # the norm in front of a layer, a prompt batch with tokens first
        {"name": "norm_prompt", "op": "norm_fwd", "dtype": "bf16", "B": 4, "L": 2048, "C": 4096, "channel_major": False},
        # a training step of the norm on channel-major activations
        {"name": "norm_train", "op": "norm_train", "dtype": "bf16", "B": 4, "L": 2048, "C": 2048, "channel_major": True},
        # the same in fp32 with tokens first and odd sizes
        {"name": "norm_train_odd", "op": "norm_train", "dtype": "f32", "B": 3, "L": 371, "C": 1001,
         "channel_major": False},
        # the input projection of a prompt batch, written channel-major for the convolution
        {"name": "f8_prompt", "op": "f8", "dtype": "bf16", "B": 4, "L": 2048, "C": 4096, "O": 8192,
         "channel_major": True, "bias": False},
        # an output projection of odd sizes, tokens first
        {"name": "f8_odd", "op": "f8", "dtype": "f32", "B": 1, "L": 1111, "C": 1000, "O": 1777,
         "channel_major": False, "bias": True},
        # a few new tokens: the weight's bytes
        {"name": "f8_tokens", "op": "f8", "dtype": "bf16", "B": 8, "L": 1, "C": 4096, "O": 8192,
         "channel_major": False, "bias": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_train", "delta_train", "delta_step", "norm_fwd", "norm_train",
                     "norm_train", "f8", "f8", "f8"])
    c = {"op": op, "dtype": rng.choice(["f32", "bf16"])}
    if op.startswith("delta"):
        c.update(B=_log(rng, 1, 8 if op != "delta_step" else 64), P=rng.choice([64, 128, 128, _log(rng, 16, 256)]),
                 V=rng.choice([64, 128, 128, _log(rng, 16, 256)]), Hk=_log(rng, 1, 16))
        c["Hv"] = c["Hk"] * rng.choice([1, 1, 2, 3])
        if op == "delta_step":
            c["B"] = max(1, min(c["B"], 33554432 // (c["Hv"] * c["P"] * c["V"])))
        else:
            most = 67108864 if op == "delta_train" else 134217728   # heads x steps x states
            c["L"] = _log(rng, 1, max(1, min(8192, most * 16 // (c["B"] * c["Hv"] * c["P"] * c["V"]))))
        if op == "delta_fwd":
            c["ragged"] = rng.random() < 0.4
    elif op.startswith("norm"):
        c.update(B=_log(rng, 1, 8), L=_log(rng, 1, 4096), channel_major=rng.random() < 0.5)
        c["C"] = _log(rng, 16, max(16, min(8192, 16777216 // (c["B"] * c["L"]))))
    else:
        c.update(B=_log(rng, 1, 8), L=rng.choice([1, _log(rng, 1, 2048), _log(rng, 1, 2048)]), C=_log(rng, 64, 8192),
                 channel_major=rng.random() < 0.5, bias=rng.random() < 0.5)
        c["O"] = _log(rng, 64, min(8192, 274877906944 // (c["B"] * c["L"] * c["C"])))
    return c


# ------------------------------------------------------------------ inputs

def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _lengths(gen, B, L):
    """Lengths of right-padded prompts: the longest fills the batch, one is empty, one has a token."""
    n = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = L
    if B > 1:
        n[1] = 0
    if B > 2:
        n[2] = 1
    return n


def _two_to(e):
    """2^e exactly, in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op}
    if op.startswith("delta"):
        B, Hk, Hv, P, V = (case[k] for k in ("B", "Hk", "Hv", "P", "V"))
        tail = () if op == "delta_step" else (case["L"],)
        # q, k and v are parts of the convolution's output [B, 2 Hk P + Hv V, L]
        qkv = _normal(gen, dt, B, 2 * Hk * P + Hv * V, *tail)
        s["q"], s["k"], s["v"] = qkv[:, :Hk * P], qkv[:, Hk * P:2 * Hk * P], qkv[:, 2 * Hk * P:]
        # log decays as such layers make them: -a softplus(u), a spread over heads from 0.01 to 1; step sizes in (0, 1)
        a = torch.exp(torch.rand(Hv, generator=gen, device="cuda") * math.log(100.0) - math.log(100.0))
        u = _normal(gen, torch.float32, B, Hv, *tail)
        s["g"] = -a.view(1, Hv, *(1,) * len(tail)) * torch.log1p(torch.exp(u))
        s["beta"] = torch.sigmoid(_normal(gen, torch.float32, B, Hv, *tail))
        s["heads"] = Hk
        if op == "delta_step":
            s["state"] = 0.1 * _normal(gen, torch.float32, B, Hv, P, V)
            s["state_out"] = torch.empty_like(s["state"])
        elif op == "delta_fwd":
            s["lengths"] = _lengths(gen, B, case["L"]) if case["ragged"] else None
            s["state"] = 0.1 * _normal(gen, torch.float32, B, Hv, P, V) if case["ragged"] else None
        else:
            s["dy"] = _normal(gen, dt, B, Hv * V, *tail)
    elif op.startswith("norm"):
        B, L, C = (case[k] for k in "BLC")
        shape = (B, C, L) if case["channel_major"] else (B, L, C)
        # channels differ in size and the tokens have means of their own
        size = torch.exp(0.5 * _normal(gen, torch.float32, C))
        x = torch.randn(B, L, C, generator=gen, device="cuda") * size + _normal(gen, torch.float32, B, L, 1)
        s["x"] = (x.transpose(1, 2) if case["channel_major"] else x).to(dt).contiguous()
        s["w"] = 1 + 0.2 * _normal(gen, torch.float32, C)
        s["b"] = 0.2 * _normal(gen, torch.float32, C)
        s["channel_major"] = case["channel_major"]
        if op == "norm_train":
            s["dy"] = _normal(gen, dt, *shape)
    else:
        B, L, C, O = (case[k] for k in "BLCO")
        s.update(dims=(B, L, C, O), dtype=dt, channel_major=case["channel_major"])
        s["x"] = _normal(gen, dt, B * L, C) * torch.exp(_normal(gen, torch.float32, B * L, 1)).to(dt)
        w = _normal(gen, torch.float32, O, C) / math.sqrt(C)
        # the weight is quantised once, its rows padded with zeros to a multiple of 128
        pad = -(-C // 128) * 128
        blocks = torch.nn.functional.pad(w, (0, pad - C)).view(O, pad // 128, 128)
        m, x = torch.frexp(blocks.abs().amax(2))
        e = torch.clamp(torch.where(m > 0.875, x - 8, x - 9), min=-127)
        s["wq"] = (blocks * _two_to(-e)[..., None]).float().view(O, pad).to(torch.float8_e4m3fn)
        s["ws"] = (e + 127).t().contiguous().to(torch.uint8).view(torch.float8_e8m0fnu)
        s["bias"] = 0.1 * _normal(gen, torch.float32, O) if case["bias"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import convolution_implicit_gemm_nchw_amd as mc
    op = s["op"]
    if op == "delta_fwd":
        final = torch.empty(s["g"].shape[:2] + (s["q"].shape[1] // s["heads"], s["v"].shape[1] // s["g"].shape[1]),
                            dtype=torch.float32, device="cuda")
        y = mc.gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], key_heads=s["heads"], l2norm=True,
                               initial_state=s["state"], lengths=s["lengths"], final_state=final)
        return {"y": y, "state": final}
    if op == "delta_train":
        saved = mc.gated_delta_states(s["q"], s["v"], s["g"], key_heads=s["heads"])
        y = mc.gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], key_heads=s["heads"], l2norm=True,
                               states=saved)
        grads = mc.gated_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], saved, key_heads=s["heads"],
                                   l2norm=True)
        return {"y": y, **grads}
    if op == "delta_step":
        y = mc.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], key_heads=s["heads"],
                                l2norm=True, state_out=s["state_out"])
        return {"y": y, "state": s["state_out"]}
    if op == "norm_fwd":
        return {"y": mc.layer_norm_fwd(s["x"], s["w"], s["b"], channel_major=s["channel_major"])}
    if op == "norm_train":
        stats = mc.layer_norm_stats(s["x"], channel_major=s["channel_major"])
        y = mc.layer_norm_fwd(s["x"], s["w"], s["b"], channel_major=s["channel_major"], stats=stats)
        dx, dw, db = mc.layer_norm_bwd(s["x"], s["dy"], stats, s["w"], s["b"], channel_major=s["channel_major"])
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    q, scale = mc.quantize_f8(s["x"])
    return {"y": mc.matmul_f8(q, scale, s["wq"], s["ws"], bias=s["bias"], out_dtype=s["dtype"],
                              length=s["dims"][1] if s["channel_major"] else None)}


EPS = 1e-5          # layer norm
EPS_HEAD = 1e-6     # the normalisation of queries and keys


def _plain(s):
    op = s["op"]
    if op.startswith("norm"):
        return _plain_norm(s)
    if op == "f8":
        return {"y": _plain_f8(s)}
    if op == "delta_step":
        return _plain_step(s)
    return _plain_delta(s)


def _heads(t, heads, repeat=1):
    """[B, heads * d, L] as [B, heads * repeat, L, d] in 32 bits."""
    return t.float().unflatten(1, (heads, -1)).transpose(2, 3).repeat_interleave(repeat, 1)


def _plain_step(s):
    Hk, Hv = s["heads"], s["g"].shape[1]
    q, k = (_heads(s[n][..., None], Hk, Hv // Hk)[:, :, 0] for n in "qk")
    v = _heads(s["v"][..., None], Hv)[:, :, 0]
    q = q * torch.rsqrt((q * q).sum(2, keepdim=True) + EPS_HEAD)
    k = k * torch.rsqrt((k * k).sum(2, keepdim=True) + EPS_HEAD)
    S = torch.exp(s["g"])[..., None, None] * s["state"]
    u = s["beta"][..., None] * (v - (k[..., None] * S).sum(2))
    S = S + k[..., None] * u[:, :, None]
    y = (q[..., None] * S).sum(2) * q.shape[2] ** -0.5
    return {"y": y.flatten(1).to(s["v"].dtype), "state": S}


CHUNK = 64


def _chunks(t):
    """[B, H, L, ...] as [B, H, n, CHUNK, ...], zeros past L."""
    L = t.shape[2]
    n = -(-L // CHUNK)
    full = t.new_zeros(t.shape[:2] + (n * CHUNK,) + t.shape[3:])
    full[:, :, :L] = t
    return full.unflatten(2, (n, CHUNK))


def _plain_delta(s):
    """The delta rule by chunks of 64 steps: within a chunk the steps' updates u solve a triangular system, whose
    inverse is a product of powers; the state goes from chunk to chunk."""
    Hk, Hv = s["heads"], s["g"].shape[1]
    rep, L, out = Hv // Hk, s["q"].shape[2], s["v"].dtype
    raw_q, raw_k, v = _heads(s["q"], Hk, rep), _heads(s["k"], Hk, rep), _heads(s["v"], Hv)
    B, _, _, P = raw_q.shape
    rq = torch.rsqrt((raw_q * raw_q).sum(3, keepdim=True) + EPS_HEAD)
    rk = torch.rsqrt((raw_k * raw_k).sum(3, keepdim=True) + EPS_HEAD)
    q, k, g, beta = raw_q * rq, raw_k * rk, s["g"], s["beta"]
    lengths = s.get("lengths")
    if lengths is not None:
        inside = torch.arange(L, device="cuda") < lengths[:, None, None]
        q, k, v = (t * inside[..., None] for t in (q, k, v))
        g, beta = g * inside, beta * inside
    scale = P ** -0.5
    q, k, v, g, beta = (_chunks(t) for t in (q * scale, k, v, g.double(), beta))
    beta = beta[..., None]
    G = g.cumsum(3)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    D = (G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf).exp().float()
    e, f = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    kk = (k @ k.transpose(3, 4)) * D.tril(-1)          # without the step sizes
    power = -(kk * beta.transpose(3, 4)).double()
    inverse = torch.eye(CHUNK, dtype=torch.float64, device="cuda") + power
    for _ in range(5):
        power = power @ power
        inverse = inverse + inverse @ power
    inverse, attn = inverse.float(), (q @ k.transpose(3, 4)) * D
    S = v.new_zeros(B, Hv, P, v.shape[4]) if s.get("state") is None else s["state"]
    n, entry, y, Z = v.shape[2], [], torch.empty_like(v), torch.empty_like(v)
    for i in range(n):
        entry.append(S)
        Z[:, :, i] = inverse[:, :, i] @ (v[:, :, i] - e[:, :, i] * (k[:, :, i] @ S))
        U = beta[:, :, i] * Z[:, :, i]
        y[:, :, i] = e[:, :, i] * (q[:, :, i] @ S) + attn[:, :, i] @ U
        S = e[:, :, i, -1:] * S + (f[:, :, i] * k[:, :, i]).transpose(2, 3) @ U
    flat = lambda t: t.flatten(2, 3)[:, :, :L]                                    # noqa: E731
    rows = lambda t: t.transpose(2, 3).flatten(1, 2).to(out)                      # noqa: E731
    r = {"y": rows(flat(y))}
    if s["op"] == "delta_fwd":
        return {**r, "state": S}
    dy = _chunks(_heads(s["dy"], Hv))
    U, back = beta * Z, attn.transpose(3, 4) @ dy
    up, dS, after = torch.empty_like(v), torch.zeros_like(S), [None] * n
    for i in reversed(range(n)):
        after[i] = dS
        dU = back[:, :, i] + f[:, :, i] * (k[:, :, i] @ dS)
        up[:, :, i] = inverse[:, :, i].transpose(2, 3) @ (beta[:, :, i] * dU)
        dS = (e[:, :, i, -1:] * dS + (e[:, :, i] * q[:, :, i]).transpose(2, 3) @ dy[:, :, i]
              - (e[:, :, i] * k[:, :, i]).transpose(2, 3) @ up[:, :, i])
        back[:, :, i] = dU
    entry, after = torch.stack(entry, 2), torch.stack(after, 2)
    dD = (dy @ U.transpose(3, 4)) * D
    dA = -(up @ U.transpose(3, 4)) * D.tril(-1)
    dq = e * (dy @ entry.transpose(3, 4)) + dD @ k
    read = dA @ k - e * (up @ entry.transpose(3, 4))
    ends = f * (U @ after.transpose(3, 4))
    write = ends + dD.transpose(3, 4) @ q + dA.transpose(3, 4) @ k
    dbeta = (Z * (back - kk.transpose(3, 4) @ up)).sum(4)
    dG = (q * dq + k * read - k * write).sum(4).double()
    last = (k * ends).sum((3, 4)).double() + G[..., -1].exp() * (entry * after).sum((3, 4)).double()
    dg = dG.flip(3).cumsum(3).flip(3) + last[..., None]
    nq, nk, dq, dk = flat(q), flat(k), flat(dq) * scale, flat(read + write)
    group = lambda t: t.unflatten(1, (Hk, rep)).sum(2)                            # noqa: E731
    # through the normalisation: r (d - n (n . d))
    nq = nq / scale
    dq = rq * (dq - nq * (nq * dq).sum(3, keepdim=True))
    dk = rk * (dk - nk * (nk * dk).sum(3, keepdim=True))
    return {**r, "dq": rows(group(dq)), "dk": rows(group(dk)), "dv": rows(flat(up)), "dg": flat(dg).float(),
            "dbeta": flat(dbeta)}


def _plain_norm(s):
    axis = 1 if s["channel_major"] else 2
    x, w, b = s["x"].float(), s["w"], s["b"]
    if s["channel_major"]:
        w, b = w[:, None], b[:, None]
    d = x - x.mean(axis, keepdim=True)
    r = torch.rsqrt((d * d).mean(axis, keepdim=True) + EPS)
    n = d * r
    y = (n * w + b).to(s["x"].dtype)
    if s["op"] == "norm_fwd":
        return {"y": y}
    dy = s["dy"].float()
    h = dy * w
    dx = r * (h - h.mean(axis, keepdim=True) - n * (h * n).mean(axis, keepdim=True))
    rest = (0, 3 - axis)
    return {"y": y, "dx": dx.to(s["x"].dtype), "dw": (dy * n).sum(rest), "db": dy.sum(rest)}


def _plain_f8(s):
    B, L, C, O = s["dims"]
    pad = s["wq"].shape[1]
    x = s["x"].float()
    full = x.new_zeros(B * L, pad)
    full[:, :C] = x
    blocks = full.view(B * L, pad // 128, 128)
    m, e = torch.frexp(blocks.abs().amax(2))
    # the least power of two that brings the block to 448 = 0.875 * 2^9 or below
    e = torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-127)
    q = (blocks * _two_to(-e)[..., None]).float().to(torch.float8_e4m3fn).double() * _two_to(e)[..., None]
    w = s["wq"].double().view(O, pad // 128, 128) * _two_to(s["ws"].view(torch.uint8).t().int() - 127)[..., None]
    y = q.float().view(B * L, pad) @ w.float().view(O, pad).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["channel_major"]:
        y = y.unflatten(0, (B, L)).transpose(1, 2).contiguous()
    return y.to(s["dtype"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    op = c["op"]
    if op == "f8":
        t = c["B"] * c["L"]
        pad = -(-c["C"] // 128) * 128
        return {"bytes": t * c["C"] * e + c["O"] * pad * 129 // 128 + t * c["O"] * e + c["O"] * 4 * int(c["bias"]),
                "flops": 2 * t * c["C"] * c["O"]}
    if op.startswith("norm"):
        n = c["B"] * c["L"] * c["C"]
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * c["C"], "flops": 8 * n}
        # x is needed again only after all of dy's sums: forward x and y, backward x, dy and dx
        return {"bytes": 5 * n * e + 16 * c["C"], "flops": 22 * n}
    B, Hk, Hv, P, V, L = c["B"], c["Hk"], c["Hv"], c["P"], c["V"], c.get("L", 1)
    rows = B * L * ((2 * Hk * P + 2 * Hv * V) * e + 8 * Hv)
    state = B * Hv * P * V * 4
    if op == "delta_step":
        return {"bytes": rows + 2 * state, "flops": B * Hv * 7 * P * V}
    # a step of a head reads the state with key and query and updates it; in chunks of 64 the steps meet in pairs
    fwd = B * Hv * L * (6 * P * V + 64 * (2 * P + 2 * V))
    if op == "delta_fwd":
        return {"bytes": rows + state * (2 if c["ragged"] else 1), "flops": fwd}
    grads = B * L * ((4 * Hk * P + 3 * Hv * V) * e + 16 * Hv)
    return {"bytes": rows + grads, "flops": fwd * 3}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "f8":
        B, L, C, O = s["dims"]
        y = torch.zeros(B * L, O, dtype=f64, device="cuda")
        power = torch.tensor([2.0 ** i for i in range(-200, 200)], dtype=f64, device="cuda")
        two = lambda e: power[e.long() + 200]  # noqa: E731
        wunit = two(s["ws"].view(torch.uint8).int() - 127)
        for k in range(0, C, 128):
            x = s["x"][:, k:k + 128].to(f64)
            top = x.abs().max(dim=1, keepdim=True).values
            unit = torch.full_like(top, 2.0 ** -127)     # no block has a smaller one
            # the least power of two >= top / 448, by its definition
            grow = torch.ceil(torch.log2(torch.clamp(top / 448, min=2.0 ** -127)))
            for d in (-1, 0, 1):
                c = two(torch.clamp(grow + d, min=-127))
                unit = torch.where((unit * 448 < top) & (c * 448 >= top), c, unit)
            v = x / unit
            # steps of 2^(floor(log2 |v|) - 3), 2^-9 below 2^-6; halves to the even neighbour
            size = torch.clamp(torch.frexp(v).exponent.to(f64) - 1, min=-6) - 3
            step = two(size)
            q = torch.round(v / step) * step * unit
            w = s["wq"][:, k:k + 128].float().to(f64)[:, :x.shape[1]] * wunit[k // 128][:, None]
            y += q @ w.t()
        if s["bias"] is not None:
            y = y + s["bias"].to(f64)[None]
        return {"y": y.view(B, L, O).permute(0, 2, 1).contiguous() if s["channel_major"] else y}
    if op.startswith("norm"):
        cm = s["channel_major"]
        x = s["x"].to(f64).movedim(1, 2) if cm else s["x"].to(f64)
        w, b = s["w"].to(f64), s["b"].to(f64)
        var, mean = torch.var_mean(x, 2, correction=0, keepdim=True)
        inv = 1 / torch.sqrt(var + EPS)
        back = lambda t: t.movedim(2, 1).contiguous() if cm else t  # noqa: E731
        r = {"y": back((x - mean) * inv * w + b)}
        if op == "norm_fwd":
            return r
        dy = s["dy"].to(f64).movedim(1, 2) if cm else s["dy"].to(f64)
        t = dy * w
        dvar = (t * (x - mean)).sum(2, keepdim=True) * (-0.5) * inv ** 3
        dmean = -(t * inv).sum(2, keepdim=True)
        n = x.shape[2]
        return {**r, "dx": back(t * inv + dvar * 2 * (x - mean) / n + dmean / n),
                "dw": torch.einsum("blc,blc->c", dy, (x - mean) * inv), "db": dy.sum((0, 1))}
    B, Hk, Hv, P, V = (case[k] for k in ("B", "Hk", "Hv", "P", "V"))
    L, rep = case.get("L", 1), Hv // Hk
    train = op == "delta_train"
    if train and B * Hv * P * V * L * 8 > 24e9:
        return None
    view = lambda t, h: t.to(f64).reshape(B, h, -1, L).permute(3, 0, 1, 2)  # noqa: E731
    q0, k0, v = view(s["q"], Hk), view(s["k"], Hk), view(s["v"], Hv)
    g, beta = (s[n].to(f64).reshape(B, Hv, L).permute(2, 0, 1) for n in ("g", "beta"))
    nq, nk = ((t * t).sum(3, keepdim=True).add(EPS_HEAD).sqrt() for t in (q0, k0))
    wide = lambda t: t[:, :, :, None].expand(L, B, Hk, rep, t.shape[3]).reshape(L, B, Hv, t.shape[3])  # noqa: E731
    q, k = wide(q0 / nq) / math.sqrt(P), wide(k0 / nk)
    S = torch.zeros(B, Hv, P, V, dtype=f64, device="cuda") if s.get("state") is None else s["state"].to(f64)
    y = torch.zeros(L, B, Hv, V, dtype=f64, device="cuda")
    lengths = s.get("lengths")
    hist = torch.empty(L + 1, B, Hv, P, V, dtype=f64, device="cuda") if train else None
    miss = torch.empty_like(y)
    if train:
        hist[0] = S
    for t in range(L):
        kept = S * g[t].exp()[..., None, None]
        miss[t] = v[t] - torch.einsum("bhp,bhpv->bhv", k[t], kept)
        new = kept + torch.einsum("bhp,bhv->bhpv", k[t], beta[t][..., None] * miss[t])
        o = torch.einsum("bhp,bhpv->bhv", q[t], new)
        if lengths is not None:
            on = (lengths > t).view(B, 1, 1)
            new, o = torch.where(on[..., None], new, S), torch.where(on, o, torch.zeros_like(o))
        S, y[t] = new, o
        if train:
            hist[t + 1] = S
    rows = lambda t: t.permute(1, 2, 3, 0).reshape(B, -1, L).contiguous()  # noqa: E731
    if op == "delta_step":
        return {"y": rows(y)[..., 0], "state": S}
    if op == "delta_fwd":
        return {"y": rows(y), "state": S}
    do = view(s["dy"], Hv)
    dS = torch.zeros_like(S)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    for t in reversed(range(L)):
        dS = dS + torch.einsum("bhp,bhv->bhpv", q[t], do[t])
        dq[t] = torch.einsum("bhpv,bhv->bhp", hist[t + 1], do[t])
        du = torch.einsum("bhpv,bhp->bhv", dS, k[t])
        dbeta[t] = (du * miss[t]).sum(2)
        dv[t] = du * beta[t][..., None]
        dk[t] = torch.einsum("bhpv,bhv->bhp", dS, beta[t][..., None] * miss[t])
        decay = g[t].exp()[..., None, None]
        dk[t] -= torch.einsum("bhpv,bhv->bhp", hist[t] * decay, dv[t])
        dS = dS - torch.einsum("bhp,bhv->bhpv", k[t], dv[t])
        dg[t] = (dS * hist[t] * decay).sum((2, 3))
        dS = dS * decay
    narrow = lambda t: t.reshape(L, B, Hk, rep, P).sum(3)  # noqa: E731
    dq, dk = narrow(dq) / math.sqrt(P), narrow(dk)
    # d of x / |x|: (d - x (x . d) / |x|^2) / |x|
    dq = (dq - q0 * (q0 * dq).sum(3, keepdim=True) / nq ** 2) / nq
    dk = (dk - k0 * (k0 * dk).sum(3, keepdim=True) / nk ** 2) / nk
    return {"y": rows(y), "dq": rows(dq), "dk": rows(dk), "dv": rows(dv), "dg": dg.permute(1, 2, 0).contiguous(),
            "dbeta": dbeta.permute(1, 2, 0).contiguous()}
