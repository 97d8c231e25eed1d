"""Workloads of the state-space language-model operators: the short causal convolution, the
selective scan and the 8-bit integer product, each as a user's program calls it.

``run`` computes one pass: with ``own`` false from elementary torch operations, with ``own`` true
through this package's entry points.  ``exact`` gives the same outputs from the definitions in
64 bits.  Activations are [B, D, L] (channel-major, time fastest), as in the rest of the package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a prompt batch through the convolution in front of the scan, inputs a half of the projection
        {"name": "conv_prompt", "op": "conv_fwd", "dtype": "bf16", "B": 4, "D": 4096, "L": 2048, "K": 4,
         "ragged": False},
        # its gradients in fp32 training, sizes that divide by nothing
        {"name": "conv_train_odd", "op": "conv_bwd", "dtype": "f32", "B": 3, "D": 1001, "L": 1533, "K": 3,
         "ragged": False},
        # one new token of one sequence: latency
        {"name": "conv_token", "op": "conv_step", "dtype": "bf16", "B": 1, "D": 2048, "K": 4},
        # one long prompt through the scan
        {"name": "scan_prompt", "op": "scan_fwd", "dtype": "bf16", "B": 1, "D": 4096, "L": 4096, "N": 16, "G": 1,
         "gate": True, "ragged": False},
        # ragged prompts (one empty, one of a single token) that continue from saved states
        {"name": "scan_ragged", "op": "scan_fwd", "dtype": "f32", "B": 6, "D": 777, "L": 531, "N": 8, "G": 1,
         "gate": False, "ragged": True},
        # a training step of the scan: forward and backward
        {"name": "scan_train", "op": "scan_train", "dtype": "bf16", "B": 2, "D": 4096, "L": 2048, "N": 16, "G": 1,
         "gate": True},
        # the same in fp32 with two groups of B and C and odd sizes
        {"name": "scan_train_odd", "op": "scan_train", "dtype": "f32", "B": 1, "D": 1538, "L": 999, "N": 16, "G": 2,
         "gate": True},
        # one new token for each of many sequences: the states' bytes
        {"name": "scan_tokens", "op": "scan_step", "dtype": "bf16", "B": 256, "D": 4096, "N": 16, "G": 1,
         "gate": True},
        # one new token of one sequence: latency
        {"name": "scan_token", "op": "scan_step", "dtype": "f32", "B": 1, "D": 2048, "N": 16, "G": 1, "gate": True},
        # the input projection of a prompt batch, written channel-major for the convolution
        {"name": "i8_prompt", "op": "i8", "dtype": "bf16", "B": 4, "L": 2048, "C": 4096, "O": 8192,
         "channel_major": True, "bias": False},
        # an output projection of odd sizes, tokens first
        {"name": "i8_odd", "op": "i8", "dtype": "f32", "B": 1, "L": 1111, "C": 1000, "O": 1777,
         "channel_major": False, "bias": True},
        # a few new tokens: the weight's bytes
        {"name": "i8_tokens", "op": "i8", "dtype": "bf16", "B": 8, "L": 1, "C": 4096, "O": 8192,
         "channel_major": False, "bias": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_train", "scan_train",
                     "scan_step", "i8", "i8", "i8"])
    c = {"op": op, "dtype": rng.choice(["f32", "bf16"])}
    if op in ("conv_fwd", "conv_bwd"):
        c.update(B=_log(rng, 1, 16), L=_log(rng, 1, 8192), K=rng.choice([2, 3, 4, 4, 5, 8]))
        c["D"] = _log(rng, 16, max(16, min(8192, 33554432 // (c["B"] * c["L"]))))
        c["ragged"] = rng.random() < 0.3
    elif op == "conv_step":
        c.update(B=_log(rng, 1, 256), D=_log(rng, 64, 8192), K=rng.choice([2, 3, 4, 4, 8]))
    elif op in ("scan_fwd", "scan_train", "scan_step"):
        c.update(B=_log(rng, 1, 8 if op != "scan_step" else 256), N=rng.choice([1, 5, 8, 16, 16, 16, 32, 64]),
                 G=rng.choice([1, 1, 1, 2, 4]), gate=rng.random() < 0.7)
        if op == "scan_step":
            c["D"] = c["G"] * _log(rng, 16, max(16, min(8192, 16777216 // (c["B"] * c["N"])) // c["G"]))
        else:
            c["L"] = _log(rng, 1, 8192)
            most = 268435456 // (c["B"] * c["L"] * c["N"])
            c["D"] = c["G"] * _log(rng, 16, max(16, min(8192, most) // c["G"]))
        if op == "scan_fwd":
            c["ragged"] = rng.random() < 0.4
    else:
        c.update(B=_log(rng, 1, 8), L=rng.choice([1, _log(rng, 1, 2048), _log(rng, 1, 2048)]), C=_log(rng, 64, 8192),
                 O=_log(rng, 64, 4096), channel_major=rng.random() < 0.5, bias=rng.random() < 0.5)
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op}
    if op in ("conv_fwd", "conv_bwd"):
        B, D, L, K = (case[k] for k in "BDLK")
        # x is the first half of the input projection [B, 2D, L]: its batches are 2 D L apart
        s["x"] = _normal(gen, dt, B, 2 * D, L)[:, :D]
        s["w"] = (_normal(gen, torch.float32, D, K) / math.sqrt(K)).to(dt)
        s["bias"] = 0.1 * _normal(gen, torch.float32, D)
        s["lengths"] = _lengths(gen, B, L) if case["ragged"] else None
        s["state"] = _normal(gen, dt, B, D, K - 1) if case["ragged"] else None
        if op == "conv_bwd":
            s["dy"] = _normal(gen, dt, B, D, L)
    elif op == "conv_step":
        B, D, K = (case[k] for k in "BDK")
        s["x"] = _normal(gen, dt, B, D)
        s["w"] = (_normal(gen, torch.float32, D, K) / math.sqrt(K)).to(dt)
        s["bias"] = 0.1 * _normal(gen, torch.float32, D)
        s["state"] = _normal(gen, dt, B, D, K - 1)
        s["state_out"] = torch.empty_like(s["state"])
    elif op in ("scan_fwd", "scan_train", "scan_step"):
        B, D, N, G = (case[k] for k in "BDNG")
        n = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
        s["A"] = -n * torch.exp(0.1 * _normal(gen, torch.float32, D, N))
        s["D"] = 1 + 0.1 * _normal(gen, torch.float32, D)
        # softplus(bias) is spread over 0.001 .. 0.1, as such layers are initialised
        step = torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
        s["bias"] = step + torch.log(-torch.expm1(-step))
        tail = () if op == "scan_step" else (case["L"],)
        s["x"] = _normal(gen, dt, B, D, *tail)
        s["delta"] = (0.5 * _normal(gen, torch.float32, B, D, *tail)).to(dt)
        s["z"] = _normal(gen, dt, B, 2 * D, *tail)[:, D:] if case["gate"] else None
        # B and C are slices of one small projection [B, 2 G N, L]
        bc = _normal(gen, dt, B, 2 * G * N, *tail)
        s["B"], s["C"] = bc[:, :G * N].unflatten(1, (G, N)), bc[:, G * N:].unflatten(1, (G, N))
        if op == "scan_step":
            s["state"] = _normal(gen, torch.float32, B, D, N)
            s["state_out"] = torch.empty_like(s["state"])
        elif op == "scan_fwd":
            s["lengths"] = _lengths(gen, B, case["L"]) if case["ragged"] else None
            s["state"] = _normal(gen, torch.float32, B, D, N) if case["ragged"] else None
        else:
            s["dy"] = _normal(gen, dt, B, D, *tail)
    else:
        B, L, C, O = (case[k] for k in "BLCO")
        s.update(dims=(B, L, C, O), dtype=dt, channel_major=case["channel_major"])
        s["x"] = _normal(gen, dt, B * L, C)
        w = _normal(gen, torch.float32, O, C).double() / math.sqrt(C)
        top = w.abs().amax(1, keepdim=True)
        # the weight is quantised once, its rows padded with zeros to a multiple of 128
        s["wq"] = torch.zeros(O, -(-C // 128) * 128, dtype=torch.int8, device="cuda")
        s["wq"][:, :C] = torch.round(w * 127 / top).to(torch.int8)
        s["ws"] = (top[:, 0] / 127).float()
        s["bias"] = 0.1 * _normal(gen, torch.float32, O) if case["bias"] else None
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import convolution_implicit_gemm_nchw_amd as mc
    op = s["op"]
    if op == "conv_fwd":
        final = torch.empty(s["x"].shape[0], s["x"].shape[1], s["w"].shape[1] - 1, dtype=s["x"].dtype, device="cuda")
        y = mc.causal_conv1d_fwd(s["x"], s["w"], bias=s["bias"], silu=True, initial_state=s["state"],
                                 lengths=s["lengths"], final_state=final)
        return {"y": y, "state": final}
    if op == "conv_bwd":
        dx, dw, db = mc.causal_conv1d_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], silu=True,
                                          initial_state=s["state"], lengths=s["lengths"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "conv_step":
        y = mc.causal_conv1d_step(s["x"], s["state"], s["w"], bias=s["bias"], silu=True, state_out=s["state_out"])
        return {"y": y, "state": s["state_out"]}
    if op == "scan_step":
        y = mc.selective_scan_step(s["x"], s["delta"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                                   delta_bias=s["bias"], softplus=True, state_out=s["state_out"])
        return {"y": y, "state": s["state_out"]}
    if op == "scan_fwd":
        final = torch.empty(s["x"].shape[:2] + s["A"].shape[1:], dtype=torch.float32, device="cuda")
        y = mc.selective_scan_fwd(s["x"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                  delta_bias=s["bias"], softplus=True, initial_state=s["state"],
                                  lengths=s["lengths"], final_state=final)
        return {"y": y, "state": final}
    if op == "scan_train":
        states = mc.selective_scan_states(s["x"], s["A"])
        y = mc.selective_scan_fwd(s["x"], s["delta"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                  delta_bias=s["bias"], softplus=True, states=states)
        grads = mc.selective_scan_bwd(s["x"], s["delta"], s["A"], s["B"], s["C"], s["dy"], states, D=s["D"],
                                      z=s["z"], delta_bias=s["bias"], softplus=True)
        return {"y": y, **{k: v for k, v in grads.items() if v is not None}}
    q, scale = mc.quantize_tokens(s["x"])
    return {"y": mc.matmul_i8(q, scale, s["wq"], s["ws"], bias=s["bias"], out_dtype=s["dtype"],
                              length=s["dims"][1] if s["channel_major"] else None)}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20))))


def _valid(lengths, L):
    """1 where a time step is inside its sequence, [B, 1, L]."""
    return (torch.arange(L, device="cuda") < lengths[:, None])[:, None]


def _first_order(a, b):
    """h_t = a_t h_{t-1} + b_t along the last axis, from zero, by doubling."""
    a, b, step = a.clone(), b.clone(), 1
    while step < b.shape[-1]:
        add = a[..., step:] * b[..., :-step]
        b[..., step:] += add
        mul = a[..., step:] * a[..., :-step]
        a[..., step:] = mul
        step *= 2
    return b


def _conv_parts(s):
    """The windows of the padded input [B, D, L, K], the pre-activation and the padded input."""
    x, w = s["x"].float(), s["w"].float()
    B, D, L = x.shape
    K = w.shape[1]
    if s["lengths"] is not None:
        x = x * _valid(s["lengths"], L)
    head = x.new_zeros(B, D, K - 1) if s["state"] is None else s["state"].float()
    full = torch.cat([head, x], 2)
    windows = full.unfold(2, K, 1)
    return windows, (windows * w[:, None]).sum(3) + s["bias"][:, None], full


def _plain(s):
    op = s["op"]
    if op == "conv_fwd":
        _, u, full = _conv_parts(s)
        y, (B, D, L), K1 = _silu(u), u.shape, s["w"].shape[1] - 1
        n = torch.full((B,), L, device="cuda") if s["lengths"] is None else s["lengths"].long()
        if s["lengths"] is not None:
            y = y * _valid(s["lengths"], L)
        last = (n[:, None] + torch.arange(K1, device="cuda"))[:, None].expand(B, D, K1)
        return {"y": y.to(s["x"].dtype), "state": full.gather(2, last).to(s["x"].dtype)}
    if op == "conv_bwd":
        windows, u, _ = _conv_parts(s)
        K, L = windows.shape[3], u.shape[2]
        sig = 1 / (1 + torch.exp(-u))
        du = s["dy"].float() * (sig * (1 + u * (1 - sig)))
        if s["lengths"] is not None:
            du = du * _valid(s["lengths"], L)
        later = torch.cat([du, du.new_zeros(du.shape[0], du.shape[1], K - 1)], 2).unfold(2, K, 1)
        dx = (later * s["w"].float().flip(1)[:, None]).sum(3)
        if s["lengths"] is not None:
            dx = dx * _valid(s["lengths"], L)
        return {"dx": dx.to(s["x"].dtype), "dw": (windows * du[..., None]).sum((0, 2)), "db": du.sum((0, 2))}
    if op == "conv_step":
        full = torch.cat([s["state"].float(), s["x"].float()[:, :, None]], 2)
        y = _silu((full * s["w"].float()).sum(2) + s["bias"])
        return {"y": y.to(s["x"].dtype), "state": full[:, :, 1:].to(s["x"].dtype)}
    if op == "i8":
        return {"y": _plain_i8(s)}
    D = s["A"].shape[0]
    x, G = s["x"].float(), s["B"].shape[1]
    raw = s["delta"].float()
    raw = raw + (s["bias"] if op == "scan_step" else s["bias"][:, None])
    dt = _softplus(raw)
    Bd, Cd = (s[k].float().repeat_interleave(D // G, 1) for k in "BC")
    z = None if s["z"] is None else s["z"].float()
    if op == "scan_step":
        h = torch.exp(dt[..., None] * s["A"]) * s["state"] + (dt * x)[..., None] * Bd
        y = (Cd * h).sum(2) + s["D"] * x
        return {"y": (y if z is None else y * _silu(z)).to(s["x"].dtype), "state": h}
    L = x.shape[2]
    if op == "scan_fwd" and s["lengths"] is not None:
        inside = _valid(s["lengths"], L)
        dt, x = dt * inside, x * inside
    a = torch.exp(dt[:, :, None] * s["A"][:, :, None])
    b = (dt * x)[:, :, None] * Bd
    if op == "scan_fwd" and s["state"] is not None:
        b[..., 0] += a[..., 0] * s["state"]
    h = _first_order(a, b)
    v = (Cd * h).sum(2) + s["D"][:, None] * x
    y = v if z is None else v * _silu(z)
    if op == "scan_fwd":
        if s["lengths"] is not None:
            y = y * inside
        return {"y": y.to(s["x"].dtype), "state": h[..., -1].clone()}
    dy, out = s["dy"].float(), s["x"].dtype
    e = dy if z is None else dy * _silu(z)
    later = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], 3)
    g = _first_order(later.flip(3), (Cd * e[:, :, None]).flip(3)).flip(3)
    del later
    gB = (g * Bd).sum(2)
    gah = g * (h - b)
    ddt = (gah * s["A"][:, :, None]).sum(2) + gB * x
    # the derivative of softplus is the logistic function
    ddelta = ddt / (1 + torch.exp(-raw))
    group = lambda t: t.unflatten(1, (G, D // G)).sum(2)  # noqa: E731
    r = {"y": y.to(out), "dx": (dt * gB + s["D"][:, None] * e).to(out), "ddelta": ddelta.to(out),
         "dA": (gah * dt[:, :, None]).sum((0, 3)), "dB": group(g * (dt * x)[:, :, None]),
         "dC": group(h * e[:, :, None]), "dD": (e * x).sum((0, 2)), "ddelta_bias": ddelta.sum((0, 2))}
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        r["dz"] = (dy * v * (sig * (1 + z * (1 - sig)))).to(out)
    return r


def _plain_i8(s):
    B, L, C, O = s["dims"]
    x = s["x"].double()                       # 64 bits: the roundings to 8 bits and sums past 2^24
    top = x.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(x * 127 / top), 0.0)
    total = q @ s["wq"][:, :C].double().t()
    y = total.float() * (top / 127).float() * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["channel_major"]:
        y = y.unflatten(0, (B, L)).transpose(1, 2).contiguous()
    return y.to(s["dtype"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    op = c["op"]
    if op in ("conv_fwd", "conv_bwd"):
        n = c["B"] * c["D"] * c["L"]
        small = c["D"] * c["K"] * e + c["D"] * 4
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + small, "flops": n * (2 * c["K"] + 5)}
        return {"bytes": 3 * n * e + small + c["D"] * (c["K"] + 1) * 4, "flops": n * (6 * c["K"] + 12)}
    if op == "conv_step":
        n = c["B"] * c["D"]
        return {"bytes": 2 * n * c["K"] * e + c["D"] * (c["K"] * e + 4), "flops": n * (2 * c["K"] + 5)}
    if op == "i8":
        t = c["B"] * c["L"]
        return {"bytes": t * c["C"] * e + c["O"] * c["C"] + t * c["O"] * e + c["O"] * 8,
                "flops": 2 * t * c["C"] * c["O"]}
    gate = int(c["gate"])
    if op == "scan_step":
        n = c["B"] * c["D"]
        return {"bytes": n * (3 + gate) * e + 2 * n * c["N"] * 4 + 2 * c["B"] * c["G"] * c["N"] * e
                + c["D"] * (c["N"] + 2) * 4, "flops": n * (7 * c["N"] + 12)}
    n, bc = c["B"] * c["D"] * c["L"], 2 * c["B"] * c["G"] * c["N"] * c["L"]
    par = c["D"] * (c["N"] + 2) * 4
    fwd = {"bytes": n * (3 + gate) * e + bc * e + par + c["B"] * c["D"] * c["N"] * 4, "flops": n * (7 * c["N"] + 12)}
    if op == "scan_fwd":
        return fwd
    # forward, then the backward pass over x, delta, z, dy, B, C and the gradients
    return {"bytes": fwd["bytes"] + n * (5 + 2 * gate) * e + bc * (e + 4) + 2 * par,
            "flops": fwd["flops"] + n * (20 * c["N"] + 30)}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "i8":
        B, L, C, O = s["dims"]
        x = s["x"].to(torch.float64)
        top = x.abs().max(dim=1).values
        scaled = x / torch.where(top == 0, torch.ones_like(top), top)[:, None] * 127
        near = scaled.floor()
        part = scaled - near
        # halves go to the even neighbour; a quotient within 1e-12 of one is one
        half = (part - 0.5).abs() < 1e-12
        q = torch.where(half, 2 * torch.round((near + 0.5) / 2), near + (part > 0.5))
        y = torch.zeros(B * L, O, dtype=torch.float64, device="cuda")
        for k in range(0, C, 1024):
            m = min(C, k + 1024)
            y += q[:, k:m] @ s["wq"][:, k:m].to(torch.float64).t()
        y = y * (top / 127)[:, None] * s["ws"].to(torch.float64)[None]
        if s["bias"] is not None:
            y = y + s["bias"].to(torch.float64)[None]
        return {"y": y.view(B, L, O).permute(0, 2, 1).contiguous() if s["channel_major"] else y}
    f = {k: (v.to(torch.float64) if torch.is_tensor(v) and v.is_floating_point() else v) for k, v in s.items()}
    sigma = torch.sigmoid
    if op == "conv_step":
        B, D, K = case["B"], case["D"], case["K"]
        u = f["bias"][None] + f["w"][None, :, K - 1] * f["x"]
        for k in range(K - 1):
            u = u + f["w"][None, :, k] * f["state"][:, :, k]
        state = torch.cat([f["state"], f["x"][:, :, None]], 2)[:, :, 1:]
        return {"y": u * sigma(u), "state": state}
    if op in ("conv_fwd", "conv_bwd"):
        B, D, L, K = (case[k] for k in "BDLK")
        n = [L] * B if s["lengths"] is None else s["lengths"].tolist()
        y, state = torch.zeros(B, D, L, dtype=torch.float64, device="cuda"), []
        dx, dw, db = torch.zeros_like(y), torch.zeros_like(f["w"]), torch.zeros_like(f["bias"])
        for b in range(B):
            head = torch.zeros(D, K - 1, dtype=torch.float64, device="cuda") if s["state"] is None else f["state"][b]
            full = torch.cat([head, f["x"][b, :, :n[b]]], 1)
            state.append(full[:, n[b]:])
            if n[b] == 0:
                continue
            u = f["bias"][:, None] + sum(f["w"][:, k:k + 1] * full[:, k:k + n[b]] for k in range(K))
            y[b, :, :n[b]] = u * sigma(u)
            if op == "conv_bwd":
                du = f["dy"][b, :, :n[b]] * (sigma(u) + u * sigma(u) * sigma(-u))
                dfull = torch.zeros_like(full)
                for k in range(K):
                    dfull[:, k:k + n[b]] += f["w"][:, k:k + 1] * du
                    dw[:, k] += (du * full[:, k:k + n[b]]).sum(1)
                db += du.sum(1)
                dx[b, :, :n[b]] = dfull[:, K - 1:]
        return {"y": y, "state": torch.stack(state)} if op == "conv_fwd" else {"dx": dx, "dw": dw, "db": db}
    B, D, N, G = (case[k] for k in "BDNG")
    A, P = f["A"], D // G
    if op == "scan_step":
        v = f["delta"] + f["bias"]
        dt = torch.logaddexp(v, torch.zeros_like(v))
        h = f["state"] * (dt[:, :, None] * A).exp()
        for g in range(G):
            h[:, g * P:(g + 1) * P] += (dt * f["x"])[:, g * P:(g + 1) * P, None] * f["B"][:, g, None]
        y = torch.cat([(h[:, g * P:(g + 1) * P] * f["C"][:, g, None]).sum(2) for g in range(G)], 1) + f["D"] * f["x"]
        return {"y": y * f["z"] * sigma(f["z"]) if s["z"] is not None else y, "state": h}
    L = case["L"]
    if 3 * B * D * L * N * 8 > 24e9:
        return None
    v = f["delta"] + f["bias"][:, None]
    dt = torch.logaddexp(v, torch.zeros_like(v))
    x, dtx = f["x"], dt * f["x"]
    lengths = s.get("lengths")
    h0 = torch.zeros(B, D, N, dtype=torch.float64, device="cuda") if s.get("state") is None else f["state"]
    hs, h = torch.empty(L + 1, B, G, P, N, dtype=torch.float64, device="cuda"), h0.reshape(B, G, P, N)
    hs[0] = h
    part = lambda t, i: t[:, :, i].reshape(B, G, P, 1)  # noqa: E731
    Ag = A.reshape(G, P, N)
    y = torch.zeros(B, D, L, dtype=torch.float64, device="cuda")
    for t in range(L):
        new = h * (part(dt, t) * Ag).exp() + part(dtx, t) * f["B"][:, :, None, :, t]
        h = new if lengths is None else torch.where((lengths > t).view(B, 1, 1, 1), new, h)
        hs[t + 1] = h
        y[:, :, t] = (h * f["C"][:, :, None, :, t]).sum(3).reshape(B, D)
    y += f["D"][:, None] * x
    gate = f["z"] * sigma(f["z"]) if s["z"] is not None else torch.ones_like(x)
    if op == "scan_fwd":
        out = y * gate
        for b in range(B if lengths is not None else 0):
            out[b, :, int(lengths[b]):] = 0
        return {"y": out, "state": h.reshape(B, D, N)}
    e = f["dy"] * gate
    r = {"y": y * gate}
    g = torch.zeros(B, G, P, N, dtype=torch.float64, device="cuda")
    gB, gA = torch.empty_like(x), torch.empty_like(x)
    dA = torch.zeros(G, P, N, dtype=torch.float64, device="cuda")
    dB = torch.empty(B, G, N, L, dtype=torch.float64, device="cuda")
    dC = torch.empty_like(dB)
    for t in reversed(range(L)):
        g = g + part(e, t) * f["C"][:, :, None, :, t]
        dC[..., t] = (hs[t + 1] * part(e, t)).sum(2)
        dB[..., t] = (g * part(dtx, t)).sum(2)
        gB[:, :, t] = (g * f["B"][:, :, None, :, t]).sum(3).reshape(B, D)
        decay = (part(dt, t) * Ag).exp()
        g = g * decay                         # now the gradient of the state before this step
        gA[:, :, t] = (g * hs[t] * Ag).sum(3).reshape(B, D)
        dA += (g * hs[t] * part(dt, t)).sum(0)
    ddelta = (gA + gB * x) * sigma(v)
    r.update(dx=dt * gB + f["D"][:, None] * e, ddelta=ddelta, dA=dA.reshape(D, N), dB=dB, dC=dC,
             dD=(e * x).sum((0, 2)), ddelta_bias=ddelta.sum((0, 2)))
    if s["z"] is not None:
        r["dz"] = f["dy"] * y * (sigma(f["z"]) + f["z"] * sigma(f["z"]) * sigma(-f["z"]))
    return r
