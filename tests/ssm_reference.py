"""Plain 64-bit forms of the state-space operators (numpy, one time step after the other) with,
beside each value, a bound on what fp32 arithmetic may lose on it.

The bounds follow the formulas: every fp32 operation rounds by at most U = 2^-24 of its result, the
exponential, logistic and softplus functions by a few U, and each bound adds these up over the path of
the value, with magnitudes (sums of absolute values) where terms may cancel.  A sum of n terms in any
order is off by at most n U of the sum of magnitudes.  Kernels that reassociate round a comparable
number of times; SLACK = 2 covers that.
"""
import numpy as np

U = 2.0 ** -24
SLACK = 2.0
OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}     # half a step of the stored type, relative


def logistic(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return v * logistic(v)


def dsilu(v):
    s = logistic(v)
    return s * (1 + v * (1 - s))


# ------------------------------------------------------------------ causal convolution

def conv(x, w, bias=None, act=False, h0=None, lengths=None, dy=None, dfs=None):
    """{name: (value, bound)} of the forward pass, or of the backward pass when dy is given."""
    B, D, L = x.shape
    K = w.shape[1]
    n = np.full(B, L) if lengths is None else np.clip(lengths, 0, L)
    bias = np.zeros(D) if bias is None else bias
    r = {k: np.zeros(s) for k, s in (("y", (B, D, L)), ("dx", (B, D, L)), ("fs", (B, D, K - 1)), ("dw", (D, K)),
                                     ("db", D), ("dh0", (B, D, K - 1)))}
    m = {k: np.zeros_like(v) for k, v in r.items()}
    count = {"dw": 1, "db": 1}
    for b in range(B):
        head = np.zeros((D, K - 1)) if h0 is None else h0[b]
        full = np.concatenate([head, x[b, :, :n[b]]], 1)
        r["fs"][b] = full[:, n[b]:]
        dfull, mfull = np.zeros_like(full), np.zeros_like(full)
        for t in range(n[b]):
            win = full[:, t:t + K]
            u, mu = (win * w).sum(1) + bias, (np.abs(win * w)).sum(1) + np.abs(bias)
            # a change of u changes silu(u) by at most 1.1 and its derivative by at most 0.5 of it
            r["y"][b, :, t] = silu(u) if act else u
            m["y"][b, :, t] = (K + 1) * mu * (1.1 if act else 1) + 12 * np.abs(u)
            if dy is not None:
                g = dy[b, :, t]
                du = g * dsilu(u) if act else g
                mdu = np.abs(g) * ((K + 1) * mu * 0.5 + 12 * (1 + np.abs(u))) if act else 0 * g
                dfull[:, t:t + K] += w * du[:, None]
                mfull[:, t:t + K] += np.abs(w) * (mdu + (K + 1) * np.abs(du))[:, None]
                r["dw"] += win * du[:, None]
                m["dw"] += np.abs(win) * (mdu + n.sum() * np.abs(du))[:, None]
                r["db"] += du
                m["db"] += mdu + n.sum() * np.abs(du)
        if dfs is not None:
            dfull[:, n[b]:] += dfs[b]
            mfull[:, n[b]:] += np.abs(dfull[:, n[b]:])
        r["dh0"][b], m["dh0"][b] = dfull[:, :K - 1], mfull[:, :K - 1]
        r["dx"][b, :, :n[b]], m["dx"][b, :, :n[b]] = dfull[:, K - 1:], mfull[:, K - 1:]
    return {k: (r[k], SLACK * U * m[k]) for k in r}


# ------------------------------------------------------------------ selective scan

def scan(x, delta, A, Bm, Cm, D=None, z=None, bias=None, sp=True, h0=None, lengths=None, dy=None, dfs=None):
    """{name: (value, bound)}: y, fs, and with dy the gradients."""
    nb, nd, L = x.shape
    N, G = A.shape[1], Bm.shape[1]
    n = np.full(nb, L) if lengths is None else np.clip(lengths, 0, L)
    inside = np.arange(L)[None, :] < n[:, None]
    x, delta = np.where(inside[:, None], x, 0), np.where(inside[:, None], delta, 0)
    Bm, Cm = (np.where(inside[:, None, None], v, 0) for v in (Bm, Cm))
    z = None if z is None else np.where(inside[:, None], z, 0)
    D = np.zeros(nd) if D is None else D
    raw = delta + (0 if bias is None else bias[:, None])
    dt = np.where(inside[:, None], softplus(raw) if sp else raw, 0)
    rdt = (10 + np.abs(raw)) * U if sp else U * np.abs(raw) / np.maximum(np.abs(dt), 1e-300) + U
    rep = lambda v: np.repeat(v, nd // G, axis=1)  # noqa: E731
    Be, Ce = rep(Bm), rep(Cm)                                    # [nb, nd, N, L]
    a = np.exp(dt[:, :, None] * A[None, :, :, None])
    ra = np.abs(dt[:, :, None] * A[None, :, :, None]) * (rdt[:, :, None] + 3 * U) + 3 * U
    bt = (dt * x)[:, :, None] * Be
    rb = rdt[:, :, None] + 4 * U
    H, mH, eH = (np.zeros((L + 1, nb, nd, N)) for _ in range(3))
    H[0] = 0 if h0 is None else h0
    mH[0] = np.abs(H[0])
    for t in range(L):
        at = a[..., t]
        H[t + 1] = at * H[t] + bt[..., t]
        mH[t + 1] = at * mH[t] + np.abs(bt[..., t])
        step = inside[:, None, None, t]
        eH[t + 1] = at * eH[t] + step * ((ra[..., t] + 3 * U) * at * mH[t] + rb[..., t] * np.abs(bt[..., t]))
    Hs, mHs, eHs = (np.moveaxis(v[1:], 0, 3) for v in (H, mH, eH))   # [nb, nd, N, L]
    v = (Ce * Hs).sum(2) + D[:, None] * x
    mv = (np.abs(Ce) * mHs).sum(2) + np.abs(D[:, None] * x)
    ev = (np.abs(Ce) * eHs).sum(2) + (N + 3) * U * mv
    gate, egate = (1.0, 0.0) if z is None else (silu(z), 12 * U * np.abs(silu(z)))
    r = {"y": (np.where(inside[:, None], v * gate, 0), np.abs(gate) * ev + egate * mv + U * np.abs(v * gate)),
         "fs": (H[L], eH[L])}
    if dy is not None:
        dy = np.where(inside[:, None], dy, 0)
        e = dy * gate
        ee = 14 * U * np.abs(e)
        g, mg, eg = (np.zeros((nb, nd, N, L)) for _ in range(3))
        Gn = np.zeros((nb, nd, N)) if dfs is None else dfs.astype(float)
        mGn, eGn = np.abs(Gn), np.zeros_like(Gn)
        for t in reversed(range(L)):
            ce = Ce[..., t] * e[:, :, None, t]
            step = inside[:, None, None, t]
            g[..., t] = ce + Gn
            mg[..., t] = np.abs(ce) + mGn
            eg[..., t] = eGn + np.abs(Ce[..., t]) * ee[:, :, None, t] + step * 2 * U * mg[..., t]
            Gn, mGn = a[..., t] * g[..., t], a[..., t] * mg[..., t]
            eGn = a[..., t] * eg[..., t] + step * (ra[..., t] + 3 * U) * mGn
        P = nd // G
        group = lambda q: q.reshape(nb, G, P, N, L).sum(2)  # noqa: E731
        e4, ma4 = np.abs(e[:, :, None]), np.abs((dt * x)[:, :, None])
        r["dC"] = (group(e[:, :, None] * Hs), group(e4 * eHs + ((P + 3) * U * e4 + ee[:, :, None]) * mHs))
        r["dB"] = (group(g * (dt * x)[:, :, None]), group(ma4 * eg + ((P + 3) * U + rdt[:, :, None]) * ma4 * mg))
        gB = (g * Be).sum(2)
        mgB = (mg * np.abs(Be)).sum(2)
        egB = (eg * np.abs(Be)).sum(2) + (N + 3) * U * mgB
        r["dx"] = (dt * gB + D[:, None] * e, dt * egB + (rdt + 3 * U) * dt * mgB + np.abs(D[:, None]) * (ee + 3 * U * np.abs(e)))
        hp, mhp, ehp = (np.moveaxis(q[:L], 0, 3) for q in (H, mH, eH))
        ah, mah = a * hp, a * mhp
        eah = a * ehp + (ra + 3 * U) * mah
        w, mw = g * ah, mg * mah
        ew = eg * mah + mg * eah + 3 * U * mw
        A4 = np.abs(A[None, :, :, None])
        ddt = (w * A[None, :, :, None]).sum(2) + x * gB
        mddt = (mw * A4).sum(2) + np.abs(x) * mgB
        eddt = (ew * A4).sum(2) + np.abs(x) * egB + (N + 4) * U * mddt
        sg = logistic(raw) if sp else np.ones_like(raw)
        dd = np.where(inside[:, None], ddt * sg, 0)
        edd = np.where(inside[:, None], sg * eddt + 14 * U * sg * mddt, 0)
        r["ddelta"] = (dd, edd)
        terms = n.sum()
        r["ddelta_bias"] = (dd.sum((0, 2)), (edd + terms * U * np.where(inside[:, None], sg * mddt, 0)).sum((0, 2)))
        r["dD"] = ((e * x).sum((0, 2)), (np.abs(x) * (ee + (terms + 2) * U * np.abs(e))).sum((0, 2)))
        d4 = dt[:, :, None]
        r["dA"] = ((w * d4).sum((0, 3)), (np.abs(d4) * (ew + ((terms + 3) * U + rdt[:, :, None]) * mw)).sum((0, 3)))
        r["dh0"] = (Gn, eGn)
        if z is not None:
            s = dsilu(z)
            r["dz"] = (dy * v * s, np.abs(dy) * (np.abs(s) * ev + 14 * U * (1 + np.abs(z)) * mv))
    return {k: (val, SLACK * err) for k, (val, err) in r.items()}


# ------------------------------------------------------------------ 8-bit products

def quantize(x):
    """q and scale of tokens x [T, C]; the quotient is rounded as the exact one would be."""
    top = np.abs(x).max(1)
    ok = np.isfinite(top)
    with np.errstate(all="ignore"):
        q = np.where((ok & (top > 0))[:, None], np.rint(x * 127.0 / top[:, None]), 0)
    scale = np.where(ok, top.astype(np.float32) / np.float32(127), np.float32(np.nan)).astype(np.float32)
    return np.nan_to_num(q).astype(np.int8), scale


def within(got, ref, bound, kind, extra=0.0):
    """Largest (|got - ref|) / (bound + half a step of the stored type); fails where got is not finite."""
    got = np.asarray(got, np.float64)
    # the smallest normal numbers are the limit below which the stored type and the exponential flush
    room = bound + OUT[kind] * (np.abs(ref) + bound) + 1e-37 + extra
    assert got.shape == np.shape(ref), (got.shape, np.shape(ref))
    return float(np.max(np.abs(got - ref) / room)) if got.size and np.isfinite(got).all() else (0.0 if got.size == 0 else np.inf)
