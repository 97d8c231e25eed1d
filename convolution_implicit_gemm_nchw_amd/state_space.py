"""A state-space block: the operators of this package put together as a language model uses them.

For hidden values h [B, L, M] (tokens first) with width D, N states and a step-size rank R:

  x, z   = halves of W_in h                       [B, 2D, L]
  u      = silu(causal_conv1d(x))                 short depthwise convolution over time
  dt     = W_dt (W_r u),  B, C = halves of W_bc u
  y      = selective_scan(u, dt, A, B, C) * silu(z)
  out    = W_out y                                [B, L, M]

``prompt`` and ``token`` serve with the two large projections in 8-bit integers (weights quantised once,
by channel, activations per token); ``train_step`` runs the projections as 1x1 convolutions in bf16
and returns every gradient.  The small projections are 1x1 convolutions throughout.
"""
import math

import torch

import convolution_implicit_gemm_nchw_amd as mc


class StateSpaceBlock:
    def __init__(self, M, D, N=16, K=4, R=None, device="cuda", seed=0):
        R = R or max(1, D // 16)
        self.M, self.D, self.N, self.K, self.R = M, D, N, K, R
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(device)
        bf = torch.bfloat16
        self.w_in = normal(2 * D, M, scale=M ** -0.5).to(bf)
        self.w_out = normal(M, D, scale=D ** -0.5).to(bf)
        self.w_conv = normal(D, K, scale=K ** -0.5).to(bf)
        self.b_conv = normal(D, scale=0.1)
        self.w_r = normal(R, D, scale=D ** -0.5).to(bf)
        self.w_bc = normal(2 * N, D, scale=D ** -0.5).to(bf)
        self.w_dt = normal(D, R, scale=R ** -0.5).to(bf)
        self.A = -torch.arange(1, N + 1, device=device, dtype=torch.float32).repeat(D, 1)
        self.skip = torch.ones(D, device=device)
        step = torch.exp(torch.rand(D, generator=gen) * math.log(100.0) + math.log(1e-3)).to(device)
        self.b_dt = step + torch.log(-torch.expm1(-step))       # softplus(b_dt) = step
        self.q_in, self.q_out = mc.quantize_tokens(self.w_in), mc.quantize_tokens(self.w_out)

    # -------------------------------------------------------------- serving

    def states(self, B):
        """(convolution state, scan state) of B sequences that have not begun."""
        dev = self.A.device
        return (torch.zeros(B, self.D, self.K - 1, dtype=torch.bfloat16, device=dev),
                torch.zeros(B, self.D, self.N, device=dev))

    def prompt(self, h, states, lengths=None):
        """out [B, L, M] of right-padded prompts h [B, L, M] that continue from `states`, which are updated.
        `lengths` int32 [B]; what lies past a length does not count."""
        B, L, _ = h.shape
        q, s = mc.quantize_tokens(h)
        xz = mc.matmul_i8(q, s, *self.q_in, out_dtype=h.dtype, length=L)
        x, z = xz[:, :self.D], xz[:, self.D:]
        conv, scan = states
        conv_out, scan_out = torch.empty_like(conv), torch.empty_like(scan)
        u = mc.causal_conv1d_fwd(x, self.w_conv, bias=self.b_conv, silu=True, initial_state=conv, lengths=lengths,
                                 final_state=conv_out)
        delta, Bm, Cm = self._project(u)
        y = mc.selective_scan_fwd(u, delta, self.A, Bm, Cm, D=self.skip, z=z, delta_bias=self.b_dt, softplus=True,
                                  initial_state=scan, lengths=lengths, final_state=scan_out)
        conv.copy_(conv_out)
        scan.copy_(scan_out)
        q, s = mc.quantize_tokens(y, channel_major=True)
        return mc.matmul_i8(q, s, *self.q_out, out_dtype=h.dtype).view(B, L, self.M)

    def token(self, h, states, slots=None):
        """out [B, M] of one token per sequence, h [B, M]; `states` are updated in place.  With slots (int32
        [B]) the states are a pool and sequence b owns states slots[b]."""
        q, s = mc.quantize_tokens(h)
        xz = mc.matmul_i8(q, s, *self.q_in, out_dtype=h.dtype)
        x, z = xz[:, :self.D], xz[:, self.D:]
        u = mc.causal_conv1d_step(x, states[0], self.w_conv, bias=self.b_conv, silu=True, slots=slots)
        delta, Bm, Cm = self._project(u[:, :, None])
        y = mc.selective_scan_step(u, delta[:, :, 0], self.A, Bm[..., 0], Cm[..., 0], states[1], D=self.skip, z=z,
                                   delta_bias=self.b_dt, softplus=True, slots=slots)
        q, s = mc.quantize_tokens(y)
        return mc.matmul_i8(q, s, *self.q_out, out_dtype=h.dtype)

    def _project(self, u):
        """delta [B, D, L] and B, C [B, 1, N, L] of u [B, D, L]."""
        low = _conv(u, self.w_r)
        bc = _conv(u, self.w_bc)
        return _conv(low, self.w_dt), bc[:, None, :self.N], bc[:, None, self.N:]

    # -------------------------------------------------------------- training

    def train_step(self, h, dout):
        """(out, gradients) for h [B, M, L] (channel-major, bf16) and the gradient dout [B, M, L] of
        out [B, M, L]; gradients by name, of the weights in fp32 and of h in bf16."""
        xz = _conv(h, self.w_in)
        x, z = xz[:, :self.D], xz[:, self.D:]
        u = mc.causal_conv1d_fwd(x, self.w_conv, bias=self.b_conv, silu=True)
        low, bc = _conv(u, self.w_r), _conv(u, self.w_bc)
        delta = _conv(low, self.w_dt)
        Bm, Cm = bc[:, None, :self.N], bc[:, None, self.N:]
        scan = dict(D=self.skip, z=z, delta_bias=self.b_dt, softplus=True)
        states = mc.selective_scan_states(u, self.A)
        y = mc.selective_scan_fwd(u, delta, self.A, Bm, Cm, states=states, **scan)
        out = _conv(y, self.w_out)

        dy = _conv_data(dout, self.w_out)
        dxz = torch.empty_like(xz)                # its halves are written in place
        g = mc.selective_scan_bwd(u, delta, self.A, Bm, Cm, dy, states, dz=dxz[:, self.D:], **scan)
        dbc = torch.cat([g["dB"], g["dC"]], 2)[:, 0].to(h.dtype)
        dlow = _conv_data(g["ddelta"], self.w_dt)
        # u reaches the scan directly and through both projections: one sum
        du = _conv_data(dbc, self.w_bc, into=_conv_data(dlow, self.w_r, into=g["dx"]))
        _, dw_conv, db_conv = mc.causal_conv1d_bwd(x, self.w_conv, du, bias=self.b_conv, silu=True,
                                                   dx=dxz[:, :self.D])
        return out, {"h": _conv_data(dxz, self.w_in), "w_in": _conv_filter(h, dxz), "w_out": _conv_filter(y, dout),
                     "w_conv": dw_conv, "b_conv": db_conv, "w_r": _conv_filter(u, dlow), "w_bc": _conv_filter(u, dbc),
                     "w_dt": _conv_filter(low, g["ddelta"]), "A": g["dA"], "skip": g["dD"],
                     "b_dt": g["ddelta_bias"]}


def _conv(x, w):
    """W x over the channels: a 1x1 convolution of [B, C, L] in bf16."""
    return mc.conv2d_fwd_ex(x[:, :, None], w[:, :, None, None], out_dtype=x.dtype)[:, :, 0]


def _conv_data(dy, w, into=None):
    """The gradient of _conv in x; added to `into` when given."""
    shape = (1, dy.shape[2])
    if into is None:
        return mc.conv2d_bwd_data_ex(dy[:, :, None], w[:, :, None, None], shape, out_dtype=dy.dtype)[:, :, 0]
    mc.conv2d_bwd_data_ex(dy[:, :, None], w[:, :, None, None], shape, beta=1.0, dx=into[:, :, None])
    return into


def _conv_filter(x, dy):
    return mc.conv2d_bwd_filter(x[:, :, None], dy[:, :, None], (1, 1))[:, :, 0, 0]


def main():
    """Serves two ragged prompts and some tokens, then takes one training step."""
    block = StateSpaceBlock(M=256, D=512)
    gen = torch.Generator().manual_seed(1)
    h = torch.randn(2, 40, 256, generator=gen).to("cuda", torch.bfloat16)
    states = block.states(2)
    out = block.prompt(h, states, lengths=torch.tensor([40, 23], dtype=torch.int32, device="cuda"))
    last = out[[0, 1], [39, 22]]
    for _ in range(4):
        last = block.token(last, states)
    print("4 tokens after prompts of 40 and 23:", tuple(last.shape), "norms", last.float().norm(dim=1).tolist())
    x = h.transpose(1, 2).contiguous()
    _, grads = block.train_step(x, torch.ones_like(x))
    for name, g in grads.items():
        print(f"  d{name}: {tuple(g.shape)} norm {float(g.float().norm()):.4g}")


if __name__ == "__main__":
    main()
