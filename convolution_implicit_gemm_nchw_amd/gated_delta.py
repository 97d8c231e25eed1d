"""A gated delta block: layer norm, 8-bit floating-point products, the causal convolution and the gated delta rule
put together as a language model uses them.

For hidden values h [B, L, M] (tokens first), Hk key heads of P channels and Hv value heads of V:

  n       = layer_norm(h)
  x, a, b = parts of W_in n                       [B, 2 Hk P + Hv V, L], [B, Hv, L] twice
  q, k, v = parts of silu(causal_conv1d(x))       short depthwise convolution over time
  g       = -exp(decay) softplus(a + a0)          log decays;   beta = logistic(b)
  y       = gated_delta(q, k, v, g, beta)         queries and keys normalised
  out     = h + W_out layer_norm(y)               [B, L, M]

``prompt`` and ``token`` serve with both products in 8-bit floating point (weights quantised once);
``train_step`` runs the projections as 1x1 convolutions in bf16 and returns every gradient.
"""
import math

import torch

import convolution_implicit_gemm_nchw_amd as mc
from convolution_implicit_gemm_nchw_amd.state_space import _conv, _conv_data, _conv_filter


class GatedDeltaBlock:
    def __init__(self, M, Hk, Hv, P, V, K=4, device="cuda", seed=0):
        self.M, self.Hk, self.Hv, self.P, self.V, self.K = M, Hk, Hv, P, V, K
        self.parts = [Hk * P, Hk * P, Hv * V]
        self.D = D = sum(self.parts)
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(device)
        bf = torch.bfloat16
        self.w_in = normal(D + 2 * Hv, M, scale=M ** -0.5).to(bf)
        self.w_out = normal(M, Hv * V, scale=(Hv * V) ** -0.5).to(bf)
        self.w_conv = normal(D, K, scale=K ** -0.5).to(bf)
        self.b_conv = normal(D, scale=0.1)
        self.w_norm, self.b_norm = 1 + normal(M, scale=0.1), normal(M, scale=0.1)
        self.w_mix = 1 + normal(Hv * V, scale=0.1)
        self.decay = (torch.rand(Hv, generator=gen) * math.log(100.0) - math.log(100.0)).to(device)
        self.a0 = normal(Hv, scale=0.5)
        self.q_in, self.q_out = mc.quantize_f8(self.w_in), mc.quantize_f8(self.w_out)

    def _gates(self, xab):
        """(x, g, beta) of W_in n [B, D + 2 Hv, ...]."""
        a, b = xab[:, self.D:self.D + self.Hv].float(), xab[:, self.D + self.Hv:].float()
        tail = (1,) * (a.dim() - 2)
        g = -torch.exp(self.decay).view(-1, *tail) * torch.nn.functional.softplus(a + self.a0.view(-1, *tail))
        return xab[:, :self.D], g, torch.sigmoid(b)

    # -------------------------------------------------------------- serving

    def states(self, B):
        """(convolution state, delta state) of B sequences that have not begun."""
        dev = self.w_norm.device
        return (torch.zeros(B, self.D, self.K - 1, dtype=torch.bfloat16, device=dev),
                torch.zeros(B, self.Hv, self.P, self.V, device=dev))

    def prompt(self, h, states, lengths=None):
        """out [B, L, M] of right-padded prompts h [B, L, M] that continue from `states`, which are updated.
        `lengths` int32 [B]; what lies past a length does not count."""
        B, L, _ = h.shape
        n = mc.layer_norm_fwd(h, self.w_norm, self.b_norm, lengths=lengths)
        xab = mc.matmul_f8(*mc.quantize_f8(n), *self.q_in, out_dtype=h.dtype, length=L)
        x, g, beta = self._gates(xab)
        conv, delta = states
        conv_out, delta_out = torch.empty_like(conv), torch.empty_like(delta)
        u = mc.causal_conv1d_fwd(x, self.w_conv, bias=self.b_conv, silu=True, initial_state=conv, lengths=lengths,
                                 final_state=conv_out)
        y = mc.gated_delta_fwd(*u.split(self.parts, 1), g, beta, key_heads=self.Hk, l2norm=True, initial_state=delta,
                               lengths=lengths, final_state=delta_out)
        conv.copy_(conv_out)
        delta.copy_(delta_out)
        y = mc.layer_norm_fwd(y, self.w_mix, channel_major=True, lengths=lengths)
        q, s = mc.quantize_f8(y, channel_major=True)
        return h + mc.matmul_f8(q, s, *self.q_out, out_dtype=h.dtype).view(B, L, self.M)

    def token(self, h, states, slots=None):
        """out [B, M] of one token per sequence, h [B, M]; `states` are updated in place.  With slots (int32
        [B]) the states are a pool and sequence b owns states slots[b]."""
        n = mc.layer_norm_fwd(h, self.w_norm, self.b_norm)
        x, g, beta = self._gates(mc.matmul_f8(*mc.quantize_f8(n), *self.q_in, out_dtype=h.dtype))
        u = mc.causal_conv1d_step(x, states[0], self.w_conv, bias=self.b_conv, silu=True, slots=slots)
        y = mc.gated_delta_step(*u.split(self.parts, 1), g, beta, states[1], key_heads=self.Hk, l2norm=True, slots=slots)
        y = mc.layer_norm_fwd(y, self.w_mix)
        return h + mc.matmul_f8(*mc.quantize_f8(y), *self.q_out, out_dtype=h.dtype)

    # -------------------------------------------------------------- training

    def train_step(self, h, dout):
        """(out, gradients) for h [B, M, L] (channel-major, bf16) and the gradient dout [B, M, L] of
        out [B, M, L]; gradients by name, of the weights in fp32 and of h in bf16."""
        stats = mc.layer_norm_stats(h, channel_major=True)
        n = mc.layer_norm_fwd(h, self.w_norm, self.b_norm, channel_major=True, stats=stats)
        xab = _conv(n, self.w_in)
        x, g, beta = self._gates(xab)
        u = mc.causal_conv1d_fwd(x, self.w_conv, bias=self.b_conv, silu=True)
        q, k, v = u.split(self.parts, 1)
        rule = dict(key_heads=self.Hk, l2norm=True)
        states = mc.gated_delta_states(q, v, g, key_heads=self.Hk)
        y = mc.gated_delta_fwd(q, k, v, g, beta, states=states, **rule)
        mix_stats = mc.layer_norm_stats(y, channel_major=True)
        mixed = mc.layer_norm_fwd(y, self.w_mix, channel_major=True, stats=mix_stats)
        out = h + _conv(mixed, self.w_out)

        dy, dw_mix, _ = mc.layer_norm_bwd(y, _conv_data(dout, self.w_out), mix_stats, self.w_mix, channel_major=True)
        du, dxab = torch.empty_like(u), torch.empty_like(xab)          # their parts are written in place
        dq, dk, dv = du.split(self.parts, 1)
        d = mc.gated_delta_bwd(q, k, v, g, beta, dy, states, dq=dq, dk=dk, dv=dv, **rule)
        # g = -exp(decay) softplus(s), s = a + a0;  beta = logistic(b)
        s = xab[:, self.D:self.D + self.Hv].float() + self.a0.view(-1, 1)
        ds = -torch.exp(self.decay).view(-1, 1) * torch.sigmoid(s) * d["dg"]
        dxab[:, self.D:self.D + self.Hv] = ds
        dxab[:, self.D + self.Hv:] = d["dbeta"] * beta * (1 - beta)
        _, dw_conv, db_conv = mc.causal_conv1d_bwd(x, self.w_conv, du, bias=self.b_conv, silu=True, dx=dxab[:, :self.D])
        dh, dw_norm, db_norm = mc.layer_norm_bwd(h, _conv_data(dxab, self.w_in), stats, self.w_norm, self.b_norm,
                                                 channel_major=True)
        return out, {"h": dh + dout, "w_in": _conv_filter(n, dxab), "w_out": _conv_filter(mixed, dout), "w_conv": dw_conv,
                     "b_conv": db_conv, "w_norm": dw_norm, "b_norm": db_norm, "w_mix": dw_mix,
                     "decay": (g * d["dg"]).sum((0, 2)), "a0": ds.sum((0, 2))}


def main():
    """Serves two ragged prompts and some tokens, then takes one training step."""
    block = GatedDeltaBlock(M=256, Hk=2, Hv=4, P=64, V=64)
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
