"""A gated delta rule block on this library's operators: an example of how they are
used together, for prompts, single tokens and gradients.

    s = h + residual;  n = layer_norm(s)
    q, k, v = silu(causal_conv(in_proj(n)));  z = z_proj(n);  dt, beta = gate_proj(n)
    o = gated_delta_rule(q, k, v, dt, A, beta)
    out = out_proj(group_norm(o, heads) * silu(z))

The residual stream is s; the next block (or the head) adds ``out`` to it. The
projections are those of ssm_block.py, so activations are fp16. The backward pass
covers the norms, the convolution and the delta rule with fixed projections, whose
input gradients are 1x1 convolutions with the filter transposed.

``python -m conv2d_batchnorm_silu_amd.delta_block`` takes the tokens of a group-normed
strided 3x3 stem convolution through two blocks, as one prompt and as a shorter
prompt followed by single tokens, and one backward pass.
"""
from __future__ import annotations

import math

import torch

from . import sequence as seq
from .binding import ConvBnSilu
from .ssm_block import F16, F32, Projection


class DeltaBlock:
    """C channels in the residual stream, HK key heads of K and HV value heads of V
    columns, ``taps`` of the convolution."""

    def __init__(self, C, HK=2, HV=4, K=32, V=32, taps=4, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).to(device)

        self.C, self.HK, self.HV, self.K, self.V, self.taps = C, HK, HV, K, V, taps
        self.D = 2 * HK * K + HV * V
        self.gamma, self.beta = 1 + rand(C, scale=0.1), rand(C, scale=0.1)
        self.in_proj = Projection(rand(self.D, C, scale=C ** -0.5))
        self.z_proj = Projection(rand(HV * V, C, scale=C ** -0.5))
        self.gate_proj = Projection(rand(2 * HV, C, scale=C ** -0.5))
        self.w, self.b = rand(taps, self.D, scale=taps ** -0.5), rand(self.D, scale=0.1)
        self.norm = 1 + rand(HV * V, scale=0.1)
        self.out_proj = Projection(rand(C, HV * V, scale=(HV * V) ** -0.5))
        # Decay rates from 1 to 16, step sizes from 0.001 to 0.1 at dt = 0.
        self.A = -(1 + 15 * torch.rand(HV, generator=g)).to(device)
        step = torch.exp(torch.rand(HV, generator=g) * math.log(100.0) + math.log(0.001))
        self.dt_bias = (step + torch.log(-torch.expm1(-step))).to(device)

    def new_state(self, num_slots):
        """Room for the states of num_slots sequences: (conv rows, delta rule states)."""
        dev = self.A.device
        return (torch.zeros(num_slots, self.taps - 1, self.D, dtype=F16, device=dev),
                torch.zeros(num_slots, self.HV, self.K, self.V, dtype=F32, device=dev))

    def _rule_inputs(self, x, gates):
        kw, heads = self.HK * self.K, (self.HK, self.K)
        return (x[..., :kw].unflatten(-1, heads), x[..., kw:2 * kw].unflatten(-1, heads),
                x[..., 2 * kw:].unflatten(-1, (self.HV, self.V)), gates[..., :self.HV], self.A,
                gates[..., self.HV:])

    def _head_norm(self, o, z):
        """Over each head of each token, with the gate."""
        flat = o.flatten(-2)
        y = seq.group_norm(flat.view(-1, flat.shape[-1]), self.HV, self.norm, act="none",
                           z=z.view(-1, z.shape[-1]))
        return y.view(flat.shape)

    def prompt(self, h, residual, state=None, offsets=None):
        """h, residual [S, L, C] (or packed [T, C] with offsets) -> (out, s, state)."""
        n, s = seq.layer_norm(h, self.gamma, self.beta, residual=residual)
        conv0, rule0 = state or (None, None)
        x, conv1 = seq.causal_conv(self.in_proj(n), self.w, self.b, initial_state=conv0,
                                   offsets=offsets, return_state=True)
        o, rule1 = seq.gated_delta_rule(*self._rule_inputs(x, self.gate_proj(n)),
                                        dt_bias=self.dt_bias, initial_state=rule0,
                                        offsets=offsets, return_state=True)
        return self.out_proj(self._head_norm(o, self.z_proj(n))), s, (conv1, rule1)

    def step(self, h, residual, state, slots=None):
        """One token of each of n sequences, h, residual [n, C] -> (out, s); the
        states (new_state, or a prompt's) move on in place."""
        n, s = seq.layer_norm(h, self.gamma, self.beta, residual=residual)
        x = seq.causal_conv_step(self.in_proj(n), state[0], self.w, self.b, slots=slots)
        o = seq.gated_delta_rule_step(*self._rule_inputs(x, self.gate_proj(n)), state[1],
                                      dt_bias=self.dt_bias, slots=slots)
        return self.out_proj(self._head_norm(o, self.z_proj(n))), s

    def forward_backward(self, h, residual, dout, ds):
        """Outputs and gradients of a training step with fixed projections, from
        the gradients of ``out`` and of s: (out, s, dh, {name: gradient})."""
        n, s, mean, rstd = seq.layer_norm_train(h, self.gamma, self.beta, residual=residual)
        x0, z, gates = self.in_proj(n), self.z_proj(n), self.gate_proj(n)
        x = seq.causal_conv(x0, self.w, self.b)
        args = self._rule_inputs(x, gates)
        o, saved = seq.gated_delta_rule_train(*args, dt_bias=self.dt_bias)
        rows = lambda t: t.reshape(-1, self.HV * self.V)  # noqa: E731
        y, m, r = seq.group_norm_train(rows(o), self.HV, self.norm, act="none", z=rows(z))
        out = self.out_proj(y.view(z.shape))

        g = seq.group_norm_backward(rows(self.out_proj.input_gradient(dout)), rows(o), self.HV,
                                    self.norm, m, r, act="none", z=rows(z))
        d = seq.gated_delta_rule_backward(g.dx.view(o.shape), *args, saved, dt_bias=self.dt_bias)
        dx = torch.cat([d.dq.flatten(-2), d.dk.flatten(-2), d.dv.flatten(-2)], -1)
        dx0, dw, db, _ = seq.causal_conv_backward(dx, x0, self.w, self.b)
        dn = (self.in_proj.input_gradient(dx0) + self.z_proj.input_gradient(g.dz.view(z.shape))
              + self.gate_proj.input_gradient(torch.cat([d.ddt, d.dbeta], -1)))
        dh, dgamma, dbeta = seq.layer_norm_backward(dn, s, self.gamma, mean, rstd, dsum=ds)
        return out, s, dh, dict(gamma=dgamma, beta=dbeta, w=dw, b=db, norm=g.dgamma, A=d.dA,
                                dt_bias=d.ddt_bias)


def main():
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(1)
    S, side, C = 2, 64, 64
    # Tokens: a 3x3 stride-2 stem over RGB images and its group norm, one token for
    # each pixel row by row.
    stem = ConvBnSilu(S, side, side, 3, C, 3, stride=2, pad=1)
    x = torch.randn(S, side, side, 3, generator=g).to(dev, F16)
    w = (torch.randn(C, 3, 3, 3, generator=g) * 27 ** -0.5).to(dev, F16)
    one, zero = torch.ones(C, device=dev), torch.zeros(C, device=dev)
    tokens = seq.group_norm(stem.run(x, w, one, zero), 8, one).view(S, -1, C)
    L, tail = tokens.shape[1], 8
    blocks = [DeltaBlock(C, seed=i, device=dev) for i in range(2)]

    def prompt(t):
        h, res, states = t, torch.zeros_like(t), []
        for b in blocks:
            h, res, state = b.prompt(h, res)
            states.append(state)
        return h + res, states

    whole, _ = prompt(tokens)
    first, states = prompt(tokens[:, :L - tail].contiguous())
    ys = [first]
    for t in range(L - tail, L):
        h = tokens[:, t].contiguous()
        res = torch.zeros_like(h)
        for b, state in zip(blocks, states):
            h, res = b.step(h, res, state)
        ys.append((h + res).unsqueeze(1))
    off = float((torch.cat(ys, 1).float() - whole.float()).abs().max())
    print("%d images, %d tokens of %d channels, 2 blocks: prompt and %d steps against one prompt: "
          "largest difference %.2g of %.2g" % (S, L, C, tail, off, float(whole.abs().max())))
    out, s, dh, grads = blocks[0].forward_backward(tokens, torch.zeros_like(tokens),
                                                   torch.randn_like(tokens), torch.zeros_like(tokens))
    print("gradients:", ", ".join("%s %.3g" % (k, float(v.norm())) for k, v in
                                  dict(grads, h=dh.float()).items()))


if __name__ == "__main__":
    main()
