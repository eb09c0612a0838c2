"""A state space block on this library's operators: an example of how they are
used together, for prompts, single tokens and gradients.

    s = h + residual;  n = layer_norm(s)
    x, z = in_proj(n);  x = silu(causal_conv(x))
    r, B, C = low_proj(x), b_proj(x), c_proj(x);  dt = dt_proj(r)
    out = out_proj(selective_scan(x, dt, A, B, C, D, z))

The residual stream is s; the next block (or the head) adds ``out`` to it. The
projections are 1x1 convolutions over tokens with the epilogue's identity
activation (ConvBnSilu), so activations are fp16. The backward pass covers the
norm, the convolution and the scan with fixed projections, whose input
gradients are 1x1 convolutions with the filter transposed.

``python -m conv2d_batchnorm_silu_amd.ssm_block`` takes the tokens of a strided
3x3 stem convolution through two blocks, as one prompt and as a shorter
prompt followed by single tokens, and one backward pass.
"""
from __future__ import annotations

import math

import torch

from . import sequence as seq
from .binding import ConvBnSilu

F16, F32 = torch.float16, torch.float32


class Projection:
    """A linear map of tokens, w [C_out, C_in], as a 1x1 convolution."""

    def __init__(self, w):
        self.w = w.to(F16).contiguous()
        out, inn = self.w.shape
        self.scale = torch.ones(out, dtype=F32, device=w.device)
        self.bias = torch.zeros(out, dtype=F32, device=w.device)
        self._plans = {}
        self._transposed = None

    def __call__(self, x):
        out, inn = self.w.shape
        rows = x.numel() // inn
        plan = self._plans.get(rows)
        if plan is None:
            plan = self._plans[rows] = ConvBnSilu(1, 1, rows, inn, out, 1, act="none")
        y = plan.run(x.contiguous().view(1, 1, rows, inn), self.w.view(out, 1, 1, inn), self.scale,
                     self.bias)
        return y.view(x.shape[:-1] + (out,))

    def input_gradient(self, dy):
        if self._transposed is None:
            self._transposed = Projection(self.w.t())
        return self._transposed(dy)


class SsmBlock:
    """C channels in the residual stream, D inside, N states, K taps."""

    def __init__(self, C, D, N=16, K=4, rank=None, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rank = rank or max(8, -(-D // 16) // 8 * 8)

        def rand(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).to(device)

        self.C, self.D, self.N, self.K = C, D, N, K
        self.gamma, self.beta = 1 + rand(C, scale=0.1), rand(C, scale=0.1)
        self.in_proj = Projection(rand(2 * D, C, scale=C ** -0.5))
        self.w, self.b = rand(K, D, scale=K ** -0.5), rand(D, scale=0.1)
        self.low_proj = Projection(rand(rank, D, scale=D ** -0.5))
        self.dt_proj = Projection(rand(D, rank, scale=rank ** -0.5))
        self.b_proj = Projection(rand(N, D, scale=D ** -0.5))
        self.c_proj = Projection(rand(N, D, scale=D ** -0.5))
        self.out_proj = Projection(rand(C, D, scale=D ** -0.5))
        # Decay rates 1 .. N, step sizes from 0.001 to 0.1 at dt = 0.
        self.A = -torch.arange(1, N + 1, dtype=F32).repeat(D, 1).to(device)
        step = torch.exp(torch.rand(D, generator=g) * math.log(100.0) + math.log(0.001))
        self.dt_bias = (step + torch.log(-torch.expm1(-step))).to(device)
        self.skip = torch.ones(D, device=device)

    def new_state(self, num_slots):
        """Room for the states of num_slots sequences: (conv rows, scan states)."""
        dev = self.A.device
        return (torch.zeros(num_slots, self.K - 1, self.D, dtype=F16, device=dev),
                torch.zeros(num_slots, self.D, self.N, dtype=F32, device=dev))

    def _scan_inputs(self, x):
        group = (1, self.N)
        return (x, self.dt_proj(self.low_proj(x)), self.A, self.b_proj(x).unflatten(-1, group),
                self.c_proj(x).unflatten(-1, group))

    def prompt(self, h, residual, state=None, offsets=None):
        """h, residual [S, L, C] (or packed [T, C] with offsets) -> (out, s, state)."""
        n, s = seq.layer_norm(h, self.gamma, self.beta, residual=residual)
        xz = self.in_proj(n)
        conv0, scan0 = state or (None, None)
        x, conv1 = seq.causal_conv(xz[..., :self.D], self.w, self.b, initial_state=conv0,
                                   offsets=offsets, return_state=True)
        y, scan1 = seq.selective_scan(*self._scan_inputs(x), D=self.skip, z=xz[..., self.D:],
                                      dt_bias=self.dt_bias, initial_state=scan0, offsets=offsets,
                                      return_state=True)
        return self.out_proj(y), s, (conv1, scan1)

    def step(self, h, residual, state, slots=None):
        """One token of each of n sequences, h, residual [n, C] -> (out, s); the
        states (new_state, or a prompt's) move on in place."""
        n, s = seq.layer_norm(h, self.gamma, self.beta, residual=residual)
        xz = self.in_proj(n)
        x = seq.causal_conv_step(xz[..., :self.D], state[0], self.w, self.b, slots=slots)
        y = seq.selective_scan_step(*self._scan_inputs(x), state[1], D=self.skip,
                                    z=xz[..., self.D:], dt_bias=self.dt_bias, slots=slots)
        return self.out_proj(y), s

    def forward_backward(self, h, residual, dout, ds):
        """Outputs and gradients of a training step with fixed projections, from
        the gradients of ``out`` and of s: (out, s, dh, {name: gradient})."""
        n, s, mean, rstd = seq.layer_norm_train(h, self.gamma, self.beta, residual=residual)
        xz = self.in_proj(n)
        x0, z = xz[..., :self.D], xz[..., self.D:]
        x = seq.causal_conv(x0, self.w, self.b)
        args = self._scan_inputs(x)
        more = dict(D=self.skip, z=z, dt_bias=self.dt_bias)
        y, saved = seq.selective_scan_train(*args, **more)
        out = self.out_proj(y)

        d = seq.selective_scan_backward(self.out_proj.input_gradient(dout), *args, saved, **more)
        dx = (d.dx + self.b_proj.input_gradient(d.dB.flatten(-2))
              + self.c_proj.input_gradient(d.dC.flatten(-2))
              + self.low_proj.input_gradient(self.dt_proj.input_gradient(d.ddt)))
        dx0, dw, db, _ = seq.causal_conv_backward(dx, x0, self.w, self.b)
        dn = self.in_proj.input_gradient(torch.cat([dx0, d.dz], -1))
        dh, dgamma, dbeta = seq.layer_norm_backward(dn, s, self.gamma, mean, rstd, dsum=ds)
        return out, s, dh, dict(gamma=dgamma, beta=dbeta, w=dw, b=db, A=d.dA, skip=d.dD,
                                dt_bias=d.ddt_bias)


def main():
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(1)
    S, side, C, D = 2, 64, 64, 128
    # Tokens: a 3x3 stride-2 stem over RGB images, then one token for each pixel row by row.
    stem = ConvBnSilu(S, side, side, 3, C, 3, stride=2, pad=1)
    x = torch.randn(S, side, side, 3, generator=g).to(dev, F16)
    w = (torch.randn(C, 3, 3, 3, generator=g) * 27 ** -0.5).to(dev, F16)
    one, zero = torch.ones(C, device=dev), torch.zeros(C, device=dev)
    tokens = stem.run(x, w, one, zero).view(S, -1, C)
    L, tail = tokens.shape[1], 8
    blocks = [SsmBlock(C, D, seed=i, device=dev) for i in range(2)]

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
