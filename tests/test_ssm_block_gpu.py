"""The state space block of ssm_block.py: prompts against prompts in pieces and
single tokens, packed against dense, and its gradients against autograd of the
same formulas in 64 bits.

The block's tensors are fp16, rounded at 9 places between input and output, so
two ways through it may differ by that many roundings of 2^-11, each
carried on by maps of about unit gain: 9 * 2^-11 * 4 (four times: a sum over
128 channels of roundings in one direction or the other reaches a few standard
deviations) of the largest value, which is what TOL stands for; the gradients
pass through 9 more."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 9 * 2.0 ** -11 * 4


def _near(a, b, tol=TOL):
    a, b = a.double().cpu(), b.double().cpu()
    assert a.shape == b.shape
    assert float((a - b).abs().max()) <= tol * float(b.abs().max())


def _block(C=64, D=128):
    from conv2d_batchnorm_silu_amd.ssm_block import SsmBlock
    return SsmBlock(C, D, seed=3)


def _tokens(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).half().cuda()


def test_prompt_in_pieces_and_steps():
    b = _block()
    h, res = _tokens(3, 70, 64), _tokens(3, 70, 64, seed=1)
    out, s, _ = b.prompt(h, res)
    o1, s1, state = b.prompt(h[:, :33].contiguous(), res[:, :33].contiguous())
    o2, s2, state = b.prompt(h[:, 33:65].contiguous(), res[:, 33:65].contiguous(), state)
    outs, sums = [o1, o2], [s1, s2]
    # The sequences move to a larger cache, in another order.
    cache = b.new_state(5)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    for c, t in zip(cache, state):
        c[slots.long()] = t
    for t in range(65, 70):
        o, r = b.step(h[:, t].contiguous(), res[:, t].contiguous(), cache, slots)
        outs.append(o.unsqueeze(1))
        sums.append(r.unsqueeze(1))
    _near(torch.cat(outs, 1), out)
    assert torch.equal(torch.cat(sums, 1), s)


def test_packed_equals_dense():
    b = _block()
    h, res = _tokens(3, 20, 64), _tokens(3, 20, 64, seed=1)
    out, s, state = b.prompt(h, res)
    off = torch.arange(0, 61, 20, dtype=torch.int32, device="cuda")
    po, ps, pstate = b.prompt(h.view(60, 64), res.view(60, 64), offsets=off)
    assert torch.equal(po.view_as(out), out) and torch.equal(ps.view_as(s), s)
    assert all(torch.equal(a, c) for a, c in zip(state, pstate))


def test_gradients():
    b = _block()
    S, L = 2, 24
    h, res = _tokens(S, L, 64), _tokens(S, L, 64, seed=1)
    dout, ds = _tokens(S, L, 64, seed=2), _tokens(S, L, 64, seed=3)
    out, s, dh, grads = b.forward_backward(h, res, dout, ds)

    p = {k: getattr(b, k).double().cpu().requires_grad_() for k in grads}
    lin = {k: getattr(b, k).w.double().cpu() for k in
           ("in_proj", "low_proj", "dt_proj", "b_proj", "c_proj", "out_proj")}
    hd = h.double().cpu().requires_grad_()
    sd = hd + res.double().cpu()
    var, mean = torch.var_mean(sd, -1, unbiased=False, keepdim=True)
    n = (sd - mean) / torch.sqrt(var + 1e-5) * p["gamma"] + p["beta"]
    xz = n @ lin["in_proj"].t()
    x0, z = xz[..., :128], xz[..., 128:]
    pad = torch.cat([torch.zeros(S, 3, 128, dtype=torch.float64), x0], 1)
    x = torch.nn.functional.silu(p["b"] + sum(p["w"][k] * pad[:, k:k + L] for k in range(4)))
    d = torch.nn.functional.softplus((x @ lin["low_proj"].t()) @ lin["dt_proj"].t() + p["dt_bias"])
    B, C = x @ lin["b_proj"].t(), x @ lin["c_proj"].t()
    state, ys = torch.zeros(S, 128, 16, dtype=torch.float64), []
    for t in range(L):
        state = torch.exp(d[:, t, :, None] * p["A"]) * state + (d * x)[:, t, :, None] * B[:, t, None]
        ys.append((state * C[:, t, None]).sum(-1))
    y = (torch.stack(ys, 1) + p["skip"] * x) * torch.nn.functional.silu(z)
    od = y @ lin["out_proj"].t()
    _near(out, od.detach())
    loss = (od * dout.double().cpu()).sum() + (sd * ds.double().cpu()).sum()
    want = torch.autograd.grad(loss, [hd] + [p[k] for k in grads])
    _near(dh, want[0], 2 * TOL)
    for (name, got), w in zip(grads.items(), want[1:]):
        _near(got, w, 2 * TOL)


def test_example_runs(capsys):
    from conv2d_batchnorm_silu_amd import ssm_block
    ssm_block.main()
    assert "gradients" in capsys.readouterr().out
