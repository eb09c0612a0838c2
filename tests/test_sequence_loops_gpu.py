"""The sequence operators' long loops against the 64-bit references of seq_ref.py:
rows, strips and rounds enough that every buffer is used again and every
prefetch is taken, with tails. Sizes follow the kernels' own splitting: a workgroup
of the layer norm takes 4 rows or more one after another, a strip of the convolution
9 rows or more, a workgroup of the scan 5 rounds or more, and a part of a sequence 3."""
from __future__ import annotations

import pytest

import conv2d_batchnorm_silu_amd as tg
import seq_ref as R
from gpu_cases import note
from test_sequence_gpu import Rand, ScanCase, _bounds, _cat, f64, up

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64


# ---- layer norm

@pytest.mark.parametrize("rows,C,dtype,residual", [
    (25003, 48, F16, True),     # a wave for each row, 2048 workgroups of 4
    (26000, 63, F32, False),    # the same by single elements
    (6200, 1024, F16, True),    # 128 threads
    (3500, 2048, BF16, True),   # 256 threads
    (3300, 1001, BF16, False),  # 256 threads, 4 single elements each
    (1700, 4096, BF16, True),   # 512 threads
    (820, 8192, F16, True),     # 1024 threads
    (810, 16390, F32, True)], ids=str)  # rows too long to be held
def test_norm_many_rows(rows, C, dtype, residual, monkeypatch):
    note("norm %d x %d %s" % (rows, C, dtype))
    # At most 16 values in a thread's chain, or C/1024 where rows are too long to be held.
    monkeypatch.setattr(R, "norm_sums", lambda C: max(16, C // 1024 + 1) + 22)
    r = Rand(rows + C)
    x = r(rows, C, dtype=dtype, shift=3.0)
    res = r(rows, C, dtype=dtype, scale=2.0) if residual else None
    gamma, beta = r(C, shift=1.0, scale=0.3), r(C)
    s = x if res is None else (x.float() + res.float()).to(dtype)
    y, s2, mean, rstd = tg.layer_norm_train(up(x), up(gamma), up(beta), 1e-5, up(res))
    want = R.norm(s.double(), gamma.double(), beta.double(), 1e-5)
    assert torch.equal(s2.cpu(), s)
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        R.check(name, got, *want[name])
    dy = r(rows, C, dtype=dtype)
    dsum = r(rows, C, dtype=dtype) if residual else None
    got = tg.layer_norm_backward(up(dy), s2, up(gamma), mean, rstd, up(dsum))
    want = R.norm_grads(dy.double(), s.double(), gamma.double(), 1e-5, f64(dsum))
    for name, g in zip(("dx", "dgamma", "dbeta"), got):
        R.check(name, g, *want[name])


# ---- short causal convolution

@pytest.mark.parametrize("lengths,packed,D,K,dtype", [
    ([10001, 10001], False, 260, 4, BF16), ([19000, 1, 0, 3, 996, 17], True, 260, 4, F16),
    ([40000], False, 130, 3, F32), ([7, 30000, 9993], True, 67, 8, F16)], ids=str)
def test_conv_long_strips(lengths, packed, D, K, dtype):
    note("conv %s D=%d K=%d" % (lengths, D, K))
    r, T, S, b = Rand(D + K), sum(lengths), len(lengths), _bounds(lengths)
    x, w, bias, init = r(T, D, dtype=dtype), r(K, D, scale=0.5), r(D), r(S, K - 1, D, dtype=dtype)
    dy, dlast = r(T, D, dtype=dtype), r(S, K - 1, D, dtype=dtype)
    shape = (T, D) if packed else (S, T // S, D)
    off = torch.tensor(b, dtype=torch.int32).cuda() if packed else None
    args = (up(x.reshape(shape)), up(w), up(bias), "silu", up(init), off)
    y, state = tg.causal_conv(*args, return_state=True)
    dx, dw, db, d0 = tg.causal_conv_backward(up(dy.reshape(shape)), *args, dstate=up(dlast))
    fwd, grads = [], []
    for i in range(S):
        cut = lambda t: t[b[i]:b[i + 1]].double()  # noqa: E731
        v, last, _ = R.conv(cut(x), w.double(), bias.double(), True, init[i].double())
        fwd.append(v)
        assert torch.equal(state[i].cpu().double(), last)
        grads.append(R.conv_grads(cut(dy), cut(x), w.double(), bias.double(), True, init[i].double(), dlast[i].double()))
    R.check("y", y.reshape(T, D), *_cat(fwd))
    R.check("dx", dx.reshape(T, D), *_cat([g["dx"] for g in grads]))
    R.check("dinit", d0, torch.stack([g["dinit"][0] for g in grads]), torch.stack([g["dinit"][1] for g in grads]))
    for name, got in (("dw", dw), ("dbias", db)):
        v = sum(g[name][0] for g in grads)
        mag = sum(g[name][0].abs() + g[name][1] / R.E for g in grads)
        R.check(name, got, v, sum(g[name][1] for g in grads) + 2 * S * R.E * mag)


# ---- selective scan

SCAN = [
    # Rounds: sequences not cut into parts, for each number of states a lane holds.
    ([700] * 4, False, 4, "f32"), ([700] * 4, False, 8, "bf16"), ([700] * 4, False, 16, "f32"),
    ([700, 3, 0, 1290, 1, 64, 129, 333], True, 16, "bf16"), ([350] * 4, False, 24, "f32"),
    ([0, 350, 1, 65, 420, 7], True, 32, "f16"), ([90] * 8, False, 64, "f32"), ([45] * 16, False, 128, "f32"),
    # Parts of three rounds or more.
    ([6157], False, 16, "bf16"), ([6157], False, 8, "f32"), ([3, 6150], True, 3, "f32"), ([3083], False, 24, "f32"),
    ([1543], False, 64, "f32"), ([1543], False, 128, "f32"),
]


@pytest.mark.parametrize("lengths,packed,N,dtype", SCAN, ids=str)
def test_scan_many_rounds(lengths, packed, N, dtype):
    """16 groups of 32 channels; the first and the last group, which share nothing
    with the others, against the reference."""
    note("scan %s N=%d %s" % (lengths, N, dtype))
    G, W = 16, 32
    c = ScanCase((lengths, packed, G * W, N, G, dtype, True, True, True, 0))
    dy, dstate = c.r(*c.x.shape, dtype=c.dtype), c.r(c.S, c.D, N)
    y, state, saved = tg.selective_scan_train(*c.args(), return_state=True, **c.more())
    got = tg.selective_scan_backward(c.dev(dy), *c.args(), saved, dstate=up(dstate), **c.more())
    for g in (0, G - 1):
        at = slice(g * W, (g + 1) * W)
        fwd, grads = [], []
        cut = lambda t: t[c.b[i]:c.b[i + 1], at].double()  # noqa: E731
        bc = lambda t: t[c.b[i]:c.b[i + 1], g:g + 1].double()  # noqa: E731
        for i in range(c.S):
            ref = (cut(c.x), cut(c.dt), c.A[at].double(), bc(c.B), bc(c.C), c.skip[at].double(), cut(c.z),
                   c.bias[at].double(), True, c.init[i, at].double())
            v, h, _ = R.scan(*ref)
            fwd.append((v, h))
            grads.append(R.scan_grads(cut(dy), *ref, dfinal=dstate[i, at].double()))
        R.check("y", y.reshape(c.T, c.D)[:, at], *_cat([v for v, _ in fwd]))
        R.check("state", state[:, at], torch.stack([h[0] for _, h in fwd]), torch.stack([h[1] for _, h in fwd]))
        for name in ("dx", "ddt", "dz"):
            R.check(name, getattr(got, name).reshape(c.T, c.D)[:, at], *_cat([r[name] for r in grads]))
        for name in ("dB", "dC"):
            R.check(name, getattr(got, name).reshape(c.T, G, N)[:, g:g + 1], *_cat([r[name] for r in grads]))
        for name, key in (("dA", "dA"), ("dD", "dD"), ("ddt_bias", "dbias")):
            v, e = sum(r[key][0] for r in grads), sum(r[key][1] for r in grads)
            R.check(name, getattr(got, name)[at], v, e + (c.S + 1) * R.E * sum(r[key][0].abs() for r in grads))
        # The hardware's exponential is zero below 2^-126, which seq_ref.py does not count: a
        # token's decay (here at most 1) is off by that, and what it multiplies is at most
        # the sum of all that the adjoint takes up.
        flush = []
        for i in range(c.S):
            most = dstate[i, at].double().abs() + ((cut(dy) * cut(c.z)).abs()[..., None] * bc(c.C).abs()).sum(0)
            flush.append(most * (c.b[i + 1] - c.b[i]) * 2.0 ** -126)
        R.check("dinit", got.dinitial_state[:, at], torch.stack([r["dinit"][0] for r in grads]),
                torch.stack([r["dinit"][1] for r in grads]) + torch.stack(flush))
