"""The C entry points of the gated delta rule and of group norm on the host: every
argument error is found before a launch (no call here reaches the GPU), sizes are
what the header says, and the Python layer refuses tensors that are not on a
device."""
from __future__ import annotations

import ctypes

import pytest
import torch

import conv2d_batchnorm_silu_amd as tg
from conv2d_batchnorm_silu_amd import sequence as S
from test_sequence_abi import ALIGN, BF16, F16, F32, F8, INVAL, OK, P, UNSUP, WS, _rows

BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    return S._lib()


def _delta(**kw):
    """Two value heads of 16 columns on one key head of 8, four rows."""
    a = S._DeltaArgs(S._Seqs(kw.pop("seqs", 1), kw.pop("rows", 4), kw.pop("offsets", 0)), 1, 2, 8, 16, F16)
    a.q = a.k = _rows(seq=32, row=8)
    a.v = a.y = _rows(seq=128, row=32)
    a.dt = a.beta = _rows(seq=8, row=2)
    a.A, a.scale = P, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD = [(dict(seqs=0), INVAL), (dict(rows=-1), INVAL), (dict(seqs=3), INVAL), (dict(HK=0), INVAL), (dict(HV=0), INVAL),
       (dict(HK=2, HV=3), INVAL), (dict(K=0), INVAL), (dict(V=0), INVAL), (dict(K=257), UNSUP), (dict(dtype=F8), UNSUP),
       (dict(V=1 << 20), UNSUP), (dict(rows=1 << 30, offsets=P), UNSUP), (dict(offsets=P + 2), ALIGN), (dict(A=0), INVAL),
       (dict(A=P + 2), ALIGN), (dict(dt_bias=P + 1), ALIGN), (dict(initial=P + 2), ALIGN), (dict(final=P + 2), ALIGN),
       (dict(q=_rows(0)), INVAL), (dict(k=_rows(0)), INVAL), (dict(v=_rows(0)), INVAL), (dict(dt=_rows(0)), INVAL),
       (dict(beta=_rows(0)), INVAL), (dict(q=_rows(P + 1, 32)), ALIGN), (dict(k=_rows(row=-8)), INVAL),
       (dict(v=_rows(seq=1 << 30, row=1 << 25)), UNSUP)]


@pytest.mark.parametrize("bad,want", BAD + [(dict(y=_rows(0)), INVAL), (dict(y=_rows(seq=128, row=31)), INVAL)])
def test_delta_arguments(lib, bad, want):
    assert lib.tg_gated_delta_rule(ctypes.byref(_delta(**bad)), P, BIG, 0, 0, 0) == want


def _sizes(lib, a):
    v = [ctypes.c_size_t() for _ in range(3)]
    assert lib.tg_gated_delta_rule_sizes(ctypes.byref(a), *(ctypes.byref(t) for t in v)) == OK
    return [t.value for t in v]


def test_delta_workspaces(lib):
    a = _delta()
    work, saved, back = _sizes(lib, a)
    assert work > 0 and saved >= 2 * (8 + 4) * 16 * 4 and back > saved
    call = lib.tg_gated_delta_rule
    assert call(ctypes.byref(a), P, work - 1, 0, 0, 0) == WS and call(ctypes.byref(a), 0, 0, 0, 0, 0) == WS
    assert call(ctypes.byref(a), P, work, P, saved - 1, 0) == WS and call(ctypes.byref(a), P + 4, work, 0, 0, 0) == ALIGN
    # A packed batch has room for every split of its rows into sequences.
    assert _sizes(lib, _delta(seqs=9, rows=1000, offsets=P))[1] >= _sizes(lib, _delta(rows=1000))[1]
    for dt in (F16, BF16, F32):
        for K in (8, 100, 200):
            assert all(n > 0 for n in _sizes(lib, _delta(K=K, dtype=dt)))


def _grads(**kw):
    g = S._DeltaGrads()
    full = dict(dy=_rows(seq=128, row=32), dq=_rows(seq=32, row=8), dk=_rows(seq=32, row=8), dv=_rows(seq=128, row=32),
                ddt=_rows(seq=8, row=2), dbeta=_rows(seq=8, row=2), dA=P)
    for k, v in dict(full, **kw).items():
        setattr(g, k, v)
    return g


@pytest.mark.parametrize("bad,want", BAD)
def test_delta_backward_arguments(lib, bad, want):
    g = _grads()
    assert lib.tg_gated_delta_rule_backward(ctypes.byref(_delta(**bad)), ctypes.byref(g), P, BIG, P, BIG, 0) == want


def test_delta_backward_gradients(lib):
    _, saved, back = _sizes(lib, _delta())

    def call(sv=P, svn=saved, ws=P, wsn=back, **kw):
        g = _grads(**kw)
        return lib.tg_gated_delta_rule_backward(ctypes.byref(_delta()), ctypes.byref(g), sv, svn, ws, wsn, 0)
    for name in ("dy", "dq", "dk", "dv", "ddt", "dbeta"):
        assert call(**{name: _rows(0)}) == INVAL, name
    assert call(dA=0) == INVAL and call(dq=_rows(seq=32, row=7)) == INVAL
    assert call(sv=0) == WS and call(svn=saved - 1) == WS and call(ws=0) == WS and call(wsn=back - 1) == WS
    assert call(dinitial=P + 2) == ALIGN and call(dk=_rows(P + 1, 32, 8)) == ALIGN and call(ws=P + 8) == ALIGN


def test_delta_step_arguments(lib):
    def call(state=P, num=4, slots=0, **kw):
        a = _delta(**dict(dict(seqs=4, rows=4), **kw))
        return lib.tg_gated_delta_rule_step(ctypes.byref(a), state, num, slots, 0)
    assert call(state=0) == INVAL and call(num=3) == INVAL and call(rows=8) == INVAL and call(offsets=P) == INVAL
    assert call(num=-1) == INVAL and call(state=P + 2) == ALIGN and call(slots=P + 1) == ALIGN
    assert call(K=300) == UNSUP and call(y=_rows(0)) == INVAL and call(A=0) == INVAL
    assert call(seqs=0, rows=0) == OK


def test_delta_more_than_a_launch_holds(lib):
    n = 1 << 23
    a = _delta(seqs=n, rows=n)
    assert lib.tg_gated_delta_rule(ctypes.byref(a), P, BIG, 0, 0, 0) == UNSUP
    assert lib.tg_gated_delta_rule_step(ctypes.byref(a), P, n, 0, 0) == UNSUP
    a = _delta(rows=(1 << 30) - 1)
    assert lib.tg_gated_delta_rule(ctypes.byref(a), P, BIG, 0, 0, 0) == UNSUP


def _group(**kw):
    a = S._GroupNormArgs(2, 5, 8, 2, F16, 0, 1e-5, P, 8, 0, 0, P, P, P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_GROUP = [(dict(N=-1), INVAL), (dict(L=0), INVAL), (dict(C=0), INVAL), (dict(G=0), INVAL), (dict(G=3), INVAL),
             (dict(eps=-1.0), INVAL), (dict(eps=float("nan")), INVAL), (dict(dtype=F8), UNSUP), (dict(act=1), UNSUP),
             (dict(C=1 << 21), UNSUP), (dict(C=10000, G=5000), UNSUP), (dict(L=1 << 30), UNSUP), (dict(N=1 << 30), UNSUP),
             (dict(N=1 << 20, L=1 << 20), UNSUP), (dict(gamma=0), INVAL), (dict(x=0), INVAL), (dict(x_stride=7), INVAL),
             (dict(z=P, z_stride=-8), INVAL), (dict(x=P + 1), ALIGN), (dict(gamma=P + 2), ALIGN), (dict(beta=P + 1), ALIGN),
             (dict(N=1 << 25, L=1, C=1024, G=1), UNSUP)]


@pytest.mark.parametrize("bad,want", BAD_GROUP + [(dict(y=0), INVAL), (dict(mean=P), INVAL), (dict(N=0, x=0, y=0), OK)])
def test_group_norm_arguments(lib, bad, want):
    assert lib.tg_group_norm(ctypes.byref(_group(**bad)), P, BIG, 0) == want


@pytest.mark.parametrize("bad,want", BAD_GROUP + [(dict(mean=0, rstd=0), INVAL), (dict(z=P, z_stride=8), INVAL)])
def test_group_norm_backward_arguments(lib, bad, want):
    a = _group(mean=P, rstd=P)
    for k, v in bad.items():
        setattr(a, k, v)
    g = S._GroupNormGrads(P, 8, P, 0, P, P)
    assert lib.tg_group_norm_backward(ctypes.byref(a), ctypes.byref(g), P, BIG, 0) == want


def test_group_norm_workspaces(lib):
    a, work, back = _group(mean=P, rstd=P), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.tg_group_norm_sizes(ctypes.byref(a), ctypes.byref(work), ctypes.byref(back)) == OK
    assert work.value > 0 and back.value > 0
    assert lib.tg_group_norm(ctypes.byref(a), P, work.value - 1, 0) == WS

    def grads(ws=P, size=back.value, **kw):
        g = S._GroupNormGrads(P, 8, P, 0, P, P)
        for k, v in kw.items():
            setattr(g, k, v)
        return lib.tg_group_norm_backward(ctypes.byref(a), ctypes.byref(g), ws, size, 0)
    assert grads(size=back.value - 1) == WS and grads(ws=0) == WS and grads(ws=P + 4) == ALIGN
    assert grads(dy=0) == INVAL and grads(dx=0) == INVAL and grads(dgamma=0) == INVAL and grads(dy_stride=5) == INVAL
    assert grads(dz=P) == INVAL and grads(dx=P + 1) == ALIGN
    heads = _group(L=1, N=10)
    assert lib.tg_group_norm_sizes(ctypes.byref(heads), ctypes.byref(work), None) == OK and work.value == 0


def test_python_refuses_host_tensors():
    q, v, d, A = (torch.zeros(s) for s in ((2, 3, 1, 4), (2, 3, 2, 5), (2, 3, 2), (2,)))
    x, w = torch.zeros(2, 3, 8), torch.zeros(8)
    for f in (lambda: tg.gated_delta_rule(q, q, v, d, A, d), lambda: tg.gated_delta_rule_train(q, q, v, d, A, d),
              lambda: tg.gated_delta_rule_backward(v, q, q, v, d, A, d, A),
              lambda: tg.gated_delta_rule_step(q[0], q[0], v[0], d[0], A, d[0], A),
              lambda: tg.group_norm(x, 2, w), lambda: tg.group_norm_train(x, 2, w),
              lambda: tg.group_norm_backward(x, x, 2, w, w, w)):
        with pytest.raises(ValueError, match="device tensor"):
            f()


def test_symbols_are_declared():
    names = tg.exported_symbols()
    for n in ("tg_gated_delta_rule", "tg_gated_delta_rule_backward", "tg_gated_delta_rule_step", "tg_group_norm",
              "tg_group_norm_backward"):
        assert n in names
