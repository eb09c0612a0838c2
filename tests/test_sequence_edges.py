"""The sequence operators' edges on the host: sizes that no launch holds are
refused before one, and which tensors share memory. No call here reaches the GPU."""
from __future__ import annotations

import ctypes
import itertools
import random

import pytest
import torch

from conv2d_batchnorm_silu_amd import sequence as S
from test_sequence_abi import F16, F32, P, UNSUP, _conv, _rows, _scan


@pytest.fixture(scope="module")
def lib():
    return S._lib()


@pytest.mark.parametrize("D,dtype,n", [(8, F16, 1 << 28), (130, F32, 1 << 26), (516, F32, 1 << 24),
                                       (513, F16, 1 << 24), (129, F16, 1 << 24)])
def test_conv_more_than_a_launch_holds(lib, D, dtype, n):
    """n rows, one to a sequence: with their states to write, or as single
    tokens, 2^32 threads or more along one axis."""
    rows = _rows(seq=D, row=D)
    a = _conv(seqs=n, rows=n, D=D, dtype=dtype, x=rows, y=rows, final=P)
    assert lib.tg_causal_conv(ctypes.byref(a), 0) == UNSUP
    assert lib.tg_causal_conv_backward(ctypes.byref(a), rows, rows, P, P, 0, P, P, 1 << 62, 0) == UNSUP
    assert lib.tg_causal_conv_step(P, D, P, n, 0, P, 0, n, D, 4, dtype, 0, P, 0) == UNSUP


@pytest.mark.parametrize("D,n", [(8, 1 << 24), (48, 1 << 24), (128, 1 << 23), (1000, 1 << 20)])
def test_scan_step_more_than_a_launch_holds(lib, D, n):
    rows, bc = _rows(seq=D, row=D), _rows(seq=16, row=16)
    a = _scan(seqs=n, rows=n, D=D, x=rows, dt=rows, z=rows, y=rows, B=bc, C=bc)
    assert lib.tg_selective_scan_step(ctypes.byref(a), P, n, 0, 0) == UNSUP


def _bytes(t):
    w = t.element_size()
    return {t.data_ptr() + w * sum(i * st for i, st in zip(at, t.stride())) + k
            for at in itertools.product(*map(range, t.shape)) for k in range(w)}


def test_overlap_is_exact():
    """Views of one buffer, with strides that nest, interleave and repeat,
    against their sets of bytes."""
    rng, seen = random.Random(3), [0, 0]
    for _ in range(6000):
        buf = torch.zeros(400, dtype=rng.choice([torch.float16, torch.float32]))
        views = []
        for _ in range(2):
            shape = [rng.randint(1, 4) for _ in range(rng.randint(1, 3))]
            strides = [rng.choice([0, 1, 2, 5, 8, 16, 30]) for _ in shape[:-1]] + [1]
            v = buf.as_strided(shape, strides, rng.randint(0, 120))
            views.append(v.view(torch.int16) if rng.random() < 0.2 and shape[-1] > 0 else v)
        want = bool(_bytes(views[0]) & _bytes(views[1]))
        seen[want] += 1
        assert S._overlap(*views) == want, [(v.shape, v.stride(), v.storage_offset(), v.dtype) for v in views]
    assert min(seen) > 500
    x = torch.zeros(3, 40, 16)
    assert not S._overlap(x[..., :8], x[..., 8:]) and S._overlap(x[..., :8], x[..., 7:])
    assert not S._overlap(x[:, :20], x[:, 20:]) and S._overlap(x[:, :21], x[:, 20:])
    assert not S._overlap(x[:0], x) and S._overlap(x[0, 0].expand(3, 40, 16), x)
    big = torch.empty(1 << 20, 1 << 10, 2, device="meta")
    assert not S._overlap(big[..., :1], big[..., 1:]) and S._overlap(big, big[5:, 7:])
