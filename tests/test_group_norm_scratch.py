"""Sizes of workspaces on the host (no call here reaches the GPU)."""
from __future__ import annotations

import ctypes

import pytest

from conv2d_batchnorm_silu_amd import sequence as S
from test_delta_abi import _group
from test_sequence_abi import F16, F32, OK, P


@pytest.mark.parametrize("N,L,C,G,dtype", [(1000000, 1, 512, 1, F16), (16384, 1, 4096, 1, F16), (4000000, 1, 300, 1, F32),
                                           (500000, 4, 64, 4, F16), (3000, 49, 128, 8, F32), (2000, 1, 257, 1, F16)])
def test_group_norm_scratch_does_not_outgrow_the_tensors(N, L, C, G, dtype):
    """Channels' sums of at most 2048 chunks, or 64 MB, one row more for each of so many, and
    a pair of floats for each chunk and group."""
    a = _group(N=N, L=L, C=C, G=G, dtype=dtype, x_stride=C, mean=P, rstd=P)
    back = ctypes.c_size_t()
    assert S._lib().tg_group_norm_sizes(ctypes.byref(a), None, ctypes.byref(back)) == OK
    chunks = N * ((L + 255) // 256 + 1)
    assert back.value <= max(2048 * 8 * C, 1 << 26) + (chunks // 2048 + 1) * 8 * C + chunks * G * 8 + 1024
