"""Sequence operators of libtgconv.so (include/tg_sequence.h): layer norm, group
norm, the short causal convolution with SiLU, the selective state space scan and
the gated delta rule.

Like ``binding``, this is argument checking and ctypes marshalling: the HIP
kernels behind the C ABI compute every step, and PyTorch supplies device
memory and streams. Gradients are functions of their own (``*_backward``);
nothing is recorded by autograd.

Activations are fp16, bf16 or fp32 device tensors, channels contiguous.
Parameters are fp32. A batch is dense, ``[S, L, C]`` (any batch and row
strides, so a slice of a wider projection is taken as it is), or packed,
``[T, C]`` with ``offsets``, an int32 device tensor of S + 1 row numbers
(non-decreasing, from 0 to T; sequences may be empty). Outputs are dense new
tensors unless ``out`` is given. ``out`` shares no memory with an argument,
but for the ones that a function's text says it may be: that tensor itself,
with its strides. Any other overlap raises ValueError.

``stream`` is a ``torch.cuda.Stream`` (default: the current one). New
outputs and scratch are allocated for that stream; making the inputs ready on
it, and its results ready elsewhere, is the caller's part as with any stream.
"""
from __future__ import annotations

import collections
import ctypes
import struct

import torch

from .binding import Activation, Dtype, _check, library

i32, i64, vp, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t

_F32, _I32, _DENSE = torch.float32, torch.int32, torch.contiguous_format
_DTYPES = {torch.float16: int(Dtype.F16), torch.bfloat16: int(Dtype.BF16),
           torch.float32: int(Dtype.F32)}


class _Rows(ctypes.Structure):
    _fields_ = [("p", vp), ("seq_stride", i64), ("row_stride", i64)]


class _Seqs(ctypes.Structure):
    _fields_ = [("seqs", i64), ("rows", i64), ("offsets", vp)]


class _ConvArgs(ctypes.Structure):
    _fields_ = [("seqs", _Seqs), ("D", i32), ("K", i32), ("dtype", i32), ("act", i32),
                ("x", _Rows), ("y", _Rows), ("w", vp), ("bias", vp), ("initial", vp),
                ("final", vp)]


class _ScanArgs(ctypes.Structure):
    _fields_ = [("seqs", _Seqs), ("D", i32), ("N", i32), ("G", i32), ("dtype", i32),
                ("softplus", i32), ("x", _Rows), ("dt", _Rows), ("B", _Rows), ("C", _Rows),
                ("z", _Rows), ("y", _Rows), ("A", vp), ("D_skip", vp), ("dt_bias", vp),
                ("initial", vp), ("final", vp)]


class _ScanGrads(ctypes.Structure):
    _fields_ = [("dy", _Rows), ("dfinal", vp), ("dx", _Rows), ("ddt", _Rows), ("dB", _Rows),
                ("dC", _Rows), ("dz", _Rows), ("dA", vp), ("dD", vp), ("ddt_bias", vp),
                ("dinitial", vp)]


class _DeltaArgs(ctypes.Structure):
    _fields_ = [("seqs", _Seqs), ("HK", i32), ("HV", i32), ("K", i32), ("V", i32), ("dtype", i32),
                ("softplus", i32), ("sigmoid", i32), ("normalize", i32), ("scale", ctypes.c_float),
                ("q", _Rows), ("k", _Rows), ("v", _Rows), ("dt", _Rows), ("beta", _Rows),
                ("y", _Rows), ("A", vp), ("dt_bias", vp), ("initial", vp), ("final", vp)]


class _DeltaGrads(ctypes.Structure):
    _fields_ = [("dy", _Rows), ("dfinal", vp), ("dq", _Rows), ("dk", _Rows), ("dv", _Rows),
                ("ddt", _Rows), ("dbeta", _Rows), ("dA", vp), ("ddt_bias", vp), ("dinitial", vp)]


class _GroupNormArgs(ctypes.Structure):
    _fields_ = [("N", i64), ("L", i64), ("C", i32), ("G", i32), ("dtype", i32), ("act", i32),
                ("eps", ctypes.c_float), ("x", vp), ("x_stride", i64), ("z", vp), ("z_stride", i64),
                ("gamma", vp), ("beta", vp), ("y", vp), ("mean", vp), ("rstd", vp)]


class _GroupNormGrads(ctypes.Structure):
    _fields_ = [("dy", vp), ("dy_stride", i64), ("dx", vp), ("dz", vp), ("dgamma", vp),
                ("dbeta", vp)]


# The same layouts as flat numbers: filling a ctypes structure field by field
# takes several microseconds, which a single token's call would mostly consist of.
_CONV = struct.Struct("3q4i10q")
_SCAN = struct.Struct("3q5i4x23q")
_DELTA = struct.Struct("3q8if4x22q")
_GROUP = struct.Struct("2q4if4x9q")
assert _CONV.size == ctypes.sizeof(_ConvArgs) and _SCAN.size == ctypes.sizeof(_ScanArgs)
assert _DELTA.size == ctypes.sizeof(_DeltaArgs) and _GROUP.size == ctypes.sizeof(_GroupNormArgs)

ScanGradients = collections.namedtuple(
    "ScanGradients", "dx ddt dA dB dC dD dz ddt_bias dinitial_state")
DeltaGradients = collections.namedtuple(
    "DeltaGradients", "dq dk dv ddt dA dbeta ddt_bias dinitial_state")
GroupNormGradients = collections.namedtuple("GroupNormGradients", "dx dgamma dbeta dz")

_loaded = None


def _lib():
    global _loaded
    if _loaded is not None:
        return _loaded
    lib = library()
    f, psz = ctypes.c_float, ctypes.POINTER(sz)
    conv = scan = delta = group = vp  # structures, or bytes of their layout
    grads = ctypes.POINTER(_ScanGrads)
    lib.tg_layer_norm.argtypes = [vp, i64, vp, i64, vp, vp, f, i64, i32, i32, vp, vp, vp, vp, vp]
    lib.tg_layer_norm_backward_workspace.argtypes = [i64, i32, i32, psz]
    lib.tg_layer_norm_backward.argtypes = ([vp, i64, vp, i64, vp, vp, vp, vp, i64, i64, i32, i32]
                                           + [vp] * 4 + [sz, vp])
    lib.tg_causal_conv.argtypes = [conv, vp]
    lib.tg_causal_conv_backward_workspace.argtypes = [conv, psz]
    lib.tg_causal_conv_backward.argtypes = [conv, _Rows, _Rows, vp, vp, vp, vp, vp, sz, vp]
    lib.tg_causal_conv_step.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, i32, i32, i32, i32,
                                        vp, vp]
    lib.tg_selective_scan_sizes.argtypes = [scan, psz, psz, psz]
    lib.tg_selective_scan.argtypes = [scan, vp, sz, vp, sz, vp]
    lib.tg_selective_scan_backward.argtypes = [scan, grads, vp, sz, vp, sz, vp]
    lib.tg_selective_scan_step.argtypes = [scan, vp, i64, vp, vp]
    lib.tg_group_norm_sizes.argtypes = [group, psz, psz]
    lib.tg_group_norm.argtypes = [group, vp, sz, vp]
    lib.tg_group_norm_backward.argtypes = [group, ctypes.POINTER(_GroupNormGrads), vp, sz, vp]
    lib.tg_gated_delta_rule_sizes.argtypes = [delta, psz, psz, psz]
    lib.tg_gated_delta_rule.argtypes = [delta, vp, sz, vp, sz, vp]
    lib.tg_gated_delta_rule_backward.argtypes = [delta, ctypes.POINTER(_DeltaGrads), vp, sz, vp,
                                                 sz, vp]
    lib.tg_gated_delta_rule_step.argtypes = [delta, vp, i64, vp, vp]
    _loaded = lib
    return lib


def _dtype(t, name):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError("%s must be float16, bfloat16 or float32, got %s" % (name, t.dtype))
    return d


def _device(t, name):
    """The device number of the tensor that the others are held against."""
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.get_device()


def _refuse(t, name, dev, shape, dtype, contiguous):
    """Say what is wrong with an argument; the checks before only saw that
    something is."""
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)


def _flat(t, name, dev, shape, dtype=_F32):
    """A dense argument's address; None gives 0."""
    if t is None:
        return 0
    if not (t.dtype is dtype and t.is_cuda and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        _refuse(t, name, dev, shape, dtype, True)
    return t.data_ptr()


def _some(t, name):
    if t is None:
        raise ValueError("%s is required" % name)
    return t


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _elsewhere(dev, stream):
    """A context that makes ``stream``, or device ``dev``, torch's current one
    if it is not: the call then starts over inside, so that outputs and
    scratch are allocated for that stream."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream is on %s, the tensors on cuda:%d" % (stream.device, dev))
        return torch.cuda.stream(stream)
    return None if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def _batch(x, offsets, dev):
    """(seqs, rows, offsets address) of a dense or packed batch."""
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("x must be [S, L, C], or [T, C] with offsets; got %s"
                             % (tuple(x.shape),))
        S, L = x.shape[0], x.shape[1]
        if S < 1:
            raise ValueError("x must hold at least one sequence")
        return S, S * L, 0
    if x.dim() != 2:
        raise ValueError("x must be [T, C] with offsets, got %s" % (tuple(x.shape),))
    if (not offsets.is_cuda or offsets.get_device() != dev or offsets.dtype != _I32
            or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 tensor of at least 2 elements on "
                         "cuda:%d" % dev)
    return offsets.numel() - 1, x.shape[0], offsets.data_ptr()


_NO_ROWS = (0, 0, 0)


def _rows(t, name, dev, shape, dtype, packed, width):
    """The tg_rows of a batch's tensor, as a tuple; ``width``: elements of a row."""
    if t is None:
        return _NO_ROWS
    st = t.stride()
    if not (t.dtype is dtype and t.is_cuda and t.get_device() == dev and t.shape == shape
            and (st[-1] == 1 or shape[-1] == 1)):
        _refuse(t, name, dev, shape, dtype, False)
    return _place(t, st, packed, width)


def _place(t, st, packed, width):
    # The stride of a dimension of one element means nothing.
    if packed:
        return t.data_ptr(), 0, st[0] if t.shape[0] > 1 else width
    row = st[1] if t.shape[1] > 1 else width
    return t.data_ptr(), st[0] if t.shape[0] > 1 else row * t.shape[1], row


def _span(t):
    """(first byte, bytes in a run, [(bytes apart, how many)] of the runs)."""
    run, steps = t.element_size(), []
    for step, n in sorted((st * t.element_size(), n) for st, n in zip(t.stride(), t.shape) if n > 1):
        if step == run and not steps:
            run *= n
        elif step:
            steps.append((step, n))
    return t.data_ptr(), run, steps


def _overlap(a, b):
    """Whether two tensors have a byte in common: whether a whole number of
    each of their strides leads from a run of one into a run of the other. A
    search that does not end soon (strides that do not nest) counts as yes."""
    if a.numel() == 0 or b.numel() == 0:
        return False
    (pa, wa, sa), (pb, wb, sb) = _span(a), _span(b)
    reach = {}
    for step, n in sa:
        lo, hi = reach.get(step, (0, 0))
        reach[step] = lo, hi + n - 1
    for step, n in sb:
        lo, hi = reach.get(step, (0, 0))
        reach[step] = lo - (n - 1), hi
    terms = sorted(reach.items(), reverse=True)
    rest = [(0, 0)]  # least and most that the terms from here on add up to
    for step, (lo, hi) in reversed(terms):
        rest.append((rest[-1][0] + step * lo, rest[-1][1] + step * hi))
    rest.reverse()
    left = 10000

    def search(i, lo, hi):  # sum of the terms from i on within lo .. hi
        nonlocal left
        left -= 1
        if hi < rest[i][0] or lo > rest[i][1]:
            return False
        if i == len(terms) or left < 0:
            return True
        step, (least, most) = terms[i]
        first = max(least, -((rest[i + 1][1] - lo) // step))
        last = min(most, (hi - rest[i + 1][0]) // step)
        return any(search(i + 1, lo - k * step, hi - k * step) for k in range(first, last + 1))
    return search(0, pb - pa - wa + 1, pb - pa + wb - 1)


def _is(a, b):
    return (a.data_ptr() == b.data_ptr() and a.shape == b.shape
            and all(n == 1 or x == y for n, x, y in zip(a.shape, a.stride(), b.stride())))


def _new(like):
    return torch.empty_like(like, memory_format=_DENSE)


def _given(out, like, dev, dense, may, apart):
    """``out`` if it fits ``like``: it may be one of ``may`` and shares memory with
    none of ``apart`` ({name: argument})."""
    _refuse(out, "out", dev, like.shape, like.dtype, dense)
    held = out.untyped_storage()
    lo = held.data_ptr()
    hi = lo + held.nbytes()
    for names in (may, apart):
        for name, t in names.items():
            if t is None:
                continue
            held = t.untyped_storage()
            p = held.data_ptr()
            # Strides are looked at only within one allocation.
            if (p < hi and lo < p + held.nbytes() and not (name in may and _is(out, t))
                    and _overlap(out, t)):
                raise ValueError("out shares memory with %s" % name)
    return out


# -------------------------------------------------------------- layer norm

def _norm_rows(t, name, dev, shape, dtype):
    """(address, row stride) of [..., C] whose leading dimensions are one row
    stride apart."""
    if t is None:
        return 0, 0
    if not (t.dtype is dtype and t.is_cuda and t.get_device() == dev and t.shape == shape):
        _refuse(t, name, dev, shape, dtype, False)
    C = shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), C
    _refuse(t, name, dev, shape, dtype, False)
    stride = step = None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n != 1:
            if step is not None and st != step:
                raise ValueError("%s: the rows must be one stride apart (make it contiguous)" % name)
            stride = st if stride is None else stride
            step = st * n
    return t.data_ptr(), C if stride is None else stride


def _norm_shape(x, name):
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("%s must be [..., C] with C >= 1, got %s" % (name, tuple(x.shape)))
    shape, C = x.shape, x.shape[-1]
    return shape, C, x.numel() // C, x.dtype


def _norm_forward(x, gamma, beta, eps, residual, train, out, dev):
    dt = _dtype(x, "x")
    shape, C, rows, dtype = _norm_shape(x, "x")
    xp, xs = _norm_rows(x, "x", dev, shape, dtype)
    rp, rs = _norm_rows(residual, "residual", dev, shape, dtype)
    gp = _flat(_some(gamma, "gamma"), "gamma", dev, (C,))
    bp = _flat(beta, "beta", dev, (C,))
    # Training hands x back as s where there is no residual.
    y = _new(x) if out is None else _given(
        out, x, dev, True, {} if train and residual is None else dict(x=x, residual=residual),
        dict(x=x, residual=residual, gamma=gamma, beta=beta))
    total, tp, mean, rstd, mp, qp = None, 0, None, None, 0, 0
    if residual is not None:
        total = torch.empty_like(x, memory_format=_DENSE)
        tp = total.data_ptr()
    if train:
        mean = torch.empty(shape[:-1], dtype=_F32, device=x.device)
        rstd = torch.empty_like(mean)
        mp, qp = mean.data_ptr(), rstd.data_ptr()
    st = _lib().tg_layer_norm(xp, xs, rp, rs, gp, bp, eps, rows, C, dt, y.data_ptr(), tp, mp, qp,
                              _raw_stream(dev))
    if st:
        _check(st, "tg_layer_norm")
    return y, total, mean, rstd


def layer_norm(x, gamma, beta=None, eps=1e-5, residual=None, out=None, stream=None):
    """Layer norm over the last dimension: y, or with ``residual`` (x's shape
    and type) the pair (y, x + residual), the norm taken of the sum. ``out``
    may be x or residual."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return layer_norm(x, gamma, beta, eps, residual, out)
    y, total, _, _ = _norm_forward(x, gamma, beta, eps, residual, False, out, dev)
    return y if residual is None else (y, total)


def layer_norm_train(x, gamma, beta=None, eps=1e-5, residual=None, out=None, stream=None):
    """(y, s, mean, rstd): layer norm and what its backward pass takes. s is
    the normalised input: x itself, or x + residual, and then ``out`` may be x
    or residual."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return layer_norm_train(x, gamma, beta, eps, residual, out)
    y, total, mean, rstd = _norm_forward(x, gamma, beta, eps, residual, True, out, dev)
    return y, x if residual is None else total, mean, rstd


def layer_norm_backward(dy, s, gamma, mean, rstd, dsum=None, out=None, stream=None):
    """(dx, dgamma, dbeta) from dy and layer_norm_train's s, mean and rstd.
    ``dsum``: a gradient that reaches s past the norm (the residual stream's),
    added to dx. dx is the gradient of x and of the residual alike. ``out``
    (dx) may be dy, s or dsum."""
    dev = _device(s, "s")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return layer_norm_backward(dy, s, gamma, mean, rstd, dsum, out)
    dt = _dtype(s, "s")
    shape, C, rows, dtype = _norm_shape(s, "s")
    sp, ss = _norm_rows(s, "s", dev, shape, dtype)
    gp, gs = _norm_rows(_some(dy, "dy"), "dy", dev, shape, dtype)
    dp, ds = _norm_rows(dsum, "dsum", dev, shape, dtype)
    wp = _flat(_some(gamma, "gamma"), "gamma", dev, (C,))
    mp = _flat(_some(mean, "mean"), "mean", dev, shape[:-1])
    qp = _flat(_some(rstd, "rstd"), "rstd", dev, shape[:-1])
    lib = _lib()
    need = sz()
    _check(lib.tg_layer_norm_backward_workspace(rows, C, dt, ctypes.byref(need)),
           "tg_layer_norm_backward_workspace")
    dx = _new(s) if out is None else _given(out, s, dev, True, dict(dy=dy, s=s, dsum=dsum),
                                            dict(gamma=gamma, mean=mean, rstd=rstd))
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
    ws = torch.empty(need.value, dtype=torch.uint8, device=s.device)
    _check(lib.tg_layer_norm_backward(
        gp, gs, sp, ss, wp, mp, qp, dp, ds, rows, C, dt, dx.data_ptr(), dgamma.data_ptr(),
        dbeta.data_ptr(), ws.data_ptr(), need.value, _raw_stream(dev)), "tg_layer_norm_backward")
    return dx, dgamma, dbeta


# -------------------------------------------------------------- group norm

def _group_args(x, groups, gamma, beta, eps, act, z, dev):
    """A function of (y's, mean's and rstd's addresses) that gives the call's
    arguments; the statistics' shape."""
    dt = _dtype(x, "x")
    if x.dim() < 2 or x.shape[-1] < 1:
        raise ValueError("x must be [N, ..., C] with C >= 1, got %s" % (tuple(x.shape),))
    shape, N, C, dtype = x.shape, x.shape[0], x.shape[-1], x.dtype
    if groups < 1 or C % groups:
        raise ValueError("the %d groups must divide the %d channels" % (groups, C))
    L = 1
    for n in shape[1:-1]:
        L *= n
    if L < 1:
        raise ValueError("x must hold a row for each of its N, got %s" % (tuple(shape),))
    xp, xs = _norm_rows(x, "x", dev, shape, dtype)
    zp, zs = _norm_rows(z, "z", dev, shape, dtype)
    head = (N, L, C, groups, dt, _activation(act), eps, xp, xs, zp, zs,
            _flat(_some(gamma, "gamma"), "gamma", dev, (C,)), _flat(beta, "beta", dev, (C,)))
    return (lambda y, mean, rstd: _GROUP.pack(*head, y, mean, rstd)), (N, groups)


def _group_forward(x, groups, gamma, beta, eps, act, z, train, out, dev):
    args, stats = _group_args(x, groups, gamma, beta, eps, act, z, dev)
    # The backward pass takes x and z again.
    y = _new(x) if out is None else _given(
        out, x, dev, True, {} if train else dict(x=x, z=z), dict(x=x, z=z, gamma=gamma, beta=beta))
    mean = rstd = None
    mp = rp = 0
    if train:
        mean = torch.empty(stats, dtype=_F32, device=x.device)
        rstd = torch.empty_like(mean)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    a = args(y.data_ptr(), mp, rp)
    lib = _lib()
    work = sz()
    _check(lib.tg_group_norm_sizes(a, ctypes.byref(work), None), "tg_group_norm_sizes")
    ws, wp = None, 0
    if work.value:
        ws = torch.empty(work.value, dtype=torch.uint8, device=x.device)
        wp = ws.data_ptr()
    _check(lib.tg_group_norm(a, wp, work.value, _raw_stream(dev)), "tg_group_norm")
    return y, mean, rstd


def group_norm(x, groups, gamma, beta=None, eps=1e-5, act="silu", z=None, out=None, stream=None):
    """Group norm of x [N, ..., C], channels last, then ``act`` ("silu" or
    "none") and the gate: y = act(h * gamma + beta) * silu(z), where h is x less its
    mean, divided by its standard deviation, over each n and each of ``groups``
    groups of neighbouring channels. Maps are [N, H, W, C]; with x [N, C] the groups
    are the heads of single tokens. gamma, beta [C]; z like x. ``out`` may be x or z."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return group_norm(x, groups, gamma, beta, eps, act, z, out)
    return _group_forward(x, groups, gamma, beta, eps, act, z, False, out, dev)[0]


def group_norm_train(x, groups, gamma, beta=None, eps=1e-5, act="silu", z=None, out=None,
                     stream=None):
    """(y, mean, rstd): group norm and what its backward pass takes, [N, groups]."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return group_norm_train(x, groups, gamma, beta, eps, act, z, out)
    return _group_forward(x, groups, gamma, beta, eps, act, z, True, out, dev)


def group_norm_backward(dy, x, groups, gamma, mean, rstd, beta=None, act="silu", z=None, out=None,
                        stream=None):
    """GroupNormGradients (dx, dgamma, dbeta, dz) of group_norm_train's y with the
    same arguments and its mean and rstd; dz is None without z. ``out`` (dx) may be
    x or dy."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return group_norm_backward(dy, x, groups, gamma, mean, rstd, beta, act, z, out)
    args, stats = _group_args(x, groups, gamma, beta, 0.0, act, z, dev)
    a = args(0, _flat(_some(mean, "mean"), "mean", dev, stats),
             _flat(_some(rstd, "rstd"), "rstd", dev, stats))
    gp, gs = _norm_rows(_some(dy, "dy"), "dy", dev, x.shape, x.dtype)
    lib = _lib()
    need = sz()
    _check(lib.tg_group_norm_sizes(a, None, ctypes.byref(need)), "tg_group_norm_sizes")
    dx = _new(x) if out is None else _given(out, x, dev, True, dict(x=x, dy=dy),
                                            dict(x=x, dy=dy, z=z, gamma=gamma, beta=beta, mean=mean,
                                                 rstd=rstd))
    dz = None if z is None else _new(x)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(gamma)
    ws = torch.empty(need.value, dtype=torch.uint8, device=x.device)
    g = _GroupNormGrads(gp, gs, dx.data_ptr(), 0 if dz is None else dz.data_ptr(),
                        dgamma.data_ptr(), dbeta.data_ptr())
    _check(lib.tg_group_norm_backward(a, ctypes.byref(g), ws.data_ptr(), need.value,
                                      _raw_stream(dev)), "tg_group_norm_backward")
    return GroupNormGradients(dx, dgamma, dbeta, dz)


# -------------------------------------------------- short causal convolution

_ACTS = {"silu": int(Activation.SILU), "none": int(Activation.NONE),
         Activation.SILU: int(Activation.SILU), Activation.NONE: int(Activation.NONE)}


def _activation(act):
    a = _ACTS.get(act.lower() if isinstance(act, str) else act)
    if a is None:
        raise ValueError("act must be silu or none, got %s" % (act,))
    return a


def _taps(w):
    if w is None or w.dim() != 2:
        raise ValueError("w must be [K, D]")
    return w.shape[0]


def _conv_args(x, w, bias, act, initial_state, offsets, dev):
    """A function of (y's rows, address of the final states) that gives the
    call's arguments; whether the batch is packed; the states' shape; D."""
    dt, dtype = _dtype(x, "x"), x.dtype
    seqs = _batch(x, offsets, dev)
    packed, D, K = offsets is not None, x.shape[-1], _taps(w)
    held = (seqs[0], K - 1, D)
    head = (*seqs, D, K, dt, _activation(act), *_rows(x, "x", dev, x.shape, dtype, packed, D))
    tail = (_flat(w, "w", dev, (K, D)), _flat(bias, "bias", dev, (D,)),
            _flat(initial_state, "initial_state", dev, held, dtype))
    return (lambda y, final: _CONV.pack(*head, *y, *tail, final)), packed, held, D


def causal_conv(x, w, bias=None, act="silu", initial_state=None, offsets=None, return_state=False,
                out=None, stream=None):
    """Depthwise causal convolution over each sequence's rows, then ``act``
    ("silu" or "none"): v[t] = bias + sum_k w[k] * x[t-K+1+k].

    w: [K, D] (2 <= K <= 8), oldest tap first. ``initial_state`` [S, K-1, D]:
    the rows before each sequence (default zeros). Returns y, or with
    ``return_state`` (y, state): the last K-1 rows of each sequence, as a
    next chunk's initial state or causal_conv_step's state."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return causal_conv(x, w, bias, act, initial_state, offsets, return_state, out)
    args, packed, held, D = _conv_args(x, w, bias, act, initial_state, offsets, dev)
    y = _new(x) if out is None else _given(
        out, x, dev, False, {}, dict(x=x, w=w, bias=bias, initial_state=initial_state,
                                     offsets=offsets))
    state, final = None, 0
    if return_state:
        state = torch.empty(held, dtype=x.dtype, device=x.device)
        final = state.data_ptr()
    _check(_lib().tg_causal_conv(args(_place(y, y.stride(), packed, D), final), _raw_stream(dev)),
           "tg_causal_conv")
    return (y, state) if return_state else y


def causal_conv_backward(dy, x, w, bias=None, act="silu", initial_state=None, offsets=None,
                         dstate=None, stream=None):
    """(dx, dw, dbias, dinitial_state) of causal_conv's y with the same x, w,
    bias, act, initial_state and offsets. ``dstate`` [S, K-1, D]: the gradient
    of the returned state. dinitial_state is None without an initial_state."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return causal_conv_backward(dy, x, w, bias, act, initial_state, offsets, dstate)
    args, packed, held, D = _conv_args(x, w, bias, act, initial_state, offsets, dev)
    a = args(_NO_ROWS, 0)
    g = _rows(_some(dy, "dy"), "dy", dev, x.shape, x.dtype, packed, D)
    df = _flat(dstate, "dstate", dev, held, x.dtype)
    lib = _lib()
    need = sz()
    _check(lib.tg_causal_conv_backward_workspace(a, ctypes.byref(need)),
           "tg_causal_conv_backward_workspace")
    dx = torch.empty_like(x, memory_format=_DENSE)
    dw, db = torch.empty_like(w), torch.empty(D, dtype=_F32, device=x.device)
    d0, d0p = None, 0
    if initial_state is not None:
        d0 = torch.empty(held, dtype=x.dtype, device=x.device)
        d0p = d0.data_ptr()
    ws = torch.empty(need.value, dtype=torch.uint8, device=x.device)
    _check(lib.tg_causal_conv_backward(
        a, _Rows(*g), _Rows(*_place(dx, dx.stride(), packed, D)), dw.data_ptr(),
        db.data_ptr(), df, d0p, ws.data_ptr(), need.value,
        _raw_stream(dev)), "tg_causal_conv_backward")
    return dx, dw, db, d0


def causal_conv_step(x, state, w, bias=None, act="silu", slots=None, out=None, stream=None):
    """One token of each of n sequences: x [n, D] -> y [n, D]; ``state``
    [num_slots, K-1, D] moves on in place. ``slots`` (int32 [n]): each
    sequence's place in ``state`` (default: its number); a slot outside the
    state marks a row without a sequence (y zero, nothing updated). ``out`` may
    be x."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return causal_conv_step(x, state, w, bias, act, slots, out)
    dt, dtype = _dtype(x, "x"), x.dtype
    if x.dim() != 2:
        raise ValueError("x must be [n, D], got %s" % (tuple(x.shape),))
    (n, D), K, num = x.shape, _taps(w), state.shape[0]
    xp, _, xs = _rows(x, "x", dev, x.shape, dtype, True, D)
    hp = _flat(state, "state", dev, (num, K - 1, D), dtype)
    sp = _flat(slots, "slots", dev, (n,), _I32)
    wp, bp = _flat(w, "w", dev, (K, D)), _flat(bias, "bias", dev, (D,))
    y = _new(x) if out is None else _given(out, x, dev, True, dict(x=x),
                                           dict(state=state, slots=slots, w=w, bias=bias))
    st = _lib().tg_causal_conv_step(xp, xs, hp, num, sp, wp, bp, n, D, K, dt, _activation(act),
                                    y.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "tg_causal_conv_step")
    return y


# ---------------------------------------------------------- selective scan

def _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seqs, packed, dev):
    """A function of (y's rows, address of the final states) that gives the
    call's arguments; channels, N, G."""
    d, dtype, shape = _dtype(x, "x"), x.dtype, x.shape
    lead, width = shape[:-1], shape[-1]
    if A is None or A.dim() != 2:
        raise ValueError("A must be [channels, N]")
    N = A.shape[1]
    if B.dim() != len(lead) + 2:
        raise ValueError("B must be %s + [G, N], got %s" % (tuple(lead), tuple(B.shape)))
    G = B.shape[-2]
    if G < 1 or width % G:
        raise ValueError("the %d groups of B must divide the %d channels" % (G, width))
    gn = lead + (G, N)
    if G > 1:
        for name, t in (("B", B), ("C", C)):
            if t.dim() == len(gn) and t.stride(-2) != N:
                raise ValueError("%s: the groups of a row must lie one after another" % name)
    head = (*seqs, width, N, G, d, 1 if softplus else 0,
            *_rows(x, "x", dev, shape, dtype, packed, width),
            *_rows(dt, "dt", dev, shape, dtype, packed, width),
            *_rows(B, "B", dev, gn, dtype, packed, G * N),
            *_rows(C, "C", dev, gn, dtype, packed, G * N),
            *_rows(z, "z", dev, shape, dtype, packed, width))
    tail = (_flat(A, "A", dev, (width, N)), _flat(D, "D", dev, (width,)),
            _flat(dt_bias, "dt_bias", dev, (width,)),
            _flat(initial_state, "initial_state", dev, (seqs[0], width, N)))
    return (lambda y, final: _SCAN.pack(*head, *y, *tail, final)), width, N, G


def _scan_forward(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, offsets, want_state,
                  train, out, dev):
    packed, seqs = offsets is not None, _batch(x, offsets, dev)
    args, width, N, _ = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seqs,
                                   packed, dev)
    # A token's x, dt and z are read by the thread that writes its y.
    y = _new(x) if out is None else _given(
        out, x, dev, False, {} if train else dict(x=x, dt=dt, z=z),
        dict(x=x, dt=dt, z=z, A=A, B=B, C=C, D=D, dt_bias=dt_bias, initial_state=initial_state,
             offsets=offsets))
    state, final = None, 0
    if want_state:
        state = torch.empty((seqs[0], width, N), dtype=_F32, device=x.device)
        final = state.data_ptr()
    a = args(_place(y, y.stride(), packed, width), final)
    lib = _lib()
    work, keep = sz(), sz()
    _check(lib.tg_selective_scan_sizes(a, ctypes.byref(work), ctypes.byref(keep), None),
           "tg_selective_scan_sizes")
    saved = ws = None
    wp = kp = 0
    if train:
        saved = torch.empty(keep.value // 4, dtype=_F32, device=x.device)
        kp = saved.data_ptr()
    if work.value:
        ws = torch.empty(work.value, dtype=torch.uint8, device=x.device)
        wp = ws.data_ptr()
    _check(lib.tg_selective_scan(a, wp, work.value, kp, keep.value if train else 0,
                                 _raw_stream(dev)), "tg_selective_scan")
    return y, state, saved


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, initial_state=None,
                   offsets=None, return_state=False, out=None, stream=None):
    """The selective state space scan over each sequence's rows:

        d = softplus(dt + dt_bias)            (d = dt + dt_bias if not softplus)
        h[n] = exp(d * A[c, n]) * h[n] + d * B[g, n] * x
        y = (sum_n C[g, n] * h[n] + D[c] * x) * silu(z)

    x, dt, z: [S, L, channels] or packed [T, channels]; A [channels, N], N <=
    128; B, C [..., G, N], each group shared by channels/G neighbouring channels;
    D, dt_bias [channels]. ``initial_state`` fp32 [S, channels, N] (default
    zeros). Returns y, or with ``return_state`` (y, state). ``out`` may be x, dt
    or z."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return selective_scan(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, offsets,
                                  return_state, out)
    y, state, _ = _scan_forward(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, offsets,
                                return_state, False, out, dev)
    return (y, state) if return_state else y


def selective_scan_train(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True,
                         initial_state=None, offsets=None, return_state=False, out=None,
                         stream=None):
    """selective_scan for training: (y, saved) or (y, state, saved); ``saved``
    holds the states that selective_scan_backward starts from."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return selective_scan_train(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state,
                                        offsets, return_state, out)
    y, state, saved = _scan_forward(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state,
                                    offsets, return_state, True, out, dev)
    return (y, state, saved) if return_state else (y, saved)


def selective_scan_backward(dy, x, dt, A, B, C, saved, D=None, z=None, dt_bias=None, softplus=True,
                            initial_state=None, offsets=None, dstate=None, stream=None):
    """ScanGradients (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinitial_state) of
    selective_scan_train's y with the same arguments and its ``saved``;
    entries are None for arguments that were not given. ``dstate`` fp32 [S,
    channels, N]: the gradient of the returned state."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return selective_scan_backward(dy, x, dt, A, B, C, saved, D, z, dt_bias, softplus,
                                           initial_state, offsets, dstate)
    packed, seqs = offsets is not None, _batch(x, offsets, dev)
    args, width, N, G = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seqs,
                                   packed, dev)
    a, S, gn = args(_NO_ROWS, 0), seqs[0], G * N
    g = _ScanGrads(_rows(_some(dy, "dy"), "dy", dev, x.shape, x.dtype, packed, width),
                   _flat(dstate, "dstate", dev, (S, width, N)))
    lib = _lib()
    keep, need = sz(), sz()
    _check(lib.tg_selective_scan_sizes(a, None, ctypes.byref(keep), ctypes.byref(need)),
           "tg_selective_scan_sizes")
    sp = _flat(_some(saved, "saved"), "saved", dev, (keep.value // 4,))

    def rows_like(t, w):
        o = torch.empty_like(t, memory_format=_DENSE)
        return o, _place(o, o.stride(), packed, w)

    def params(*shape):
        return torch.empty(shape, dtype=_F32, device=x.device)

    dx, g.dx = rows_like(x, width)
    ddt, g.ddt = rows_like(x, width)
    dB, g.dB = rows_like(B, gn)
    dC, g.dC = rows_like(C, gn)
    dz = dD = db = d0 = None
    if z is not None:
        dz, g.dz = rows_like(x, width)
    dA = params(width, N)
    g.dA = dA.data_ptr()
    if D is not None:
        dD = params(width)
        g.dD = dD.data_ptr()
    if dt_bias is not None:
        db = params(width)
        g.ddt_bias = db.data_ptr()
    if initial_state is not None:
        d0 = params(S, width, N)
        g.dinitial = d0.data_ptr()
    ws = torch.empty(need.value, dtype=torch.uint8, device=x.device)
    _check(lib.tg_selective_scan_backward(a, ctypes.byref(g), sp, keep.value, ws.data_ptr(),
                                          need.value, _raw_stream(dev)),
           "tg_selective_scan_backward")
    return ScanGradients(dx, ddt, dA, dB, dC, dD, dz, db, d0)


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus=True,
                        slots=None, out=None, stream=None):
    """One token of each of n sequences: x, dt, z [n, channels], B, C [n, G, N]
    -> y [n, channels]; ``state`` fp32 [num_slots, channels, N] is updated in
    place. ``slots`` as in causal_conv_step. ``out`` may be x, dt or z."""
    dev = _device(x, "x")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return selective_scan_step(x, dt, A, B, C, state, D, z, dt_bias, softplus, slots, out)
    if x.dim() != 2:
        raise ValueError("x must be [n, channels], got %s" % (tuple(x.shape),))
    n = x.shape[0]
    args, width, N, _ = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, None, (n, n, 0), True,
                                   dev)
    num = state.shape[0]
    hp = _flat(state, "state", dev, (num, width, N))
    sp = _flat(slots, "slots", dev, (n,), _I32)
    y = _new(x) if out is None else _given(
        out, x, dev, False, dict(x=x, dt=dt, z=z),
        dict(A=A, B=B, C=C, D=D, dt_bias=dt_bias, state=state, slots=slots))
    st = _lib().tg_selective_scan_step(args(_place(y, y.stride(), True, width), 0), hp, num, sp,
                                       _raw_stream(dev))
    if st:
        _check(st, "tg_selective_scan_step")
    return y


# -------------------------------------------------------- gated delta rule

def _heads(t, name, lead):
    """(heads, width) of a tensor of rows of heads, one head after another."""
    if t.dim() != len(lead) + 2 or t.shape[:-2] != lead:
        raise ValueError("%s must be %s + [heads, width], got %s"
                         % (name, tuple(lead), tuple(t.shape)))
    H, W = t.shape[-2:]
    if H < 1 or W < 1:
        raise ValueError("%s must hold a head of one column at the least, got %s"
                         % (name, tuple(t.shape)))
    if H > 1 and t.stride(-2) != W:
        raise ValueError("%s: the heads of a row must lie one after another" % name)
    return H, W


def _delta_batch(v, offsets, dev):
    """As _batch, for rows of heads."""
    if v.dim() != (4 if offsets is None else 3):
        raise ValueError("v must be [S, L, heads, V], or [T, heads, V] with offsets; got %s"
                         % (tuple(v.shape),))
    return _batch(v.select(-2, 0) if v.shape[-2] else v.flatten(-2), offsets, dev)


def _delta_args(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize, scale, initial_state,
                seqs, packed, dev):
    """A function of (y's rows, address of the final states) that gives the
    call's arguments; value heads, V; the states' shape."""
    d, dtype, shape = _dtype(v, "v"), v.dtype, v.shape
    lead, dims = shape[:-2], len(shape)
    HV, V = shape[-2], shape[-1]
    # Each tensor of heads in full only if something is wrong with it.
    if HV < 1 or V < 1 or (HV > 1 and v.stride(-2) != V):
        _heads(v, "v", lead)
    if k is None or k.dim() != dims or k.shape[:-2] != lead or k.shape[-1] < 1 or k.shape[-2] < 1:
        _heads(_some(k, "k"), "k", lead)
    HK, K = k.shape[-2], k.shape[-1]
    if HK > 1 and k.stride(-2) != K:
        _heads(k, "k", lead)
    if HV % HK:
        raise ValueError("the %d heads of k must divide the %d of v" % (HK, HV))
    if HK > 1 and q is not None and q.dim() == dims and q.stride(-2) != K:
        _heads(q, "q", lead)
    held = (seqs[0], HV, K, V)
    gates = shape[:-1]
    if scale is None:
        scale = K ** -0.5
    head = (*seqs, HK, HV, K, V, d, 1 if softplus else 0, 1 if sigmoid else 0,
            1 if normalize else 0, scale,
            *_rows(_some(q, "q"), "q", dev, k.shape, dtype, packed, HK * K),
            *_rows(k, "k", dev, k.shape, dtype, packed, HK * K),
            *_rows(v, "v", dev, v.shape, dtype, packed, HV * V),
            *_rows(_some(dt, "dt"), "dt", dev, gates, dtype, packed, HV),
            *_rows(_some(beta, "beta"), "beta", dev, gates, dtype, packed, HV))
    tail = (_flat(_some(A, "A"), "A", dev, (HV,)), _flat(dt_bias, "dt_bias", dev, (HV,)),
            _flat(initial_state, "initial_state", dev, held))
    return (lambda y, final: _DELTA.pack(*head, *y, *tail, final)), HV, V, held


def _delta_forward(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize, scale,
                   initial_state, offsets, want_state, train, out, dev):
    packed, seqs = offsets is not None, _delta_batch(v, offsets, dev)
    args, HV, V, held = _delta_args(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize,
                                    scale, initial_state, seqs, packed, dev)
    # A workgroup reads its columns of v for 64 tokens before it writes their y.
    y = _new(v) if out is None else _given(
        out, v, dev, False, {} if train else dict(v=v),
        dict(q=q, k=k, v=v, dt=dt, A=A, beta=beta, dt_bias=dt_bias, initial_state=initial_state,
             offsets=offsets))
    if out is not None:
        _heads(y, "out", v.shape[:-2])
    state, final = None, 0
    if want_state:
        state = torch.empty(held, dtype=_F32, device=v.device)
        final = state.data_ptr()
    a = args(_place(y, y.stride(), packed, HV * V), final)
    lib = _lib()
    work, keep = sz(), sz()
    _check(lib.tg_gated_delta_rule_sizes(a, ctypes.byref(work), ctypes.byref(keep), None),
           "tg_gated_delta_rule_sizes")
    saved, kp = None, 0
    if train:
        saved = torch.empty(keep.value // 4, dtype=_F32, device=v.device)
        kp = saved.data_ptr()
    ws = torch.empty(work.value, dtype=torch.uint8, device=v.device)
    _check(lib.tg_gated_delta_rule(a, ws.data_ptr(), work.value, kp, keep.value if train else 0,
                                   _raw_stream(dev)), "tg_gated_delta_rule")
    return y, state, saved


def gated_delta_rule(q, k, v, dt, A, beta, dt_bias=None, softplus=True, sigmoid=True,
                     normalize=True, scale=None, initial_state=None, offsets=None,
                     return_state=False, out=None, stream=None):
    """The gated delta rule over each sequence's tokens, a K x V matrix S for
    each value head:

        d = softplus(dt + dt_bias)            (d = dt + dt_bias if not softplus)
        b = sigmoid(beta)                     (b = beta if not sigmoid)
        q, k = q / sqrt(sum q^2 + 1e-6), k / sqrt(sum k^2 + 1e-6)  (if normalize)
        S = exp(d * A) * S
        S = S + b * k (v - k S)
        y = scale * q S                       (scale: default K ** -0.5)

    q, k: [S, L, key heads, K] or packed [T, key heads, K], K <= 256; v [...,
    value heads, V], each key head shared by value heads / key heads neighbouring
    ones; dt, beta [..., value heads]; A, dt_bias [value heads]. The heads of a
    row lie one after another. ``initial_state`` fp32 [S, value heads, K, V]
    (default zeros). Returns y, or with ``return_state`` (y, state). ``out`` may
    be v.

    The states are computed to fp32's 24 bits, in training and without. Decays above 1
    (A > 0) are taken as they are while the product over any tokens in a row stays
    within fp32. What is infinite or NaN in a token (a sum of squares of q or k past
    fp32 too) reaches its own y and, but for q, later ones of its head."""
    dev = _device(v, "v")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return gated_delta_rule(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize,
                                    scale, initial_state, offsets, return_state, out)
    y, state, _ = _delta_forward(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize, scale,
                                 initial_state, offsets, return_state, False, out, dev)
    return (y, state) if return_state else y


def gated_delta_rule_train(q, k, v, dt, A, beta, dt_bias=None, softplus=True, sigmoid=True,
                           normalize=True, scale=None, initial_state=None, offsets=None,
                           return_state=False, out=None, stream=None):
    """gated_delta_rule for training: (y, saved) or (y, state, saved); ``saved``
    holds the states and corrections that gated_delta_rule_backward starts from."""
    dev = _device(v, "v")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return gated_delta_rule_train(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid,
                                          normalize, scale, initial_state, offsets, return_state,
                                          out)
    y, state, saved = _delta_forward(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize,
                                     scale, initial_state, offsets, return_state, True, out, dev)
    return (y, state, saved) if return_state else (y, saved)


def gated_delta_rule_backward(dy, q, k, v, dt, A, beta, saved, dt_bias=None, softplus=True,
                              sigmoid=True, normalize=True, scale=None, initial_state=None,
                              offsets=None, dstate=None, stream=None):
    """DeltaGradients (dq, dk, dv, ddt, dA, dbeta, ddt_bias, dinitial_state) of
    gated_delta_rule_train's y with the same arguments and its ``saved``; entries
    are None for arguments that were not given. ``dstate`` fp32 [S, value heads,
    K, V]: the gradient of the returned state."""
    dev = _device(v, "v")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return gated_delta_rule_backward(dy, q, k, v, dt, A, beta, saved, dt_bias, softplus,
                                             sigmoid, normalize, scale, initial_state, offsets,
                                             dstate)
    packed, seqs = offsets is not None, _delta_batch(v, offsets, dev)
    args, HV, V, held = _delta_args(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize,
                                    scale, initial_state, seqs, packed, dev)
    a = args(_NO_ROWS, 0)
    if _some(dy, "dy").shape == v.shape:
        _heads(dy, "dy", v.shape[:-2])
    g = _DeltaGrads(_rows(dy, "dy", dev, v.shape, v.dtype, packed, HV * V),
                    _flat(dstate, "dstate", dev, held))
    lib = _lib()
    keep, need = sz(), sz()
    _check(lib.tg_gated_delta_rule_sizes(a, None, ctypes.byref(keep), ctypes.byref(need)),
           "tg_gated_delta_rule_sizes")
    sp = _flat(_some(saved, "saved"), "saved", dev, (keep.value // 4,))

    def rows_like(t):
        o = torch.empty_like(t, memory_format=_DENSE)
        return o, _place(o, o.stride(), packed, o.shape[-1] * (o.shape[-2] if t.dim() == v.dim() else 1))

    dq, g.dq = rows_like(q)
    dk, g.dk = rows_like(k)
    dv, g.dv = rows_like(v)
    ddt, g.ddt = rows_like(dt)
    dbeta, g.dbeta = rows_like(beta)
    dA = torch.empty_like(A)
    g.dA = dA.data_ptr()
    db = d0 = None
    if dt_bias is not None:
        db = torch.empty_like(dt_bias)
        g.ddt_bias = db.data_ptr()
    if initial_state is not None:
        d0 = torch.empty_like(initial_state)
        g.dinitial = d0.data_ptr()
    ws = torch.empty(need.value, dtype=torch.uint8, device=v.device)
    _check(lib.tg_gated_delta_rule_backward(a, ctypes.byref(g), sp, keep.value, ws.data_ptr(),
                                            need.value, _raw_stream(dev)),
           "tg_gated_delta_rule_backward")
    return DeltaGradients(dq, dk, dv, ddt, dA, dbeta, db, d0)


def gated_delta_rule_step(q, k, v, dt, A, beta, state, dt_bias=None, softplus=True, sigmoid=True,
                          normalize=True, scale=None, slots=None, out=None, stream=None):
    """One token of each of n sequences: q, k [n, key heads, K], v [n, value
    heads, V], dt, beta [n, value heads] -> y like v; ``state`` fp32 [num_slots,
    value heads, K, V] is updated in place. ``slots`` as in causal_conv_step."""
    dev = _device(v, "v")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return gated_delta_rule_step(q, k, v, dt, A, beta, state, dt_bias, softplus, sigmoid,
                                         normalize, scale, slots, out)
    if v.dim() != 3:
        raise ValueError("v must be [n, heads, V], got %s" % (tuple(v.shape),))
    n = v.shape[0]
    args, HV, V, held = _delta_args(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, normalize,
                                    scale, None, (n, n, 0), True, dev)
    num = _some(state, "state").shape[0]
    hp = _flat(state, "state", dev, (num,) + held[1:])
    sp = _flat(slots, "slots", dev, (n,), _I32)
    y = _new(v) if out is None else _given(
        out, v, dev, False, {}, dict(q=q, k=k, v=v, dt=dt, A=A, beta=beta, dt_bias=dt_bias,
                                     state=state, slots=slots))
    if out is not None:
        _heads(y, "out", v.shape[:-2])
    st = _lib().tg_gated_delta_rule_step(args(_place(y, y.stride(), True, HV * V), 0), hp, num, sp,
                                         _raw_stream(dev))
    if st:
        _check(st, "tg_gated_delta_rule_step")
    return y
