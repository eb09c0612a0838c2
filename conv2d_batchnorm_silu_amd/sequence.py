"""Sequence operators of libtgconv.so (include/tg_sequence.h): layer norm, the
short causal convolution with SiLU and the selective state space scan.

Like ``binding``, this is argument checking and ctypes marshalling: the HIP
kernels behind the C ABI compute every step, and PyTorch supplies device
memory and streams. Gradients are functions of their own (``*_backward``);
nothing is recorded by autograd.

Activations are fp16, bf16 or fp32 device tensors, channels contiguous.
Parameters are fp32. A batch is dense, ``[S, L, C]`` (any batch and row
strides, so a slice of a wider projection is taken as it is), or packed,
``[T, C]`` with ``offsets``, an int32 device tensor of S + 1 row numbers
(non-decreasing, from 0 to T; sequences may be empty). Outputs are dense new
tensors unless ``out`` is given.

``stream`` is a ``torch.cuda.Stream`` (default: the current one). New
outputs and scratch are allocated for that stream; making the inputs ready on
it, and its results ready elsewhere, is the caller's part as with any stream.
"""
from __future__ import annotations

import collections
import ctypes

from .binding import Activation, Dtype, _check, library

i32, i64, vp, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


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


ScanGradients = collections.namedtuple(
    "ScanGradients", "dx ddt dA dB dC dD dz ddt_bias dinitial_state")

_ready = False


def _lib():
    global _ready
    lib = library()
    if not _ready:
        f = ctypes.c_float
        psz = ctypes.POINTER(sz)
        conv, scan, grads = (ctypes.POINTER(t) for t in (_ConvArgs, _ScanArgs, _ScanGrads))
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
        _ready = True
    return lib


def _dtypes():
    import torch
    return {torch.float16: int(Dtype.F16), torch.bfloat16: int(Dtype.BF16),
            torch.float32: int(Dtype.F32)}


_DTYPES = None


def _dtype(t, name):
    global _DTYPES
    if _DTYPES is None:
        _DTYPES = _dtypes()
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError("%s must be float16, bfloat16 or float32, got %s" % (name, t.dtype))
    return d


def _device(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    return t.device


def _tensor(t, name, like, shape, dtype=None):
    """Device, type and shape of an argument; its last dimension contiguous."""
    if t.device != like.device:
        raise ValueError("%s must be on %s, got %s" % (name, like.device, t.device))
    want = like.dtype if dtype is None else dtype
    if t.dtype != want:
        raise ValueError("%s must be %s, got %s" % (name, want, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)


def _flat(t, name, like, shape, dtype):
    """A dense argument's address; None gives 0."""
    if t is None:
        return 0
    _tensor(t, name, like, shape, dtype)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _param(t, name, like, *shape):
    import torch
    return _flat(t, name, like, shape, torch.float32)


def _row_stride(t, width):
    return t.stride(-2) if t.shape[-2] > 1 else width


class _Launch:
    """The stream of a call, and its device and stream as torch's current ones
    while outputs are allocated (only entered where they are not already)."""

    def __init__(self, x, stream):
        import torch
        cur = torch.cuda.current_stream(x.device)
        self.contexts = []
        if stream is not None and stream != cur:
            if stream.device != x.device:
                raise ValueError("stream is on %s, the tensors on %s" % (stream.device, x.device))
            self.contexts.append(torch.cuda.stream(stream))
            cur = stream
        elif x.device.index != torch.cuda.current_device():
            self.contexts.append(torch.cuda.device(x.device))
        self.handle = cur.cuda_stream

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _batch(x, offsets, name="x"):
    """(_Seqs, leading shape, number of sequences) of a dense or packed batch."""
    import torch
    _device(x, name)
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("%s must be [S, L, C], or [T, C] with offsets; got %s"
                             % (name, tuple(x.shape)))
        S, L = x.shape[0], x.shape[1]
        if S < 1:
            raise ValueError("%s must hold at least one sequence" % name)
        return _Seqs(S, S * L, 0), x.shape[:2], S
    if x.dim() != 2:
        raise ValueError("%s must be [T, C] with offsets, got %s" % (name, tuple(x.shape)))
    if (offsets.device != x.device or offsets.dtype != torch.int32 or offsets.dim() != 1
            or offsets.numel() < 2 or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 tensor of at least 2 elements on %s"
                         % x.device)
    S = offsets.numel() - 1
    return _Seqs(S, x.shape[0], offsets.data_ptr()), x.shape[:1], S


def _rows(t, name, like, shape, packed, width=None):
    """_Rows of a batch's tensor; ``width``: elements of a row."""
    if t is None:
        return _Rows(0, 0, 0)
    _tensor(t, name, like, shape)
    return _rows_unchecked(t, packed, width or shape[-1], len(shape) - (1 if packed else 2))


def _rows_unchecked(t, packed, width, inner=1):
    if packed:
        return _Rows(t.data_ptr(), 0, t.stride(0) if t.shape[0] > 1 else width)
    row = t.stride(1) if t.shape[1] > 1 else width
    return _Rows(t.data_ptr(), t.stride(0) if t.shape[0] > 1 else row * t.shape[1], row)


def _out(out, like, name, shape):
    import torch
    if out is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    _tensor(out, name, like, shape)
    return out


def _slots(slots, like, n):
    import torch
    if slots is None:
        return 0
    return _flat(slots, "slots", like, (n,), torch.int32)


# -------------------------------------------------------------- layer norm

def _norm_rows(t, name, like):
    """(address, row stride) of [..., C] whose leading dimensions are one row
    stride apart."""
    _tensor(t, name, like, like.shape)
    C = t.shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), C
    if t.numel() == 0:
        return t.data_ptr(), C
    stride, step = None, 0
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = s
            step = s * n
        elif s != step:
            raise ValueError("%s: the rows must be one stride apart (make it contiguous)" % name)
        else:
            step = s * n
    return t.data_ptr(), C if stride is None else stride


def _norm_forward(x, gamma, beta, eps, residual, train, out, stream):
    import torch
    _device(x, "x")
    dt = _dtype(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., C] with C >= 1, got %s" % (tuple(x.shape),))
    C = x.shape[-1]
    rows = x.numel() // C
    xp, xs = _norm_rows(x, "x", x)
    rp, rs = (0, 0) if residual is None else _norm_rows(residual, "residual", x)
    if gamma is None:
        raise ValueError("gamma is required")
    gp, bp = _param(gamma, "gamma", x, C), _param(beta, "beta", x, C)
    lib = _lib()
    with _Launch(x, stream) as st:
        y = _out(out, x, "out", x.shape)
        if out is not None and not y.is_contiguous():
            raise ValueError("out must be contiguous")
        total = None if residual is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        mean = rstd = None
        if train:
            mean, rstd = torch.empty((2,) + x.shape[:-1], dtype=torch.float32, device=x.device)
        _check(lib.tg_layer_norm(
            xp, xs, rp, rs, gp, bp, eps, rows, C, dt, y.data_ptr(),
            0 if total is None else total.data_ptr(), 0 if mean is None else mean.data_ptr(),
            0 if rstd is None else rstd.data_ptr(), st), "tg_layer_norm")
    return y, total, mean, rstd


def layer_norm(x, gamma, beta=None, eps=1e-5, residual=None, out=None, stream=None):
    """Layer norm over the last dimension: y, or with ``residual`` (x's shape
    and type) the pair (y, x + residual), the norm taken of the sum."""
    y, total, _, _ = _norm_forward(x, gamma, beta, eps, residual, False, out, stream)
    return y if residual is None else (y, total)


def layer_norm_train(x, gamma, beta=None, eps=1e-5, residual=None, out=None, stream=None):
    """(y, s, mean, rstd): layer norm and what its backward pass takes. s is
    the normalised input: x itself, or x + residual."""
    y, total, mean, rstd = _norm_forward(x, gamma, beta, eps, residual, True, out, stream)
    return y, x if residual is None else total, mean, rstd


def layer_norm_backward(dy, s, gamma, mean, rstd, dsum=None, out=None, stream=None):
    """(dx, dgamma, dbeta) from dy and layer_norm_train's s, mean and rstd.
    ``dsum``: a gradient that reaches s past the norm (the residual stream's),
    added to dx. dx is the gradient of x and of the residual alike."""
    import torch
    _device(s, "s")
    dt = _dtype(s, "s")
    C = s.shape[-1]
    rows = s.numel() // C
    sp, ss = _norm_rows(s, "s", s)
    gp, gs = _norm_rows(dy, "dy", s)
    dp, ds = (0, 0) if dsum is None else _norm_rows(dsum, "dsum", s)
    if gamma is None:
        raise ValueError("gamma is required")
    wp = _param(gamma, "gamma", s, C)
    mp = _param(mean, "mean", s, *s.shape[:-1])
    qp = _param(rstd, "rstd", s, *s.shape[:-1])
    lib = _lib()
    need = sz()
    _check(lib.tg_layer_norm_backward_workspace(rows, C, dt, ctypes.byref(need)),
           "tg_layer_norm_backward_workspace")
    with _Launch(s, stream) as st:
        dx = _out(out, s, "out", s.shape)
        if out is not None and not dx.is_contiguous():
            raise ValueError("out must be contiguous")
        dw = torch.empty((2, C), dtype=torch.float32, device=s.device)
        ws = torch.empty(need.value, dtype=torch.uint8, device=s.device)
        _check(lib.tg_layer_norm_backward(
            gp, gs, sp, ss, wp, mp, qp, dp, ds, rows, C, dt, dx.data_ptr(), dw[0].data_ptr(),
            dw[1].data_ptr(), ws.data_ptr(), need.value, st), "tg_layer_norm_backward")
    return dx, dw[0], dw[1]


# -------------------------------------------------- short causal convolution

def _activation(act):
    a = act if isinstance(act, Activation) else Activation[str(act).upper()]
    if a not in (Activation.SILU, Activation.NONE):
        raise ValueError("act must be silu or none, got %s" % act)
    return int(a)


def _conv_args(x, w, bias, act, initial_state, offsets):
    import torch
    dt = _dtype(x, "x")
    seqs, lead, S = _batch(x, offsets)
    packed = offsets is not None
    D = x.shape[-1]
    if w is None or w.dim() != 2:
        raise ValueError("w must be [K, D]")
    K = w.shape[0]
    a = _ConvArgs(seqs, D, K, dt, _activation(act))
    a.x = _rows(x, "x", x, x.shape, packed)
    a.w, a.bias = _param(w, "w", x, K, D), _param(bias, "bias", x, D)
    a.initial = _flat(initial_state, "initial_state", x, (S, K - 1, D), x.dtype)
    return a, packed, (S, K - 1, D)


def causal_conv(x, w, bias=None, act="silu", initial_state=None, offsets=None, return_state=False,
                out=None, stream=None):
    """Depthwise causal convolution over each sequence's rows, then ``act``
    ("silu" or "none"): v[t] = bias + sum_k w[k] * x[t-K+1+k].

    w: [K, D] (2 <= K <= 8), oldest tap first. ``initial_state`` [S, K-1, D]:
    the rows before each sequence (default zeros). Returns y, or with
    ``return_state`` (y, state): the last K-1 rows of each sequence, as a
    next chunk's initial state or causal_conv_step's state."""
    import torch
    a, packed, held = _conv_args(x, w, bias, act, initial_state, offsets)
    lib = _lib()
    with _Launch(x, stream) as st:
        y = _out(out, x, "out", x.shape)
        a.y = _rows_unchecked(y, packed, a.D)
        state = torch.empty(held, dtype=x.dtype, device=x.device) if return_state else None
        if return_state:
            a.final = state.data_ptr()
        _check(lib.tg_causal_conv(ctypes.byref(a), st), "tg_causal_conv")
    return (y, state) if return_state else y


def causal_conv_backward(dy, x, w, bias=None, act="silu", initial_state=None, offsets=None,
                         dstate=None, stream=None):
    """(dx, dw, dbias, dinitial_state) of causal_conv's y with the same x, w,
    bias, act, initial_state and offsets. ``dstate`` [S, K-1, D]: the gradient
    of the returned state. dinitial_state is None without an initial_state."""
    import torch
    a, packed, held = _conv_args(x, w, bias, act, initial_state, offsets)
    g = _rows(dy, "dy", x, x.shape, packed)
    df = _flat(dstate, "dstate", x, held, x.dtype)
    lib = _lib()
    need = sz()
    _check(lib.tg_causal_conv_backward_workspace(ctypes.byref(a), ctypes.byref(need)),
           "tg_causal_conv_backward_workspace")
    with _Launch(x, stream) as st:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty((a.K + 1, a.D), dtype=torch.float32, device=x.device)
        d0 = (None if initial_state is None
              else torch.empty(held, dtype=x.dtype, device=x.device))
        ws = torch.empty(need.value, dtype=torch.uint8, device=x.device)
        _check(lib.tg_causal_conv_backward(
            ctypes.byref(a), g, _rows_unchecked(dx, packed, a.D), dw.data_ptr(),
            dw[a.K].data_ptr(), df, 0 if d0 is None else d0.data_ptr(), ws.data_ptr(), need.value,
            st), "tg_causal_conv_backward")
    return dx, dw[:a.K], dw[a.K], d0


def causal_conv_step(x, state, w, bias=None, act="silu", slots=None, out=None, stream=None):
    """One token of each of n sequences: x [n, D] -> y [n, D]; ``state``
    [num_slots, K-1, D] moves on in place. ``slots`` (int32 [n]): each
    sequence's place in ``state`` (default: its number); a slot outside the
    state marks a row without a sequence (y zero, nothing updated)."""
    _device(x, "x")
    dt = _dtype(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [n, D], got %s" % (tuple(x.shape),))
    n, D = x.shape
    if w is None or w.dim() != 2:
        raise ValueError("w must be [K, D]")
    K = w.shape[0]
    if state.dim() != 3:
        raise ValueError("state must be [num_slots, K-1, D]")
    num = state.shape[0]
    _tensor(x, "x", x, x.shape)
    hp = _flat(state, "state", x, (num, K - 1, D), x.dtype)
    sp = _slots(slots, x, n)
    wp, bp = _param(w, "w", x, K, D), _param(bias, "bias", x, D)
    a = _activation(act)
    lib = _lib()
    with _Launch(x, stream) as st:
        y = _out(out, x, "out", x.shape)
        if out is not None and not y.is_contiguous():
            raise ValueError("out must be contiguous")
        _check(lib.tg_causal_conv_step(x.data_ptr(), _row_stride(x, D), hp, num, sp, wp, bp, n, D,
                                       K, dt, a, y.data_ptr(), st), "tg_causal_conv_step")
    return y


# ---------------------------------------------------------- selective scan

def _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seqs, lead, S, packed):
    import torch
    d = _dtype(x, "x")
    width = x.shape[-1]
    if A is None or A.dim() != 2:
        raise ValueError("A must be [D, N]")
    N = A.shape[1]
    if B.dim() != len(lead) + 2:
        raise ValueError("B must be %s + [G, N], got %s" % (tuple(lead), tuple(B.shape)))
    G = B.shape[-2]
    if G < 1 or width % G:
        raise ValueError("the %d groups of B must divide the %d channels" % (G, width))
    a = _ScanArgs(seqs, width, N, G, d, 1 if softplus else 0)
    a.x = _rows(x, "x", x, x.shape, packed)
    a.dt = _rows(dt, "dt", x, x.shape, packed)
    gn = lead + (G, N)
    for name, t in (("B", B), ("C", C)):
        if t.dim() == len(gn) and G > 1 and t.stride(-2) != N:
            raise ValueError("%s: the groups of a row must lie one after another" % name)
        setattr(a, name, _rows(t, name, x, gn, packed, G * N))
    a.z = _rows(z, "z", x, x.shape, packed)
    a.A, a.D_skip = _param(A, "A", x, width, N), _param(D, "D", x, width)
    a.dt_bias = _param(dt_bias, "dt_bias", x, width)
    a.initial = _param(initial_state, "initial_state", x, S, width, N)
    return a


def _scan_forward(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, offsets, want_state,
                  train, out, stream):
    import torch
    seqs, lead, S = _batch(x, offsets)
    packed = offsets is not None
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seqs, lead, S, packed)
    lib = _lib()
    work, keep = sz(), sz()
    _check(lib.tg_selective_scan_sizes(ctypes.byref(a), ctypes.byref(work), ctypes.byref(keep),
                                       None), "tg_selective_scan_sizes")
    with _Launch(x, stream) as st:
        y = _out(out, x, "out", x.shape)
        a.y = _rows_unchecked(y, packed, a.D)
        state = saved = ws = None
        if want_state:
            state = torch.empty((S, a.D, a.N), dtype=torch.float32, device=x.device)
            a.final = state.data_ptr()
        if train:
            saved = torch.empty(keep.value // 4, dtype=torch.float32, device=x.device)
        if work.value:
            ws = torch.empty(work.value, dtype=torch.uint8, device=x.device)
        _check(lib.tg_selective_scan(
            ctypes.byref(a), 0 if ws is None else ws.data_ptr(), work.value,
            0 if saved is None else saved.data_ptr(), keep.value if train else 0, st),
            "tg_selective_scan")
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
    zeros). Returns y, or with ``return_state`` (y, state)."""
    y, state, _ = _scan_forward(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, offsets,
                                return_state, False, out, stream)
    return (y, state) if return_state else y


def selective_scan_train(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True,
                         initial_state=None, offsets=None, return_state=False, out=None,
                         stream=None):
    """selective_scan for training: (y, saved) or (y, state, saved); ``saved``
    holds the states that selective_scan_backward starts from."""
    y, state, saved = _scan_forward(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state,
                                    offsets, return_state, True, out, stream)
    return (y, state, saved) if return_state else (y, saved)


def selective_scan_backward(dy, x, dt, A, B, C, saved, D=None, z=None, dt_bias=None, softplus=True,
                            initial_state=None, offsets=None, dstate=None, stream=None):
    """ScanGradients (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dinitial_state) of
    selective_scan_train's y with the same arguments and its ``saved``;
    entries are None for arguments that were not given. ``dstate`` fp32 [S,
    channels, N]: the gradient of the returned state."""
    import torch
    seqs, lead, S = _batch(x, offsets)
    packed = offsets is not None
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, initial_state, seqs, lead, S, packed)
    g = _ScanGrads()
    g.dy = _rows(dy, "dy", x, x.shape, packed)
    g.dfinal = _param(dstate, "dstate", x, S, a.D, a.N)
    lib = _lib()
    keep, need = sz(), sz()
    _check(lib.tg_selective_scan_sizes(ctypes.byref(a), None, ctypes.byref(keep),
                                       ctypes.byref(need)), "tg_selective_scan_sizes")
    sp = _flat(saved, "saved", x, (keep.value // 4,), torch.float32)
    with _Launch(x, stream) as st:
        def new(shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=x.device)
        dx, ddt = new(x.shape, x.dtype), new(x.shape, x.dtype)
        dz = None if z is None else new(x.shape, x.dtype)
        dB, dC = new(B.shape, x.dtype), new(C.shape, x.dtype)
        dA = new((a.D, a.N))
        dD = None if D is None else new((a.D,))
        db = None if dt_bias is None else new((a.D,))
        d0 = None if initial_state is None else new((S, a.D, a.N))
        ws = new((need.value,), torch.uint8)
        for name, t, w in (("dx", dx, a.D), ("ddt", ddt, a.D), ("dz", dz, a.D),
                           ("dB", dB, a.G * a.N), ("dC", dC, a.G * a.N)):
            if t is not None:
                setattr(g, name, _rows_unchecked(t, packed, w))
        g.dA = dA.data_ptr()
        g.dD = 0 if dD is None else dD.data_ptr()
        g.ddt_bias = 0 if db is None else db.data_ptr()
        g.dinitial = 0 if d0 is None else d0.data_ptr()
        _check(lib.tg_selective_scan_backward(ctypes.byref(a), ctypes.byref(g), sp, keep.value,
                                              ws.data_ptr(), need.value, st),
               "tg_selective_scan_backward")
    return ScanGradients(dx, ddt, dA, dB, dC, dD, dz, db, d0)


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus=True,
                        slots=None, out=None, stream=None):
    """One token of each of n sequences: x, dt, z [n, channels], B, C [n, G, N]
    -> y [n, channels]; ``state`` fp32 [num_slots, channels, N] is updated in
    place. ``slots`` as in causal_conv_step."""
    import torch
    _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [n, channels], got %s" % (tuple(x.shape),))
    n = x.shape[0]
    a = _scan_args(x, dt, A, B, C, D, z, dt_bias, softplus, None, _Seqs(n, n, 0), x.shape[:1], n,
                   True)
    if state.dim() != 3:
        raise ValueError("state must be [num_slots, channels, N]")
    num = state.shape[0]
    hp = _param(state, "state", x, num, a.D, a.N)
    sp = _slots(slots, x, n)
    lib = _lib()
    with _Launch(x, stream) as st:
        y = _out(out, x, "out", x.shape)
        a.y = _rows_unchecked(y, True, a.D)
        _check(lib.tg_selective_scan_step(ctypes.byref(a), hp, num, sp, st),
               "tg_selective_scan_step")
    return y
