"""Fused conv2d + BatchNorm + SiLU for AMD Instinct MI355X (gfx950).

The compute path is a C-ABI shared library (``libtgconv.so``, built from
``csrc/``) of hand-written HIP kernels; ``binding`` wraps it with ctypes and
uses PyTorch only for device memory and streams; ``sequence`` does the same
for the sequence operators (layer norm, group norm, causal convolution, selective
scan, gated delta rule).
``inputs`` holds the seeded
synthetic data recipes shared by tests and the benchmark.

Importing this package does not load the shared library; the first use of a
binding name does, and fails loudly if the library is missing.
"""
from __future__ import annotations

_BINDING_NAMES = {
    "ConvBnSilu", "bn_fold", "library", "Kernel", "Dtype", "TgError", "status_string",
    "kernel_name", "library_path", "build_library", "exported_symbols", "Table", "dispatch_choose",
}
_SEQUENCE_NAMES = {
    "layer_norm", "layer_norm_train", "layer_norm_backward", "causal_conv",
    "causal_conv_backward", "causal_conv_step", "selective_scan", "selective_scan_train",
    "selective_scan_backward", "selective_scan_step", "ScanGradients",
    "gated_delta_rule", "gated_delta_rule_train", "gated_delta_rule_backward",
    "gated_delta_rule_step", "DeltaGradients", "group_norm", "group_norm_train",
    "group_norm_backward", "GroupNormGradients",
}


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import binding
        return getattr(binding, name)
    if name in _SEQUENCE_NAMES:
        from . import sequence
        return globals().setdefault(name, getattr(sequence, name))
    raise AttributeError(name)
