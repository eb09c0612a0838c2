"""Where packed sequences lie (SeqMap), on the host: tests/sanitize/seq_map_driver.hip,
built with sanitizers on the host pass, holds right and wrong offsets against
the bounds that the kernels rely on. No GPU is used."""
import os
import subprocess

import pytest

from conv2d_batchnorm_silu_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_offsets_stay_in_range(tmp_path):
    if not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "seq_map")
    cmd = [B.hipcc(), "--offload-arch=" + B.ARCH, "-O1", "-g", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-I", B.INCLUDE, "-I", B.CSRC,
           os.path.join(HERE, "sanitize", "seq_map_driver.hip"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="halt_on_error=1"))
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout + r.stderr[-3000:]
