"""Static checks of the sequence operators' compiled code, from the built library (CPU
only). The delta rule's walks wait for LDS by hand before a barrier that does not wait for
global memory; a generic (flat) access counts on both and is neither. Memory is written
through vector stores only, and fp32 arithmetic is never packed."""
import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

import conv2d_batchnorm_silu_amd as tg
from conv2d_batchnorm_silu_amd import build as B

isa = pytest.importorskip("test_isa")

FLAT = re.compile(r"^\s*flat_\w+\s")
PACKED = re.compile(r"^\s*v_pk_(add|mul|fma)_f32\b")
# Kernels that every build has, each in a code object of its own source.
KERNELS = ["delta_prep", "delta_step", "delta_forward", "delta_backward", "delta_grads", "delta_join", "map_stats", "map_apply",
           "map_sums", "map_grads", "heads", "column_sums"]


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    """{file: disassembly lines} of the library's device code objects."""
    d = tmp_path_factory.mktemp("isa")
    tg.library()
    shutil.copy(B.LIB_PATH, d / "lib.so")
    dump = os.path.join(os.path.dirname(os.path.dirname(B.hipcc())), "llvm", "bin", "llvm-objdump")
    subprocess.run([dump, "--offloading", "lib.so"], cwd=d, check=True, capture_output=True)

    def read(name):
        r = subprocess.run([dump, "-d", "--no-show-raw-insn", name], cwd=d, check=True, capture_output=True, text=True)
        found = {"scalar stores": [], "packed": [], "flat": [], "kernels": set()}
        kernel = ""
        for line in r.stdout.splitlines():
            if line.endswith(">:"):
                kernel = line.split("<")[1][:-2]
                found["kernels"].add(kernel)
            elif isa.SCALAR_STORE.match(line):
                found["scalar stores"].append((kernel, line.strip()))
            elif PACKED.match(line):
                found["packed"].append((kernel, line.strip()))
            elif FLAT.match(line):
                found["flat"].append((kernel, line.strip()))
        return found
    with cf.ThreadPoolExecutor(max_workers=min(6, os.cpu_count() or 1)) as ex:
        return list(ex.map(read, [n for n in sorted(os.listdir(d)) if B.ARCH in n]))


def test_all_kernels_are_seen(objects):
    names = {k for o in objects for k in o["kernels"]}
    for want in KERNELS:
        assert any(("%d%s" % (len(want), want)) in k for k in names), want


def test_no_scalar_stores_and_no_packed_arithmetic(objects):
    for o in objects:
        assert not o["scalar stores"] and not o["packed"], (o["scalar stores"] + o["packed"])[:5]


def test_no_flat_accesses_of_the_delta_rule(objects):
    bad = [f for o in objects for f in o["flat"] if "delta_" in f[0]]
    assert not bad, bad[:5]
