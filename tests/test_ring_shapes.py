"""Host check of the rings that the layer norm's kernels are launched with
(tests/cuda/ring_shapes.cu): what the host sizes is what the kernel lays out."""

import os
import subprocess

from dense_int8_matrix_gb300 import build as build_mod

HERE = os.path.dirname(os.path.abspath(__file__))


def test_rings_are_the_kernels(tmp_path):
    exe = str(tmp_path / "ring_shapes")
    subprocess.run([build_mod.nvcc_path(), *build_mod.ARCH, "-std=c++17", "-I" + build_mod.CSRC, "-I" + build_mod.INCLUDE, "-o", exe,
                    os.path.join(HERE, "cuda", "ring_shapes.cu")], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
