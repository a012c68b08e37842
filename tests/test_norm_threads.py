"""The norms' calls from two host threads at once, in a plain C program
(tests/c_abi/norm_threads.c): Python's own threads hardly ever run two calls side
by side."""

import os
import subprocess

import pytest

from tensor_transformer_mlp_forward_gb300 import build
from tests.test_c_abi import OUT_DIR, cuda_lib_dir, cuda_root

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "norm_threads.c")
EXE = os.path.join(OUT_DIR, "norm_threads")


@pytest.fixture(scope="module")
def exe():
    build.build()
    os.makedirs(OUT_DIR, exist_ok=True)
    root = cuda_root()
    libdir, pkg = cuda_lib_dir(root), os.path.dirname(build.LIB)
    cmd = ["gcc", "-std=c99", "-D_POSIX_C_SOURCE=200809L", "-Wall", "-Wextra", "-Werror", "-O2", "-I", build.INCLUDE,
           "-I", os.path.join(root, "include"), SRC, "-o", EXE, "-L", pkg, "-ltpmlp", "-L", libdir, "-lcudart",
           "-lpthread", f"-Wl,-rpath,{pkg}:{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, " ".join(cmd) + "\n" + r.stdout + r.stderr
    return EXE


def test_rejects_bad_arguments(exe):
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 2 and "usage" in r.stderr
    assert subprocess.run([exe, "backward", "0", "8", "8"], capture_output=True).returncode == 2


@pytest.mark.gpu
# the same kernel with other amounts of shared memory: three and two CTAs an
# SM, clusters of few and of many warps a CTA
@pytest.mark.parametrize("widths", [(2560, 4096), (10240, 16384)])
def test_two_threads_of_other_widths(exe, widths):
    r = subprocess.run([exe, "backward", "100000", *map(str, widths)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_two_threads_of_residual_norms(exe):
    # rows staged in shared memory, of different sizes
    r = subprocess.run([exe, "residual", "100000", "32776", "49152"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
