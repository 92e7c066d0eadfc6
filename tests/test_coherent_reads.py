"""Kernels are launched while the stream's previous kernel may still run, and wait for it before they read what it wrote.  A
read through the non-coherent path (ld.global.nc: __ldg, const __restrict__ parameters) may be served by what was cached since
the kernel's start, that is before the wait: no kernel has one."""
import glob
import os
import re

import pytest

from dense_tiled_gemm_04_gb300 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "**", "*.cu*"), recursive=True))


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.relpath(p, build.CSRC) for p in SOURCES])
def test_no_read_takes_the_non_coherent_path(path):
    with open(path) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"__ldg\b|__restrict__|ld\.global\S*\.nc|tex\.", code)
