"""The linear-layer entry points without a GPU: struct layouts, workspace sizes, null handles."""
import ctypes
import os
import subprocess
import threading
import time

import pytest
import torch

from conftest import ROOT

STRUCTS = ["gemm_linear_args_t", "gemm_dgrad_args_t", "gemm_wgrad_args_t", "gemm_act_grad_args_t"]


@pytest.fixture(scope="module")
def lib():
    from dense_tiled_gemm_04_gb300 import build, native

    build.build()
    return native


def test_structs_are_laid_out_as_the_c_compiler_does(lib, tmp_path):
    lines = []
    for s in STRUCTS:
        lines.append(f'printf("%zu\\n", sizeof({s}));')
        lines += [f'printf("%zu\\n", offsetof({s}, {f}));' for f, _ in getattr(lib, s)._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"gemm.h\"\nint main(void) {\n" + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in STRUCTS:
        cls = getattr(lib, s)
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


@pytest.mark.parametrize("M,cols,want", [(0, 5, 0), (5, 0, 0), (-1, 8, 0), (1, 1, 256), (32, 64, 256), (33, 65, 1024),
                                         (16384, 8192, 4 * 512 * 8192), ((1 << 31) - 1, 1 << 20, 4 << 46)])
def test_workspace_bytes(lib, M, cols, want):
    assert lib.bias_grad_workspace_bytes(M, cols) == want


@pytest.mark.parametrize("M,cols", [(0, 5), (5, 0), (1, 1), (31, 63), (32, 64), (33, 65), (4097, 40), (16384, 8192), (1 << 30, 1000)])
def test_workspace_bytes_in_the_binding(lib, M, cols):
    assert lib._sums_bytes(M, cols) == lib.bias_grad_workspace_bytes(M, cols)


def test_null_handles_and_arguments(lib):
    so = lib.load()
    for name, cls in (("gemm_run_linear", lib.gemm_linear_args_t), ("gemm_run_linear_dgrad", lib.gemm_dgrad_args_t),
                      ("gemm_run_linear_wgrad", lib.gemm_wgrad_args_t), ("gemm_run_act_grad", lib.gemm_act_grad_args_t)):
        assert getattr(so, name)(None, None, None) == lib.ERR_INVALID_ARG
        assert getattr(so, name)(None, ctypes.byref(cls()), None) == lib.ERR_INVALID_ARG


def test_activation_codes_match_the_header(lib):
    text = open(os.path.join(ROOT, "include", "gemm.h")).read()
    for name, code in lib.ACTS.items():
        if name:
            assert f"GEMM_ACT_{name.upper()} = {code}" in text


def test_every_name_that_the_package_lists_resolves():
    import dense_tiled_gemm_04_gb300 as package

    assert [n for n in package.__all__ if not hasattr(package, n)] == []
    names = {}
    exec("from dense_tiled_gemm_04_gb300 import *", names)
    assert set(package.__all__) <= set(names)


class FakeGemm:
    """A handle that records its calls, as native.Gemm's stand-in; creating one takes a while."""

    made = []

    def __init__(self, device):
        time.sleep(0.02)
        self.device, self.inside, self.overlaps, self.calls = device, 0, 0, 0
        FakeGemm.made.append(self)

    def linear_dgrad(self, *args):
        self.overlaps += self.inside
        self.inside += 1
        time.sleep(0.002)
        self.inside -= 1
        self.calls += 1
        return self


class FakeTensor:
    def get_device(self):
        return 0


@pytest.fixture
def fake(lib, monkeypatch):
    monkeypatch.setattr(lib, "Gemm", FakeGemm)
    monkeypatch.setattr(lib, "_default", {})
    FakeGemm.made = []
    return lib


def test_module_functions_use_a_handle_per_stream(fake):
    # Calls on streams that are not ordered share no workspace.
    t = FakeTensor()
    a, b = fake.linear_dgrad(t, None, stream=64), fake.linear_dgrad(t, None, stream=128)
    assert a is not b and fake.linear_dgrad(t, None, stream=64) is a
    assert len(FakeGemm.made) == 2


def test_module_functions_from_several_threads(fake):
    # One handle per stream is made however many threads ask first, and its calls (two launches each) do not interleave.
    t = FakeTensor()
    threads = [threading.Thread(target=lambda s=s: [fake.linear_dgrad(t, None, stream=s) for _ in range(5)])
               for s in (64, 128) for _ in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert len(FakeGemm.made) == 2
    assert [h.calls for h in FakeGemm.made] == [20, 20] and [h.overlaps for h in FakeGemm.made] == [0, 0]


def test_module_functions_refuse_host_tensors(lib):
    x = torch.zeros((8, 8), dtype=torch.float16)
    for call in (lambda: lib.linear(x, x), lambda: lib.linear_dgrad(x, x), lambda: lib.linear_wgrad(x, x), lambda: lib.act_grad(x)):
        with pytest.raises(ValueError):
            call()
