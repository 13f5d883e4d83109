"""The list operators from a plain C11 program (tests/c_list_demo.c), which checks
its own results against double arithmetic."""
import os
import subprocess

import pytest

import precision_adam_optimizer_amd as pk  # noqa: F401  (the library is built)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "precision_adam_optimizer_amd")


def build(tmp_path) -> str:
    exe = str(tmp_path / "c_list_demo")
    r = subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
                        f"-I{os.path.join(ROOT, 'include')}", "-I/opt/rocm/include",
                        os.path.join(ROOT, "tests", "c_list_demo.c"), f"-L{PKG}", "-lfp8adam", "-L/opt/rocm/lib",
                        "-lamdhip64", "-lm", f"-Wl,-rpath,{PKG}", "-Wl,-rpath,/opt/rocm/lib", "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_c_list_caller_compiles_and_links(tmp_path):
    libs = subprocess.run(["ldd", build(tmp_path)], check=True, capture_output=True, text=True).stdout
    assert "libfp8adam.so" in libs and "torch" not in libs


@pytest.mark.gpu
def test_c_list_caller(tmp_path):
    r = subprocess.run([build(tmp_path)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "c list demo ok" in r.stdout, r.stdout + r.stderr
