"""Errors of the HIP runtime in the layer operators, on a stand-in runtime (tests/stub_hip.h), without
a GPU: launches are judged by their own result, a call that fails leaves no error behind, and the
calls allocate, copy and wait for nothing."""
import os
import subprocess

import precision_adam_optimizer_amd as pk  # noqa: F401  (the library is built)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "precision_adam_optimizer_amd")


def test_layer_launch_errors(tmp_path):
    exe = str(tmp_path / "driver")
    r = subprocess.run(["gcc", "-std=c11", "-O1", "-g", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(ROOT, 'tests')}", "-I/opt/rocm/include",
                        os.path.join(ROOT, "tests", "layer_launch_error_driver.c"), f"-L{PKG}", "-lfp8adam", "-L/opt/rocm/lib",
                        "-lamdhip64", "-lm", "-Wl,--export-dynamic", f"-Wl,-rpath,{PKG}", "-Wl,-rpath,/opt/rocm/lib",
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "launch errors ok" in r.stdout, r.stdout + r.stderr
