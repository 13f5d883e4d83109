"""The plan builders' host code under AddressSanitizer: the library's units are
built again with the sanitizer on the host side only, and
tests/list_abi_sanitize_driver.c builds plans over long mixed lists and lists that
are refused.  No GPU is needed."""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from precision_adam_optimizer_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang"


@pytest.mark.slow
@pytest.mark.skipif(not os.path.exists(CLANG) or shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                    reason="ROCm compilers not available")
def test_list_host_code_is_clean_under_asan(tmp_path):
    host_asan = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fno-omit-frame-pointer"]

    def run(cmd, **kw):
        r = subprocess.run(cmd, capture_output=True, text=True, **kw)
        assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
        return r

    def compile_unit(src):
        out = str(tmp_path / (os.path.basename(src) + ".o"))
        cmd = b.compile_command(src, out)
        cmd[cmd.index("-O3")] = "-O1"
        run(cmd[:-3] + host_asan + cmd[-3:])
        return out

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_unit, b.UNITS))
    lib = str(tmp_path / "libfp8adam.so")
    link = b.link_command(objs, lib)
    run(link[:1] + ["-Xarch_host", "-fsanitize=address"] + link[1:])
    exe = str(tmp_path / "list_driver")
    run([CLANG, "-std=c11", "-g", "-O1", "-fsanitize=address", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
         f"-I{os.path.join(ROOT, 'include')}", "-I/opt/rocm/include",
         os.path.join(ROOT, "tests", "list_abi_sanitize_driver.c"), f"-L{tmp_path}", "-lfp8adam", "-L/opt/rocm/lib",
         "-lamdhip64", f"-Wl,-rpath,{tmp_path}", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    r = run([exe], timeout=300)
    assert "list abi driver done, 0 failures" in r.stdout
    assert "Sanitizer" not in r.stderr, r.stderr[-4000:]
