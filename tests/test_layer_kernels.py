"""Which kernel a call of the layer operators takes, on a stand-in runtime without a GPU: the calls that the GPU
tests make to reach a kernel (tests/layer_kernels.py) do reach it."""
import os
import re
import subprocess

import pytest

import layer_kernels as lk
import precision_adam_optimizer_amd as pk  # noqa: F401  (the library is built)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "precision_adam_optimizer_amd")
DTYPES = {"fp32": 0, "bf16": 1, "fp16": 2}
FORMATS = {"e4m3": 0, "e5m2": 1}


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """launches(lines): the kernels that each call launches, as (name, template arguments)."""
    exe = str(tmp_path_factory.mktemp("kernels") / "driver")
    r = subprocess.run(["gcc", "-std=c11", "-O1", "-g", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{os.path.join(ROOT, 'tests')}", "-I/opt/rocm/include",
                        os.path.join(ROOT, "tests", "layer_kernels_driver.c"), f"-L{PKG}", "-lfp8adam", "-L/opt/rocm/lib",
                        "-lamdhip64", "-lm", "-Wl,--export-dynamic", f"-Wl,-rpath,{PKG}", "-Wl,-rpath,/opt/rocm/lib",
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
        got = [line.split() for line in r.stdout.splitlines()]
        assert len(got) == len(lines)
        return [[kernel(name) for name in names] for names in got]
    return ask


def kernel(mangled):
    """(name, template arguments that are numbers) of a kernel's mangled name."""
    name = re.search(r"\d(k_[a-z_]+?)(?:I|E|P|v|$)", mangled)
    assert name, mangled
    return name[1], tuple(-int(x) if minus else int(x) for minus, x in re.findall(r"L[ib](n?)(\d+)E", mangled))


def product_line(c):
    return (f"{'gated8' if c.gated else 'linear8'} {c.tokens} {c.rows} {c.cols} {FORMATS[c.x]} {FORMATS[c.w]} "
            f"{-1 if c.packed else DTYPES[c.dtype]} {DTYPES[c.dtype]} {int(c.keep)} {-1 if c.pack is None else FORMATS[c.pack]} {int(c.exact)}")


def test_forward_tiles(launches):
    cases = lk.products()
    reached = set()
    for (tt, wide, c), got in zip(cases, launches([product_line(c) for _, _, c in cases])):
        assert got[-1] == ("k_product", (FORMATS[c.x], FORMATS[c.w], int(c.gated), tt, int(wide))), c
        reached.add(got[-1])
    assert len(reached) == 40  # of 2 x 2 formats, linear and gated, three tiles and two with widened codes


def test_few_tokens(launches):
    cases = lk.few()
    reached = set()
    for (nt, waves, c), got in zip(cases, launches([product_line(c) for _, _, c in cases])):
        packs = c.tokens <= 4  # the product packs x itself
        assert len(got) == (1 if packs else 2)
        assert got[-1] == ("k_product_few", (FORMATS[c.x], FORMATS[c.w], int(c.gated), nt, DTYPES[c.dtype] if packs else -1, waves)), c
        reached.add(got[-1])
    # of 2 x 2 formats, linear and gated, four waves and eight: one, two and four blocks of tokens, and three types
    # that are packed here
    assert len(reached) == 8 * 2 * 6


def test_gradients(launches):
    cases = lk.gradients()
    reached = set()
    lines = [f"{'input' if c.n else 'weight'}_grad8 {c.tokens} {c.rows} {c.cols} {c.n or 1} {FORMATS[c.fmt]} {DTYPES[c.dtype]} {int(c.exact)}" for _, _, c in cases]
    for (tile, parts, c), got in zip(cases, launches(lines)):
        got = [k for k in got if k[0] != "k_split"]
        assert got[0] == ("k_grad", (int(not c.n), FORMATS[c.fmt], tile, tile, 4 if tile == 256 else 2)), c
        assert len(got) == 1 + parts and (not parts or got[1][0] == "k_grad_join"), c
        reached.add((got[0], parts))
    assert sum(k[1][2] == 256 for k, _ in reached) == 8  # either direction and format, with the sum in parts and in one
