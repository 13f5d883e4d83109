"""The layer operators' refusals, before any device work: argument errors of the C ABI
(include/fp8adam_layer.h) come back as codes with a message, those of the binding as
ValueError; the binding's structs, nested and packed, have the header's layout."""
import ctypes
import os
import subprocess
from types import SimpleNamespace

import pytest
import torch

import precision_adam_optimizer_amd as pk
from precision_adam_optimizer_amd import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EALIGN = -1, -2
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
U8 = torch.uint8


def test_structs_match_the_header(tmp_path):
    structs = {"fp8adam_matrix": layers.MatrixArg, "fp8adam_matrix8": layers.Matrix8Arg, "fp8adam_product8": layers.Product8Arg,
               "fp8adam_act_backward8": layers.ActBackward8Arg, "fp8adam_grad8": layers.Grad8Arg}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fp8adam_layer.h"', "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    names = {"FP8ADAM_LAYER_MAX_COLS": layers.LAYER_MAX_COLS, "FP8ADAM_LAYER_MAX_LD": layers.LAYER_MAX_LD,
             "FP8ADAM_ACT_NONE": layers.ACT_NONE, "FP8ADAM_ACT_RELU": layers.ACT_RELU, "FP8ADAM_ACT_SILU": layers.ACT_SILU,
             "FP8ADAM_ACT_GELU": layers.ACT_GELU, "FP8ADAM_SCALES_E8M0": layers.SCALES_E8M0, "FP8ADAM_SCALES_F32": layers.SCALES_F32}
    lines += [f'  printf("{n} value %d\\n", (int){n});' for n in names] + ["  return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", f"-I{os.path.join(ROOT, 'include')}",
                    "-I/opt/rocm/include", "-o", str(exe), str(src)], check=True, capture_output=True)
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in
           subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()}
    for n, v in names.items():
        assert got[(n, "value")] == v, n
    for cname, py in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, f"{cname}.{f}"


def flat(s):
    """The leaves of a ctypes struct, in order."""
    out = []
    for name, _ in s._fields_:
        v = getattr(s, name)
        for x in (list(v) if isinstance(v, ctypes.Array) else [v]):
            out += flat(x) if isinstance(x, ctypes.Structure) else [x or 0]
    return out


@pytest.mark.parametrize("packed, struct", [(layers._PRODUCT8, layers.Product8Arg), (layers._ACT_BACKWARD8, layers.ActBackward8Arg),
                                            (layers._GRAD8, layers.Grad8Arg)])
def test_packed_structs_are_the_same(packed, struct):
    assert packed.size == ctypes.sizeof(struct)
    n = len(packed.unpack(bytes(packed.size)))
    args = struct.from_buffer_copy(packed.pack(*range(1, n + 1)))
    assert flat(args) == list(range(1, n + 1))


# ------------------------------------------------------------------------ the C ABI

T, N, K = 100, 256, 300  # tokens, rows, cols


def at(i):
    return (i + 1) << 32  # far apart; nothing is read or written


def mat(i, rows, cols, dtype=pk.BF16, **kw):
    d = dict(data=at(i), ld=cols, dtype=dtype, reserved=0)
    d.update(kw)
    return layers.MatrixArg(**d)


def mat8(i, rows, cols, **kw):
    nb = -(-cols // 128)
    d = dict(codes=at(i), scales=at(i) + (1 << 31), ld=nb * 128, ld_scale=-(-nb // 4) * 4, format=pk.E4M3, scale_type=layers.SCALES_E8M0)
    d.update(kw)
    return layers.Matrix8Arg(**d)


def product(**kw):
    d = dict(tokens=T, rows=N, cols=K, x_in=mat(0, T, K), x=mat8(1, T, K), w=mat8(2, N, K), y=mat(5, T, N),
             activation=layers.ACT_GELU)
    d.update(kw)
    return layers.Product8Arg(**d)


def gated(**kw):
    return product(**{"w_up": mat8(3, N, K), **kw})


def back(**kw):
    d = dict(tokens=T, rows=N, dy=mat(0, T, N), keep=mat8(1, T, N), dz=mat(3, T, N), activation=layers.ACT_GELU)
    d.update(kw)
    return layers.ActBackward8Arg(**d)


def gated_back(**kw):
    return back(**{"keep_up": mat8(2, T, N), "dup": mat(4, T, N), **kw})


def grad(weights, **kw):
    d = dict(tokens=T, rows=N, cols=K, n=1, dy=(layers.MatrixArg * 2)(mat(0, T, N), mat(1, T, N)),
             b=(layers.Matrix8Arg * 2)(mat8(2, T if weights else N, K), mat8(3, N, K)),
             out=mat(4, N if weights else T, K, pk.F32), workspace=at(5), workspace_bytes=1 << 31)
    d.update(kw)
    return layers.Grad8Arg(**d)


def two(a, b):
    return (type(a) * 2)(a, b)


def refused(fn, args, code, text):
    assert getattr(layers._lib(), fn)(ctypes.byref(args) if args is not None else None, None) == code, (text, pk.fp8adam_last_error())
    assert text in pk.fp8adam_last_error()


MAX = layers.LAYER_MAX_COLS
SIZES = [(dict(tokens=-1), "number of tokens"), (dict(tokens=1 << 31), "number of tokens"), (dict(rows=0), "rows and cols"),
         (dict(rows=MAX + 1), "rows and cols")]


@pytest.mark.parametrize("make, fn", [(product, "fp8adam_linear8"), (gated, "fp8adam_gated8")])
@pytest.mark.parametrize("kw, code, text", [(kw, EINVAL, t) for kw, t in SIZES] + [
    (dict(cols=0), EINVAL, "rows and cols"), (dict(cols=MAX + 1), EINVAL, "rows and cols"),
    (dict(activation=-1), EINVAL, "bad activation"), (dict(activation=4), EINVAL, "bad activation"),
    (dict(x_in=mat(0, T, K, ld=K - 1)), EINVAL, "ld of x_in"), (dict(x_in=mat(0, T, K, ld=(1 << 21) + 1)), EINVAL, "ld of x_in"),
    (dict(x_in=mat(0, T, K, dtype=3)), EINVAL, "bad dtype of x_in"), (dict(x_in=mat(0, T, K, data=at(0) + 1)), EALIGN, "x_in"),
    (dict(x=mat8(1, T, K, codes=None)), EINVAL, "x is null"), (dict(x=mat8(1, T, K, scales=None)), EINVAL, "x is null"),
    (dict(x=mat8(1, T, K, codes=at(1) + 8)), EALIGN, "codes of x"), (dict(x=mat8(1, T, K, scales=at(1) + 2)), EALIGN, "scales of x"),
    (dict(x=mat8(1, T, K, ld=256)), EINVAL, "ld of x"), (dict(x=mat8(1, T, K, ld=392)), EINVAL, "ld of x"),
    (dict(x=mat8(1, T, K, ld_scale=3)), EINVAL, "ld_scale of x"), (dict(x=mat8(1, T, K, ld_scale=6)), EINVAL, "ld_scale of x"),
    (dict(x=mat8(1, T, K, scale_type=layers.SCALES_F32)), EINVAL, "must be E8M0"),
    (dict(x=mat8(1, T, K, scale_type=2)), EINVAL, "bad scale_type of x"),
    (dict(w=mat8(2, N, K, format=2)), EINVAL, "bad format of w"), (dict(w=mat8(2, N, K, format=-1)), EINVAL, "bad format of w"),
    (dict(w=mat8(2, N, K, scale_type=layers.SCALES_F32, ld_scale=2)), EINVAL, "ld_scale of w"),
    (dict(y=layers.MatrixArg()), EINVAL, "y and y8 are null"),
    (dict(y=mat(5, T, N, ld=N - 1)), EINVAL, "ld of y"), (dict(y=mat(5, T, N, pk.F32, data=at(5) + 2)), EALIGN, "y is not"),
    (dict(y8=mat8(6, T, N, ld=128)), EINVAL, "ld of y8"), (dict(keep=mat8(6, T, N, format=9)), EINVAL, "bad format of keep"),
    (dict(y=mat(0, T, N)), EINVAL, "x_in and y"),          # over the input
    (dict(y=mat(5, T, N, data=at(2))), EINVAL, "w and y"),  # over the weights
    (dict(y8=mat8(1, T, N)), EINVAL, "overlaps"),
])
def test_products_refuse(make, fn, kw, code, text):
    if make is gated and "keep" in kw:
        kw = {**kw, "keep_up": mat8(7, T, N, format=9)}
    refused(fn, make(**kw), code, text)


@pytest.mark.parametrize("make, fn, kw, text", [
    (product, "fp8adam_linear8", dict(w_up=mat8(3, N, K)), "takes no w_up"),
    (product, "fp8adam_linear8", dict(keep_up=mat8(3, T, N)), "takes no w_up"),
    (product, "fp8adam_linear8", dict(bias=mat(7, 1, N, dtype=5)), "bad dtype of bias"),
    (product, "fp8adam_linear8", dict(residual=mat(7, T, N, ld=N - 1)), "ld of residual"),
    (product, "fp8adam_linear8", dict(residual=mat(5, T, N, ld=N + 1)), "residual and y"),           # another ld
    (product, "fp8adam_linear8", dict(residual=mat(5, T, N, data=at(5) + 2)), "residual and y"),      # an element off
    (product, "fp8adam_linear8", dict(residual=mat(5, T, N, pk.F16)), "residual and y"),              # another type
    (product, "fp8adam_linear8", dict(bias=mat(5, 1, N, data=at(5) + 64)), "bias and y"),
    (product, "fp8adam_linear8", dict(keep=mat8(5, T, N)), "y and keep"),
    (gated, "fp8adam_gated8", dict(w_up=layers.Matrix8Arg()), "ld of w_up"),
    (gated, "fp8adam_gated8", dict(w_up=mat8(3, N, K, format=pk.E5M2)), "one format"),
    (gated, "fp8adam_gated8", dict(w_up=mat8(3, N, K, scale_type=layers.SCALES_F32)), "one type of scales"),
    (gated, "fp8adam_gated8", dict(bias=mat(7, 1, N)), "no bias"),
    (gated, "fp8adam_gated8", dict(residual=mat(7, T, N)), "no residual"),
    (gated, "fp8adam_gated8", dict(keep=mat8(7, T, N)), "together"),
    (gated, "fp8adam_gated8", dict(keep_up=mat8(7, T, N)), "together"),
    (gated, "fp8adam_gated8", dict(keep=mat8(7, T, N), keep_up=mat8(8, T, N, format=pk.E5M2)), "one format"),
    (gated, "fp8adam_gated8", dict(keep=mat8(7, T, N), keep_up=mat8(7, T, N)), "keep and keep_up"),
])
def test_products_refuse_what_is_not_theirs(make, fn, kw, text):
    refused(fn, make(**kw), EINVAL, text)


@pytest.mark.parametrize("make, fn, kw, code, text", [(back, "fp8adam_linear8_backward", kw, EINVAL, t) for kw, t in SIZES] + [
    (gated_back, "fp8adam_gated8_backward", kw, EINVAL, t) for kw, t in SIZES] + [
    (back, "fp8adam_linear8_backward", dict(activation=7), EINVAL, "bad activation"),
    (back, "fp8adam_linear8_backward", dict(dy=mat(0, T, N, data=None)), EINVAL, "dy is null"),
    (back, "fp8adam_linear8_backward", dict(dz=mat(3, T, N, pk.F32)), EINVAL, "dy's dtype"),
    (back, "fp8adam_linear8_backward", dict(dz=mat(0, T, N, ld=N + 1)), EINVAL, "dy and dz"),
    (back, "fp8adam_linear8_backward", dict(keep=layers.Matrix8Arg()), EINVAL, "ld of keep"),
    (back, "fp8adam_linear8_backward", dict(keep_up=mat8(2, T, N)), EINVAL, "takes no keep_up"),
    (back, "fp8adam_linear8_backward", dict(dup=mat(4, T, N)), EINVAL, "no dup"),
    (back, "fp8adam_linear8_backward", dict(activation=0), EINVAL, "dz is dy"),
    (back, "fp8adam_linear8_backward", dict(activation=0, keep=layers.Matrix8Arg(), dz=layers.MatrixArg()), EINVAL, "nothing to do"),
    (back, "fp8adam_linear8_backward", dict(bias_grad=mat(6, 1, N), workspace_bytes=1 << 20), EINVAL, "workspace is null"),
    (back, "fp8adam_linear8_backward", dict(bias_grad=mat(6, 1, N), workspace=at(7), workspace_bytes=2047), EINVAL, "fewer than 2048"),
    (back, "fp8adam_linear8_backward", dict(bias_grad=mat(6, 1, N), workspace=at(7) + 8, workspace_bytes=2048), EALIGN, "16-byte"),
    (back, "fp8adam_linear8_backward", dict(bias_grad=mat(6, 1, N), workspace=at(3), workspace_bytes=2048), EINVAL, "dz and workspace"),
    (back, "fp8adam_linear8_backward", dict(bias_grad=mat(0, 1, N), workspace=at(7), workspace_bytes=2048), EINVAL, "dy and bias_grad"),
    (gated_back, "fp8adam_gated8_backward", dict(bias_grad=mat(6, 1, N), workspace=at(7), workspace_bytes=1 << 20), EINVAL, "no bias_grad"),
    (gated_back, "fp8adam_gated8_backward", dict(dup=mat(3, T, N)), EINVAL, "dz and dup"),
    (gated_back, "fp8adam_gated8_backward", dict(dz=mat(0, T, N), dup=mat(0, T, N)), EINVAL, "dz and dup"),
    (gated_back, "fp8adam_gated8_backward", dict(dup=mat(4, T, N, pk.F16)), EINVAL, "dy's dtype"),
    (gated_back, "fp8adam_gated8_backward", dict(keep_up=layers.Matrix8Arg()), EINVAL, "ld of keep_up"),
    (gated_back, "fp8adam_gated8_backward", dict(keep=mat8(3, T, N)), EINVAL, "keep and dz"),
])
def test_backward_refuses(make, fn, kw, code, text):
    refused(fn, make(**kw), code, text)


GRADS = [("fp8adam_weight_grad8", True), ("fp8adam_input_grad8", False)]


@pytest.mark.parametrize("fn, weights", GRADS)
@pytest.mark.parametrize("kw, code, text", [(kw, EINVAL, t) for kw, t in SIZES] + [
    (dict(cols=0), EINVAL, "rows and cols"), (dict(n=0), EINVAL, "n must be 1"), (dict(n=3), EINVAL, "n must be 1"),
    (dict(dy=two(mat(0, T, N, dtype=8), mat(1, T, N))), EINVAL, "dtype of dy"),
    (dict(dy=two(mat(0, T, N, data=None), mat(1, T, N))), EINVAL, "dy is null"),
    (dict(dy=two(mat(0, T, N, ld=N - 8), mat(1, T, N))), EINVAL, "ld of dy"),
    (dict(b=two(mat8(2, T, K, ld=256), mat8(3, N, K))), EINVAL, "ld of"),
    (dict(out=mat(4, 1, K, data=None)), EINVAL, "out is null"), (dict(out=mat(4, 1, K, ld=K - 1)), EINVAL, "ld of out"),
    (dict(out=mat(4, 1, K, data=at(4) + 1)), EALIGN, "out is not"), (dict(out=mat(0, 1, K)), EINVAL, "dy and out"),
    (dict(out=mat(2, 1, K)), EINVAL, "overlaps"),
    (dict(workspace=None, dy=two(mat(0, T, N, pk.F32), mat(1, T, N, pk.F32))), EINVAL, "workspace is null"),
    (dict(workspace_bytes=100, dy=two(mat(0, T, N, pk.F32), mat(1, T, N, pk.F32))), EINVAL, "workspace has fewer"),
    (dict(workspace=at(5) + 4, dy=two(mat(0, T, N, pk.F32), mat(1, T, N, pk.F32))), EALIGN, "16-byte"),
    (dict(workspace=at(4), dy=two(mat(0, T, N, pk.F32), mat(1, T, N, pk.F32))), EINVAL, "out and workspace"),
])
def test_gradients_refuse(fn, weights, kw, code, text):
    refused(fn, grad(weights, **kw), code, text)


def test_pairs_of_layers_refuse():
    for kw, text in ((dict(dy=two(mat(0, T, N), mat(1, T, N, pk.F32))), "more than one"),
                     (dict(b=two(mat8(2, N, K), mat8(3, N, K, format=pk.E5M2))), "one format"),
                     (dict(b=two(mat8(2, N, K), mat8(3, N, K, scale_type=layers.SCALES_F32))), "one type of scales"),
                     (dict(b=two(mat8(2, N, K), layers.Matrix8Arg())), "ld of")):
        refused("fp8adam_input_grad8", grad(False, n=2, **kw), EINVAL, text)
    refused("fp8adam_weight_grad8", grad(True, n=2), EINVAL, "n must be 1")


def test_packing_refuses():
    L = layers._lib()

    def call(fn, a, b, rows, cols, code, text):
        order = (a, b) if fn == "fp8adam_pack8" else (b, a)
        assert getattr(L, fn)(*(None if v is None else ctypes.byref(v) for v in order), rows, cols, None) == code, text
        assert text in pk.fp8adam_last_error()
    for fn in ("fp8adam_pack8", "fp8adam_unpack8"):
        ok, ok8 = mat(0, T, K), mat8(1, T, K)
        call(fn, None, ok8, T, K, EINVAL, "null")
        call(fn, ok, None, T, K, EINVAL, "null")
        call(fn, ok, ok8, -1, K, EINVAL, "tokens")
        call(fn, ok, ok8, T, 0, EINVAL, "rows and cols")
        call(fn, ok, ok8, T, MAX + 1, EINVAL, "rows and cols")
        call(fn, mat(0, T, K, dtype=3), ok8, T, K, EINVAL, "dtype of x")
        call(fn, mat(0, T, K, data=None), ok8, T, K, EINVAL, "x is null")
        call(fn, mat(0, T, K, data=at(0) + 1), ok8, T, K, EALIGN, "x is not")
        call(fn, ok, mat8(1, T, K, codes=at(1) + 4), T, K, EALIGN, "codes")
        call(fn, ok, mat8(0, T, K), T, K, EINVAL, "overlaps")
    call("fp8adam_pack8", mat(0, T, K), mat8(1, T, K, scale_type=layers.SCALES_F32), T, K, EINVAL, "must be E8M0")


def test_null_arguments():
    for fn in layers.LAYER_EXPORTS[2:]:
        L = layers._lib()
        code = getattr(L, fn)(None) if fn.endswith("_workspace") else getattr(L, fn)(None, None)
        assert code == EINVAL and "args is null" in pk.fp8adam_last_error()


def test_workspaces():
    """What a call needs, from sizes and types alone; a negative code for arguments that are refused."""
    L = layers._lib()
    ask = lambda fn, a: getattr(L, fn + "_workspace")(ctypes.byref(a))  # noqa: E731
    assert ask("fp8adam_linear8_backward", back()) == 0
    assert ask("fp8adam_linear8_backward", back(bias_grad=mat(6, 1, N))) == 2 * 256 * 4  # two chunks of 64 tokens
    assert ask("fp8adam_linear8_backward", back(tokens=0, bias_grad=mat(6, 1, N))) == 0
    assert ask("fp8adam_linear8_backward", back(tokens=-1)) == EINVAL
    for fn, weights in GRADS:
        assert ask(fn, grad(weights, tokens=0)) == 0
        assert ask(fn, grad(weights, n=4)) == EINVAL
        base = ask(fn, grad(weights))
        split = ask(fn, grad(weights, dy=two(mat(0, T, N, pk.F32), mat(1, T, N))))
        assert split - base >= 2 * T * N * 2  # both bf16 parts of dy
        one = ask(fn, grad(weights, dy=two(mat(0, T, N, data=at(0) + 2), mat(1, T, N))))
        assert one - base >= T * N * 2  # a copy whose rows are whole 16-byte pieces


# ---------------------------------------------------------------------- the binding

def u8(*shape):
    return torch.zeros(shape, dtype=U8)


def packed(rows, cols, **kw):
    nb = -(-cols // 128)
    return pk.Packed8(u8(rows, nb * 128), u8(rows, nb), cols, **kw)


@pytest.mark.parametrize("args, text", [
    ((torch.zeros(4, 128), u8(4, 1), 128), "codes must be a matrix"), ((u8(4 * 128), u8(4, 1), 128), "codes must be a matrix"),
    ((u8(4, 128), u8(4, 1), 0), "cols must be positive"), ((u8(4, 128), u8(4, 1), 129), "codes must have 256 columns"),
    ((u8(4, 100), u8(4, 1), 100), "codes must have 128 columns"), ((u8(4, 128), u8(3, 1), 128), "scales must be"),
    ((u8(4, 256), u8(4, 1), 200), "scales must be"), ((u8(4, 128), u8(4), 128), "scales must be"),
    ((u8(4, 128), torch.zeros(4, 1, dtype=F16), 128), "scales must be"),
    ((u8(128, 4).t(), u8(4, 1), 128), "rows of codes"), ((u8(1, 128).expand(4, 128), u8(4, 1), 128), "rows of codes"),
    ((u8(4, 256), u8(2, 4).t(), 256), "rows of scales"),
])
def test_packed8_refuses(args, text):
    with pytest.raises(ValueError, match=text):
        pk.Packed8(*args)
    with pytest.raises(KeyError):
        pk.Packed8(u8(4, 128), u8(4, 1), 128, "e3m4")


def test_packed8_types():
    """float8 tensors give their own format; float8 scales are bytes; rows of scales become whole dwords."""
    p = pk.Packed8(u8(3, 256).view(torch.float8_e5m2), u8(3, 2).view(torch.float8_e8m0fnu), 200)
    assert p.fmt == "e5m2" and p.scale_type == layers.SCALES_E8M0 and p.scales.shape == (3, 4)
    codes, scales = p.values()
    assert codes.shape == (3, 200) and codes.dtype == torch.float8_e5m2 and scales.shape == (3, 2) and scales.dtype == torch.float8_e8m0fnu
    q = pk.Packed8(u8(3, 256), torch.ones(3, 2), 256)
    assert q.scale_type == layers.SCALES_F32 and q.values()[1].dtype == F32
    wide = u8(3, 8)
    assert pk.Packed8(u8(3, 512), wide[:, :4], 512).scales.data_ptr() == wide.data_ptr()


def test_from_quantizer_refuses():
    def q(v, granularity="block128", mode="pow2"):
        return SimpleNamespace(values=[v], codes=[u8(v.numel())], scales=[torch.ones(-(-v.numel() // 128))], formats=["e4m3"],
                               granularity=granularity, scale_mode=mode)
    assert pk.Packed8.from_quantizer(q(torch.zeros(4, 256)), 0).rows == 4
    for v, kw, text in ((torch.zeros(4, 256), dict(granularity="tensor"), "block128"), (torch.zeros(4, 256), dict(mode="exact"), "block128"),
                        (torch.zeros(4, 100), {}, "multiple of 128"), (torch.zeros(512), {}, "contiguous matrix"),
                        (torch.zeros(128, 4).t(), {}, "contiguous matrix"), (torch.zeros(0, 128), {}, "contiguous matrix")):
        with pytest.raises(ValueError, match=text):
            pk.Packed8.from_quantizer(q(v, **kw), 0)


def bf(*shape):
    return torch.zeros(shape, dtype=BF16)


@pytest.mark.parametrize("call, text", [
    (lambda: pk.pack8(bf(4)), "at least two dimensions"), (lambda: pk.pack8(bf(4, 6).double()), "must be float32"),
    (lambda: pk.pack8(bf(6, 4).t()), "rows of x must be contiguous"), (lambda: pk.pack8(bf(4, 6, 8).transpose(0, 1)), "do not fold"),
    (lambda: pk.pack8(bf(4, 6)), "on a GPU"), (lambda: pk.unpack8(packed(4, 6)), "on a GPU"),
    (lambda: pk.unpack8(packed(4, 6), torch.float64), "dtype must be"), (lambda: pk.unpack8(packed(4, 6), out=bf(4, 7)), "out must have 4 rows of 6"),
    (lambda: pk.linear8(bf(4, 6), bf(8, 6)), "weights must be a Packed8"),
    (lambda: pk.linear8(bf(4, 7), packed(8, 6)), "x must have 4 rows of 6"),
    (lambda: pk.linear8(packed(4, 7), packed(8, 6)), "x must have 4 rows of 6"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), bias=bf(7)), "bias must be contiguous, with 8"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), bias=bf(16)[::2]), "bias must be contiguous"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), bias=bf(8).double()), "bias must be float32"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), residual=bf(4, 7)), "residual must have 4 rows of 8"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), activation="tanh"), "activation must be one of"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), dtype=None), "nothing to write"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), dtype=torch.float64), "dtype must be"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), out=bf(4, 9)), "out must have 4 rows of 8"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6), out=bf(8, 4).t()), "rows of out must be contiguous"),
    (lambda: pk.linear8(bf(4, 6), packed(8, 6)), "on a GPU"),
    (lambda: pk.gated8(bf(4, 6), packed(8, 6), None), "weights must be a Packed8"),
    (lambda: pk.gated8(bf(4, 6), packed(8, 6), packed(9, 6)), "w_up must have 8 rows of 6"),
    (lambda: pk.gated8(bf(4, 6), packed(8, 6), packed(8, 6)), "on a GPU"),
    (lambda: pk.gated8_backward(bf(4, 8), packed(4, 8), packed(4, 9)), "up must have 4 rows of 8"),
    (lambda: pk.gated8_backward(bf(4, 9), packed(4, 8), packed(4, 8)), "dy must have 4 rows of 8"),
    (lambda: pk.gated8_backward(bf(4, 8), packed(4, 8), packed(4, 8), outs=(bf(4, 8), bf(4, 7))), "dup must have"),
    (lambda: pk.gated8_backward(bf(4, 8), packed(4, 8), packed(4, 8)), "on a GPU"),
    (lambda: pk.linear8_backward(bf(4, 8), packed(4, 8)), "z is given with an activation"),
    (lambda: pk.linear8_backward(bf(4, 8), activation="gelu"), "z is given with an activation"),
    (lambda: pk.linear8_backward(bf(4, 8), out=bf(4, 8)), "out must be None"),
    (lambda: pk.linear8_backward(bf(4, 8), packed(4, 9), activation="gelu"), "z must have 4 rows of 8"),
    (lambda: pk.linear8_backward(bf(4, 8), packed(4, 8), activation="gelu", bias_grad=bf(9)), "bias_grad must be"),
    (lambda: pk.linear8_backward(bf(4, 8), packed(4, 8), activation="gelu"), "on a GPU"),
    (lambda: pk.weight_grad8(bf(4, 8), bf(4, 6)), "x must be a Packed8"),
    (lambda: pk.weight_grad8(bf(5, 8), packed(4, 6)), "dy must have 4 rows"),
    (lambda: pk.weight_grad8(bf(4, 8), packed(4, 6), accumulate=True), "accumulate needs out"),
    (lambda: pk.weight_grad8(bf(4, 8), packed(4, 6), bf(8, 7)), "out must have 8 rows of 6"),
    (lambda: pk.weight_grad8(bf(4, 8), packed(4, 6)), "on a GPU"),
    (lambda: pk.input_grad8([bf(4, 8)], [packed(8, 6)] * 2), "one gradient per layer"),
    (lambda: pk.input_grad8([bf(4, 8)] * 3, [packed(8, 6)] * 3), "one gradient per layer"),
    (lambda: pk.input_grad8([], []), "one gradient per layer"),
    (lambda: pk.input_grad8(bf(4, 8), bf(8, 6)), "weights must be a Packed8"),
    (lambda: pk.input_grad8([bf(4, 8)] * 2, [packed(8, 6), packed(9, 6)]), "second weights must have"),
    (lambda: pk.input_grad8([bf(4, 8)] * 2, [packed(8, 6), packed(8, 6, fmt="e5m2")]), "one format"),
    (lambda: pk.input_grad8([bf(4, 8), bf(4, 8).float()], [packed(8, 6)] * 2), "one type of dy"),
    (lambda: pk.input_grad8(bf(4, 8), packed(8, 6), accumulate=True), "accumulate needs out"),
    (lambda: pk.input_grad8(bf(4, 9), packed(8, 6)), "dy must have 4 rows of 8"),
    (lambda: pk.input_grad8(bf(4, 8), packed(8, 6)), "on a GPU"),
])
def test_the_binding_refuses(call, text):
    with pytest.raises(ValueError, match=text):
        call()
