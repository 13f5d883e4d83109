"""The list operators' refusals, before any device work: argument errors of the
C ABI (include/fp8adam_list.h) come back as codes with a message, those of the
binding as ValueError; and the binding's structs have the header's layout."""
import ctypes
import os
import subprocess

import pytest
import torch

import precision_adam_optimizer_amd as pk
from precision_adam_optimizer_amd import lists

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EALIGN = -1, -2
MOST = (((1 << 32) - 1) // 256 & ~7) * 1024  # elements of one plan


def test_structs_match_the_header(tmp_path):
    structs = {"fp8adam_adamw_tensor": pk.AdamwTensorArg, "fp8adam_adamw_config": pk.AdamwConfigArg,
               "fp8adam_adamw_hparams": pk.AdamwHParamsArg, "fp8adam_clip_tensor": pk.ClipTensorArg,
               "fp8adam_quant_tensor": pk.QuantTensorArg, "fp8adam_quant_config": pk.QuantConfigArg}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fp8adam_list.h"', "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    lines += ['  printf("max groups %d\\n", FP8ADAM_MAX_GROUPS);', "  return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines) + "\n")
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", f"-I{os.path.join(ROOT, 'include')}",
                    "-I/opt/rocm/include", "-o", str(exe), str(src)], check=True, capture_output=True)
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in
           subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()}
    assert got.pop(("max", "groups")) == pk.MAX_GROUPS
    for cname, py in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, f"{cname}.{f}"


def refused(fn, struct, tensors, cfg, code, text):
    L = lists._lib()
    h = ctypes.c_void_p(1)
    arr = (struct * max(1, len(tensors)))(*tensors)
    args = [ctypes.byref(h), arr, len(tensors)] + ([] if cfg is None else [ctypes.byref(cfg)]) + [None]
    assert getattr(L, fn)(*args) == code, (text, pk.fp8adam_last_error())
    assert text in pk.fp8adam_last_error()
    assert h.value is None  # no handle


def adamw_tensor(**kw):
    d = dict(param=1 << 12, grad=2 << 12, copy=None, m=3 << 12, v=4 << 12, m_scale=5 << 12, v_scale=6 << 12, numel=100,
             param_dtype=pk.F32, grad_dtype=pk.BF16, copy_dtype=0, moments=pk.MOMENTS_32, group=0, reserved=0)
    d.update(kw)
    return pk.AdamwTensorArg(**d)


@pytest.mark.parametrize("kw, cfg, code, text", [
    (dict(param=None), (1, 0, 1), EINVAL, "param of tensor 0 is null"),
    (dict(grad=None), (1, 0, 1), EINVAL, "grad of tensor 0 is null"),
    (dict(v=None), (1, 0, 1), EINVAL, "v of tensor 0 is null"),
    (dict(moments=pk.MOMENTS_8, v_scale=None), (1, 0, 1), EINVAL, "v_scale of tensor 0 is null"),
    (dict(param=(1 << 12) + 2), (1, 0, 1), EALIGN, "param of tensor 0 is not aligned"),
    (dict(grad=(2 << 12) + 1), (1, 0, 1), EALIGN, "grad of tensor 0 is not aligned"),
    (dict(moments=pk.MOMENTS_8, m_scale=(5 << 12) + 2), (1, 0, 1), EALIGN, "m_scale of tensor 0 is not aligned"),
    (dict(numel=-1), (1, 0, 1), EINVAL, "negative"),
    (dict(numel=MOST + 1), (1, 0, 1), EINVAL, "too many elements"),
    (dict(numel=1 << 62), (1, 0, 1), EINVAL, "too many elements"),
    (dict(param_dtype=3), (1, 0, 1), EINVAL, "bad dtype of tensor 0"),
    (dict(grad_dtype=-1), (1, 0, 1), EINVAL, "bad dtype of tensor 0"),
    (dict(copy=7 << 12, copy_dtype=pk.F32), (1, 0, 1), EINVAL, "copy of tensor 0"),
    (dict(copy=7 << 12, copy_dtype=pk.BF16, param_dtype=pk.BF16), (1, 0, 1), EINVAL, "copy of tensor 0"),
    (dict(moments=2), (1, 0, 1), EINVAL, "bad moments of tensor 0"),
    (dict(group=1), (1, 0, 1), EINVAL, "group of tensor 0"),
    (dict(group=-1), (2, 0, 1), EINVAL, "group of tensor 0"),
    (dict(), (0, 0, 1), EINVAL, "n_groups"),
    (dict(), (pk.MAX_GROUPS + 1, 0, 1), EINVAL, "n_groups"),
    (dict(), (1, 2, 1), EINVAL, "m_format"),
    # memory a step writes overlaps other memory of the list
    (dict(m=(1 << 12) + 396), (1, 0, 1), EINVAL, "overlaps"),
    (dict(grad=(3 << 12) + 4, grad_dtype=pk.F32), (1, 0, 1), EINVAL, "overlaps"),
    (dict(v=3 << 12), (1, 0, 1), EINVAL, "overlaps"),
])
def test_adamw_plan_refuses(kw, cfg, code, text):
    refused("fp8adam_adamw_plan", pk.AdamwTensorArg, [adamw_tensor(**kw)], pk.AdamwConfigArg(*cfg, 0), code, text)


def test_adamw_plan_refuses_lists():
    cfg = pk.AdamwConfigArg(1, 0, 1, 0)
    refused("fp8adam_adamw_plan", pk.AdamwTensorArg, [], cfg, EINVAL, "n must be positive")
    refused("fp8adam_adamw_plan", pk.AdamwTensorArg, [adamw_tensor(), adamw_tensor()], cfg, EINVAL, "overlaps")
    # the sum of the list, and the list rounded up to whole work-groups
    far = [adamw_tensor(numel=MOST // 2 + 64, **{k: (i * 20 + j) << 40 for j, k in enumerate(
        ("param", "grad", "m", "v"), 1)}) for i in range(2)]
    refused("fp8adam_adamw_plan", pk.AdamwTensorArg, far, cfg, EINVAL, "too many elements")
    L = lists._lib()
    assert L.fp8adam_adamw_plan(None, None, 1, None, None) == EINVAL
    h = ctypes.c_void_p()
    assert L.fp8adam_adamw_plan(ctypes.byref(h), None, 1, ctypes.byref(cfg), None) == EINVAL
    assert L.fp8adam_adamw_plan(ctypes.byref(h), (pk.AdamwTensorArg * 1)(adamw_tensor()), 1, None, None) == EINVAL


def test_clip_plan_refuses():
    def one(**kw):
        d = dict(src=1 << 12, dst=2 << 12, numel=100, src_dtype=pk.F32, dst_dtype=pk.BF16)
        d.update(kw)
        return pk.ClipTensorArg(**d)
    for kw, code, text in ((dict(src=None), EINVAL, "src of tensor 0 is null"), (dict(src=4098), EALIGN, "src of tensor 0"),
                           (dict(dst=8193), EALIGN, "dst of tensor 0"), (dict(dst_dtype=5), EINVAL, "bad dtype"),
                           (dict(dst=1 << 12), EINVAL, "is src itself"), (dict(dst=(1 << 12) + 200), EINVAL, "overlaps"),
                           (dict(numel=-3), EINVAL, "negative"), (dict(numel=MOST + 1), EINVAL, "too many elements")):
        refused("fp8adam_clip_plan", pk.ClipTensorArg, [one(**kw)], None, code, text)
    refused("fp8adam_clip_plan", pk.ClipTensorArg, [], None, EINVAL, "n must be positive")
    same = one(dst=1 << 12, dst_dtype=pk.F32)  # in place, but twice in the list
    refused("fp8adam_clip_plan", pk.ClipTensorArg, [same, same], None, EINVAL, "overlaps")


def test_quant_plan_refuses():
    def one(**kw):
        d = dict(values=1 << 12, codes=2 << 12, scale=3 << 12, numel=100, dtype=pk.F32, format=pk.E4M3)
        d.update(kw)
        return pk.QuantTensorArg(**d)
    ok = (pk.SCALE_BLOCK128, pk.SCALE_POW2)
    for kw, cfg, code, text in (
            (dict(values=None), ok, EINVAL, "values of tensor 0 is null"), (dict(codes=None), ok, EINVAL, "codes"),
            (dict(scale=None), ok, EINVAL, "scale of tensor 0 is null"), (dict(scale=12290), ok, EALIGN, "scale"),
            (dict(dtype=9), ok, EINVAL, "bad dtype"), (dict(format=2), ok, EINVAL, "bad format"),
            (dict(), (2, 0), EINVAL, "granularity"), (dict(), (0, 2), EINVAL, "scale_mode"),
            (dict(codes=(1 << 12) + 8), ok, EINVAL, "overlaps"), (dict(scale=(2 << 12) + 96), ok, EINVAL, "overlaps"),
            (dict(numel=MOST + 1), ok, EINVAL, "too many elements")):
        refused("fp8adam_quant_plan", pk.QuantTensorArg, [one(**kw)], pk.QuantConfigArg(*cfg), code, text)


def test_calls_refuse_a_null_plan():
    L = lists._lib()
    hp = (pk.AdamwHParamsArg * 1)(pk.AdamwHParamsArg(1e-3, 0.9, 0.999, 1e-8, 0.0))
    amp = pk.AmpConfigArg(1.0, 2.0, 0.5, 2000)
    assert L.fp8adam_adamw_step(None, hp, 1, 1, None) == EINVAL
    assert L.fp8adam_adamw_step_amp(None, hp, 1, ctypes.byref(amp), 64, None) == EINVAL
    assert L.fp8adam_clip_grads(None, 1.0, 64, None) == EINVAL
    assert L.fp8adam_quantize(None, None) == EINVAL and L.fp8adam_dequantize(None, None) == EINVAL
    assert "plan is null" in pk.fp8adam_last_error()
    L.fp8adam_plan_destroy(None)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(n):
    return torch.zeros(n, dtype=torch.uint8)


@pytest.mark.parametrize("args, kw, text", [
    (([torch.zeros(4)], []), {}, "one gradient per parameter"),
    (([], []), {}, "at least one parameter"),
    (([torch.zeros(4).double()], [bf(4)]), {}, "weights must be"),
    (([torch.zeros(4)], [torch.zeros(4).int()]), {}, "gradients must be"),
    (([torch.zeros(4)], [bf(5)]), {}, "size and order"),
    (([torch.zeros(8)[::2]], [bf(4)]), {}, "dense"),
    (([torch.zeros(4, 6)[:, :5]], [bf(4, 5)]), {}, "dense"),
    (([torch.zeros(1).expand(4)], [bf(4)]), {}, "dense"),
    (([torch.zeros(4, 6).t()], [bf(6, 4)]), {}, "size and order"),
    (([torch.zeros(4)], [bf(4)]), dict(copies=[torch.zeros(4)]), "copy must be"),
    (([bf(4)], [bf(4)]), dict(copies=[bf(4)]), "copy must be"),
    (([torch.zeros(4)], [bf(4)]), dict(copies=[bf(5)]), "copy must have"),
    (([torch.zeros(4)], [bf(4)]), dict(copies=[]), "one entry per parameter"),
    (([torch.zeros(4)], [bf(4)]), dict(state_bits=16), "32 or 8"),
    (([torch.zeros(4)], [bf(4)]), dict(groups=[1], n_groups=1), "groups must lie"),
    (([torch.zeros(4)], [bf(4)]), dict(groups=[-1]), "groups must lie"),
    (([torch.zeros(4)], [bf(4)]), dict(groups=[40]), "groups must lie"),
    (([torch.zeros(4)], [bf(4)]), dict(state=([torch.zeros(4)],)), "state must be"),
    (([torch.zeros(4)], [bf(4)]), dict(state=([torch.zeros(5)], [torch.zeros(4)])), "32-bit moments"),
    (([torch.zeros(4)], [bf(4)]), dict(state=([bf(4)], [torch.zeros(4)])), "32-bit moments"),
    (([torch.zeros(4)], [bf(4)]), dict(state_bits=8, state=([u8(4)], [u8(4)])), "need scales"),
    (([torch.zeros(4)], [bf(4)]), dict(state_bits=8, state=([u8(3)], [u8(4)], [torch.ones(1)], [torch.ones(1)])), "4 elements"),
    (([torch.zeros(129)], [bf(129)]), dict(state_bits=8, state=([u8(129)], [u8(129)], [torch.ones(2)], [torch.ones(1)])),
     "at least 2 elements"),
    (([torch.zeros(4)], [bf(4)]), {}, "on a GPU"),
])
def test_adamw_binding_refuses(args, kw, text):
    with pytest.raises(ValueError, match=text):
        pk.AdamW(*args, **kw)


def test_clip_and_quantizer_bindings_refuse():
    for args, text in ((([],), "at least one gradient"), (([bf(3)], []), "one entry of outs"),
                       (([bf(3).double()],), "must be float32"), (([bf(3)], [bf(4)]), "size and order"),
                       (([bf(6)[::2]],), "dense"), (([bf(3)],), "on a GPU")):
        with pytest.raises(ValueError, match=text):
            pk.GradClip(*args)
    for args, kw, text in (([], {}, "at least one tensor"), ([u8(3)], {}, "values must be"), ([bf(6)[::2]], {}, "dense"),
                           ([bf(3)], dict(codes=[u8(2)]), "codes must have 3"),
                           ([bf(300)], dict(scales=[torch.ones(2)]), "scales must have at least 3"),
                           ([bf(300)], dict(scales=[torch.ones(0)], granularity="tensor"), "scales must have at least 1"),
                           ([bf(3)], dict(fmt=["e4m3", "e5m2"]), "one entry per tensor"), ([bf(3)], {}, "on a GPU")):
        with pytest.raises(ValueError, match=text):
            pk.Quantizer(args, **kw)
    with pytest.raises(KeyError):
        pk.Quantizer([bf(3)], granularity="row")
