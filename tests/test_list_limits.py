"""The number of elements that one plan of the list operators holds: the largest list is taken (up
to the first call that needs a GPU), one element more is refused."""
import ctypes

import pytest

import precision_adam_optimizer_amd as pk
from precision_adam_optimizer_amd import lists

EINVAL, EHIP = -1, -4
# work-groups of 256 lanes in a grid of 2^32 - 1 lanes, in whole runs of 32 on each of the 8 XCDs, 1024 elements each
MOST = ((2 ** 32 - 1) // 256 // 256 * 256) * 1024


def plan(fn, struct, tensors, cfg):
    L = lists._lib()
    h = ctypes.c_void_p()
    rc = getattr(L, fn)(ctypes.byref(h), (struct * len(tensors))(*tensors), len(tensors),
                        *([] if cfg is None else [ctypes.byref(cfg)]), None)
    if h.value:
        pk.fp8adam_plan_destroy(h.value)
    return rc, pk.fp8adam_last_error() if rc else ""


def adamw(sizes, **kw):
    d = dict(param_dtype=pk.F32, grad_dtype=pk.BF16, moments=pk.MOMENTS_32)
    d.update(kw)
    names = ("param", "grad", "m", "v", "m_scale", "v_scale")
    return [pk.AdamwTensorArg(numel=n, **{k: (8 * i + j + 1) << 44 for j, k in enumerate(names)}, **d)
            for i, n in enumerate(sizes)]


def clip(sizes):
    return [pk.ClipTensorArg((2 * i + 1) << 44, (2 * i + 2) << 44, n, pk.F32, pk.BF16) for i, n in enumerate(sizes)]


def quant(sizes):
    return [pk.QuantTensorArg((3 * i + 1) << 44, (3 * i + 2) << 44, (3 * i + 3) << 44, n, pk.BF16, pk.E5M2)
            for i, n in enumerate(sizes)]


PLANS = {
    "adamw": lambda sizes: plan("fp8adam_adamw_plan", pk.AdamwTensorArg, adamw(sizes), pk.AdamwConfigArg(1, 0, 1, 0)),
    "adamw 8 bits": lambda sizes: plan("fp8adam_adamw_plan", pk.AdamwTensorArg,
                                       adamw(sizes, moments=pk.MOMENTS_8, param_dtype=pk.BF16), pk.AdamwConfigArg(1, 0, 1, 0)),
    "clip": lambda sizes: plan("fp8adam_clip_plan", pk.ClipTensorArg, clip(sizes), None),
    "quant": lambda sizes: plan("fp8adam_quant_plan", pk.QuantTensorArg, quant(sizes), pk.QuantConfigArg(1, 0)),
    "quant by tensors": lambda sizes: plan("fp8adam_quant_plan", pk.QuantTensorArg, quant(sizes), pk.QuantConfigArg(0, 0)),
}


@pytest.mark.parametrize("kind", list(PLANS))
def test_most_elements_of_a_plan(kind):
    for sizes in ([MOST], [MOST - 1024, 1024], [0, MOST]):
        rc, msg = PLANS[kind](sizes)
        assert rc in (0, EHIP), (sizes, msg)  # taken; without a GPU the device calls fail
    for sizes in ([MOST + 1], [MOST, 1], [MOST - 5, 0, 6]):
        rc, msg = PLANS[kind](sizes)
        assert rc == EINVAL and "too many elements" in msg, (sizes, rc, msg)


def test_most_work_groups_of_a_plan():
    """A tensor whose last work-group holds one element counts it whole."""
    rc, msg = PLANS["adamw"]([MOST // 2 + 1, MOST // 2 - 1024])  # as many work-groups as the largest tensor
    assert rc in (0, EHIP), msg
    rc, msg = PLANS["adamw"]([MOST // 2 + 1, MOST // 2 - 1])
    assert rc == EINVAL and "whole parts" in msg, (rc, msg)
