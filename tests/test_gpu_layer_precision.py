"""What the layer operators' sums keep of small products beside large ones."""
import pytest
import torch

import layer_util as u
import precision_adam_optimizer_amd as pk

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def beside_large(rows, cols):
    """A matrix whose products with itself's like have, in every eight of consecutive columns, one large product and seven 2^-16
    of it; the large ones cancel in pairs.  Of the sums over all columns 7 * 2^-16 * cols / 8 is left, which every
    type holds exactly, as 32 bits do each partial sum."""
    x = torch.full((rows, cols), 2.0 ** -8, device="cuda")
    x[:, ::8] = 1.0
    sign = torch.ones(cols, device="cuda")
    sign[::16] = -1.0
    return x, x * sign


def outputs(gated, tokens, rows, dtype, **kw):
    """{name: values} of one call on these matrices."""
    a, b = beside_large(tokens, 256)[0], beside_large(rows, 256)[1]
    w = pk.pack8(b)
    if gated:
        one = torch.zeros(rows, 256, device="cuda")
        one[:, 1] = 2.0 ** 8  # the up projection: 1 everywhere
        r = pk.gated8(a.to(dtype), w, pk.pack8(one), activation="none", dtype=dtype, **kw)
        got = {"y": r.y, "gate": r.gate}
    else:
        r = pk.linear8(a.to(dtype), w, dtype=dtype, **kw)
        got = {"y": r.y, "z": r.z}
    got["y8"] = r.y8
    return {k: u.values(v) if isinstance(v, pk.Packed8) else v.double() for k, v in got.items() if v is not None}


EXACT = 7 * 2.0 ** -16 * 32


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("tokens", [1, 4, 5, 16, 17, 40, 64])
def test_few_tokens_keep_small_products(tokens, dtype, gated):
    """Whether or not something is kept or packed."""
    for kw in ({}, dict(keep="e4m3"), dict(pack="e5m2"), dict(keep="e5m2", pack="e4m3")):
        for name, v in outputs(gated, tokens, 130, dtype, **kw).items():
            assert (v == EXACT).all(), (name, kw)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("tokens", [3, 65, 300])
def test_exact_keeps_small_products(tokens, dtype, gated):
    """Of any number of tokens, whatever is written."""
    for kw in ({}, dict(keep="e4m3"), dict(pack="e5m2"), dict(keep="e5m2", pack="e4m3")):
        for name, v in outputs(gated, tokens, 130, dtype, exact=True, **kw).items():
            assert (v == EXACT).all(), (name, kw)
