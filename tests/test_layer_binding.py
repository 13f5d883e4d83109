"""The layer operators' binding, without a GPU: what a Packed8 holds of the tensors that it was made of, and refusals."""
import ctypes

import pytest
import torch

import precision_adam_optimizer_amd as pk
from precision_adam_optimizer_amd import layers

U8 = torch.uint8


def made(rows, cols, scales):
    """(codes, scales, Packed8) whose values are all 1."""
    nb = -(-cols // 128)
    codes = torch.full((rows, 128 * nb), 0x38, dtype=U8)  # 1.0 in E4M3
    return codes, scales, pk.Packed8(codes, scales, cols)


def values(p):
    c, s = p.values()
    if p.scale_type == 0:
        s = torch.exp2(s.view(U8).float() - 127)
    return c.float() * s.repeat_interleave(128, 1)[:, :p.cols]


@pytest.mark.parametrize("make", [
    lambda: torch.full((5, 6), 127, dtype=U8),                       # six blocks: not whole dwords
    lambda: torch.full((5, 6), 127, dtype=U8).view(torch.float8_e8m0fnu),
    lambda: torch.full((5, 11), 127, dtype=U8)[:, 2:8],              # rows 11 bytes apart, off a dword
    lambda: torch.full((5, 8), 127, dtype=U8)[:, :6],                # whole dwords apart, not as long
    lambda: torch.full((41,), 127, dtype=U8)[1:].view(5, 8),         # whole dwords long, off a dword
])
def test_copied_scales_come_with_copied_codes(make):
    """Scales whose rows are not whole dwords are copied.  Codes and scales rewritten in place later are
    then seen together or not at all: never new codes with old scales."""
    codes, scales, p = made(5, 768, make())
    assert (values(p) == 1).all()
    assert p.scales.data_ptr() != scales.data_ptr() and p.codes.data_ptr() != codes.data_ptr()
    codes.fill_(0x40)  # 2.0
    scales.view(U8).fill_(129)
    assert (values(p) == 1).all()
    assert p.arg()[:2] == (p.codes.data_ptr(), p.scales.data_ptr())


@pytest.mark.parametrize("make", [lambda: torch.full((5, 8), 127, dtype=U8), lambda: torch.ones(5, 6), lambda: torch.ones(5, 9)[:, 1:7]])
def test_other_scales_are_seen_with_their_codes(make):
    codes, scales, p = made(5, 768, make())
    assert p.scales.data_ptr() == scales.data_ptr() and p.codes.data_ptr() == codes.data_ptr()
    codes.fill_(0x40)
    scales.fill_(128 if scales.dtype == U8 else 2.0)
    assert (values(p) == 4).all()


def test_exact_is_a_truth_value():
    for fn in ("fp8adam_linear8", "fp8adam_gated8"):
        for exact in (-1, 2):
            args = layers.Product8Arg(tokens=1, rows=1, cols=1, exact=exact)
            assert getattr(layers._lib(), fn)(ctypes.byref(args), None) == -1
            assert "exact must be 0 or 1" in pk.fp8adam_last_error()
    for fn in ("fp8adam_weight_grad8", "fp8adam_input_grad8"):
        for exact in (-1, 2):
            args = layers.Grad8Arg(tokens=1, rows=1, cols=1, n=1, exact=exact)
            assert getattr(layers._lib(), fn)(ctypes.byref(args), None) == -1
            assert "exact must be 0 or 1" in pk.fp8adam_last_error()
            assert getattr(layers._lib(), fn + "_workspace")(ctypes.byref(args)) == -1


def test_workspace_of_fp32_gradients():
    """Two bf16 parts of dy, and with `exact` three."""
    for fn in ("fp8adam_weight_grad8_workspace", "fp8adam_input_grad8_workspace"):
        for n in (1, 2) if "input" in fn else (1,):
            size = []
            for exact in (0, 1):
                dy = layers.MatrixArg(data=1 << 32, ld=128, dtype=pk.F32)
                args = layers.Grad8Arg(tokens=64, rows=128, cols=128, n=n, dy=(layers.MatrixArg * 2)(dy, dy), exact=exact)
                size.append(getattr(layers._lib(), fn)(ctypes.byref(args)))
            assert size[1] - size[0] >= n * 64 * 128 * 2


def test_packed_inputs_give_their_shape_to_the_output(monkeypatch):
    """A matrix packed from a tensor of more dimensions, by pack8 or as a call's output or input, stands for that tensor:
    what is made of it has the leading dimensions that it would have from the tensor itself."""
    monkeypatch.setattr(layers, "_run", lambda *args: None)
    w, w2 = (pk.Packed8(torch.zeros(r, 128 * -(-c // 128), dtype=U8), torch.full((r, 4), 127, dtype=U8), c) for r, c in ((24, 40), (40, 24)))
    for lead in ((3, 5), (2, 3, 5), (15,), (0, 4), (2, 0, 4)):
        x = torch.zeros(*lead, 40, dtype=torch.bfloat16)
        for src in (x, pk.pack8(x)):
            for r in (pk.linear8(src, w, keep="e4m3", pack="e4m3", activation="silu"), pk.gated8(src, w, w, keep="e4m3", pack="e5m2")):
                assert r.y.shape == (*lead, 24)
                assert pk.linear8(r.y8, w2, residual=x).y.shape == x.shape
                assert pk.linear8(r.x, w, dtype=torch.float32).y.shape == (*lead, 24)
                assert pk.gated8(r.x, w, w).y.shape == (*lead, 24)
                for p in (r.x, r.y8):
                    assert p.rows == x.numel() // 40
                out = torch.zeros(p.rows, 24, dtype=torch.bfloat16)
                assert pk.linear8(src, w, out=out).y is out
    by_hand = pk.Packed8(torch.zeros(15, 128, dtype=U8), torch.full((15, 4), 127, dtype=U8), 40)
    assert pk.linear8(by_hand, w).y.shape == (15, 24) and pk.unpack8(pk.pack8(torch.zeros(3, 5, 40))).shape == (15, 40)


def needs_gradient(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, requires_grad=True)


@pytest.mark.parametrize("call", [
    lambda x, w: pk.pack8(x(4, 6)), lambda x, w: pk.linear8(x(4, 6), w(8, 6)), lambda x, w: pk.gated8(x(4, 6), w(8, 6), w(8, 6)),
    lambda x, w: pk.linear8(w(4, 6), w(8, 6), bias=x(8)), lambda x, w: pk.linear8(w(4, 6), w(8, 6), residual=x(4, 8)),
    lambda x, w: pk.linear8_backward(x(4, 8), w(4, 8), activation="gelu"), lambda x, w: pk.gated8_backward(x(4, 8), w(4, 8), w(4, 8)),
    lambda x, w: pk.weight_grad8(x(4, 8), w(4, 6)), lambda x, w: pk.input_grad8(x(4, 8), w(8, 6)),
    lambda x, w: pk.unpack8(w(4, 6), out=x(4, 6)),
])
def test_inputs_that_require_a_gradient(call, monkeypatch):
    """Nothing is recorded, so a result would be cut off from its input without a word: refused, but where nothing is to
    be recorded."""
    monkeypatch.setattr(layers, "_run", lambda *args: None)
    packed = lambda r, c: pk.Packed8(torch.zeros(r, 128 * -(-c // 128), dtype=U8), torch.full((r, 4), 127, dtype=U8), c)  # noqa: E731
    with pytest.raises(ValueError, match="requires a gradient"):
        call(needs_gradient, packed)
    with torch.no_grad():
        call(needs_gradient, packed)
    call(lambda *shape: needs_gradient(*shape).detach(), packed)


def test_inside_a_function_of_autograd(monkeypatch):
    """torch.autograd.Function runs its own forward and backward passes with nothing recorded."""
    monkeypatch.setattr(layers, "_run", lambda *args: None)
    w = pk.Packed8(torch.zeros(8, 128, dtype=U8), torch.full((8, 4), 127, dtype=U8), 6)

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return pk.linear8(x, w).y

        @staticmethod
        def backward(ctx, dy):
            return pk.input_grad8(dy, w)
    x = needs_gradient(4, 6)
    Layer.apply(x).square().sum().backward()
    assert x.grad.shape == x.shape
