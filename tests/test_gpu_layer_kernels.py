"""Every kernel of the layer operators' products (tests/layer_kernels.py says which call reaches which), against
the formulas in 64 bits: sums longer than the loops' unrolled part, ragged tokens, rows and columns, every type and format."""
import pytest
import torch

import layer_kernels as lk
import layer_util as u
import precision_adam_optimizer_amd as pk
from test_gpu_layer import BF16, F16, F32, check, check_packed, product_bound

pytestmark = pytest.mark.gpu
DTYPES = {"fp32": F32, "bf16": BF16, "fp16": F16}


def weights(rows, cols, seed, fmt):
    w = pk.pack8(u.randn((rows, cols), seed) / cols ** 0.5, fmt)
    return w, u.values(w)


def rounded(t, y, dtype):
    """What a value known to t may be off once it is rounded to dtype."""
    return t + u.half_step(dtype) * (y.abs() + t) + torch.finfo(dtype).smallest_normal * u.half_step(dtype) * 2


def check_product(c, eights):
    dtype = DTYPES[c.dtype]
    x = u.randn((c.tokens, c.cols), c.cols + c.tokens, dtype=dtype, spread=1.0)
    codes, scales = u.pack(x.float(), c.x)
    xv = u.decode(codes, scales, c.cols, c.x)
    w, wv = weights(c.rows, c.cols, 2, c.w)
    src = pk.pack8(x, c.x) if c.packed else x
    kw = dict(activation=c.activation, dtype=dtype, fmt=c.x, keep="e4m3" if c.keep else None, pack=c.pack, exact=c.exact)
    z = xv @ wv.t()
    if c.gated:
        w_up, wv_up = weights(c.rows, c.cols, 3, c.w)
        def call():
            return pk.gated8(src, w, w_up, **kw)
        got = call()
        up, zero = xv @ wv_up.t(), torch.zeros_like(z)
        tz, ta = product_bound(xv, wv, z, c.activation, zero, eights)
        tu, _ = product_bound(xv, wv_up, up, "none", zero, eights)
        y = u.act(z, c.activation) * up
        ty = ta * (up.abs() + tu) + u.act(z, c.activation).abs() * tu + 2.0 ** -23 * y.abs()
        kept = [(got.gate, z, tz), (got.up, up, tu)]
    else:
        b = u.randn((c.rows,), 4, dtype=F32) if c.bias else None
        r = u.randn((c.tokens, c.rows), 5, dtype=dtype) if c.residual else None
        def call():
            return pk.linear8(src, w, bias=b, residual=r, **kw)
        got = call()
        extra = torch.zeros_like(z)
        if c.bias:
            z, extra = z + b.double(), extra + b.double().abs()
        if c.residual:
            extra = extra + r.double().abs()
        tz, ty = product_bound(xv, wv, z, c.activation, extra, eights)
        y = u.act(z, c.activation) + (r.double() if c.residual else 0.0)
        kept = [(got.z, z, tz)]
    assert torch.equal(got.x.codes, codes) and torch.equal(got.x.scales[:, :u.blocks(c.cols)], scales)
    check(got.y, y, rounded(ty, y, dtype))
    assert all(torch.equal(call().y, got.y) for _ in range(3))  # the same bits every time
    if c.keep:
        for p, v, t in kept:
            check_packed(p, v, t, "e4m3")
    if c.pack:
        check_packed(got.y8, y, ty, c.pack)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tt, wide", [(64, False), (128, False), (256, False), (64, True), (128, True)])
def test_forward_tiles(tt, wide, gated):
    for _, _, c in [k for k in lk.products() if (k[0], k[1], k[2].gated) == (tt, wide, gated)]:
        print(c, flush=True)
        check_product(c, not wide)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("waves", [4, 8])
@pytest.mark.parametrize("nt", [1, 2, 4])
def test_few_tokens(nt, waves, gated):
    for _, _, c in [k for k in lk.few() if (k[0], k[1], k[2].gated) == (nt, waves, gated)]:
        print(c, flush=True)
        check_product(c, False)


@pytest.mark.parametrize("tile, parts, n", sorted({(tile, parts, c.n) for tile, parts, c in lk.gradients()}))
def test_gradients(tile, parts, n):
    cases = [k[2] for k in lk.gradients() if k[:2] == (tile, parts) and k[2].n == n]
    for c in cases:
        print(c, flush=True)
        dtype = DTYPES[c.dtype]
        dys = [u.randn((c.tokens, c.rows), 1 + i, dtype=dtype) for i in range(c.n or 1)]
        if c.n:
            ws, wv = zip(*(weights(c.rows, c.cols, 5 + i, c.fmt) for i in range(c.n)))
            a, b, shape = torch.cat([d.double() for d in dys], 1), torch.cat(wv), (c.tokens, c.cols)
            call = lambda *args, **kw: pk.input_grad8(dys, list(ws), *args, exact=c.exact, **kw)  # noqa: E731
        else:
            x = pk.pack8(u.randn((c.tokens, c.cols), 9, spread=1.0), c.fmt)
            a, b, shape = dys[0].double().t(), u.values(x), (c.rows, c.cols)
            call = lambda *args, **kw: pk.weight_grad8(dys[0], x, *args, exact=c.exact, **kw)  # noqa: E731
        want, terms = a @ b, a.abs() @ b.abs()
        # up to three terms for each product; of fp32 gradients in two terms it is off by 2^-16 of itself
        t = u.sum_bound(terms, 3 * a.shape[1] + 2) + (0.0 if dtype != F32 or c.exact else 2.0 ** -16 * terms)
        got = call(dtype=F32)
        check(got, want, t)
        assert all(torch.equal(call(dtype=F32), got) for _ in range(3))  # the same bits every time
        for out_dtype in (F32, BF16):
            old = u.randn(shape, 7, dtype=out_dtype)
            out = u.strided(old, 5, 1)
            assert call(out, accumulate=True) is out
            total = want + old.double()
            check(out, total, rounded(t + 2.0 ** -23 * total.abs(), total, out_dtype))
            assert out._base.isnan().sum() == out._base.numel() - out.numel()  # nothing between the rows was written
