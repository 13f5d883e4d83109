"""The layer operators at their calls' edges: few tokens at every alignment, one matrix in two places of a
call, outputs in place and inside larger buffers, sums in many parts, other streams."""
import pytest
import torch

import layer_util as u
import precision_adam_optimizer_amd as pk

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DTYPES = (F32, BF16, F16)


def close(got, want, tol):
    assert got.shape == want.shape
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, by up to {((got.double() - want).abs() / tol).max().item():.3g} of the tolerance"


def rounded(t, y, dtype):
    """A sum known to t, rounded to dtype."""
    return t + u.half_step(dtype) * (y.abs() + t) + torch.finfo(dtype).smallest_normal


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 127, 130, 256, 1001, 4100])
@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 8, 15, 16, 17])
def test_few_tokens_at_every_alignment(tokens, cols, dtype):
    """The product that packs its input itself, and the one that has it packed, from rows at odd elements: the codes are
    pack8's bit for bit and the sums those of the packed input."""
    x = u.randn((tokens, cols), 3, dtype=dtype, spread=2.0)
    w = pk.pack8(u.randn((50, cols), 4) / cols ** 0.5, "e5m2")
    codes, scales = u.pack(x.float(), "e4m3")
    xv, wv = u.decode(codes, scales, cols, "e4m3"), u.values(w)
    want, t = xv @ wv.t(), u.sum_bound(xv.abs() @ wv.abs().t(), cols + 2)
    first = None
    for pad, off in ((0, 0), (1, 0), (2, 1), (8, 3), (7, 8)):
        got = pk.linear8(u.strided(x, pad, off), w, dtype=F32)
        assert torch.equal(got.x.codes, codes) and torch.equal(got.x.scales[:, :u.blocks(cols)], scales)
        close(got.y, want, t)
        first = got.y if first is None else first
        assert torch.equal(got.y, first)
    assert torch.equal(pk.linear8(pk.pack8(x), w, dtype=F32).y, first)


def test_not_finite_in_few_tokens():
    """The product that packs its input itself: a NaN, Infs, zeros, subnormals and the largest numbers, as pack8 has them."""
    for dtype in DTYPES:
        x = u.randn((4, 512), 1, dtype=dtype)
        x[0, 3], x[1, 200], x[1, 201] = float("nan"), float("inf"), float("-inf")
        x[2, :128] = 0
        x[2, 128:256] = torch.finfo(dtype).smallest_normal / 4
        x[3, 256:384] = torch.finfo(dtype).max
        w = pk.pack8(u.randn((32, 512), 2))
        got, p = pk.linear8(x, w, dtype=F32), pk.pack8(x)
        assert torch.equal(got.x.codes, p.codes) and torch.equal(got.x.scales, p.scales)
        assert got.y[0].isnan().all()
        # (128 products of the largest number pass it: where the sizes of a sum's terms do not, it is finite)
        held = u.values(p)[1:].abs() @ u.values(w).abs().t() < torch.finfo(F32).max
        assert held[:2].all() and got.y[1:][held].isfinite().all()
        other = pk.linear8(p, w, dtype=F32).y
        assert torch.equal(got.y.isnan(), other.isnan()) and torch.equal(got.y.nan_to_num(), other.nan_to_num())


@pytest.mark.parametrize("tokens", [3, 64, 200])
def test_one_matrix_in_two_places(tokens):
    """Both projections of one weight, one gradient for both layers, a matrix times itself."""
    w = pk.pack8(u.randn((256, 256), 1) / 16)
    wv = u.values(w)
    x = u.randn((tokens, 256), 2, dtype=BF16)
    g = pk.gated8(x, w, w, activation="none", dtype=F32)
    xv = u.values(g.x)
    z, t = xv @ wv.t(), u.sum_bound(xv.abs() @ wv.abs().t(), 258)
    close(g.y, z * z, 2 * t * z.abs() + t * t + 2.0 ** -23 * z * z)
    close(pk.linear8(w, w, dtype=F32).y, wv @ wv.t(), u.sum_bound(wv.abs() @ wv.abs().t(), 258))
    one, both = pk.input_grad8(x, w, dtype=F32), pk.input_grad8([x, x], [w, w], dtype=F32)
    terms = x.double().abs() @ wv.abs()
    close(both, 2 * (x.double() @ wv), u.sum_bound(2 * terms, 514))
    close(one, x.double() @ wv, u.sum_bound(terms, 258))


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_and_inside_larger_buffers(dtype):
    """dy's own memory takes a gradient; nothing outside an output's rows and columns changes."""
    T, N = 70, 200
    z, up = (pk.pack8(u.randn((T, N), s)) for s in (1, 2))
    dy = u.randn((T, N), 3, dtype=dtype)
    want = pk.gated8_backward(dy, z, up)
    for k in range(2):
        room = torch.full((T + 2, N + 9), 7.0, dtype=dtype, device="cuda")
        view = room[1:-1, 4:4 + N]
        view.copy_(dy)
        other = torch.empty_like(dy)
        outs = (view, other) if k == 0 else (other, view)
        pk.gated8_backward(view, z, up, outs=outs)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        view.fill_(7.0)
        assert (room == 7).all()
    single = pk.linear8_backward(dy, z, activation="silu")
    mine = dy.clone()
    assert pk.linear8_backward(mine, z, activation="silu", out=mine) is mine and torch.equal(mine, single)
    w = pk.pack8(u.randn((N, 136), 5))
    for T2 in (1, 5, 64, 70):
        room = torch.full((T2 + 3, N + 5), 7.0, dtype=dtype, device="cuda")
        out = room[1:T2 + 1, 2:2 + N]
        x = u.randn((T2, 136), 6, dtype=dtype)
        assert pk.linear8(x, w, out=out).y is out
        assert torch.equal(out, pk.linear8(x, w, dtype=dtype).y)
        out.fill_(7.0)
        assert (room == 7).all()
        d = u.randn((T2, N), 8, dtype=dtype)
        for fn, args, shape in ((pk.input_grad8, (d, w), (T2, 136)), (pk.weight_grad8, (d, pk.pack8(x)), (N, 136))):
            room = torch.full((shape[0] + 2, 150), 7.0, dtype=dtype, device="cuda")
            out = room[1:-1, 7:7 + 136]
            fn(*args, out)
            assert torch.equal(out, fn(*args, dtype=dtype))
            out.fill_(7.0)
            assert (room == 7).all()


@pytest.mark.parametrize("tokens, rows, cols, n", [
    (20000, 8, 100, 1), (20000, 130, 16, 1), (63, 5000, 100, 2), (64, 4097, 128, 2), (65, 1030, 300, 2), (129, 8200, 17, 2),
    (4000, 1024, 256, 2), (64, 64, 128, 2), (1, 3000, 128, 2), (16, 16384, 256, 2)])
def test_sums_in_many_parts(tokens, rows, cols, n):
    """Few tiles and long sums: parts that begin and end inside either pair, and inside a step."""
    x, dys = pk.pack8(u.randn((tokens, cols), 1)), [u.randn((tokens, rows), 2 + i, dtype=BF16) for i in range(n)]
    xv, d = u.values(x), dys[0].double()
    close(pk.weight_grad8(dys[0], x), d.t() @ xv, u.sum_bound(d.abs().t() @ xv.abs(), 2 * tokens + 2))
    ws = [pk.pack8(u.randn((rows, cols), 5 + i) / rows ** 0.5, "e5m2") for i in range(n)]
    wv = torch.cat([u.values(w) for w in ws])
    d = torch.cat(dys, 1).double()
    want, t = d @ wv, u.sum_bound(d.abs() @ wv.abs(), 2 * n * rows + 2)
    close(pk.input_grad8(dys, ws, dtype=F32), want, t)
    old = u.randn((tokens, cols), 9, dtype=F16)
    out = old.clone()
    pk.input_grad8(dys, ws, out, accumulate=True)
    want = want + old.double()
    close(out, want, rounded(t + 2.0 ** -23 * want.abs(), want, F16))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tokens", [17, 50, 64])
def test_some_tokens_of_wide_layers(tokens, fmt):
    """17 to 64 tokens of layers with so many outputs that the tiled product takes them: sums as exact as those of few tokens."""
    cols, rows = 1100, 40003
    for n, (dtype, kind) in enumerate([(F32, "none"), (BF16, "relu"), (F16, "relu")]):
        x = u.randn((tokens, cols), n, dtype=dtype, spread=1.0)
        w = pk.pack8(u.randn((rows, cols), 4 + n) / cols ** 0.5, fmt)
        b, r = u.randn((rows,), 7, dtype=F16), u.randn((tokens, rows), 8, dtype=BF16)
        got = pk.linear8(x, w, bias=b, activation=kind, residual=r, dtype=dtype)
        xv, wv = u.values(got.x), u.values(w)
        extra = b.double().abs() + r.double().abs()
        y, t = u.act(xv @ wv.t() + b.double(), kind) + r.double(), u.sum_bound(xv.abs() @ wv.abs().t() + extra, cols + 3)
        close(got.y, y, rounded(t, y, dtype))
        half = pk.Packed8(w.codes[:20001], w.scales[:20001], cols, fmt)
        other = pk.Packed8(w.codes[20001:40002], w.scales[20001:40002], cols, fmt)
        got = pk.gated8(x, half, other, activation="none", dtype=dtype)
        g, up = xv @ wv[:20001].t(), xv @ wv[20001:40002].t()
        tg, tu = (u.sum_bound(xv.abs() @ v.abs().t(), cols + 2) for v in (wv[:20001], wv[20001:40002]))
        close(got.y, g * up, rounded(tg * (up.abs() + tu) + tu * g.abs() + 2.0 ** -23 * (g * up).abs(), g * up, dtype))


def test_on_another_stream_than_the_tensors_own():
    """Tensors made on one stream, calls on another that waits for it, results read on the first again."""
    w = pk.pack8(u.randn((384, 256), 1) / 16)
    x, dy = u.randn((500, 256), 2, dtype=BF16), u.randn((500, 384), 3, dtype=F32)

    def work():
        r = pk.linear8(x, w, activation="silu", keep="e4m3", pack="e5m2")
        dz = pk.linear8_backward(dy, r.z, activation="silu")
        return [r.y, r.y8.codes, r.z.codes, dz, pk.weight_grad8(dz, r.x), pk.input_grad8(dz, w)]
    want = work()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = work()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got


def test_packed_output_feeds_the_next_layer():
    """y8 of one layer as the next one's input: the same as its fp32 output packed, within the roundings; alone, without y."""
    for tokens in (5, 300):
        w1, w2 = pk.pack8(u.randn((640, 256), 1) / 16), pk.pack8(u.randn((100, 640), 2) / 25)
        x = u.randn((tokens, 256), 3, dtype=BF16)
        a = pk.linear8(x, w1, activation="relu", dtype=None, pack="e4m3")
        assert a.y is None
        b = pk.linear8(x, w1, activation="relu", pack="e4m3")
        assert torch.equal(a.y8.codes, b.y8.codes) and torch.equal(a.y8.scales[:, :5], b.y8.scales[:, :5])
        yv, wv = u.values(a.y8), u.values(w2)
        close(pk.linear8(a.y8, w2, dtype=F32).y, yv @ wv.t(), u.sum_bound(yv.abs() @ wv.abs().t(), 642))
        close(b.y, yv, (2 * 2.0 ** -4) * yv.abs() + torch.exp2(b.y8.scales[:, :5].double() - 127 - 9).repeat_interleave(128, 1))


def test_largest_columns():
    """The longest rows that the operators take, of few tokens and weights."""
    cols = pk.LAYER_MAX_COLS
    x, w = u.randn((3, cols), 1, dtype=BF16), pk.pack8(u.randn((17, cols), 2) / 1024)
    got = pk.linear8(x, w, dtype=F32)
    xv, wv = u.values(got.x), u.values(w)
    close(got.y, xv @ wv.t(), u.sum_bound(xv.abs() @ wv.abs().t(), cols + 2))
    dy = u.randn((3, 17), 3, dtype=BF16)
    close(pk.weight_grad8(dy, got.x), dy.double().t() @ xv, u.sum_bound(dy.double().abs().t() @ xv.abs(), 8))
    close(pk.input_grad8(dy, w, dtype=F32), dy.double() @ wv, u.sum_bound(dy.double().abs() @ wv.abs(), 36))
    assert torch.equal(pk.unpack8(got.x, F32).double(), xv)
