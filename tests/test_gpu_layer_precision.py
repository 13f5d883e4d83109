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


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_gradients_take_every_bit_of_fp32(fmt):
    """A number times 1, and what is left of two numbers that agree in their first 20 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    # 24 random bits, from sizes whose last bit bf16 still holds as a normal number up to the largest
    bits = torch.randint(0, 1 << 23, (1, 448), generator=g, device="cuda", dtype=torch.int32) | 1
    dy = (bits | torch.arange(24, 24 + 448, device="cuda", dtype=torch.int32).clamp(max=254)[None] << 23).view(F32)
    dy[:, ::3] *= -1
    one = pk.pack8(torch.ones(1, 200, device="cuda"), fmt)
    assert torch.equal(pk.weight_grad8(dy, one), dy.t().expand(448, 200))
    for n in (1, 2):  # the first layer alone, and a second whose gradient is zero
        ws = [pk.pack8(torch.eye(448, device="cuda"), fmt)] * n
        dys = [dy, torch.zeros_like(dy)][:n]
        assert torch.equal(pk.input_grad8(dys, ws, dtype=F32), dy)
        assert torch.equal(pk.input_grad8(dys[::-1], ws, dtype=F32), dy)
    near = torch.tensor([[1 + 2.0 ** -8 + 2.0 ** -20], [-1 - 2.0 ** -8]], device="cuda").expand(2, 200).contiguous()
    ones = pk.pack8(torch.ones(2, 130, device="cuda"), fmt)
    assert (pk.weight_grad8(near, ones) == 2.0 ** -20).all()
    w = pk.pack8(torch.ones(200, 130, device="cuda"), fmt)
    rest = near.clone()
    rest[:, 1:] = 0
    rest[:, 1] = -1 - 2.0 ** -8
    assert (pk.input_grad8(rest[:1], w, dtype=F32) == 2.0 ** -20).all()
    assert (pk.weight_grad8(near, ones, exact=False) == 0).all()  # 16 bits of each


def test_gradients_of_one_token_are_rounded_once():
    """One fp32 token: every element is one product, off by its rounding alone."""
    dy = u.randn((1, 300), 1)
    x = pk.pack8(u.randn((1, 500), 2))
    want = dy.double().t() @ u.values(x)
    assert ((pk.weight_grad8(dy, x).double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all()  # three terms are added


def activations(rows, cols, seed, columns_that_stand_out):
    """Normal numbers; or rows of different sizes and a hundredth of the columns eight times as large."""
    x = u.randn((rows, cols), seed, spread=0.5 if columns_that_stand_out else 0.0)
    if columns_that_stand_out:
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        x = x * torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    return x


@pytest.mark.parametrize("stand_out, typical", [(False, 1.4e-5), (True, 2.7e-5)])
@pytest.mark.parametrize("tokens, cols, rows", [(2048, 768, 2048), (1027, 1000, 2050), (1024, 4096, 2048)])
def test_what_the_fp8_instruction_cuts(tokens, cols, rows, stand_out, typical):
    """The figures that the header gives, within a factor of 1.5: the error of the sums next to their rms, read off
    what is left beside a residual that takes the sums away, and the kept codes on the other side of a border."""
    x, w = pk.pack8(activations(tokens, cols, 1, stand_out)), pk.pack8(u.randn((rows, cols), 2) / cols ** 0.5)
    z = u.values(x) @ u.values(w).t()
    codes = u.pack(z.float(), "e4m3")[0]
    for exact, most, share in ((False, 1.5 * typical, 1.5 / 640), (True, 2e-7, 1.5 / 190000)):
        r = pk.linear8(x, w, residual=-z.float(), keep="e4m3", exact=exact)  # (the residual's own rounding: 2^-24)
        error = (r.y.double().square().mean() / z.square().mean()).sqrt().item()
        differ = (r.z.codes[:, :rows] != codes[:, :rows]).double().mean().item()
        print(f"exact {exact}: error {error:.3g} of the rms, kept codes that differ 1 in {1 / differ if differ else 0:.0f}")
        assert error <= most
        assert differ <= share
        if not exact:
            assert error >= typical / 1.5 and differ >= 1 / (1.5 * 990)


@pytest.mark.parametrize("fmt, first", [("e4m3", 3), ("e5m2", 10)])
def test_smallest_scales(fmt, first):
    """Every code under the smallest scales, times a power of two: exact from the scale on whose smallest code is 2^-133, and
    below it off by half of that at most."""
    n = 126 if fmt == "e4m3" else 123
    codes = torch.zeros(n, 128, dtype=torch.uint8, device="cuda")
    codes[:, 0] = torch.arange(1, n + 1, device="cuda")
    big = 2.0 ** 100
    w = pk.pack8(torch.full((1, 128), big, device="cuda"))
    dy = torch.full((1, 1), big, dtype=BF16, device="cuda")
    for byte in (1, 2, 3, 5, 8, 9, 10, 11, 30):
        scales = torch.full((n, 4), byte, dtype=torch.uint8, device="cuda")
        x = pk.Packed8(codes, scales, 128, fmt)
        want = u.values(x)[:, 0]
        off = 0.0 if byte >= first else 2.0 ** -134
        assert torch.equal(pk.unpack8(x, F32).double()[:, 0], want)
        few = torch.cat([pk.linear8(pk.Packed8(codes[i:i + 50], scales[i:i + 50], 128, fmt), w, dtype=F32).y for i in range(0, n, 50)])
        tile = pk.linear8(x, w, dtype=F32).y  # more than 64 tokens
        grad = torch.cat([pk.weight_grad8(dy, pk.Packed8(codes[i:i + 1], scales[i:i + 1], 128, fmt))[:, :1] for i in range(n)])
        for got in (few, tile, grad):
            assert ((got.double()[:, 0] / big - want).abs() <= off).all(), byte


def exact_step(x, w, dy, out):
    """Forward with every product in fp32, kept, and both gradients of an fp32 dy."""
    r = pk.linear8(x, w, activation="silu", keep="e4m3", exact=True)
    dz = pk.linear8_backward(dy, r.z, activation="silu")
    return [r.y, r.z.codes, dz, pk.weight_grad8(dz, r.x, out, accumulate=True), pk.input_grad8([dz, dy], [w, w], dtype=F32)]


def test_exact_calls_captured_and_on_two_streams():
    """Two graphs, whose workspaces are their own, replayed in turn with eager work between; then the calls on two streams at
    once: the same bits as alone."""
    w = pk.pack8(u.randn((520, 256), 1) / 16)
    graphs = []
    for tokens in (40, 900):
        x, dy, out = (torch.zeros(s, dtype=d, device="cuda") for s, d in (((tokens, 256), BF16), ((tokens, 520), F32), ((520, 256), F32)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            exact_step(x, w, dy, out)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = exact_step(x, w, dy, out)
        graphs.append((g, x, dy, out, outs))
    for r in range(4):
        for g, x, dy, out, outs in graphs:
            x.copy_(u.randn(x.shape, 10 + r, dtype=BF16))
            dy.copy_(u.randn(dy.shape, 20 + r))
            out.zero_()
            g.replay()
            want = exact_step(x.clone(), w, dy.clone(), torch.zeros_like(out))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), r
    args = [(x.clone(), w, dy.clone()) for _, x, dy, _, _ in graphs]
    want = [exact_step(*a, torch.zeros(520, 256, device="cuda")) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(exact_step(*a, torch.zeros(520, 256, device="cuda")))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for v, x in zip(got, want) for a, b in zip(v, x))


def test_parts_of_a_gradient_past_32_bits():
    """An fp32 gradient whose parts are more than 2^32 bytes each: the sums of its last rows."""
    tokens, rows, cols = 1_100_000, 2056, 100
    dy = torch.zeros(tokens, rows, device="cuda")
    dy[-500:] = u.randn((500, rows), 1)
    x = pk.pack8(torch.ones(tokens, cols, device="cuda") * 0.5)
    d = dy[-500:].double()
    want = (d.t() @ torch.full((500, cols), 0.5, dtype=torch.float64, device="cuda"))
    assert ((pk.weight_grad8(dy, x).double() - want).abs() <= u.sum_bound(0.5 * d.abs().sum(0)[:, None], 3 * 500 + 300)).all()
    w = pk.pack8(u.randn((rows, cols), 2) / 45)
    dx = pk.input_grad8(dy, w, dtype=F32)
    wv = u.values(w)
    assert not dx[:-500].any()
    assert ((dx[-500:].double() - d @ wv).abs() <= u.sum_bound(d.abs() @ wv.abs(), 3 * rows + 300)).all()
