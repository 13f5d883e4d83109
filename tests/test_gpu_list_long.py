"""Lists long enough that a work-group's chunk of the gradient list holds more than one part, and
tensors long enough that a chunk of their maxima holds more than 8192 elements: ragged lists with
empty, tiny and odd tensors between large ones, against 64 bits.  The tolerances are those of
test_gpu_list.py."""
import math

import pytest
import torch

import precision_adam_optimizer_amd as pk
from tests.test_gpu_list import (BF16, F16, F32, F8, HALF, HP, TINY, U, Case, amp_fields, f32, filled, gen, guards_hold,
                                 optimizer, ref_codes, ref_scale)

pytestmark = pytest.mark.gpu


def ragged_sizes(total):
    """Sizes that add to about `total`: large odd tensors, with small and empty ones before, between
    and behind them."""
    big = [int(total * f) | 1 for f in (0.31, 0.02, 0.4, 0.17, 0.1)]
    small = [[1], [0, 3, 8191], [4096, 8192], [4097, 0, 0, 2], [32768 + 5], [8193, 1]]
    out = list(small[0])
    for b, s in zip(big, small[1:]):
        out += [b] + s
    return out


# totals on each side of 512 chunks of 4096, 8192, 16384 and 32768 elements
TOTALS = [4_100_000, 5_000_000, 10_000_000, 20_000_000]


@pytest.mark.parametrize("total", TOTALS)
@pytest.mark.parametrize("sd, dd", [(F32, BF16), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("place", ["apart", "in place"])
def test_clip_of_long_lists(total, sd, dd, place):
    g = gen(total + (sd == F32))
    sizes = ragged_sizes(total)
    src = [filled(n, sd, g, 10.0 ** (k % 4 - 3), k % 3) for k, n in enumerate(sizes)]
    old = [x.clone() for x in src]
    dd = sd if place == "in place" else dd
    dst = src if place == "in place" else [filled(n, dd, g, 0.0, k % 2) for k, n in enumerate(sizes)]
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in old))
    clip = pk.GradClip(src, outs=None if place == "in place" else dst)
    for limit in (norm / 3, 0.0 if place == "apart" else norm / 9):
        now = math.sqrt(sum(float(x.double().square().sum()) for x in src))
        before = [x.clone() for x in src]
        res = clip.clip(limit).cpu()
        c = min(1.0, f32(limit) / (now + 1e-6)) if limit > 0 else 1.0
        assert abs(float(res[0]) - now) <= 2 * U * now and abs(float(res[1]) - c) <= 2 * U * c
        for x, d, s in zip(before, dst, src):
            want = x.double() * c
            tol = 2 * U * want.abs()
            if dd != F32:
                tol = tol + HALF[dd] * (want.abs() + tol)
            assert bool(((d.double() - want).abs() <= tol + TINY[dd] / 2).all()), (total, x.numel())
            guards_hold(d)
            if place == "apart":
                assert torch.equal(s, x)
                guards_hold(s)
    clip.close()


@pytest.mark.parametrize("at", ["first", "last", "small"])
def test_norm_of_a_long_list_sees_every_tensor(at):
    """One gradient that is not zero, in the first, the last or a small tensor between large ones."""
    sizes = ragged_sizes(10_000_000)
    xs = [torch.zeros(n, device="cuda", dtype=BF16) for n in sizes]
    k = {"first": 0, "last": len(sizes) - 1, "small": sizes.index(8191)}[at]
    clip = pk.GradClip(xs, outs=[None] * len(xs))
    for i in (0, sizes[k] // 2, sizes[k] - 1):
        xs[k][i] = 3.0
        assert clip.clip(1.0).tolist() == [3.0, f32(1.0 / (3.0 + 1e-6))]
        xs[k][i] = 0.0
    assert clip.clip(1.0).tolist() == [0.0, 1.0]
    clip.close()


@pytest.mark.parametrize("total", TOTALS[1:])
def test_scaled_step_of_long_lists(total):
    """The norm, the decision and the step of ragged lists with both kinds of moments; then a step
    that an Inf in the last tensor has skipped."""
    g = gen(total)
    S = 256.0
    sizes = ragged_sizes(total)
    cases = [Case(n, g, F32, BF16, None, 32 if k % 2 else 8, offset=k % 2, gscale=1e-2 * S) for k, n in enumerate(sizes)]
    opt = optimizer(cases, groups=[k % 3 for k in range(len(cases))], n_groups=3)
    amp = pk.amp_state(S)
    hp = {**HP, "weight_decay": (0.1, 0.0, 0.3)}
    norm = math.sqrt(sum(float(c.g.double().square().sum()) for c in cases)) / S
    factor = f32(f32(min(1.0, 0.5 / (norm + 1e-6))) * f32(1 / S))
    for k, c in enumerate(cases):
        c.expect(1, **{**HP, "weight_decay": hp["weight_decay"][k % 3]}, factor=factor)
    opt.step_amp(amp, max_norm=0.5, **hp)
    st = amp_fields(amp)
    assert abs(st["grad_norm"] - norm) <= 2 * U * norm and st["grad_factor"] == factor and st["step"] == 1
    for c in cases:
        c.check()
    cases[-1].g[-1] = math.inf
    before = [[x.clone() for x in (c.p, c.m, c.v)] for c in cases]
    opt.step_amp(amp, max_norm=0.5, **hp)
    st = amp_fields(amp)
    assert st["found_inf"] == 1 and st["step"] == 1 and st["scale"] == S / 2
    assert all(torch.equal(x, y) for c, old in zip(cases, before) for x, y in zip((c.p, c.m, c.v), old))
    opt.close()


@pytest.mark.parametrize("pd, gd", [(F32, F32), (BF16, BF16), (F16, BF16)])
def test_clipping_a_packed_list_of_thousands(pd, gd):
    """A packed list of 3000 ragged views and the one tensor they lie in, each against its own
    coefficient."""
    g = gen(14)
    n = 300007
    gr = filled(n, gd, g, 1e-3)
    cuts = [0] + torch.randint(0, n + 1, (2999,), generator=g, device="cuda").sort().values.tolist() + [n]
    spans = list(zip(cuts[:-1], cuts[1:]))
    norm = math.sqrt(float(gr.double().square().sum()))
    for lists in ([(0, n)], spans):
        out = torch.zeros(n + 1, device="cuda", dtype=BF16)[1:]
        clip = pk.GradClip([gr[i:j] for i, j in lists], outs=[out[i:j] for i, j in lists])
        res = clip.clip(0.1).cpu()
        assert abs(float(res[0]) - norm) <= 2 * U * norm
        assert torch.equal(out, (gr.float() * float(res[1])).bfloat16())  # one fp32 product, one rounding
        clip.close()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("mode", ["pow2", "amax"])
def test_tensor_scales_of_long_tensors(dtype, fmt, mode):
    """Three long tensors of odd sizes with a small and an empty one: the largest value in the first,
    a middle and the last chunk of its tensor, in the elements before and behind the vectors; codes,
    scales and the values they stand for bit for bit."""
    g = gen(21)
    sizes = [2_097_153, 0, 4_999_999, 77, 3_100_001]
    offs = [1, 0, 0, 1, 3]
    xs = [filled(n, dtype, g, 0.5, o) for n, o in zip(sizes, offs)]
    codes = [Case.bytes(torch.zeros(n, dtype=torch.uint8), o) for n, o in zip(sizes, offs)]
    scales = [filled(1, F32, g) for _ in sizes]
    q = pk.Quantizer(xs, fmt=fmt, granularity="tensor", scale_mode=mode, codes=codes, scales=scales)
    for turn in range(6):
        # a value larger than any other by a factor of its own, so that a missed one shows in the scale
        for k, x in enumerate(xs):
            n = x.numel()
            if n:
                at = [0, n - 1, n // 2, min(n - 1, 2), n - 2, (n * 2) // 3][turn]
                x[at] = -40.0 * 3.0 ** ((turn + k) % 5) if turn % 2 else 55.0 * 2.5 ** ((turn + k) % 5)
        q.quantize()
        for x, c, s in zip(xs, codes, scales):
            guards_hold(c)
            guards_hold(s)
            if not x.numel():
                continue
            v = x.float().cpu()
            want, inv = ref_scale(v.abs().amax().view(1), fmt, mode)
            assert s.item() == want.float().item(), (x.numel(), turn)
            assert torch.equal(c.cpu(), ref_codes(v, inv.expand(v.numel()), fmt)), (x.numel(), turn)
    old = [x.clone() for x in xs]
    q.dequantize()
    for x, c, s, was in zip(xs, codes, scales, old):
        if x.numel():
            assert torch.equal(x, (c.view(F8[fmt]).float() * s).to(dtype))
        guards_hold(x)
    q.close()
