"""8-bit moments of the list AdamW over the whole range of fp32: codes and scales bit for bit
against the CPU's, at every scale exponent, from subnormal moments to the largest, at ties and a
step of fp32 beside them, and with the largest value at the border where its scale doubles.

beta1 = beta2 = 0 make the fresh moments plain functions of the gradient: m' = g and v' = g * g in
fp32, one rounding.
"""
import pytest
import torch

import precision_adam_optimizer_amd as pk
from tests.test_gpu_list import F8, FMAX, quantized, ref_scale

pytestmark = pytest.mark.gpu

F32 = torch.float32
PAIRS = [("e4m3", "e5m2"), ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2")]
HP = dict(lr=1e-3, beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0)


def neighbours(x):
    """x and the fp32 numbers next to it."""
    inf = torch.tensor(float("inf"))
    return [x, torch.nextafter(x, -inf), torch.nextafter(x, inf)]


def largest_values():
    """For every power of two of fp32: 0.875 of it (FMAX of both formats is 0.875 * 2^k) with the
    numbers beside it, and two others of its binade."""
    p = torch.ldexp(torch.ones(277), torch.arange(-149, 128))
    at = torch.cat(neighbours(0.875 * p) + [p, 0.6 * p])
    return at[at > 0]


def blocks_over_the_range(fmt):
    """Blocks of 128 in which the first value is the largest: four for each of largest_values(), one
    of values over the whole range below it, three at the ties of the format and beside them."""
    g = torch.Generator().manual_seed(3)
    top = largest_values()
    n = top.numel()
    s, _ = ref_scale(top, fmt)
    # values: magnitudes spread over their logarithm below the largest, down to the last subnormal
    e = (torch.log2(top)[:, None] + 149).clamp(min=0) * torch.rand(n, 127, generator=g)
    spread = torch.minimum(torch.exp2((e - 149).double()).float(), top[:, None])
    grid = torch.arange(256, dtype=torch.uint8).view(F8[fmt]).float()
    grid = grid[torch.isfinite(grid) & (grid >= 0)].unique()
    ties = (grid[1:] + grid[:-1]).double() / 2
    ties = (ties[None, :] * s[:, None]).float()          # exact but where it is subnormal in fp32
    ties = torch.cat([ties, ties.new_zeros(n, 127 - ties.shape[1])], 1)
    ties = torch.minimum(ties, top[:, None])
    rows = [spread] + [torch.minimum(x.clamp(min=0), top[:, None]) for x in neighbours(ties)]
    signs = torch.where(torch.rand(4, n, 127, generator=g) < 0.5, -1.0, 1.0)
    out = torch.cat([torch.cat([top[:, None], r * q], 1) for r, q in zip(rows, signs)])
    return out[torch.randperm(out.shape[0], generator=g)]


def guarded(n, dtype, fill):
    x = torch.full((n + 8,), 7, dtype=dtype, device="cuda")
    x[:n] = fill
    return x


def run(gr, sizes, fmts):
    """The fresh state of gr's pieces of those sizes, and the state after a second step that halves
    the moments (no gradient, betas of 1/2), with what lies behind every buffer checked."""
    pieces = list(gr.split(sizes))
    blocks = [-(-n // 128) for n in sizes]
    state = [[guarded(n, torch.uint8, 0) for n in sizes] for _ in range(2)] + [
        [guarded(n, F32, 1.0) for n in blocks] for _ in range(2)]
    views = [[x[:-8] for x in xs] for xs in state]
    opt = pk.AdamW([torch.zeros_like(x) for x in pieces], pieces, state_bits=8, m_format=fmts[0], v_format=fmts[1],
                   state=views)
    opt.step(step=1, **HP)
    assert all(bool((x[-8:] == 7).all()) for xs in state for x in xs)
    first = [torch.cat(xs).cpu() for xs in views]
    for x in pieces:
        x.zero_()
    opt.step(step=2, **{**HP, "beta1": 0.5, "beta2": 0.5})
    assert all(bool((x[-8:] == 7).all()) for xs in state for x in xs)
    opt.close()
    return first, [torch.cat(xs).cpu() for xs in views]


@pytest.mark.parametrize("fmts", PAIRS)
@pytest.mark.parametrize("roots", [False, True])
def test_codes_over_the_whole_range(fmts, roots):
    """roots: gradients whose squares cover the range (those of the others pass fp32 at both ends)."""
    x = blocks_over_the_range(fmts[1] if roots else fmts[0]).view(-1)
    if roots:
        x = torch.sqrt(x.abs()).copysign(x)
    sq = (x.double() * x.double()).float()
    x = x + 0.0  # m' = fma(0, 0, g): a gradient of -0 gives 0 + -0 = +0
    want = [quantized(y, f) for y, f in zip((x, sq), fmts)]
    finite = torch.isfinite(sq.view(-1, 128)).all(1).repeat_interleave(128)
    n = x.numel()
    if roots:
        assert bool(finite.all()) and bool(((sq > 0) & (sq < 2.0 ** -126)).any())
    for sizes in ([n], [896] * (n // 896) + ([n % 896] if n % 896 else [])):  # whole work-groups; parts of one
        (m, v, ms, vs), second = run(x.cuda(), sizes, fmts)
        assert torch.equal(ms, want[0][1]), "m scales"
        bad = (m != want[0][0]).nonzero().view(-1)
        assert bad.numel() == 0, ("m", bad.numel(), [(x[i].item(), ms[i // 128].item(), m[i].item(), want[0][0][i].item()) for i in bad[:5]])
        if bool(finite.all()):
            assert torch.equal(vs, want[1][1]), "v scales"
        bad = ((v != want[1][0]) & finite).nonzero().view(-1)
        assert bad.numel() == 0, ("v", bad.numel(), [(sq[i].item(), vs[i // 128].item(), v[i].item(), want[1][0][i].item()) for i in bad[:5]])
        # a square past fp32: its block takes scale 1, and an Inf saturates
        if not bool(finite.all()):
            odd = ~finite
            assert bool((vs[odd[::128]] == 1).all())
            over = v[~torch.isfinite(sq)].view(F8[fmts[1]]).float()
            assert bool((over == FMAX[fmts[1]]).all())
        # the second step: half of each decoded moment (one rounding where that is subnormal), in new codes
        for c, sc, f, got, got_s in zip((m, v), (ms, vs), fmts, second[:2], second[2:]):
            half = (c.view(F8[f]).double() * sc.double().repeat_interleave(128) / 2).float()
            half = half + 0.0  # fma(1/2, -0, 0) = +0
            want2, want2_s = quantized(half, f)
            assert torch.equal(got_s, want2_s) and torch.equal(got, want2), f
