"""The list operators (AdamW over mixed lists, clipping, conversion to 8 bits)
against plain references in 64 bits.

Tolerances, in half-steps u = 2^-24 of fp32 (a rounding is off by at most one
half-step of its result) plus, for 16-bit results, one half-step of their type:
  * 32-bit moments: m' = fma(b1, m, (1-b1)*G).  b1, 1-b1 and G carry one half-step
    each, the product one, the fma one: at most 3u|(1-b1)G| + u|b1 m| + u|m'|, held to
    4u(|b1 m| + |(1-b1)G|).  v' likewise with G twice: 6u(b2 v + (1-b2)G^2).
  * 8-bit moments: codes and scales equal, bit for bit, from the fp32 chain.
  * weights: update = step * m' / (sqrt(v'/bc2) + eps): half of v's 6, bc2 1/2, its product 1/2, the
    square root 2 (one ulp), the sum 1, the reciprocal 2, step 1 and two products 2: at
    most 12u|update|, beside m's own 4u(|b1 m| + |(1-b1)G|) through step / den; decay, its sum
    and the difference: 2u|lr wd p| + u|update| + u|p'|.
  * clipping: the coefficient (1 half-step, and none of the fp64 sum's) and the product: 2u|out|.
"""
import math

import numpy as np
import pytest
import torch

import precision_adam_optimizer_amd as pk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # smallest step
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SIZES = [1, 2, 3, 5, 31, 32, 33, 127, 128, 129, 0, 255, 1023, 1024, 1025, 4099, 20000]
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def filled(n, dtype, g, scale=1.0, offset=0, fill=None):
    """n values at an offset of that many elements into their memory, with guards behind them."""
    x = torch.full((n + offset + 8,), 7.0, dtype=F32, device="cuda")
    x[offset:offset + n] = torch.randn(n, generator=g, device="cuda") * scale if fill is None else fill
    x = x.to(dtype)
    return x[offset:offset + n]


def guards_hold(t):
    base = t._base
    n = t.numel()
    off = t.storage_offset()
    assert bool((base[:off].float() == 7).all()) and bool((base[off + n:].float() == 7).all())


def f32(x):
    return float(np.float32(x))


def ref_scale(amax, fmt, mode="pow2"):
    """(scale, inverse) in fp32 numbers (as float64 tensors) of amax (fp32 numbers)."""
    a = amax.double()
    fine = (a > 0) & torch.isfinite(a)
    if mode == "pow2":
        f, e = torch.frexp(a.float())
        k = (e - (9 if fmt == "e4m3" else 16) + (f > 0.875)).clamp(-126, 126)
        s = torch.tensor([2.0 ** int(i) for i in k.tolist()], dtype=torch.float64)
        inv = 1.0 / s
    else:
        sc = a.float() / torch.tensor(FMAX[fmt], dtype=F32)
        low = sc < 2.0 ** -126
        s = torch.where(low, torch.full_like(sc, 2.0 ** -126), sc).double()
        inv = torch.where(low, torch.full_like(sc, 2.0 ** 126), torch.tensor(FMAX[fmt], dtype=F32) / a.float()).double()
    one = torch.ones_like(a)
    return torch.where(fine, s, one), torch.where(fine, inv, one)


def ref_codes(x, inv, fmt):
    """Codes of fp32 x (CPU) at fp32 inverse scales, saturating."""
    return (x * inv.float()).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)


def blocks_of(x):
    n = x.numel()
    pad = torch.zeros(-(-n // 128) * 128 - n, dtype=x.dtype)
    return torch.cat([x, pad]).view(-1, 128)


def quantized(x, fmt, mode="pow2"):
    """(codes, scales) of fp32 x on the CPU, by blocks of 128."""
    s, inv = ref_scale(blocks_of(x.abs()).amax(1), fmt, mode)
    return ref_codes(x, inv.repeat_interleave(128)[:x.numel()], fmt), s.float()


class Case:
    """One tensor of a list: its inputs on the GPU and what a step has to give."""

    def __init__(self, n, g, pd=F32, gd=BF16, cd=None, bits=32, offset=0, fmts=("e4m3", "e5m2"), gscale=1e-3):
        self.n, self.bits, self.fmts = n, bits, fmts
        self.p = filled(n, pd, g, 0.02, offset)
        self.g = filled(n, gd, g, gscale, offset)
        self.copy = filled(n, cd, g, 0.0, offset) if cd else None
        m = torch.randn(n, generator=g, device="cuda") * gscale * 0.3
        v = (torch.randn(n, generator=g, device="cuda") * 0.3 + 1).abs() * gscale * gscale
        if bits == 32:
            self.m, self.v = filled(n, F32, g, 0, offset, m), filled(n, F32, g, 0, offset, v)
            self.ms = self.vs = None
        else:
            (cm, sm), (cv, sv) = quantized(m.cpu(), fmts[0]), quantized(v.cpu(), fmts[1])
            self.m, self.v = self.bytes(cm, offset), self.bytes(cv, offset)
            self.ms, self.vs = sm.cuda(), sv.cuda()

    @staticmethod
    def bytes(c, offset):
        x = torch.full((c.numel() + offset + 8,), 7, dtype=torch.uint8, device="cuda")
        x[offset:offset + c.numel()] = c.cuda()
        return x[offset:offset + c.numel()]

    def expect(self, t, lr, beta1, beta2, eps, weight_decay, factor=1.0):
        """References from the present state, before the step runs."""
        p, gr = self.p.double().cpu(), self.g.double().cpu()
        self.p_old = p
        if self.bits == 32:
            G = gr * factor
            am, ag = beta1 * self.m.double().cpu(), (1 - beta1) * G
            av, agg = beta2 * self.v.double().cpu(), (1 - beta2) * G * G
            m1, v1 = am + ag, av + agg
            self.m_tol = 4 * U * (am.abs() + ag.abs()) + 2.0 ** -148
            self.v_tol = 6 * U * (av + agg) + 2.0 ** -148
            self.want_m, self.want_v = m1, v1
        else:
            # the fp32 chain: products and sums exact in 64 bits, then rounded
            G = (gr * factor).float()
            dm = self.m.cpu().view(F8[self.fmts[0]]).double() * self.ms.cpu().double().repeat_interleave(128)[:self.n]
            dv = self.v.cpu().view(F8[self.fmts[1]]).double() * self.vs.cpu().double().repeat_interleave(128)[:self.n]
            gm = (f32(1 - beta1) * G.double()).float()
            gv = (f32(1 - beta2) * (G.double() * G.double()).float().double()).float()
            m1 = (f32(beta1) * dm + gm.double()).float().double()
            v1 = (f32(beta2) * dv + gv.double()).float().double()
            self.want_m, self.want_ms = quantized(m1.float(), self.fmts[0])
            self.want_v, self.want_vs = quantized(v1.float(), self.fmts[1])
            self.m_tol = torch.zeros_like(m1)
        step = lr / (1 - beta1 ** t)
        den = (v1 / (1 - beta2 ** t)).sqrt() + eps
        upd, decay = step * m1 / den, lr * weight_decay * p
        self.want_p = p - (decay + upd)
        self.p_tol = U * (13 * upd.abs() + 2 * decay.abs() + self.want_p.abs()) + step * self.m_tol / den + 2.0 ** -148

    def check(self, name=""):
        for what, got, extra in (("p", self.p, None), ("copy", self.copy, None)):
            if got is None:
                continue
            err = (got.double().cpu() - self.want_p).abs()
            tol = self.p_tol if got.dtype == F32 else (
                self.p_tol + HALF[got.dtype] * (self.want_p.abs() + self.p_tol) + TINY[got.dtype] / 2)
            assert bool((err <= tol).all()), (name, what, self.n, got.dtype, float((err - tol).max()))
            guards_hold(got)
        if self.bits == 32:
            for what, got, want, tol in (("m", self.m, self.want_m, self.m_tol), ("v", self.v, self.want_v, self.v_tol)):
                err = (got.double().cpu() - want).abs()
                assert bool((err <= tol).all()), (name, what, self.n, float((err - tol).max()))
        else:
            for what, got, want in (("m", self.m, self.want_m), ("v", self.v, self.want_v), ("m scales", self.ms, self.want_ms),
                                    ("v scales", self.vs, self.want_vs)):
                assert torch.equal(got.cpu(), want), (name, what, self.n)
        guards_hold(self.m)
        guards_hold(self.v)


def optimizer(cases, **kw):
    if any(c.bits == 8 for c in cases):
        state = ([c.m for c in cases], [c.v for c in cases], [c.ms for c in cases], [c.vs for c in cases])
    else:
        state = ([c.m for c in cases], [c.v for c in cases])
    return pk.AdamW([c.p for c in cases], [c.g for c in cases], copies=[c.copy for c in cases],
                    state_bits=[c.bits for c in cases], state=state, **kw)


WEIGHTS = [(F32, None), (F32, BF16), (F32, F16), (BF16, None), (F16, None)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gd", [F32, BF16, F16])
@pytest.mark.parametrize("pd, cd", WEIGHTS)
@pytest.mark.parametrize("offset", [0, 1])
def test_adamw_types_and_sizes(bits, gd, pd, cd, offset):
    g = gen(1)
    cases = [Case(n, g, pd, gd, cd, bits, offset) for n in SIZES]
    opt = optimizer(cases)
    for t in (1, 2):
        for c in cases:
            c.expect(t, **HP)
        opt.step(step=t, **HP)
        for c in cases:
            c.check(f"step {t}")
    opt.close()


@pytest.mark.parametrize("fmts", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2"), ("e4m3", "e5m2")])
def test_adamw_formats(fmts):
    g = gen(2)
    cases = [Case(n, g, bits=8, fmts=fmts, gscale=10.0 ** -(k % 6)) for k, n in enumerate(SIZES)]
    opt = optimizer(cases, m_format=fmts[0], v_format=fmts[1])
    for t in (7, 8):
        for c in cases:
            c.expect(t, **HP)
        opt.step(step=t, **HP)
        for c in cases:
            c.check()
    opt.close()


def test_adamw_mixed_list_and_groups():
    """Every kind in one list, in three groups with their own hyperparameters."""
    g = gen(3)
    cases = [Case(n, g, pd, gd, cd, bits, offset=(n + k) % 3)
             for k, (pd, cd) in enumerate(WEIGHTS) for gd in (F32, BF16, F16) for bits in (32, 8) for n in (77, 1500, 0)]
    groups = [k % 3 for k in range(len(cases))]
    hp = dict(lr=[1e-3, 3e-4, 0.0], beta1=[0.9, 0.0, 0.95], beta2=[0.95, 0.999, 0.0], eps=[1e-8, 1e-6, 1e-3],
              weight_decay=[0.1, 0.0, 0.5])
    opt = optimizer(cases, groups=groups)
    for t in (5, 6):
        for c, q in zip(cases, groups):
            c.expect(t, **{k: x[q] for k, x in hp.items()})
        opt.step(step=t, **hp)
        for c in cases:
            c.check()
    with pytest.raises(ValueError, match="each of the 3 groups"):
        opt.step(step=7, **{**hp, "lr": [1e-3]})
    for bad in (dict(lr=math.inf), dict(lr=1e39), dict(eps=1e39), dict(lr=1e30, weight_decay=1e30), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(weight_decay=math.nan)):
        with pytest.raises(pk.Fp8AdamError):
            opt.step(step=7, **{**hp, **bad})
    with pytest.raises(pk.Fp8AdamError, match="step"):
        opt.step(step=0, **hp)
    for c in cases:
        c.check()  # nothing that was refused ran
    opt.close()
    with pytest.raises(RuntimeError, match="closed"):
        opt.step(step=7, **hp)


def test_adamw_repeats_and_does_not_depend_on_the_list():
    """Two runs give the same bits, and a tensor's result does not depend on the list around it."""
    def run(sizes, keep):
        out = []
        for n in sizes:
            g = gen(n)
            c = Case(n, g, bits=8)
            out.append(c)
        opt = optimizer(out)
        for t in range(1, 4):
            opt.step(step=t, **HP)
        opt.close()
        return [[x.clone() for x in (c.p, c.m, c.v, c.ms, c.vs)] for c in out if c.n in keep]
    a, b, d = run([5000, 333, 129], (333,)), run([5000, 333, 129], (333,)), run([333], (333,))
    for x, y, z in zip(a[0], b[0], d[0]):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("pd", [F32, BF16])
def test_adamw8_equals_the_block_128_step(pd):
    """Codes and scales are those of FP8AdamW(granularity="block128"), bit for bit, for betas
    that are fp32 numbers; its state goes from one to the other."""
    hp = dict(lr=1e-3, beta1=f32(0.9), beta2=f32(0.95), eps=1e-8, weight_decay=0.1)
    g = gen(4)
    cases = [Case(n, g, pd, BF16, bits=8) for n in SIZES]
    p2 = [c.p.clone() for c in cases]
    st = [[x.clone() for x in xs] for xs in ([c.m for c in cases], [c.v for c in cases], [c.ms for c in cases], [c.vs for c in cases])]
    st[2] = [x if x.numel() else x.new_ones(1) for x in st[2]]
    st[3] = [x if x.numel() else x.new_ones(1) for x in st[3]]
    a = optimizer(cases)
    b = pk.FP8AdamW(p2, [c.g.clone() for c in cases], granularity="block128", state=st)
    for t in range(1, 4):
        before = [c.p.clone().float() for c in cases]
        a.step(step=t, **hp)
        b.step(step=t, **hp)
        for c, q, m, v, ms, vs, old in zip(cases, p2, b.m, b.v, b.m_scale, b.v_scale, before):
            assert torch.equal(c.m, m) and torch.equal(c.v, v)
            if c.n:
                assert torch.equal(c.ms, ms) and torch.equal(c.vs, vs)
                d = (c.p.float() - q.float()).abs()
                # p' is a difference of p and an update no larger than |p| + |p'|, each off by a few u: both
                # steps are within 1e-6 of the larger of |p| and |p'| of the exact weight (about 16u), so 2e-6
                # apart; rounded to bf16 (2^-8 each) as well, 2^-7 more
                tol = 2e-6 * torch.maximum(c.p.float().abs(), old.abs())
                tol = tol if pd == F32 else tol + 2.0 ** -7 * torch.maximum(c.p.float().abs(), q.float().abs())
                assert bool((d <= tol + 1e-30).all())
        [q.copy_(c.p) for c, q in zip(cases, p2)]
    a.close()
    b.close()


def test_adamw_orders_in_memory():
    """Weights, gradients and copies that are transposed alike; moments follow the memory."""
    g = gen(5)
    p0 = torch.randn(37, 65, generator=g, device="cuda")
    g0 = torch.randn(37, 65, generator=g, device="cuda").bfloat16()
    got = []
    for turned in (False, True):
        for bits in (32, 8):
            p, gr = (x.t().contiguous().t() if turned else x.clone() for x in (p0, g0))
            c = torch.empty_like(p, dtype=BF16)
            assert p.is_contiguous() != turned
            opt = pk.AdamW([p], [gr], state_bits=bits, copies=[c])
            opt.step(step=1, **HP)
            assert torch.equal(c, p.bfloat16())
            got.append((p, opt.m[0]))
            opt.close()
    assert torch.equal(got[0][0], got[2][0]) and torch.equal(got[0][1], got[2][1])  # 32 bits: the same numbers
    assert torch.equal(got[1][0], got[3][0])  # the first step's weights come before any rounding to 8 bits


def test_adamw_nonfinite_and_zeros():
    inf, nan = math.inf, math.nan
    vals = torch.tensor([0.0, -0.0, 1.0, inf, -inf, nan, 1e-30, -1e-38, 3e38], device="cuda")
    for bits in (32, 8):
        p = torch.ones(9, device="cuda")
        opt = pk.AdamW([p], [vals], state_bits=bits)
        opt.step(step=1, **HP)
        m, v = opt.converted_state(32)[:2] if bits == 8 else (opt.m, opt.v)
        # p: 0 gradients move nothing but the decay; an Inf gives Inf / Inf, a NaN a NaN
        assert torch.equal(p[:2].cpu(), torch.full((2,), 1 - 1e-4)), p
        assert bool(p[3:6].isnan().all()) and abs(float(p[2]) - (1 - 1e-4 - 1e-3)) < 1e-6
        # g^2 = Inf in fp32: no update is left
        assert abs(float(p[8]) - (1 - 1e-4)) < 1e-6
        if bits == 32:
            assert m[0][3] == inf and m[0][4] == -inf and m[0][5].isnan() and v[0][3] == inf and v[0][8] == inf
        else:  # the block takes scale 1: Inf saturates, NaN stays
            assert m[0][3] == 448 and m[0][4] == -448 and m[0][5].isnan()
            assert float(opt.m_scale[0]) == 1 and float(opt.v_scale[0]) == 1
        # a later tensor is untouched by it
        opt.close()
    for bits in (32, 8):  # all zero: nothing moves, scales 1
        p, gr = torch.zeros(200, device="cuda"), torch.zeros(200, device="cuda", dtype=BF16)
        opt = pk.AdamW([p], [gr], state_bits=bits)
        opt.step(step=1, **HP)
        assert not p.any() and not opt.m[0].any() and not opt.v[0].any()
        if bits == 8:
            assert bool((opt.m_scale[0] == 1).all())
        opt.close()


@pytest.mark.parametrize("eps", [0.0, 1e-25, 1e-20, 2.0 ** -38, 1e-8])
@pytest.mark.parametrize("amp", [False, True])
def test_adamw_tiny_gradients_and_eps(eps, amp):
    """Gradients whose squares are subnormal in fp32, down to none, beside large ones: the weight is
    the formula's for the moments that were stored (12u of the update, and the sum)."""
    gr = torch.tensor([10.0 ** -k for k in range(-13, 23)], device="cuda")
    p = torch.ones(gr.numel(), device="cuda")
    opt = pk.AdamW([p], [gr])
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=eps, weight_decay=0.0)
    if amp:
        opt.step_amp(pk.amp_state(1.0), **hp)
    else:
        opt.step(step=1, **hp)
    m, v = opt.m[0].double().cpu(), opt.v[0].double().cpu()
    assert float(v.min()) >= 0 and bool(((v > 0) & (v < 2.0 ** -126)).any())
    upd = 1e-3 / (1 - 0.9) * m / ((v / (1 - 0.95)).sqrt() + eps)
    some = (v > 0) | (eps > 0)
    err = (p.double().cpu() - (1 - upd)).abs()
    assert bool((err <= U * (13 * upd.abs() + 1.01) + 2.0 ** -148)[some].all()), (eps, err / U)
    opt.close()


def amp_fields(t):
    return pk.read_amp_state(t)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gd", [F32, F16, BF16])
def test_adamw_amp(bits, gd):
    """Unscale, clip, skip on Inf, count and grow: the step against the references with the
    factor that the state reports, the state against 64 bits."""
    g = gen(6)
    S = 1024.0
    cases = [Case(n, g, F32, gd, BF16, bits, gscale=1e-2 * S, offset=n % 2) for n in SIZES]
    opt = optimizer(cases, groups=[k % 2 for k in range(len(cases))])
    amp = pk.amp_state(S, "cuda")
    kw = dict(max_norm=0.5, growth_interval=2)
    hp = {**HP, "weight_decay": (0.1, 0.0)}
    taken, scale, tracker = 0, S, 0
    for call in range(5):
        grads = [c.g.clone() for c in cases]
        if call == 2:
            cases[9].g[-1] = math.inf
        if call == 3:
            cases[4].g[0] = math.nan
        bad = call in (2, 3)
        before = [[x.clone() for x in (c.p, c.copy, c.m, c.v)] for c in cases]
        norm = math.sqrt(sum(float(c.g.double().square().sum()) for c in cases)) / scale
        factor = f32(f32(min(1.0, 0.5 / (norm + 1e-6))) * f32(1 / scale)) if not bad else 0.0
        for k, c in enumerate(cases):
            c.expect(taken + 1, **{**HP, "weight_decay": hp["weight_decay"][k % 2]}, factor=factor)
        opt.step_amp(amp, **hp, **kw)
        st = amp_fields(amp)
        if bad:
            assert st["found_inf"] == 1 and math.isnan(st["grad_norm"]) and st["grad_factor"] == 0.0
            scale, tracker = scale * 0.5, 0
            for c, old in zip(cases, before):
                assert all(torch.equal(x, y) for x, y in zip((c.p, c.copy, c.m, c.v), old))
            for c, old in zip(cases, grads):
                c.g.copy_(old)
        else:
            taken, tracker = taken + 1, tracker + 1
            assert st["found_inf"] == 0 and abs(st["grad_norm"] - norm) <= 2 * U * norm
            assert abs(st["clip_coef"] - min(1.0, 0.5 / (norm + 1e-6))) <= 2 * U
            assert st["grad_factor"] == factor
            for c in cases:
                c.check(f"call {call}")
            if tracker == 2:
                scale, tracker = scale * 2, 0
        assert (st["scale"], st["growth_tracker"], st["step"]) == (scale, tracker, taken)
    with pytest.raises(ValueError, match="amp_state"):
        opt.step_amp(amp.cpu(), **hp)
    for bad in (dict(growth_factor=1.0), dict(backoff_factor=1.0), dict(growth_interval=0), dict(max_norm=math.inf)):
        with pytest.raises(pk.Fp8AdamError):
            opt.step_amp(amp, **hp, **bad)
    opt.close()


# ------------------------------------------------------------------- clipping

@pytest.mark.parametrize("sd", [F32, BF16, F16])
@pytest.mark.parametrize("dd", [F32, BF16, F16])
@pytest.mark.parametrize("soff, doff", [(0, 0), (1, 0), (0, 3), (5, 1)])
def test_clip_types_and_sizes(sd, dd, soff, doff):
    g = gen(7)
    src = [filled(n, sd, g, 0.3, soff) for n in SIZES + [70001]]
    dst = [filled(n, dd, g, 0.0, doff) for n in SIZES + [70001]]
    clip = pk.GradClip(src, outs=dst)
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in src))
    for limit in (1.0, 0.0, 1e9, norm / 2):
        [d.fill_(3.0) for d in dst]
        res = clip.clip(limit).cpu()
        c = min(1.0, f32(limit) / (norm + 1e-6)) if limit > 0 else 1.0
        assert abs(float(res[0]) - norm) <= 2 * U * norm and abs(float(res[1]) - c) <= 2 * U * c
        if c == 1.0:
            assert float(res[1]) == 1.0
        for x, d in zip(src, dst):
            want = x.double() * c
            tol = 2 * U * want.abs()
            if dd != F32:
                tol = tol + HALF[dd] * (want.abs() + tol)
            assert bool(((d.double() - want).abs() <= tol + TINY[dd] / 2).all()), (sd, dd, x.numel())
            guards_hold(d)
            guards_hold(x)
    clip.close()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_clip_in_place_and_norm_only(dtype):
    g = gen(8)
    xs = [filled(n, dtype, g, 0.1, n % 3) for n in SIZES]
    old = [x.clone() for x in xs]
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in xs))
    only = pk.GradClip(xs, outs=[None] * len(xs))
    assert abs(float(only.clip(0.01)[0]) - norm) <= 2 * U * norm
    assert all(torch.equal(x, y) for x, y in zip(xs, old))
    some = pk.GradClip(xs, outs=[x if k % 2 else None for k, x in enumerate(xs)])
    clip = pk.GradClip(xs)
    clip.clip(norm * 2)
    assert all(torch.equal(x, y) for x, y in zip(xs, old))  # under the limit: as they were
    some.clip(norm / 4)
    c = (norm / 4) / (norm + 1e-6)
    for k, (x, y) in enumerate(zip(xs, old)):
        if k % 2:
            want = y.double() * c
            tol = 2 * U * want.abs() + (0 if dtype == F32 else HALF[dtype] * 1.01 * want.abs()) + TINY[dtype] / 2
            assert bool(((x.double() - want).abs() <= tol).all())
        else:
            assert torch.equal(x, y)
        guards_hold(x)
    for o in (only, some, clip):
        o.close()


def test_clip_nonfinite_empty_and_huge():
    for value, check in ((math.inf, math.isinf), (math.nan, math.isnan)):
        x = torch.ones(5000, device="cuda")
        x[4321] = value
        out = torch.zeros(5000, device="cuda", dtype=BF16)
        clip = pk.GradClip([x], outs=[out])
        res = clip.clip(1.0).cpu()
        assert check(float(res[0])) and float(res[1]) == 1.0
        assert torch.equal(out[:4000], torch.ones(4000, device="cuda", dtype=BF16)) and check(float(out[4321]))
        clip.close()
    e = torch.zeros(0, device="cuda")
    clip = pk.GradClip([e, e])
    assert clip.clip(1.0).tolist() == [0.0, 1.0]
    clip.close()
    big = torch.full((3000,), 2.0 ** 120, device="cuda")  # squares are past fp32
    clip = pk.GradClip([big])
    res = clip.clip(1.0).tolist()
    want = math.sqrt(3000) * 2.0 ** 120
    assert abs(res[0] - want) <= 2 * U * want
    n1 = float(big.double().square().sum().sqrt())
    assert abs(n1 - 1) < 1e-6
    small = torch.full((3000,), 2.0 ** -140, device="cuda")  # and so are these
    clip2 = pk.GradClip([small])
    want = math.sqrt(3000) * 2.0 ** -140
    assert abs(clip2.clip(1.0).tolist()[0] - want) <= 2 * U * want + 2.0 ** -149
    clip.close()
    clip2.close()


# ---------------------------------------------------------- conversion to 8 bits

def values(n, dtype, g, offset, k):
    x = torch.randn(n, generator=g, device="cuda") * 10.0 ** ((k % 7) - 4)
    if n > 3:
        x[n // 2] = 0.0
        x[1] *= 50.0
    return filled(n, dtype, g, 0, offset, x)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("granularity", ["block128", "tensor"])
@pytest.mark.parametrize("mode", ["pow2", "amax"])
@pytest.mark.parametrize("offset", [0, 1])
def test_quantize_and_back(dtype, fmt, granularity, mode, offset):
    """Codes, scales and the values they stand for, bit for bit (each step is one fp32 rounding)."""
    g = gen(9)
    sizes = SIZES + [30011]
    xs = [values(n, dtype, g, offset, k) for k, n in enumerate(sizes)]
    codes = [Case.bytes(torch.zeros(n, dtype=torch.uint8), offset) for n in sizes]
    old = [x.clone() for x in xs]
    q = pk.Quantizer(xs, fmt=fmt, granularity=granularity, scale_mode=mode, codes=codes)
    q.quantize()
    for x, y, c, s in zip(xs, old, codes, q.scales):
        assert torch.equal(x, y)  # only read
        guards_hold(c)
        v = x.float().cpu()
        if not x.numel():
            continue
        if granularity == "block128":
            want, ws = quantized(v, fmt, mode)
        else:
            sc, inv = ref_scale(v.abs().amax().view(1), fmt, mode)
            want, ws = ref_codes(v, inv.expand(v.numel()), fmt), sc.float()
        assert torch.equal(s.cpu(), ws), (x.numel(), s.cpu() / ws)
        assert torch.equal(c.cpu(), want), x.numel()
    q.dequantize()
    for x, c, s in zip(xs, codes, q.scales):
        over = s.repeat_interleave(128)[:x.numel()] if granularity == "block128" else s
        want = (c.view(F8[fmt]).float() * over).to(dtype) if x.numel() else x
        assert torch.equal(x, want)
        guards_hold(x)
    q.close()


def test_quantize_mixed_list_nonfinite_and_extremes():
    dev = "cuda"
    a = torch.full((300,), 2.0 ** 127, device=dev)          # the largest scale
    b = torch.full((300,), 2.0 ** -149, device=dev)         # the smallest: codes lose it
    c = torch.ones(300, device=dev, dtype=BF16)
    c[5], c[200] = math.inf, math.nan                        # two blocks of scale 1
    z = torch.zeros(300, device=dev, dtype=F16)
    for granularity in ("block128", "tensor"):
        q = pk.Quantizer([a.clone(), b.clone(), c.clone(), z.clone()], fmt=["e5m2", "e4m3", "e4m3", "e5m2"], granularity=granularity)
        q.quantize()
        assert bool((q.scales[0] == 2.0 ** (127 - 15)).all()) and bool((q.scales[1] == 2.0 ** -126).all())
        if granularity == "block128":
            assert q.scales[2].tolist() == [1.0, 1.0, 2.0 ** -8]
        else:
            assert q.scales[2].tolist() == [1.0]
        assert bool((q.scales[3] == 1).all()) and not q.codes[3].any()
        q.dequantize()
        assert torch.equal(q.values[0], a) and not q.values[1].any() and not q.values[3].any()
        assert float(q.values[2][5]) == 448.0 and bool(q.values[2][200].isnan()) and float(q.values[2][7]) == 1.0
        q.close()
    e = torch.zeros(0, device=dev)
    q = pk.Quantizer([e])
    q.quantize()
    q.dequantize()
    q.close()


def test_state_goes_between_32_and_8_bits():
    """32-bit moments to both kinds of FP8AdamW state and to AdamW's 8-bit one, and back."""
    g = gen(10)
    cases = [Case(n, g) for n in SIZES]
    opt = optimizer(cases)
    opt.step(step=1, **HP)
    eight = opt.converted_state(8)
    for k, c in enumerate(cases):
        for j, (x, fmt) in enumerate(((c.m, "e4m3"), (c.v, "e5m2"))):
            codes, s = quantized(x.cpu(), fmt)
            assert torch.equal(eight[j][k].cpu(), codes) and (c.n == 0 or torch.equal(eight[2 + j][k].cpu(), s))
    p, gr = [c.p.clone() for c in cases], [c.g.clone() for c in cases]
    opt8 = pk.AdamW(p, gr, state_bits=8, state=eight)
    back = opt8.converted_state(32)
    for k, c in enumerate(cases):
        over = eight[2][k].repeat_interleave(128)[:c.n]
        assert torch.equal(back[0][k], eight[0][k].view(F8["e4m3"]).float() * over) and back[2][k] is None
    f = pk.FP8AdamW([x.clone() for x in p], gr, granularity="block128", state=opt8.checkpoint())
    hp = {**HP, "beta1": f32(0.9), "beta2": f32(0.95)}
    opt8.step(step=2, **hp)
    f.step(step=2, **hp)
    assert all(torch.equal(x, y) for x, y in zip(opt8.m, f.m)) and all(torch.equal(x, y) for x, y in zip(opt8.v, f.v))
    tensor = opt.converted_state(8, granularity="tensor")
    f2 = pk.FP8AdamW([x.clone() for x in p], gr, state=tensor)
    f2.step(step=2, **HP)
    with pytest.raises(ValueError, match="per-tensor"):
        opt8.converted_state(8, granularity="tensor")
    for o in (opt, opt8, f, f2):
        o.close()


# ---------------------------------------------------------------- as they are used

def test_training_step_with_all_of_them():
    """Accumulated fp32 gradients are clipped into bf16 ones, which FP8AdamW and the 8-bit list
    step both take to the same state; the new weights go to FP8 in blocks."""
    g = gen(11)
    sizes = [4099, 333, 128, 1]
    acc = [torch.zeros(n, device="cuda") for n in sizes]
    half = [torch.zeros(n, device="cuda", dtype=BF16) for n in sizes]
    p = [torch.randn(n, generator=g, device="cuda") * 0.02 for n in sizes]
    p2 = [x.clone() for x in p]
    copies = [torch.zeros(n, device="cuda", dtype=BF16) for n in sizes]
    clip = pk.GradClip(acc, outs=half)
    a = pk.AdamW(p, half, state_bits=8, copies=copies)
    b = pk.FP8AdamW(p2, half, granularity="block128")
    q = pk.Quantizer(p)
    hp = {**HP, "beta1": f32(0.9), "beta2": f32(0.95)}
    for t in range(1, 5):
        for x in acc:
            x.copy_(torch.randn(x.numel(), generator=g, device="cuda") + torch.randn(x.numel(), generator=g, device="cuda"))
        norm = math.sqrt(sum(float(x.double().square().sum()) for x in acc))
        res = clip.clip(1.0)
        old = [x.clone() for x in p]
        [x.copy_(y) for x, y in zip(p2, p)]
        a.step(step=t, **hp)
        b.step(step=t, **hp)
        q.quantize()
        assert abs(float(res[0]) - norm) <= 2 * U * norm
        for x, h in zip(acc, half):
            want = x.double() / (norm + 1e-6)
            assert bool(((h.double() - want).abs() <= 1.01 * 2.0 ** -8 * want.abs() + 1e-30).all())
        for k in range(len(sizes)):
            assert torch.equal(a.m[k], b.m[k]) and torch.equal(a.v[k], b.v[k])
            assert torch.equal(a.m_scale[k], b.m_scale[k]) and torch.equal(a.v_scale[k], b.v_scale[k])
            # as in the test of the two steps above: 2e-6 of the larger of |p| and |p'|
            assert bool(((p[k] - p2[k]).abs() <= 2e-6 * torch.maximum(p[k].abs(), old[k].abs()) + 1e-30).all())
            codes, s = quantized(p[k].cpu(), "e4m3")
            assert torch.equal(q.codes[k].cpu(), codes) and torch.equal(q.scales[k].cpu(), s)
            assert torch.equal(copies[k], p[k].bfloat16())
    for o in (clip, a, b, q):
        o.close()


def test_streams_and_graph_replays():
    """The calls on a side stream, then captured once and replayed with the program's own work
    between: every replay equals the eager call."""
    def make(seed):
        g = gen(seed)
        cases = [Case(n, g, F32, F32, BF16, bits, gscale=30.0) for n in (1000, 129, 5) for bits in (32, 8)]
        opt = optimizer(cases)
        half = [torch.zeros(c.n, device="cuda", dtype=BF16) for c in cases]
        return cases, opt, pk.GradClip([c.g for c in cases], outs=half), half, pk.Quantizer([c.p for c in cases], granularity="tensor")

    def calls(x, amp):
        x[2].clip(1.0)
        x[1].step_amp(amp, max_norm=1.0, **HP)
        x[4].quantize()

    def everything(x, amp):
        out = [amp, x[2].result] + x[3] + x[4].codes + x[4].scales
        for c in x[0]:
            out += [t for t in (c.p, c.copy, c.m, c.v, c.ms, c.vs) if t is not None]
        return [t.clone() for t in out]

    a, b = make(12), make(12)
    amp_a, amp_b = pk.amp_state(256.0), pk.amp_state(256.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(a, amp_a)
    side.synchronize()
    calls(b, amp_b)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(everything(a, amp_a), everything(b, amp_b)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(a, amp_a)
    for k in range(3):
        for x, y in zip(a[0], b[0]):
            new = torch.randn(x.n, generator=gen(100 * k + x.n), device="cuda") * 10
            if k == 1 and x.n == 129:
                new[7] = math.inf  # this step is skipped
            x.g.copy_(new)
            y.g.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        calls(b, amp_b)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in
                   zip(everything(a, amp_a), everything(b, amp_b))), k  # byte for byte: there may be a NaN
        assert pk.read_amp_state(amp_a)["found_inf"] == (k == 1)
    torch.cuda.synchronize()
    for x in (a, b):
        for o in (x[1], x[2], x[4]):
            o.close()


def ragged(total, count, g):
    """Sizes of `count` tensors, many of them empty or tiny, that fill `total` elements."""
    cuts = torch.randint(0, total + 1, (count - 1,), generator=g, device="cuda").sort().values.tolist()
    cuts = [0] + cuts + [total]
    cuts[3:6] = [cuts[3]] * 3  # some empty ones
    return list(zip(cuts[:-1], cuts[1:]))


@pytest.mark.parametrize("pd, gd", [(F32, F32), (BF16, BF16), (F16, BF16)])
def test_a_list_of_thousands_equals_one_tensor(pd, gd):
    """What is elementwise does not see where one tensor ends: a packed list of 3000 ragged views
    (any alignment) gives the bits of the one tensor they lie in."""
    g = gen(14)
    n = 300007
    p, gr = filled(n, pd, g, 0.02), filled(n, gd, g, 1e-3)
    m, v = torch.randn(n, generator=g, device="cuda") * 1e-4, torch.rand(n, generator=g, device="cuda") * 1e-6
    spans = ragged(n, 3000, g)
    one, many = [[x.clone() for x in (p, m, v)] for _ in range(2)]
    a = pk.AdamW([one[0]], [gr], state=([one[1]], [one[2]]))
    b = pk.AdamW([many[0][i:j] for i, j in spans], [gr[i:j] for i, j in spans],
                 state=([many[1][i:j] for i, j in spans], [many[2][i:j] for i, j in spans]))
    for t in (1, 2):
        a.step(step=t, **HP)
        b.step(step=t, **HP)
    assert all(torch.equal(x, y) for x, y in zip(one, many))
    out1, out2 = torch.zeros(n, device="cuda", dtype=BF16), torch.zeros(n, device="cuda", dtype=BF16)
    c1 = pk.GradClip([gr], outs=[out1])
    c2 = pk.GradClip([gr[i:j] for i, j in spans], outs=[out2[i:j] for i, j in spans])
    r1, r2 = c1.clip(0.1).clone(), c2.clip(0.1).clone()
    # the partial sums differ, in fp64: the norm by at most its rounding to fp32
    assert abs(float(r1[0]) - float(r2[0])) <= 2 * U * float(r1[0])
    if torch.equal(r1, r2):
        assert torch.equal(out1, out2)
    for o in (a, b, c1, c2):
        o.close()


def test_amp_state_goes_as_in_the_fp8_step():
    """The scaler's state after each call is FP8AdamW.step_amp's on the same gradients: taken and
    skipped calls, growth and backoff, clipped and not (the norm within its rounding: its partial
    sums differ)."""
    g = gen(18)
    grads = [filled(n, BF16, g, 20.0) for n in (5000, 300)]
    ps = [[torch.zeros(n, device="cuda") for n in (5000, 300)] for _ in range(2)]
    a, b = pk.AdamW(ps[0], grads), pk.FP8AdamW(ps[1], grads)
    sa, sb = pk.amp_state(64.0), pk.amp_state(64.0)
    for call in range(1, 9):
        for x in grads:
            x.copy_(torch.randn(x.numel(), generator=g, device="cuda") * (0.01 if call % 3 == 0 else 20.0))
        if call in (3, 6):
            grads[1][7] = math.inf
        kw = dict(max_norm=1.0, growth_interval=2, growth_factor=4.0, backoff_factor=0.25)
        a.step_amp(sa, **HP, **kw)
        b.step_amp(sb, step=call, **HP, **kw)
        x, y = amp_fields(sa), amp_fields(sb)
        for k in ("scale", "growth_tracker", "step", "found_inf"):
            assert x[k] == y[k], (call, k)
        for k in ("grad_norm", "clip_coef", "grad_factor"):
            assert x[k] == y[k] or abs(x[k] - y[k]) <= 2 * U * abs(y[k]) or (math.isnan(x[k]) and math.isnan(y[k])), (call, k)
    a.close()
    b.close()


@pytest.mark.parametrize("chunks", [1, 2, 9, 63, 64, 65, 600])
def test_amp_norm_of_every_call(chunks):
    """Lists on both sides of the one-launch rule (64 chunks of 4096): the norm of every call is that
    call's, whichever work-group ends last; the same gradients give the same bits."""
    g = gen(chunks)
    n = 4096 * chunks - 5
    gr = torch.zeros(n, device="cuda", dtype=BF16)
    opt = pk.AdamW([torch.zeros(n, device="cuda")], [gr])
    amp = pk.amp_state(1.0)
    base = torch.randn(n, generator=g, device="cuda").bfloat16()
    norm = math.sqrt(float(base.double().square().sum()))
    seen = {}
    for call in range(60):
        k = call % 5
        torch.mul(base, 2.0 ** k, out=gr)  # exact: a power of two
        opt.step_amp(amp, max_norm=1.0, growth_interval=10 ** 6, **HP)
        got = amp_fields(amp)["grad_norm"]
        assert abs(got - norm * 2.0 ** k) <= 2 * U * norm * 2.0 ** k, (call, got)
        assert seen.setdefault(k, got) == got
    assert amp_fields(amp)["step"] == 60
    opt.close()


def test_amp_over_every_kind_in_one_list():
    """One norm over gradients of three types, then every kind of tensor with the same factor."""
    g = gen(15)
    S = 512.0
    cases = [Case(n, g, pd, gd, cd, bits, offset=k % 2, gscale=1e-2 * S)
             for k, (pd, cd) in enumerate(WEIGHTS) for gd in (F32, BF16, F16) for bits in (32, 8) for n in (900, 5)]
    opt = optimizer(cases)
    amp = pk.amp_state(S)
    for t in (1, 2):
        norm = math.sqrt(sum(float(c.g.double().square().sum()) for c in cases)) / S
        factor = f32(f32(min(1.0, 0.3 / (norm + 1e-6))) * f32(1 / S))
        for c in cases:
            c.expect(t, **HP, factor=factor)
        opt.step_amp(amp, max_norm=0.3, **HP)
        assert amp_fields(amp)["grad_factor"] == factor
        for c in cases:
            c.check()
    opt.close()


def moved(t, offset):
    """t's values at that offset (in elements) into new memory."""
    out = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:]
    out.copy_(t)
    return out


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd, cd, gd", [(F32, BF16, F16), (BF16, None, F16), (F16, None, F32)])
@pytest.mark.parametrize("offs", [(1, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 1, 0, 0), (1, 1, 1, 2, 3), (1, 1, 1, 4, 4), (2, 2, 2, 3, 1)])
def test_alignment_does_not_change_the_bits(bits, pd, cd, gd, offs):
    """Weights, gradients, copies and moments each at their own offset: the aligned run's bits."""
    for n in (1, 2, 130, 2049, 9000):
        g = gen(n)
        a = Case(n, g, pd, gd, cd, bits)
        p, gr, m, v = (moved(x, o) for x, o in zip((a.p, a.g, a.m, a.v), (offs[0], offs[1], offs[3], offs[4])))
        copy = moved(a.copy, offs[2]) if cd else None
        state = ([m], [v]) if bits == 32 else ([m], [v], [moved(a.ms, 1)], [moved(a.vs, 1)])
        x = optimizer([a])
        y = pk.AdamW([p], [gr], copies=[copy], state_bits=bits, state=state)
        for t in (1, 2):
            x.step(step=t, **HP)
            y.step(step=t, **HP)
        assert torch.equal(a.p, p) and torch.equal(a.m, m) and torch.equal(a.v, v) and (not cd or torch.equal(a.copy, copy))
        x.close()
        y.close()
        for granularity in ("block128", "tensor"):
            q = [pk.Quantizer([z], granularity=granularity, codes=[moved(torch.zeros(n, dtype=torch.uint8, device="cuda"), o)])
                 for z, o in ((a.g, 0), (gr, offs[3]))]
            for k in q:
                k.quantize()
            assert torch.equal(q[0].codes[0], q[1].codes[0]) and torch.equal(q[0].scales[0], q[1].scales[0])
            for k in q:
                k.dequantize()
            assert torch.equal(a.g, gr)
            for k in q:
                k.close()


def test_two_plans_at_once():
    """Calls of different plans on two streams do not touch each other's workspace."""
    def make(seed):
        g = gen(seed)
        cases = [Case(200003, g, bits=b, gscale=3.0) for b in (32, 8)]
        half = [torch.zeros(c.n, device="cuda", dtype=BF16) for c in cases]
        return cases, optimizer(cases), pk.GradClip([c.g for c in cases], outs=half), half, \
            pk.Quantizer([c.p for c in cases], granularity="tensor"), pk.amp_state(8.0)

    def run(x):
        for _ in range(5):
            x[2].clip(1.0)
            x[1].step_amp(x[5], max_norm=1.0, **HP)
            x[4].quantize()

    def values(x):
        return [t.clone() for t in x[3] + x[4].codes + x[4].scales + [x[2].result, x[5]] + [y for c in x[0] for y in (c.p, c.m, c.v)]]

    a, b = make(16), make(17)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for x, st in zip((a, b), streams):
        with torch.cuda.stream(st):
            run(x)
    torch.cuda.synchronize()
    for x, seed in ((a, 16), (b, 17)):
        y = make(seed)
        run(y)
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(values(x), values(y)))
        for z in (x, y):
            for o in (z[1], z[2], z[4]):
                o.close()


def test_offsets_past_32_bits():
    """One tensor of more than 2^32 elements: its far end is read and written like its start."""
    n = (1 << 32) + 4099
    ends = [slice(0, 2000), slice((1 << 32) - 1000, (1 << 32) + 1000), slice(n - 1500, n)]
    g = gen(13)
    p = torch.zeros(n, device="cuda", dtype=BF16)
    gr = torch.zeros(n, device="cuda", dtype=BF16)
    small = []
    for e in ends:
        k = e.stop - e.start
        p[e], gr[e] = torch.randn(k, generator=g, device="cuda"), torch.randn(k, generator=g, device="cuda")
        small.append((p[e].clone(), gr[e].clone()))
    for bits in (8, 32):
        pp = p.clone()
        opt = pk.AdamW([pp], [gr], state_bits=bits)
        opt.step(step=1, **HP)
        for e, (q, h) in zip(ends, small):
            o = pk.AdamW([q.clone()], [h], state_bits=32)  # a first step's weights do not go by the blocks
            o.step(step=1, **HP)
            assert torch.equal(pp[e], o.params[0])
            if bits == 32:
                assert torch.equal(opt.m[0][e], o.m[0]) and torch.equal(opt.v[0][e], o.v[0])
            o.close()
        if bits == 8:
            want = opt.m[0][n - 131:].clone()  # the last blocks: n is 3 past a multiple of 128
            codes, s = quantized((f32(0.1) * gr[n - 131:].double().cpu()).float(), "e4m3")
            assert torch.equal(want.cpu(), codes) and torch.equal(opt.m_scale[0][-2:].cpu(), s)
        opt.close()
        del opt, pp
    clip = pk.GradClip([gr], outs=[p])
    norm = math.sqrt(sum(float(h.double().square().sum()) for _, h in small))
    res = clip.clip(1.0).cpu()
    assert abs(float(res[0]) - norm) <= 2 * U * norm
    for e, (_, h) in zip(ends, small):
        assert torch.equal(p[e], (h.float() * res[1].item()).bfloat16())
    clip.close()
    del p
    for granularity in ("block128", "tensor"):
        q = pk.Quantizer([gr], granularity=granularity)
        q.quantize()
        back = pk.Quantizer([torch.empty_like(gr)], granularity=granularity, codes=q.codes, scales=q.scales)
        back.dequantize()
        for e, (_, h) in zip(ends, small):
            got = back.values[0][e].float()
            scale = float(q.scales[0].max())
            assert bool(((got - h.float()).abs() <= 2.0 ** -4 * h.float().abs() + scale * 2.0 ** -10).all())
        q.close()
        back.close()
        del q, back
