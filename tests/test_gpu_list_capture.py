"""The list operators and graph captures: what a capture holds of a call, and plans that are built,
closed or dropped while a graph is captured."""
import pytest
import torch

import precision_adam_optimizer_amd as pk
from precision_adam_optimizer_amd import lists
from tests.test_gpu_list import HP, Case, gen, optimizer

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_plans_and_a_capture():
    """Building and closing are refused during a capture, a plan that is dropped is kept until later;
    the capture goes on, and its replays are right."""
    x = torch.full((5000,), 2.0, device="cuda")
    out = torch.zeros(5000, device="cuda", dtype=BF16)
    clip = pk.GradClip([x], outs=[out])
    other = pk.Quantizer([torch.ones(300, device="cuda")])
    dropped = pk.GradClip([torch.ones(300, device="cuda")])
    bits = pk.AdamW([torch.ones(300, device="cuda")], [torch.ones(300, device="cuda")])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for build in (lambda: pk.GradClip([x]), lambda: pk.Quantizer([x]), lambda: pk.AdamW([x], [x.view(-1)]),
                      lambda: bits.converted_state(8)):
            with pytest.raises(RuntimeError, match="while a graph is captured"):
                build()
        with pytest.raises(RuntimeError, match="while a graph is captured"):
            other.close()
        clip.clip(1.0)
        del dropped
        assert len(lists._kept) == 1
    for k in range(3):
        x.fill_(2.0 + k)
        graph.replay()
        torch.cuda.synchronize()
        norm = (2.0 + k) * 5000 ** 0.5
        c = float(clip.result[1])
        assert abs(float(clip.result[0]) - norm) <= 2.0 ** -23 * norm and abs(c - 1 / (norm + 1e-6)) <= 2.0 ** -23 * c
        assert torch.equal(out, (x * c).bfloat16())
    other.quantize()
    other.close()
    again = pk.GradClip([x])  # the plan that was dropped is freed with this one's building
    assert not lists._kept
    again.close()
    clip.close()
    bits.close()


def make(seed):
    g = gen(seed)
    cases = [Case(n, g, bits=bits, gscale=0.1) for n in (1500, 129) for bits in (32, 8)]
    return cases, optimizer(cases)


def state(cases):
    return [t.clone() for c in cases for t in (c.p, c.m, c.v, c.ms, c.vs) if t is not None]


def new_gradients(cases, others, k):
    for i, (x, y) in enumerate(zip(cases, others)):
        x.g.copy_(torch.randn(x.n, generator=gen(100 * k + i), device="cuda"))
        y.g.copy_(x.g)


def test_a_replayed_step_takes_its_arguments_from_the_capture():
    """Every replay is the step with the capture's t and rates on the gradients of now."""
    (a, oa), (b, ob) = make(30), make(30)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oa.step(step=2, **HP)
    oa._set(0.0, 0.0, 0.0, 1.0, 0.0)  # what the host holds now is nothing to the graph
    for k in range(3):
        new_gradients(a, b, k)
        graph.replay()
        torch.cuda.synchronize()
        ob.step(step=2, **HP)
        assert all(torch.equal(x, y) for x, y in zip(state(a), state(b))), k
    new_gradients(a, b, 3)
    graph.replay()
    ob.step(step=3, **HP)
    assert not all(torch.equal(x, y) for x, y in zip(state(a), state(b)))  # not the next step
    oa.close()
    ob.close()


def test_training_by_replays_of_the_scaled_step():
    """A scale of 1 that never grows: replays are the plain steps 1, 2, 3, ... (their factor is 1, and t
    is the device's), the eager calls among them too."""
    (a, oa), (b, ob) = make(31), make(31)
    amp = pk.amp_state(1.0)
    kw = dict(growth_interval=2 ** 31 - 1, **HP)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oa.step_amp(amp, **kw)
    for t in range(1, 7):
        new_gradients(a, b, t)
        if t == 4:
            oa.step_amp(amp, **kw)
        else:
            graph.replay()
        torch.cuda.synchronize()
        st = pk.read_amp_state(amp)
        assert (st["step"], st["scale"], st["grad_factor"]) == (t, 1.0, 1.0)
        ob.step(step=t, **HP)
        for x, y in zip(a, b):
            # moments do not see t; the weights' bias corrections come from the device's pow and the host's,
            # each within an ulp of double before it is rounded to fp32: one step of fp32 apart at most, which
            # moves the update by 2u + u and its roundings by as much as they move the plain step's (12u of
            # test_gpu_list.py, on both sides)
            assert torch.equal(x.m, y.m) and torch.equal(x.v, y.v)
            assert bool(((x.p - y.p).abs() <= 2.0 ** -24 * (27 * 10 * HP["lr"] + 2 * y.p.abs())).all())
            x.p.copy_(y.p)
    oa.close()
    ob.close()
