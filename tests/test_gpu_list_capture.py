"""The list operators and graph captures: what a capture holds of a call, and plans that are built,
closed or dropped while a graph is captured."""
import pytest
import torch

import precision_adam_optimizer_amd as pk
from precision_adam_optimizer_amd import lists

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
