"""Tensors of more dimensions through the layer operators: packed before the call, by it, or as another layer's output."""
import pytest
import torch

import layer_util as u
import precision_adam_optimizer_amd as pk

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("lead", [(3, 50), (2, 3, 7), (1, 1), (2, 0, 4), (200,)])
def test_a_block_of_a_batch(lead):
    """A gated block whose output joins the residual of the same shape; the same bits as of the folded batch."""
    wg, wu, wd = (pk.pack8(u.randn(s, i) / 14) for i, s in enumerate([(384, 200), (384, 200), (200, 384)]))
    x = u.randn((*lead, 200), 5, dtype=BF16)
    flat = x.reshape(-1, 200) if x.numel() else x.new_empty(0, 200)

    def block(x):
        h = pk.gated8(x, wg, wu, dtype=None, keep="e4m3", pack="e4m3")
        dx = pk.input_grad8(pk.gated8_backward(pk.input_grad8(x, wd), h.gate, h.up), (wg, wu))
        return pk.linear8(h.y8, wd, residual=x).y, dx
    for got, want in zip(block(x), block(flat)):
        assert got.shape == x.shape and torch.equal(got.reshape(want.shape), want)
    assert torch.equal(pk.linear8(pk.pack8(x), wg).y, pk.linear8(x, wg).y)
