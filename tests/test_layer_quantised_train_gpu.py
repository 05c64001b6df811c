"""A stack that serves through 8-bit projections trains as one that does not: its output is that of the parameters
that the gradients belong to, also after a step has changed these."""
import pytest
import torch

from examples.ssm_block import Stack
from test_layer_gpu import built  # noqa: F401

pytestmark = pytest.mark.gpu


def test_training_does_not_go_through_8_bits():
    size = dict(depth=2, D=128, N=2, G=1, K=32, V=64, seed=7)
    plain, served = Stack(**size), Stack(**size).quantise()
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(2, 50, 128, generator=gen).cuda()
    dout = torch.randn(2, 50, 128, generator=gen).to(torch.bfloat16).cuda()
    for _ in range(2):
        (a, g, _), (b, e, _) = plain.train(x, dout), served.train(x, dout)
        assert torch.equal(a, b) and g.keys() == e.keys() and all(torch.equal(g[n], e[n]) for n in g)
        assert torch.equal(a, plain.prompt(x, plain.cache(2)))
        for stack in (plain, served):  # the same step for both
            for block in stack.blocks:
                block.p["w_in"] *= 1.5
    assert not torch.equal(served.prompt(x, served.cache(2)), plain.prompt(x, plain.cache(2)))
