"""Seeded weights of the MoE sublayer, drawn without a GPU."""

import math

import torch

from mhc_residual_stream_b200.moe import MoeConfig, MoeWeights


def test_experts_drawn_one_at_a_time_are_those_drawn_at_once():
    # the host holds one expert's weights in fp32 at a time, and draws the same values
    cfg, H = MoeConfig(experts=5, intermediate=24, shared=40), 72
    got = MoeWeights.draw(cfg, H, 3, "cpu")
    g = torch.Generator()
    g.manual_seed(3)

    def w(*shape):
        return (torch.randn(*shape, generator=g) / math.sqrt(shape[-1])).to(torch.bfloat16)
    assert torch.equal(got.router, w(5, H))
    assert torch.equal(got.bias, torch.randn(5, generator=g) * 0.05)
    assert torch.equal(got.w13, w(5, 48, H)) and torch.equal(got.w2, w(5, H, 24))
    assert torch.equal(got.shared13, w(80, H)) and torch.equal(got.shared2, w(H, 40))


def test_the_largest_draw_is_one_experts(monkeypatch):
    sizes, randn = [], torch.randn

    def counted(*shape, **kw):
        sizes.append(math.prod(shape))
        return randn(*shape, **kw)
    monkeypatch.setattr(torch, "randn", counted)
    MoeWeights.draw(MoeConfig(experts=6, intermediate=16, shared=16), 32, 1, "cpu")
    assert max(sizes) == 2 * 16 * 32
