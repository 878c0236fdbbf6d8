"""GPU tests of mhc_linear and mhc_moe_experts beside their sizes and types: one
workspace for several operators, tiles that several CTAs share."""

import numpy as np
import pytest
import torch

import oracle as O
from mhc_residual_stream_b200 import mhc as M

from _sublayer import (DEV, assert_within, bf, draw_experts, experts_bound, f64, gen, i32, run_linear, run_route)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mhc_residual_stream_b200 import build
    build.build()
    M.lib()
    yield


def run_experts(x, w13, w2, prow, off, ws):
    out = torch.full((len(prow), x.shape[1]), 5.0, dtype=torch.bfloat16, device=DEV)
    M.mhc_moe_experts(x, w13, w2, prow, off, out, workspace=ws)
    return out


def test_one_workspace_serves_every_operator_in_turn():
    from mhc_residual_stream_b200 import synthetic as S
    R, k, E, H, I = 2, 2, 3, 2048, 640  # few tiles of many K blocks: the experts' tiles are shared
    x, w13, w2, e2p, prow, off = draw_experts(R, k, E, H, I, seed=41)
    exact, bound = experts_bound(f64(x), f64(w13), f64(w2), prow, off)
    ops = x.to(DEV), w13.to(DEV), w2.to(DEV), i32(prow), i32(off)
    d = S.draw_boundary(100, 512, n=4, partials=1, seed=4)
    t = {q: d[q].to(DEV) for q in ("partials", "residual", "post", "comb", "pre", "norm_weight")}
    coeff = M.Coeffs.from_weights(d["coeff"], DEV)
    mix = [torch.empty(100, *s, device=DEV) for s in ((4,), (4, 4), (4,))]
    li = torch.empty(100, 512, dtype=torch.bfloat16, device=DEV)
    res = torch.empty_like(t["residual"])
    ws = torch.zeros(max(M.mhc_moe_experts_workspace_bytes(R, R * k, I), M.mhc_workspace_bytes(100, 512, 4),
                         M.mhc_moe_route_workspace_bytes(900, 128, 8)), dtype=torch.uint8, device=DEV)
    logits = torch.randn(900, 128, generator=gen(42)).to(DEV)
    a, b = bf((24, 1024), gen(43)).to(DEV), bf((96, 1024), gen(44), 0.05).to(DEV)
    want = run_experts(*ops, M.new_moe_experts_workspace(R, R * k, I, DEV))
    assert_within(want, exact, bound, "experts")
    route, lin = run_route(logits, 8), run_linear(a, b)
    for _ in range(4):
        assert all(torch.equal(p, q) for p, q in zip(route, run_route(logits, 8, workspace=ws)))
        assert torch.equal(run_experts(*ops, ws), want)
        assert torch.equal(run_linear(a, b, workspace=ws), lin)
        M.mhc_boundary_post_pre(t["partials"], t["residual"], t["post"], t["comb"], t["pre"], t["norm_weight"], 1e-6,
                                coeff, res, layer_input=li, post_out=mix[0], comb_out=mix[1], pre_out=mix[2],
                                workspace=ws)
        assert torch.equal(run_experts(*ops, ws), want)
        assert M.mhc_get_device_status(ws) == M.OK
