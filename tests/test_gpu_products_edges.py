"""GPU tests of mhc_linear and mhc_moe_experts beside their sizes and types: one
workspace for several operators, tiles that several CTAs share."""

import pytest
import torch

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


def shares_of(tiles, kblocks, grid=148, most=4, least=24):
    """CTAs that compute each tile behind the full waves, as the schedule divides them."""
    rest = tiles % grid
    total = rest * kblocks
    parts = min(grid, rest * most, max(rest, total // least))

    def owner(w):
        return ((w + 1) * parts - 1) // total
    return {owner((t + 1) * kblocks - 1) - owner(t * kblocks) + 1 for t in range(rest)}


# one expert: hidden, intermediate, then the shares of a tile in the first and the second product
SHARED = [(7168, 2048, {4}, {2, 3}), (4096, 2048, {3, 4}, {2, 3}), (6016, 4864, {4, 5}, {4, 5}),
          (4864, 6016, {4, 5}, {4, 5}), (1152, 2560, {1}, {2, 3})]


@pytest.mark.parametrize("H,I,first,second", SHARED)
@pytest.mark.parametrize("R", [1, 13])
def test_experts_tiles_of_several_shares(H, I, first, second, R):
    got = shares_of(-(-I // 128), -(-H // 64)), shares_of(-(-H // 128), -(-I // 64))
    assert got == (first, second)
    x, w13, w2, e2p, prow, off = draw_experts(R, 1, 1, H, I, seed=H + R)
    exact, bound = experts_bound(f64(x), f64(w13), f64(w2), prow, off)
    ws = M.new_moe_experts_workspace(R, R, I, DEV)
    ops = x.to(DEV), w13.to(DEV), w2.to(DEV), i32(prow), i32(off)
    out = run_experts(*ops, ws)
    assert_within(out, exact, bound, f"{R} rows, {H} x {I}")
    for _ in range(5):
        assert torch.equal(run_experts(*ops, ws), out)
    assert M.mhc_get_device_status(ws) == M.OK


@pytest.mark.parametrize("fp8,act,R,K,N", [
    (False, "none", 1, 768, 1), (False, "none", 3, 7168, 256), (False, "none", 20, 7168, 256),
    (False, "swiglu", 2, 7168, 2048), (False, "swiglu", 32, 7168, 2048), (True, "none", 4, 7168, 7168),
    (True, "none", 64, 7168, 7168), (False, "none", 130, 128, 300), (True, "none", 700, 256, 300),
])
@pytest.mark.parametrize("budget", [1_000, 1_500_000])
def test_waits_that_run_out_leave_nothing_in_flight(fp8, act, R, K, N, budget):
    # clusters in which one CTA finishes every column (up to 4 rows) or all of them do, pairs of
    # few K blocks: the copies are expected to bring more than they do, so every wait runs out;
    # what follows directly, in the same shared memory, is right
    g = gen(R + K)
    W = 2 * N if act == "swiglu" else N
    x, w = bf((R, K), g).to(DEV), bf((W, K), g, 0.05).to(DEV)
    if fp8:
        ops = []
        for t in (x, w):
            q = torch.empty(t.shape, dtype=torch.uint8, device=DEV)
            s = torch.empty(M.mhc_mxfp8_scale_bytes(*t.shape, True), dtype=torch.uint8, device=DEV)
            M.mxfp8_quantize_rows(t, q, s, True)
            ops.append((q, s, True))
        x, w = ops
    want = run_linear(x, w, act=act)
    bad, good = M.new_linear_workspace(R, DEV), M.new_linear_workspace(R, DEV)
    out = [torch.zeros_like(want) for _ in range(6)]
    torch.cuda.synchronize()
    for k in range(0, 6, 2):
        old = M.mhc_debug_set_wait(budget, 4)
        try:
            M.mhc_linear(x, w, out[k], activation=act, workspace=bad)
        finally:
            M.mhc_debug_set_wait(old, 0)
        M.mhc_linear(x, w, out[k + 1], activation=act, workspace=good)
    assert M.mhc_get_device_status(bad) == M.DEVICE_TIMEOUT
    assert M.mhc_get_device_status(good) == M.OK
    for k in (1, 3, 5):
        assert torch.equal(out[k], want)


@pytest.mark.parametrize("R,N,K", [(24, 256, 512), (130, 300, 160), (1, 7168, 1024)])
def test_a_weight_that_is_quantized_directly_before(R, N, K):
    # the quantizer lets no kernel start early, so even a product that reads its weights ahead
    # finds them (and the padding of their scales) written
    g = gen(N)
    ws_ = [bf((N, K), g, 0.1).to(DEV) for _ in range(8)]
    x = bf((R, K), g).to(DEV)

    def buffers(t):
        return (torch.zeros(t.shape, dtype=torch.uint8, device=DEV),
                torch.zeros(M.mhc_mxfp8_scale_bytes(*t.shape, True), dtype=torch.uint8, device=DEV))
    xq, want, outs = buffers(x), [], [torch.zeros(R, N, dtype=torch.bfloat16, device=DEV) for _ in ws_]
    M.mxfp8_quantize_rows(x, *xq, True)
    ws = M.new_linear_workspace(R, DEV)
    for w in ws_:
        wq = buffers(w)
        M.mxfp8_quantize_rows(w, *wq, True)
        torch.cuda.synchronize()
        want.append(run_linear((*xq, True), (*wq, True)))
    wq = buffers(ws_[0])
    torch.cuda.synchronize()
    for w, out in zip(ws_, outs):  # one buffer, rewritten before every product
        M.mxfp8_quantize_rows(w, *wq, True)
        M.mhc_linear((*xq, True), (*wq, True), out, workspace=ws)
    torch.cuda.synchronize()
    for out, t in zip(outs, want):
        assert torch.equal(out, t)


@pytest.mark.parametrize("R", [3, 130, 300])
def test_mxfp8_rows_may_be_strided(R):
    g = gen(R)
    K, N = 160, 200
    ops = []
    for t in (bf((R, K), g), bf((N, K), g, 0.1)):
        q = torch.empty(t.shape, dtype=torch.uint8, device=DEV)
        s = torch.empty(M.mhc_mxfp8_scale_bytes(*t.shape, True), dtype=torch.uint8, device=DEV)
        M.mxfp8_quantize_rows(t.to(DEV), q, s, True)
        ops.append((q, s, True))
    want = run_linear(*ops)
    wide = torch.full((R, 256), 0x7f, dtype=torch.uint8, device=DEV)  # NaN around the rows
    wide[:, 16:16 + K] = ops[0][0]
    got = run_linear((wide[:, 16:16 + K], ops[0][1], True), ops[1])
    assert torch.equal(got, want)
