"""GPU tests of the sublayer operators (mhc_linear, mhc_moe_route,
mhc_moe_experts) against the float64 oracle, at the bounds derived in
tests/_sublayer.py."""

import math

import numpy as np
import pytest
import torch

import oracle as O
from mhc_residual_stream_b200 import mhc as M

from _sublayer import (DEV, assert_within, bf, draw_experts, experts_bound, f64, gen, i32, linear_bound, mxfp8,
                       run_linear, run_route)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mhc_residual_stream_b200 import build
    build.build()
    M.lib()
    yield


# ---------------------------------------------------------------- linear

LINEAR = [  # rows, K, N, activation, bias, residual, out
    (1, 8, 1, "none", False, False, torch.bfloat16),
    (1, 7168, 256, "none", False, False, torch.float32),
    (1, 64, 128, "silu", True, True, torch.bfloat16),
    (2, 72, 129, "relu", True, False, torch.float32),
    (3, 1000, 333, "gelu", True, True, torch.bfloat16),
    (16, 512, 1000, "none", True, True, torch.float32),
    (17, 136, 77, "swiglu", True, True, torch.bfloat16),
    (32, 7168, 256, "none", False, False, torch.float32),
    (33, 2048, 640, "swiglu", False, False, torch.float32),
    (77, 1000, 333, "gelu", True, True, torch.float32),
    (128, 256, 200, "swiglu", True, False, torch.bfloat16),
    (129, 264, 130, "swiglu", True, True, torch.bfloat16),
    (200, 520, 300, "silu", False, True, torch.bfloat16),
    (257, 128, 257, "none", True, True, torch.bfloat16),
    (300, 24, 2000, "relu", False, False, torch.bfloat16),
    (1030, 192, 1100, "none", False, True, torch.float32),
    (4099, 64, 64, "gelu", True, False, torch.bfloat16),
    (193, 72, 513, "swiglu", True, True, torch.bfloat16),
    (1000, 136, 300, "swiglu", False, False, torch.float32),
    (2500, 320, 777, "silu", True, False, torch.float32),
    (600, 200, 4501, "swiglu", True, True, torch.bfloat16),
    (200, 72, 9500, "none", True, True, torch.bfloat16),
    (700, 136, 5001, "gelu", False, True, torch.bfloat16),
    (65535, 16, 3, "none", True, False, torch.bfloat16),
]


@pytest.mark.parametrize("R,K,N,act,bias,res,out", LINEAR)
def test_linear_bf16(R, K, N, act, bias, res, out):
    g = gen(R * 7 + K)
    W = 2 * N if act == "swiglu" else N
    x, w = bf((R, K), g), bf((W, K), g, 1.5 / K ** 0.5)
    b = torch.randn(W, generator=g) * 0.3 if bias else None
    r = bf((R, N), g) if res else None
    got = run_linear(x.to(DEV), w.to(DEV), None if b is None else b.to(DEV), act, None if r is None else r.to(DEV), out)
    exact, bound = linear_bound(f64(x), f64(w), None if b is None else f64(b), act, None if r is None else f64(r), out)
    assert_within(got, exact, bound, f"linear {R}x{K}x{N} {act}")


@pytest.mark.parametrize("R,K,N,act,bias,res,out", [
    (1, 32, 1, "none", False, False, torch.float32),
    (1, 7168, 512, "none", False, False, torch.bfloat16),
    (5, 96, 200, "silu", True, True, torch.float32),
    (64, 1024, 384, "swiglu", True, False, torch.bfloat16),
    (100, 416, 333, "gelu", True, True, torch.bfloat16),
    (128, 2048, 128, "none", False, True, torch.float32),
    (129, 160, 256, "swiglu", False, True, torch.float32),
    (300, 512, 700, "relu", True, False, torch.bfloat16),
    (257, 160, 1000, "silu", True, True, torch.float32),
    (700, 1056, 2100, "none", False, True, torch.bfloat16),
    (3000, 128, 300, "gelu", True, False, torch.float32),
])
def test_linear_mxfp8(R, K, N, act, bias, res, out):
    g = gen(R * 11 + K)
    W = 2 * N if act == "swiglu" else N
    xv = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-4, 5, (R, 1), generator=g).float())
    xd, xs, x = mxfp8(xv)
    wd, wsc, w = mxfp8(torch.randn(W, K, generator=g) * (1.5 / K ** 0.5))
    b = torch.randn(W, generator=g) * 0.3 if bias else None
    r = bf((R, N), g) if res else None
    got = run_linear((xd.to(DEV), xs.to(DEV), True), (wd.to(DEV), wsc.to(DEV), True), None if b is None else b.to(DEV),
                     act, None if r is None else r.to(DEV), out)
    exact, bound = linear_bound(x, w, None if b is None else f64(b), act, None if r is None else f64(r), out)
    assert_within(got, exact, bound, f"mxfp8 linear {R}x{K}x{N} {act}")


# One product for every form the library chooses between: whole tiles, pairs, and
# clusters of 2-8 CTAs at one and two CTAs an SM.
FORMS = {
    (False, False): [(77, 64, 1), (130, 1024, 1000), (100, 768, 1500), (1, 768, 1), (17, 768, 4000), (17, 1024, 2500),
                     (1, 1536, 1), (130, 1536, 300), (1, 1536, 4000), (1, 2048, 1), (256, 2048, 1), (31, 520, 100)],
    (False, True): [(77, 64, 1), (130, 1024, 1000), (40, 1536, 4000), (17, 768, 4000), (1, 768, 1), (17, 768, 2500),
                    (17, 2048, 2500), (1, 1024, 1), (1, 1536, 4000), (1, 1536, 1), (256, 1536, 1)],
    (True, False): [(130, 64, 1), (1, 1536, 1), (1, 2048, 1), (100, 4096, 2000), (1, 4096, 1), (1, 4096, 2000),
                    (300, 4096, 2000)],
    (True, True): [(1, 1536, 128), (1, 2048, 128), (1, 4096, 128), (1, 2048, 4096), (40, 544, 256), (400, 64, 128)],
}


@pytest.mark.parametrize("fp8,gated,R,K,N", [(*k, *s) for k, v in FORMS.items() for s in v])
def test_linear_every_form(fp8, gated, R, K, N):
    g = gen(R + 3 * K + 7 * N)
    act, W = ("swiglu", 2 * N) if gated else ("silu", N)
    b, r = torch.randn(W, generator=g) * 0.3, bf((R, N), g)
    if fp8:
        xd, xs, x = mxfp8(torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-4, 5, (R, 1), generator=g).float()))
        wd, wsc, w = mxfp8(torch.randn(W, K, generator=g) * (1.5 / K ** 0.5))
        ops = [(d.to(DEV), sc.to(DEV), True) for d, sc in ((xd, xs), (wd, wsc))]
    else:
        x, w = bf((R, K), g), bf((W, K), g, 1.5 / K ** 0.5)
        ops, x, w = [x.to(DEV), w.to(DEV)], f64(x), f64(w)
    got = run_linear(*ops, b.to(DEV), act, r.to(DEV), torch.float32)
    exact, bound = linear_bound(x, w, f64(b), act, f64(r), torch.float32)
    assert_within(got, exact, bound, f"{R}x{K}x{N}")


def test_linear_takes_what_the_quantizer_writes():
    g = gen(3)
    x, w = bf((70, 384), g), bf((256, 384), g, 0.1)
    ops = []
    for t in (x, w):
        d = torch.empty(t.shape, dtype=torch.uint8, device=DEV)
        s = torch.empty(M.mhc_mxfp8_scale_bytes(*t.shape, True), dtype=torch.uint8, device=DEV)
        M.mxfp8_quantize_rows(t.to(DEV), d, s, True)
        ops.append((d, s, True))
    got = run_linear(*ops)
    exact, bound = linear_bound(mxfp8(x.float())[2], mxfp8(w.float())[2], None, "none", None, torch.bfloat16)
    assert_within(got, exact, bound, "quantized operands")


def test_linear_of_a_weight_that_the_call_before_computes():
    g = gen(30)
    a, b, x = bf((256, 4096), g, 0.02).to(DEV), bf((512, 4096), g, 0.02).to(DEV), bf((24, 512), g).to(DEV)
    ws, w = M.new_linear_workspace(256, DEV), torch.empty(256, 512, dtype=torch.bfloat16, device=DEV)
    outs = []
    for _ in range(20):
        w.zero_()
        torch.cuda.synchronize()
        M.mhc_linear(a, b, w, workspace=ws)
        out = torch.empty(24, 256, dtype=torch.bfloat16, device=DEV)
        M.mhc_linear(x, w, out, workspace=ws, read_ahead=False)
        outs.append(out)
    exact, bound = linear_bound(f64(x), f64(w), None, "none", None, torch.bfloat16)
    for out in outs:
        assert_within(out, exact, bound, "computed weight")


def test_linear_strided_rows_and_untouched_surroundings():
    g = gen(4)
    xb, rb = bf((37, 208), g).to(DEV), bf((37, 90), g).to(DEV)
    x, res = xb[:, 8:8 + 136], rb[:, 3:3 + 75]
    w = bf((75, 136), g, 0.1).to(DEV)
    ob = torch.full((40, 101), 7.0, dtype=torch.bfloat16, device=DEV)
    run_linear(x, w, residual=res, out=ob[1:38, 5:80])
    exact, bound = linear_bound(f64(x), f64(w), None, "none", f64(res), torch.bfloat16)
    assert_within(ob[1:38, 5:80], exact, bound, "strided")
    ob[1:38, 5:80] = 7.0
    assert bool((ob == 7.0).all())


@pytest.mark.parametrize("R,N", [(5, 200), (130, 700)])
def test_linear_residual_in_place(R, N):
    g = gen(5)
    x, w, r = bf((R, 512), g), bf((N, 512), g, 0.1), bf((R, N), g)
    out = r.to(DEV)
    run_linear(x.to(DEV), w.to(DEV), residual=out, out=out)
    exact, bound = linear_bound(f64(x), f64(w), None, "none", f64(r), torch.bfloat16)
    assert_within(out, exact, bound, "in place")


def test_linear_nan_and_inf_stay_in_their_row_and_feature():
    g = gen(6)
    x, w = bf((20, 640), g), bf((300, 640), g, 0.05)
    x[3, 17] = float("nan")
    x[7, 600] = float("inf")
    clean = run_linear(bf((20, 640), gen(6)).to(DEV), w.to(DEV))
    w2 = w.clone()
    w2[250, 5] = float("nan")
    got = run_linear(x.to(DEV), w2.to(DEV))
    assert bool(got[3].isnan().all()) and bool(got[:, 250].isnan().all())
    keep = [r for r in range(20) if r not in (3, 7)]
    cols = [c for c in range(300) if c != 250]
    assert torch.equal(got[keep][:, cols], clean[keep][:, cols])
    assert not bool(got[7, cols].isfinite().any())


def test_linear_is_reproducible_and_its_workspace_serves_fewer_rows():
    g = gen(8)
    ws = M.new_linear_workspace(300, DEV)
    w = bf((400, 4096), g, 0.02).to(DEV)
    for R in (300, 1, 40, 300, 129):  # shared tiles in every one of them
        x = bf((R, 4096), g).to(DEV)
        a = run_linear(x, w, workspace=ws)
        for _ in range(5):
            assert torch.equal(a, run_linear(x, w, workspace=ws))
        assert M.mhc_get_device_status(ws) == M.OK


def test_linear_on_a_side_stream_and_in_a_graph():
    g = gen(9)
    x, w = bf((24, 1024), g).to(DEV), bf((512, 1024), g, 0.05).to(DEV)
    want = run_linear(x, w)
    s = torch.cuda.Stream()
    ws, out = M.new_linear_workspace(24, DEV), torch.empty(24, 512, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    M.mhc_linear(x, w, out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graphs = []
    for _ in range(2):  # two graphs, a workspace each, replayed at once on two streams
        ws, out = M.new_linear_workspace(24, DEV), torch.zeros(24, 512, dtype=torch.bfloat16, device=DEV)
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            for _ in range(3):
                M.mhc_linear(x, w, out, workspace=ws)
        graphs.append((gr, ws, out, torch.cuda.Stream()))
    for seed in (10, 11):
        x.copy_(bf((24, 1024), gen(seed)))
        torch.cuda.synchronize()
        for gr, _, _, st in graphs:
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        want = run_linear(x, w)
        for _, _, out, _ in graphs:
            assert torch.equal(out, want)


@pytest.mark.parametrize("R,K,N,act", [(8, 512, 256, "none"), (8, 4096, 512, "swiglu"), (600, 200, 4500, "swiglu"),
                                       (4099, 64, 64, "none")])
def test_linear_wait_that_runs_out_is_reported(R, K, N, act):
    # a cluster, a pair and whole tiles: the copies are expected to bring more than they do
    g = gen(12)
    x, w = bf((R, K), g).to(DEV), bf((2 * N if act == "swiglu" else N, K), g, 0.05).to(DEV)
    want = run_linear(x, w, act=act)
    ws = M.new_linear_workspace(R, DEV)
    torch.cuda.synchronize()
    old = M.mhc_debug_set_wait(2_000_000, 4)
    try:
        run_linear(x, w, act=act, workspace=ws)
        assert M.mhc_get_device_status(ws) == M.DEVICE_TIMEOUT
    finally:
        M.mhc_debug_set_wait(old, 0)
    M.mhc_workspace_init(ws)
    assert torch.equal(run_linear(x, w, act=act, workspace=ws), want)
    assert M.mhc_get_device_status(ws) == M.OK


def test_linear_behind_a_long_call():
    # the bounded waits of a call that starts early do not run while the one before does
    g = gen(15)
    big_x, big_w = torch.zeros(16384, 8192, dtype=torch.bfloat16, device=DEV), torch.zeros(
        16384, 8192, dtype=torch.bfloat16, device=DEV)
    big_out = torch.empty(16384, 16384, dtype=torch.bfloat16, device=DEV)
    x, w = bf((8, 512), g).to(DEV), bf((256, 512), g, 0.05).to(DEV)
    want = run_linear(x, w)
    wss = [M.new_linear_workspace(16384, DEV) for _ in range(3)]
    out = [torch.empty_like(want) for _ in range(2)]
    M.mhc_linear(big_x, big_w, big_out, workspace=wss[0])
    torch.cuda.synchronize()
    old = M.mhc_debug_set_wait(1_500_000, 0)  # 1.5 ms; the long call takes about 3
    try:
        M.mhc_linear(big_x, big_w, big_out, workspace=wss[0])
        M.mhc_linear(x, w, out[0], workspace=wss[1])
        M.mhc_linear(x, w, out[1], workspace=wss[2])
        assert [M.mhc_get_device_status(ws) for ws in wss] == [M.OK] * 3
    finally:
        M.mhc_debug_set_wait(old, 0)
    assert torch.equal(out[0], want) and torch.equal(out[1], want)


def test_first_calls_may_be_captured():
    import subprocess
    import sys
    code = """
import torch
from mhc_residual_stream_b200 import mhc as M
from mhc_residual_stream_b200.moe import MoeConfig, MoeSublayer, MoeWeights
cfg = MoeConfig(experts=8, intermediate=64, top_k=2)
m, w = MoeSublayer(cfg, 40, 128), MoeWeights.draw(cfg, 128, 1, "cuda")
x = torch.randn(40, 128, device="cuda").bfloat16()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    m.run(x, w)
g.replay()
torch.cuda.synchronize()
a = [t.clone() for t in (m.logits, m.e2p, m.gemm2_permuted, m.shared_output)]
m.run(x, w)
torch.cuda.synchronize()
assert m.device_status() == M.OK
assert all(torch.equal(p, q) for p, q in zip(a, (m.logits, m.e2p, m.gemm2_permuted, m.shared_output)))
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_linear_binding_refusals():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(32, 64, dtype=torch.bfloat16, device=DEV)
    out, ws = torch.zeros(4, 32, dtype=torch.bfloat16, device=DEV), M.new_linear_workspace(4, DEV)
    d, s = torch.zeros(4, 64, dtype=torch.uint8, device=DEV), torch.zeros(512, dtype=torch.uint8, device=DEV)
    for a, kw in (((x.float(), w, out), {}), ((x, w.float(), out), {}), ((x, w, out.half()), {}), ((x.cpu(), w, out), {}),
                  (((d, s, True), w, out), {}), ((x, w, out), dict(bias=out)), ((x, w, out), dict(residual=x.float())),
                  ((x, w, out), dict(workspace=ws.float()))):
        with pytest.raises(TypeError):
            M.mhc_linear(*a, **{"workspace": ws, **kw})
    for a, kw in (((x, w[:, ::2], out), {}), ((x[:, ::2], w, out), {}), ((x, w, out[:3]), {}), ((x, w, out[:, :31]), {}),
                  ((x, w, out), dict(bias=torch.zeros(31, device=DEV))), ((x, w, out), dict(residual=out[:2])),
                  ((x, w, out), dict(activation="swiglu")), ((x[0], w, out), {}),
                  (((d, s, False), (d, s, False), out), {}), (((d, s[:511], True), (d, s, True), out), {})):
        with pytest.raises(ValueError):
            M.mhc_linear(*a, **{"workspace": ws, **kw})
    for a, kw, st in (((x, w, out), dict(workspace=None), M.WORKSPACE), ((x, w, out), dict(workspace=ws[:256]), M.WORKSPACE),
                      ((x[:, 1:57], w[:, :56].contiguous(), out), {}, M.INVALID_ARG),
                      ((x[:0], w, out[:0]), {}, M.UNSUPPORTED_SHAPE),
                      ((x, w, torch.zeros(32, dtype=torch.bfloat16, device=DEV).expand(4, 32)), {}, M.INVALID_ARG)):
        with pytest.raises(M.MhcError) as e:
            M.mhc_linear(*a, **{"workspace": ws, **kw})
        assert e.value.status == st


# ---------------------------------------------------------------- routing

def check_route(logits, k, bias=None, **kw):
    got = run_route(logits.to(DEV), k, None if bias is None else bias.to(DEV), **kw)
    w, ids, e2p, prow, off = [t.cpu() for t in got]
    ow, oids = O.moe_route(f64(logits), k, None if bias is None else f64(bias), **kw)
    oe2p, oprow, ooff = O.moe_permute(oids, logits.shape[1])
    assert np.array_equal(ids.numpy(), oids), "ids"
    assert np.array_equal(off.numpy(), ooff), "offsets"
    assert np.array_equal(e2p.numpy(), oe2p), "e2p"
    assert np.array_equal(prow.numpy(), oprow), "permuted rows"
    # scores by expf (2 steps) of an argument off by half a step of a range of at most
    # twice the largest finite logit, sums of up to 1024 terms by tree (10 levels), two divisions
    fin = logits.float()[logits.float().abs() < 1e3]
    span = float(fin.abs().max()) if fin.numel() else 0.0
    rel = (40 + 4 * span) * 2.0 ** -24
    assert np.all(np.abs(f64(w) - ow) <= rel * np.abs(ow) + 2.0 ** -126), "weights"
    return ow, oids


@pytest.mark.parametrize("R", [1, 2, 16, 17, 100, 128, 129, 700, 3001])
@pytest.mark.parametrize("E,k", [(64, 8), (200, 6)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_rows(R, E, k, scoring):
    g = gen(R + E)
    logits = torch.randn(R, E, generator=g) * 2
    check_route(logits, k, scoring=scoring, renormalize=R % 2 == 0, weight_scale=2.5)


@pytest.mark.parametrize("E,k,G,tg,gt", [
    (1, 1, 1, 1, 1), (7, 7, 1, 1, 1), (7, 3, 7, 3, 2), (33, 16, 3, 2, 2), (96, 4, 32, 5, 1), (256, 8, 8, 4, 2),
    (500, 12, 4, 1, 2), (512, 16, 1, 1, 1), (1000, 16, 8, 3, 2), (1024, 16, 32, 32, 1), (17, 1, 17, 17, 1),
])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_shapes_and_groups(E, k, G, tg, gt, scoring, biased):
    for R in (5, 150):
        g = gen(E * 3 + R)
        logits = torch.randn(R, E, generator=g) * 1.5
        bias = torch.randn(E, generator=g) * 0.2 if biased else None
        check_route(logits, k, bias, scoring=scoring, num_groups=G, top_groups=tg, group_top=gt,
                    renormalize=biased)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G", [1, 4])
def test_route_unavailable_experts_and_rows(scoring, biased, G):
    g = gen(77)
    R, E, k = 140, 40, 6
    logits = torch.randn(R, E, generator=g)
    bias = torch.randn(E, generator=g) * 0.1 if biased else None
    if biased:
        bias[4] = -math.inf
    logits[3] = -math.inf                       # nothing to choose
    logits[5, 2:] = -math.inf                   # fewer than k
    logits[6, 10:20] = -math.inf                # a whole group
    logits[7, 9] = float("nan")
    logits[8] = float("nan")
    logits[9, 11] = math.inf
    logits[10, [1, 30]] = math.inf
    logits[11] = torch.finfo(torch.float32).min
    logits[12] = -200.0 + torch.arange(E) * 0.5  # scores far below fp32's range
    logits[120:] = -math.inf                    # padding
    ow, ids = check_route(logits, k, bias, scoring=scoring, num_groups=G, top_groups=max(1, G // 2), group_top=2)
    assert (ids[3] == -1).all() and (ids[120:] == -1).all() and (ids[5] >= 0).sum() == (2 if G else 0)
    # no pair at all
    check_route(torch.full((9, 12), -math.inf), 3, scoring=scoring)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest_index(scoring):
    R, E = 64, 96
    g = gen(5)
    logits = torch.randint(0, 3, (R, E), generator=g).float()
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    bias = torch.randint(0, 2, (E,), generator=g).float()
    for G, tg in ((1, 1), (8, 3)):
        check_route(logits, 8, None, scoring=scoring, num_groups=G, top_groups=tg, group_top=2)
        check_route(logits, 8, bias, scoring=scoring, num_groups=G, top_groups=tg, group_top=2)


def test_route_near_equal_choices_do_not_depend_on_fp32_rounding():
    # choices that differ by far less than fp32 resolves: neighbouring logits at the flat
    # end of the sigmoid, under a common bias
    R, E = 40, 64
    g = gen(6)
    base = 8.0 + torch.rand(R, 1, generator=g)
    step = 2.0 ** -20 * torch.stack([torch.randperm(E, generator=g) for _ in range(R)]).float()
    check_route(base + step, 8, torch.ones(E), scoring="sigmoid")
    check_route(base + step, 8, torch.ones(E), scoring="softmax")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_groups_whose_choices_cancel(scoring):
    # a group's value is the sum of two choices a thousand away from zero on either side:
    # fp32 sums would be off by more than the groups differ
    R, G, S = 200, 8, 4
    logits = torch.randn(R, G * S, generator=gen(21))
    bias = torch.tensor([1000.0, -1000.0, -5000.0, -6000.0]).repeat(G)
    check_route(logits, 4, bias, scoring=scoring, num_groups=G, top_groups=3, group_top=2)
    bias = bias + torch.randn(G * S, generator=gen(22)) * 1e-4
    check_route(logits, 6, bias, scoring=scoring, num_groups=G, top_groups=4, group_top=2)


def test_route_many_near_winners():
    # up to all experts within fp32's reach of each other: more than a warp's lanes can hold
    g = gen(23)
    for E, k in ((64, 8), (20, 4), (40, 16), (200, 3)):
        base = torch.rand(30, 1, generator=g) * 2
        step = 2.0 ** -22 * torch.stack([torch.randperm(E, generator=g) for _ in range(30)]).float()
        check_route(base + step, k, torch.full((E,), 0.25), scoring="sigmoid")
        check_route(base + step, k, torch.full((E,), -0.25), scoring="softmax")


def test_route_bf16_logits():
    g = gen(13)
    logits = bf((130, 256), g, 2.0)
    check_route(logits, 8, torch.randn(256, generator=g) * 0.1, scoring="sigmoid", num_groups=8, top_groups=4,
                group_top=2)
    check_route(logits, 8, scoring="softmax")


def test_route_reuses_its_workspace_and_is_captured():
    g = gen(14)
    ws = M.new_moe_route_workspace(2000, 128, 8, DEV)
    for R in (2000, 3, 128, 900):
        logits = torch.randn(R, 128, generator=g).to(DEV)
        a = run_route(logits, 8, workspace=ws)
        for _ in range(3):
            assert all(torch.equal(p, q) for p, q in zip(a, run_route(logits, 8, workspace=ws)))
    for R in (60, 900):
        logits = torch.randn(R, 128, generator=g).to(DEV)
        outs = run_route(logits, 8, workspace=ws)
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            M.mhc_moe_route(logits, *outs, workspace=ws)
        logits.copy_(torch.randn(R, 128, generator=g))
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(outs, run_route(logits, 8)))


# ---------------------------------------------------------------- experts

def run_experts(x, w13, w2, prow, off, out=None, workspace=None):
    P, I = len(prow), w2.shape[2]
    out = torch.full((P, x.shape[1]), 5.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    ws = M.new_moe_experts_workspace(x.shape[0], P, I, DEV) if workspace is None else workspace
    M.mhc_moe_experts(x.to(DEV), w13.to(DEV), w2.to(DEV), i32(prow), i32(off), out, workspace=ws)
    return out, ws


@pytest.mark.parametrize("R,k,E,H,I", [
    (1, 1, 1, 8, 8), (1, 8, 64, 256, 128), (1, 2, 4, 2048, 136), (7, 3, 5, 72, 40), (16, 4, 16, 512, 264),
    (37, 3, 24, 712, 328), (50, 8, 8, 192, 200), (128, 8, 32, 320, 72), (200, 2, 3, 136, 304), (700, 4, 6, 64, 128),
    (20, 2, 300, 64, 16), (9, 16, 1000, 64, 8), (513, 4, 5, 200, 136), (1500, 2, 2, 72, 520), (2000, 3, 16, 128, 264),
])
def test_experts(R, k, E, H, I):
    x, w13, w2, e2p, prow, off = draw_experts(R, k, E, H, I, seed=R + E)
    out, ws = run_experts(x, w13, w2, prow, off)
    exact, bound = experts_bound(f64(x), f64(w13), f64(w2), prow, off)
    assert_within(out, exact, bound, f"experts {R} {k} {E} {H} {I}")
    again, _ = run_experts(x, w13, w2, prow, off, workspace=ws)
    assert torch.equal(out, again) and M.mhc_get_device_status(ws) == M.OK


@pytest.mark.parametrize("R,k", [(40, 4), (300, 2), (1100, 2)])
def test_experts_of_one_popular_expert_and_unused_places(R, k):
    E, H, I = 12, 200, 136
    ids = np.full((R, k), -1)
    ids[:, 0] = 5                         # every row to one expert
    ids[::3, 1] = 11
    x, w13, w2, e2p, prow, off = draw_experts(R, k, E, H, I, seed=R, ids=ids)
    out, ws = run_experts(x, w13, w2, prow, off)
    used = int(off[-1])
    assert used == R + (R + 2) // 3 < R * k
    exact, bound = experts_bound(f64(x), f64(w13), f64(w2), prow, off)
    assert_within(out[:used], exact[:used], bound[:used], "popular expert")
    assert bool((out[used:] == 5.0).all())  # places behind the last pair are left as they were
    none = run_experts(x, w13, w2, np.full(R * k, -1), np.zeros(E + 1))[0]
    assert bool((none == 5.0).all())


def test_experts_strided_rows():
    x, w13, w2, e2p, prow, off = draw_experts(30, 2, 6, 128, 64, seed=2)
    wide = torch.zeros(30, 152, dtype=torch.bfloat16, device=DEV)
    wide[:, 16:144] = x.to(DEV)
    out, _ = run_experts(wide[:, 16:144], w13, w2, prow, off)
    assert torch.equal(out, run_experts(x, w13, w2, prow, off)[0])


@pytest.mark.parametrize("R", [30, 600])
def test_experts_report_bad_indices(R):
    x, w13, w2, e2p, prow, off = draw_experts(R, 2, 6, 128, 64, seed=3)
    good, _ = run_experts(x, w13, w2, prow, off)
    for bad in (R, -1, 1 << 30):  # a row that x does not have reads row 0
        p = prow.copy()
        p[11] = bad
        out, ws = run_experts(x, w13, w2, p, off)
        assert M.mhc_get_device_status(ws) == M.DEVICE_INDEX
        keep = [i for i in range(2 * R) if i != 11]
        assert torch.equal(out[keep], good[keep])
    n = 2 * R
    for o in ([0, 10, 5, 20, 30, 40, n], [0, 10, 20, 30, 40, 50, n + 1], [-1, 10, 20, 30, 40, 50, n]):
        out, ws = run_experts(x, w13, w2, prow, np.array(o))  # nothing is computed
        assert M.mhc_get_device_status(ws) == M.DEVICE_INDEX
        assert bool((out == 5.0).all())


@pytest.mark.parametrize("R,k,E,H,I", [(3, 2, 8, 2048, 256), (300, 2, 4, 128, 264)])
def test_experts_wait_that_runs_out_is_reported(R, k, E, H, I):
    x, w13, w2, e2p, prow, off = draw_experts(R, k, E, H, I, seed=9)
    want, ws = run_experts(x, w13, w2, prow, off)
    torch.cuda.synchronize()
    old = M.mhc_debug_set_wait(2_000_000, 4)
    try:
        run_experts(x, w13, w2, prow, off, workspace=ws)
        assert M.mhc_get_device_status(ws) == M.DEVICE_TIMEOUT
    finally:
        M.mhc_debug_set_wait(old, 0)
    M.mhc_workspace_init(ws)
    assert torch.equal(run_experts(x, w13, w2, prow, off, workspace=ws)[0], want)
    assert M.mhc_get_device_status(ws) == M.OK


# ---------------------------------------------------------------- a run of them together

@pytest.mark.parametrize("R,padded", [(1, 0), (24, 5), (128, 0)])
def test_moe_sublayer_between_two_boundaries(R, padded):
    """Router logits, routing, the experts, the shared expert, and the boundary that
    finalizes them, against the oracle on what the library wrote stage by stage."""
    from mhc_residual_stream_b200 import synthetic as S
    H, I, E, k, n = 512, 192, 16, 4, 4
    g = gen(R)
    x = bf((R, H), g)
    router, w13, w2 = bf((E, H), g, 0.1), bf((E, 2 * I, H), g, 0.06), bf((E, H, I), g, 0.1)
    s13, s2 = bf((2 * I, H), g, 0.06), bf((H, I), g, 0.1)
    bias = torch.randn(E, generator=g) * 0.1
    d = S.draw_boundary(R, H, n=n, partials=1, seed=R)
    t = {q: d[q].to(DEV) for q in ("residual", "post", "comb", "pre", "norm_weight")}
    logits = run_linear(x.to(DEV), router.to(DEV), out_type=torch.float32)
    if padded:
        logits[R - padded:] = -math.inf
    w, ids, e2p, prow, off = run_route(logits, k, bias.to(DEV), scoring="sigmoid", num_groups=4, top_groups=2,
                                       group_top=2, weight_scale=2.0)
    perm = torch.zeros(R * k, H, dtype=torch.bfloat16, device=DEV)
    M.mhc_moe_experts(x.to(DEV), w13.to(DEV), w2.to(DEV), prow, off, perm,
                      workspace=M.new_moe_experts_workspace(R, R * k, I, DEV))
    inner = run_linear(x.to(DEV), s13.to(DEV), act="swiglu")
    shared = run_linear(inner, s2.to(DEV))
    res, li = torch.empty_like(t["residual"]), torch.empty(R, H, dtype=torch.bfloat16, device=DEV)
    ws = M.new_workspace(R, H, n, DEV)
    M.mhc_boundary_moe_finalize(perm, w, e2p, shared, t["residual"], t["post"], t["comb"], t["pre"], t["norm_weight"],
                                1e-6, None, res, layer_input=li, workspace=ws)
    assert M.mhc_get_device_status(ws) == M.OK
    # stage by stage
    ex, bd = linear_bound(f64(x), f64(router), None, "none", None, torch.float32)
    live = R - padded
    assert_within(logits[:live], ex[:live], bd[:live], "router logits")
    ow, oids = O.moe_route(f64(logits), k, f64(bias), "sigmoid", 4, 2, 2, True, 2.0)
    oe2p, oprow, ooff = O.moe_permute(oids, E)
    assert np.array_equal(e2p.cpu().numpy(), oe2p) and np.array_equal(off.cpu().numpy(), ooff)
    used = int(ooff[-1])
    ex, bd = experts_bound(f64(x), f64(w13), f64(w2), oprow, ooff)
    assert_within(perm[:used], ex[:used], bd[:used], "experts")
    ex, bd = linear_bound(f64(inner), f64(s2), None, "none", None, torch.bfloat16)
    assert_within(shared, ex, bd, "shared expert")
    # the finalize: x = shared + sum_t w gemm2[e2p], padded rows the shared output alone
    xs = f64(shared).copy()
    for i, q in enumerate(oe2p):
        if q >= 0:
            xs[i // k] += f64(w).reshape(-1)[i] * f64(perm)[q]
    want = O.post_mix(f64(d["residual"]), xs, f64(d["post"]), f64(d["comb"]))
    # both sides rounded once; fp32 sums of terms of order one
    assert np.all(np.abs(f64(res) - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -16)
