"""Helpers of the sublayer operators' tests: seeded inputs and error bounds.

Bounds, from the arithmetic the kernels state (u = 2^-24, half a step of fp32):
  * a product of K terms with exact operands, accumulated in fp32: the tensor core
    adds 16 (bf16) or 32 (MXFP8) exact products to the accumulator per step,
    each addition cut or rounded to fp32, an error of at most one step (2u) of
    the largest partial sum; K/16 steps, 16 additions in a step, at most 16
    shares joined in fp32: (K/16 + 32) * 2u * S with S = sum |x||w| + |bias|;
  * silu by the fast exponential (2 + 1.173 |v| steps of fp32, per the CUDA math
    documentation) and a division: relative (8 + 2.4 |v|) u; gelu by erff
    (2 steps) and three roundings: 8u |v| absolute; both have slopes of at most 1.13;
  * one rounding to the output type: bf16 2^-8, fp32 2^-24, relative.
"""

from __future__ import annotations

import numpy as np
import torch

import oracle as O
from mhc_residual_stream_b200 import mhc as M

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def bf(shape, g, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def mxfp8(v):
    """(data, swizzled scales, exact values) of a float tensor, by the boundary's oracle."""
    data, sc = O.mxfp8_quantize(O.bf16_round(v.double().numpy()))
    return torch.from_numpy(data), torch.from_numpy(O.swizzle_scales_128x4(sc).reshape(-1)), O.mxfp8_dequantize(data, sc)


def product_error(K, S):
    return (K / 16 + 32) * 2 * U * S


def act_error(name, v, dv):
    """Bound on the error of the activation of v, itself off by at most dv."""
    a = np.abs(v)
    if name == "silu":
        return 1.13 * dv + (8 + 2.4 * a) * U * np.abs(O.activation("silu", v)) + 2.0 ** -126
    if name == "gelu":
        return 1.13 * dv + 8 * U * a
    return dv


def linear_bound(x, w, bias, act, residual, out_type):
    """(exact result, bound on the error of the library's) for float64 operands."""
    exact = O.linear(x, w, bias, act, residual)
    y = O.linear(x, w, bias)
    S = np.abs(x) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    d = product_error(x.shape[1], S)
    if act == "swiglu":
        (g, u), (dg, du) = np.split(y, 2, axis=1), np.split(d, 2, axis=1)
        s = O.activation("silu", g)
        ds = act_error("silu", g, dg)
        err = np.abs(s) * du + ds * (np.abs(u) + du) + U * np.abs(s * u)
        val = s * u
    else:
        err, val = act_error(act, y, d), O.activation(act, y)
    if residual is not None:
        err = err + U * (np.abs(val) + np.abs(residual))
    return exact, err + HALF[out_type] * (np.abs(exact) + err)


def assert_within(got, exact, bound, what):
    got = f64(got)
    assert got.shape == exact.shape, (what, got.shape, exact.shape)
    err = np.abs(got - exact)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, worst {np.nanmax(err / bound):.3g} "
                           f"times it, first at {tuple(np.argwhere(bad)[0])}")


def experts_bound(x, w13, w2, prow, offsets):
    """(exact result with the intermediate rounded, bound). An intermediate value may round
    to another bf16 value only where the product's error spans a rounding point."""
    P, H = len(prow), x.shape[1]
    exact, bound = np.full((P, H), np.nan), np.full((P, H), np.nan)
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        rows = x[prow[a:b]]
        v = O.linear(rows, w13[e], act="swiglu")
        _, d = linear_bound(rows, w13[e], None, "swiglu", None, torch.float32)
        inner = O.bf16_round(v)
        flip = O.bf16_round(v + d) - O.bf16_round(v - d)
        exact[a:b] = inner @ w2[e].T
        S = (np.abs(inner) + flip) @ np.abs(w2[e]).T
        err = flip @ np.abs(w2[e]).T + product_error(w2[e].shape[1], S)
        bound[a:b] = err + HALF[torch.bfloat16] * (np.abs(exact[a:b]) + err)
    return exact, bound


def draw_experts(R, k, E, H, I, seed, ids=None):
    """CPU inputs of the experts' products: x, w13, w2 and the permutation of ids
    (drawn, uneven, unless given)."""
    g = gen(seed)
    x, w13, w2 = bf((R, H), g), bf((E, 2 * I, H), g, 1.5 / H ** 0.5), bf((E, H, I), g, 1.5 / I ** 0.5)
    if ids is None:
        pop = torch.randn(E, generator=g)
        ids = (torch.randn(R, E, generator=g) + pop).topk(k, dim=1).indices.numpy()
    e2p, prow, off = O.moe_permute(np.asarray(ids), E)
    return x, w13, w2, e2p, prow, off


def i32(a):
    return torch.from_numpy(np.asarray(a)).to(torch.int32).to(DEV)


def run_linear(x, w, bias=None, act="none", residual=None, out_type=torch.bfloat16, workspace=None, out=None,
               stream=None):
    R = (x if isinstance(x, torch.Tensor) else x[0]).shape[0]
    wn = (w if isinstance(w, torch.Tensor) else w[0]).shape[0]
    N = wn // 2 if act == "swiglu" else wn
    out = torch.full((R, N), float("nan"), dtype=out_type, device=DEV) if out is None else out
    workspace = M.new_linear_workspace(R, DEV) if workspace is None else workspace
    M.mhc_linear(x, w, out, bias=bias, activation=act, residual=residual, workspace=workspace, stream=stream)
    return out


def run_route(logits, k, bias=None, workspace=None, stream=None, **kw):
    R, E = logits.shape
    w = torch.full((R, k), float("nan"), device=DEV)
    ids, e2p, prow, off = (torch.full(s, -7, dtype=torch.int32, device=DEV)
                           for s in ((R, k), (R * k,), (R * k,), (E + 1,)))
    workspace = M.new_moe_route_workspace(R, E, k, DEV) if workspace is None else workspace
    M.mhc_moe_route(logits, w, ids, e2p, prow, off, bias=bias, workspace=workspace, stream=stream, **kw)
    return w, ids, e2p, prow, off
