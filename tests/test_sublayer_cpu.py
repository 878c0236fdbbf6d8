"""The sublayer operators without a GPU: refusals of bad arguments before any
launch, workspace sizes, and pins of their oracle against values worked by hand
and torch's own functions."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O
from mhc_residual_stream_b200 import build
from mhc_residual_stream_b200 import mhc as M


@pytest.fixture(scope="module")
def L():
    build.build()
    return M.lib()


def _a(addr=0x10000):
    return ctypes.c_void_p(addr)


# ---------------------------------------------------------------- refusals

def test_linear_refusals(L):
    a = _a()
    base = dict(x=a, xs=None, xst=64, w=a, wsc=None, bias=None, act=0, res=None, rst=0, out=a, fp32=0, ost=100, R=4, K=64,
                N=100, ahead=1, ws=a, wsb=1 << 30, s=None)

    def call(**kw):
        return L.mhc_linear(*{**base, **kw}.values())

    for kw in (dict(R=0), dict(R=65536), dict(K=0), dict(K=60), dict(K=65544), dict(N=0), dict(N=(1 << 20) + 1),
               dict(K=72, xs=a, wsc=a, xst=80), dict(K=64, xs=a, wsc=a, act=4)):
        assert call(**kw) == M.UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(out=None), dict(xs=a), dict(wsc=a), dict(act=5), dict(act=-1),
               dict(x=_a(0x10008)), dict(w=_a(0x10008)), dict(xs=_a(0x10008), wsc=a), dict(bias=_a(0x10002)),
               dict(res=_a(0x10001), rst=100), dict(out=_a(0x10002), fp32=1), dict(xst=56), dict(xst=68),
               dict(xs=a, wsc=a, xst=72), dict(ost=99), dict(res=a, rst=99),
               dict(res=a, rst=104), dict(res=a, rst=100, fp32=1)):  # the residual is out: same stride, bf16
        assert call(**kw) == M.INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=_a(0x10010)), dict(wsb=M.mhc_linear_workspace_bytes(4) - 1)):
        assert call(**kw) == M.WORKSPACE, kw


def test_route_refusals(L):
    a = _a()

    def call(logits=a, bf16=0, bias=None, args=(0, 1, 1, 1, 8, 1, 1.0), w=a, ids=a, e2p=a, prow=a, off=a, R=4, E=64,
             ws=a, wsb=1 << 30):
        st = None if args is None else ctypes.byref(M.RouteArgs(*args))
        return L.mhc_moe_route(logits, bf16, bias, st, w, ids, e2p, prow, off, R, E, ws, wsb, None)

    for kw in (dict(R=0), dict(R=65536), dict(E=0), dict(E=1025), dict(args=(0, 1, 1, 1, 0, 1, 1.0)),
               dict(args=(0, 1, 1, 1, 17, 1, 1.0)), dict(E=4), dict(args=(0, 0, 1, 1, 8, 1, 1.0)),
               dict(args=(0, 33, 1, 1, 8, 1, 1.0), E=66), dict(args=(0, 3, 1, 1, 8, 1, 1.0)),
               dict(args=(0, 4, 5, 1, 8, 1, 1.0)), dict(args=(0, 4, 0, 1, 8, 1, 1.0)), dict(args=(0, 4, 2, 3, 8, 1, 1.0)),
               dict(args=(0, 4, 2, 0, 8, 1, 1.0))):
        assert call(**kw) == M.UNSUPPORTED_SHAPE, kw
    for kw in (dict(args=None), dict(logits=None), dict(w=None), dict(ids=None), dict(e2p=None), dict(prow=None),
               dict(off=None), dict(args=(2, 1, 1, 1, 8, 1, 1.0)), dict(args=(0, 1, 1, 1, 8, 1, math.nan)),
               dict(args=(0, 1, 1, 1, 8, 1, math.inf)), dict(logits=_a(0x10002)), dict(logits=_a(0x10001), bf16=1),
               dict(bias=_a(0x10002)), dict(ids=_a(0x10002))):
        assert call(**kw) == M.INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=_a(0x10010)), dict(wsb=M.mhc_moe_route_workspace_bytes(4, 64, 8) - 1)):
        assert call(**kw) == M.WORKSPACE, kw


def test_experts_refusals(L):
    a = _a()
    base = dict(x=a, xst=64, w13=a, w2=a, prow=a, off=a, out=a, R=4, P=8, E=4, H=64, I=32, ws=a, wsb=1 << 30, s=None)

    def call(**kw):
        return L.mhc_moe_experts(*{**base, **kw}.values())

    for kw in (dict(R=0), dict(R=65536), dict(P=0), dict(P=16 * 65535 + 1), dict(E=0), dict(E=1025), dict(H=60),
               dict(H=0), dict(H=65544), dict(I=36), dict(I=0)):
        assert call(**kw) == M.UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=None), dict(w13=None), dict(w2=None), dict(prow=None), dict(off=None), dict(out=None),
               dict(x=_a(0x10008)), dict(out=_a(0x10008)), dict(prow=_a(0x10002)), dict(xst=56), dict(xst=68)):
        assert call(**kw) == M.INVALID_ARG, kw
    for kw in (dict(ws=None), dict(ws=_a(0x10010)), dict(wsb=M.mhc_moe_experts_workspace_bytes(4, 8, 32) - 1)):
        assert call(**kw) == M.WORKSPACE, kw


def test_workspace_sizes(L):
    sizes = [M.mhc_linear_workspace_bytes(r) for r in (1, 16, 17, 100, 127, 128, 300, 65535)]
    assert sizes == sorted(sizes) and sizes[0] >= 2048
    for bad in (0, -1, 65536):
        assert M.mhc_linear_workspace_bytes(bad) == 0
    assert M.mhc_moe_experts_workspace_bytes(4, 32, 128) >= M.mhc_linear_workspace_bytes(4) + 32 * 128 * 2
    assert M.mhc_moe_experts_workspace_bytes(0, 32, 128) == M.mhc_moe_experts_workspace_bytes(4, 0, 128) == 0
    assert M.mhc_moe_route_workspace_bytes(1, 1, 1) > 0
    for bad in ((0, 8, 2), (4, 1025, 2), (4, 8, 9), (4, 64, 17)):
        assert M.mhc_moe_route_workspace_bytes(*bad) == 0
    with pytest.raises(M.MhcError):
        M.new_linear_workspace(0, "cpu")


def test_binding_refuses_cpu_tensors_and_unknown_names(L):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        M.mhc_linear(x, x, x)
    with pytest.raises(ValueError):
        M.mhc_linear(x, x, x, activation="tanh")
    with pytest.raises(ValueError):
        M.mhc_moe_route(x, x, x, x, x, x, scoring="linear")
    with pytest.raises(TypeError):
        M.mhc_moe_experts(x, x, x, x, x, x)
    with pytest.raises(TypeError):
        M.mhc_linear(None, x, x)
    with pytest.raises(TypeError):
        M.mhc_linear((x, x, True), x, x)  # MXFP8 data are bytes


# ---------------------------------------------------------------- the oracle

def test_oracle_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    w, i = O.moe_route(l, 2)
    assert i.tolist() == [[2, 1]] and np.allclose(w, [[4 / 6, 2 / 6]])
    w, i = O.moe_route(l, 3, renormalize=False, weight_scale=8)
    assert i.tolist() == [[2, 1, 0]] and np.allclose(w, [[4, 2, 1]])  # of a sum of 8
    # sigmoid scores 0.5, 2/3, 0.8, 0.5; the bias chooses, the weight is the score
    w, i = O.moe_route(l, 2, bias=np.array([0.0, 0.0, -1.0, 0.3]), scoring="sigmoid", renormalize=False)
    assert i.tolist() == [[3, 1]] and np.allclose(w, [[0.5, 2 / 3]])
    # two groups of two: values 0.5 + 2/3 against 0.8 + 0.5
    w, i = O.moe_route(l, 2, scoring="sigmoid", num_groups=2, top_groups=1, group_top=2, renormalize=False)
    assert i.tolist() == [[2, 3]]
    w, i = O.moe_route(l[:, [0, 1, 2, 0]], 2, scoring="sigmoid", num_groups=2, top_groups=1, group_top=1)
    assert i.tolist() == [[2, 3]]
    w, i = O.moe_route(np.array([[-np.inf, 0.0, np.nan]]), 2)
    assert i.tolist() == [[1, -1]] and w.tolist() == [[1.0, 0.0]]
    w, i = O.moe_route(np.full((1, 3), -np.inf), 2, scoring="sigmoid")
    assert i.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]


def test_oracle_route_against_torch():
    l = torch.randn(50, 33, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    p, q = torch.softmax(l, 1).topk(5)
    w, i = O.moe_route(l.numpy(), 5, renormalize=False)
    assert np.array_equal(i, q.numpy()) and np.allclose(w, p.numpy(), rtol=1e-13)
    p, q = torch.sigmoid(l).topk(5)
    w, i = O.moe_route(l.numpy(), 5, scoring="sigmoid")
    assert np.array_equal(i, q.numpy()) and np.allclose(w, (p / p.sum(1, keepdim=True)).numpy(), rtol=1e-13)


def test_oracle_permutation_by_hand():
    e2p, rows, off = O.moe_permute(np.array([[2, 0], [0, -1], [2, 1]]), 4)
    assert e2p.tolist() == [3, 0, 1, -1, 4, 2]
    assert rows.tolist() == [0, 1, 2, 0, 2, -1]
    assert off.tolist() == [0, 2, 3, 5, 5]


def test_oracle_products_against_torch():
    g = torch.Generator().manual_seed(2)
    x, w, b, r = (torch.randn(*s, dtype=torch.float64, generator=g) for s in ((6, 10), (8, 10), (8,), (6, 8)))
    F = torch.nn.functional
    for name, f in (("none", lambda v: v), ("relu", F.relu), ("silu", F.silu), ("gelu", F.gelu)):
        assert np.allclose(O.linear(x.numpy(), w.numpy(), b.numpy(), name, r.numpy()), (f(F.linear(x, w, b)) + r).numpy(),
                           rtol=1e-12, atol=1e-13)
    y = F.linear(x, w, b)
    assert np.allclose(O.linear(x.numpy(), w.numpy(), b.numpy(), "swiglu"), (F.silu(y[:, :4]) * y[:, 4:]).numpy())
    # one expert of two, rows 1 and 0
    w13, w2 = torch.randn(2, 8, 10, dtype=torch.float64, generator=g), torch.randn(2, 10, 4, dtype=torch.float64, generator=g)
    got = O.moe_experts(x.numpy(), w13.numpy(), w2.numpy(), np.array([1, 0, -1]), np.array([0, 0, 2]))
    y = F.linear(x[[1, 0]], w13[1])
    inner = (F.silu(y[:, :4]) * y[:, 4:]).to(torch.bfloat16).double()
    assert np.allclose(got[:2], (inner @ w2[1].T).numpy(), rtol=1e-12) and np.isnan(got[2]).all()
