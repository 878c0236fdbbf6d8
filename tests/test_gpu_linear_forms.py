"""GPU test of a product in each form of mhc_linear that the sublayer tests do not reach."""

import pytest
import torch

import oracle as O
from mhc_residual_stream_b200 import mhc as M

from _forms import MORE_FORMS
from _sublayer import DEV, assert_within, bf, f64, gen, linear_bound, run_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mhc_residual_stream_b200 import build
    build.build()
    M.lib()
    yield


def mxfp8_operand(rows, K, g, exponent):
    """E4M3 bytes of normal values under scales of 2^exponent up to four times that, and
    the values that they stand for."""
    data = torch.randn(rows, K, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = torch.randint(127 + exponent, 130 + exponent, (rows, K // 32), generator=g, dtype=torch.uint8)
    values = O.mxfp8_dequantize(data.numpy(), scale.numpy())
    tiled = torch.from_numpy(O.swizzle_scales_128x4(scale.numpy()).reshape(-1))
    return (data.to(DEV), tiled.to(DEV), True), values


@pytest.mark.parametrize("fp8,gated,R,K,N,form", [(*kind, *c) for kind, v in MORE_FORMS.items() for c in v])
def test_linear_in_the_other_forms(fp8, gated, R, K, N, form):
    assert M.mhc_debug_linear_form(R, K, N, fp8, gated)[:3] == form
    g = gen(R + 3 * K + 7 * N)
    act, W = ("swiglu", 2 * N) if gated else ("silu", N)
    b, r = torch.randn(W, generator=g) * 0.3, bf((R, N), g)
    if fp8:
        (xo, x), (wo, w) = mxfp8_operand(R, K, g, -1), mxfp8_operand(W, K, g, -7)
    else:
        x, w = bf((R, K), g), bf((W, K), g, 1.5 / K ** 0.5)
        xo, wo, x, w = x.to(DEV), w.to(DEV), f64(x), f64(w)
    ws = M.new_linear_workspace(R, DEV)
    exact, bound = linear_bound(x, w, f64(b), act, f64(r), torch.float32)
    got = run_linear(xo, wo, b.to(DEV), act, r.to(DEV), torch.float32, workspace=ws)
    assert_within(got, exact, bound, f"{R}x{K}x{N}")
    assert torch.equal(got, run_linear(xo, wo, b.to(DEV), act, r.to(DEV), torch.float32, workspace=ws))
    assert M.mhc_get_device_status(ws) == M.OK
