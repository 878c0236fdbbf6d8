"""GPU tests of the sublayer operators at their largest sizes: offsets that pass 32 bits,
the most rows, experts and choices."""

import numpy as np
import pytest
import torch

import oracle as O
from mhc_residual_stream_b200 import mhc as M

from _sublayer import DEV, HALF, assert_within, experts_bound, f64, linear_bound, run_linear, run_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mhc_residual_stream_b200 import build
    build.build()
    M.lib()
    yield
    torch.cuda.empty_cache()


def gpu_gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(shape, g, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def some_rows(R):
    return [0, 1, R // 3, R // 2 + 1, R - 2, R - 1]


@pytest.mark.parametrize("R,K,N", [(65535, 16, 32800), (33000, 65528, 8)])
def test_linear_with_offsets_behind_32_bits(R, K, N):
    # 2.1e9 elements of out, then of x
    g = gpu_gen(R)
    x, w, b = normal((R, K), g), normal((N, K), g, K ** -0.5), torch.randn(N, generator=g, device=DEV)
    out = run_linear(x, w, b, "relu")
    at = some_rows(R)
    exact, bound = linear_bound(f64(x[at]), f64(w), f64(b), "relu", None, torch.bfloat16)
    assert_within(out[at], exact, bound, f"{R} x {K} -> {N}")
    assert bool(out.isfinite().all())


def test_experts_with_weights_behind_32_bits():
    # 300 experts of 2 x 512 x 7168: w13 has 2.2e9 elements
    E, H, I, R = 300, 7168, 512, 6
    g = gpu_gen(1)
    x, w13, w2 = normal((R, H), g), normal((E, 2 * I, H), g, H ** -0.5), normal((E, H, I), g, I ** -0.5)
    ids = np.array([[0, 299], [298, 1], [299, 150], [297, 298], [299, 0], [293, 299]])
    e2p, prow, off = O.moe_permute(ids, E)
    out = torch.full((2 * R, H), 5.0, dtype=torch.bfloat16, device=DEV)
    ws = M.new_moe_experts_workspace(R, 2 * R, I, DEV)
    i32 = [torch.from_numpy(a).to(torch.int32).to(DEV) for a in (prow, off)]
    M.mhc_moe_experts(x, w13, w2, *i32, out, workspace=ws)
    used = sorted(set(ids.reshape(-1).tolist()))
    compact = np.concatenate([[0], np.cumsum([off[e + 1] - off[e] for e in used])])
    exact, bound = experts_bound(f64(x), f64(w13[used]), f64(w2[used]), prow, compact)
    assert_within(out, exact, bound, "experts")
    assert M.mhc_get_device_status(ws) == M.OK


def test_experts_with_rows_behind_32_bits():
    # 65535 rows x 16 of 2056 columns: gemm2_permuted has 2.1e9 elements
    E, H, I, R, k = 16, 2056, 8, 65535, 16
    g = gpu_gen(2)
    x, w13, w2 = normal((R, H), g), normal((E, 2 * I, H), g, H ** -0.5), normal((E, H, I), g, I ** -0.5)
    prow = torch.arange(R, dtype=torch.int32, device=DEV).repeat(k)  # every row to every expert
    off = (torch.arange(E + 1, device=DEV) * R).to(torch.int32)
    out = torch.full((R * k, H), 5.0, dtype=torch.bfloat16, device=DEV)
    ws = M.new_moe_experts_workspace(R, R * k, I, DEV)
    M.mhc_moe_experts(x, w13, w2, prow, off, out, workspace=ws)
    at = some_rows(R)
    local = np.tile(np.arange(len(at)), E)
    exact, bound = experts_bound(f64(x[at]), f64(w13), f64(w2), local, np.arange(E + 1) * len(at))
    places = torch.tensor([e * R + r for e in range(E) for r in at], device=DEV)
    assert_within(out[places], exact, bound, "experts")
    assert M.mhc_get_device_status(ws) == M.OK


def test_route_of_the_most_rows_experts_and_choices():
    R, E, k = 65535, 1024, 16
    logits = torch.randn(R, E, generator=gpu_gen(3), device=DEV)
    w, ids, e2p, prow, off = run_route(logits, k, scoring="softmax", renormalize=True)
    want = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    p = torch.softmax(logits.gather(1, want).double(), 1)
    # as in the routing tests: (40 + 4 |largest logit|) half steps
    assert bool(((w.double() - p).abs() <= (40 + 4 * float(logits.abs().max())) * HALF[torch.float32] * p).all())
    order = torch.sort(want.reshape(-1), stable=True).indices
    assert torch.equal(prow.long(), order // k)
    assert torch.equal(e2p.long()[order], torch.arange(R * k, device=DEV))
    assert torch.equal(off.long(), torch.cat([off.new_zeros(1).long(), torch.bincount(want.reshape(-1), minlength=E).cumsum(0)]))
