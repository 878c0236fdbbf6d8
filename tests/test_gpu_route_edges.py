"""GPU tests of mhc_moe_route where its fp32 choices and the 64-bit definition part:
groups whose values carry unlike errors or leave fp32's range, scores below it."""

import numpy as np
import pytest
import torch

import oracle as O
from mhc_residual_stream_b200 import mhc as M

from _sublayer import DEV, f64, gen, run_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mhc_residual_stream_b200 import build
    build.build()
    M.lib()
    yield


def ids_agree(logits, k, bias, **kw):
    got = run_route(logits.to(DEV), k, bias.to(DEV), **kw)
    w, ids, e2p, prow, off = [t.cpu() for t in got]
    ow, oids = O.moe_route(f64(logits), k, f64(bias), **kw)
    wrong = (ids.numpy() != oids).any(1)
    assert not wrong.any(), f"{wrong.sum()} of {len(wrong)} rows, the first is {np.argwhere(wrong)[0, 0]}"
    for a, b in zip((e2p, prow, off), O.moe_permute(oids, logits.shape[1])):
        assert np.array_equal(a.numpy(), b)
    return f64(w), ow


@pytest.mark.parametrize("top_groups", [1, 2, 3])
@pytest.mark.parametrize("size", [32.0, 128.0, 1000.0])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_a_group_that_cancels_among_groups_that_do_not(scoring, size, top_groups):
    # four nearly equal groups, one of them the sum of +size and -size: its value in fp32 is
    # off by a step of `size`, the others' by a step of one, and it may stand at any rank
    R, G, S = 1500, 4, 2
    for cancels in (0, 3):
        logits = 1.0 + 1e-5 * torch.randn(R, G * S, generator=gen(int(size) + cancels))
        bias = torch.zeros(G * S)
        bias[cancels * S], bias[cancels * S + 1] = size, -size
        ids_agree(logits, 2, bias, scoring=scoring, num_groups=G, top_groups=top_groups, group_top=2)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_group_values_outside_the_range_of_fp32(sign):
    R, G, S = 20, 4, 3
    logits = torch.randn(R, G * S, generator=gen(3))
    bias = sign * torch.tensor([3.0e38, 3.2e38, 2.8e38, 3.1e38]).repeat_interleave(S)
    for tg in (1, 2, 3):
        ids_agree(logits, 3, bias, scoring="sigmoid", num_groups=G, top_groups=tg, group_top=2)
    bias[:S] = 0.0  # one group within it
    ids_agree(logits, 3, bias, scoring="sigmoid", num_groups=G, top_groups=2, group_top=2)


def test_weights_of_scores_that_only_subnormals_hold():
    # sigmoid scores of exp(-735) .. exp(-705): below exp(-708) subnormal in 64 bits, 2^-1074
    # apart, and 1 / (1 + exp(-l)) is 0 there although the score is not
    R, E, k = 40, 12, 4
    logits = -705.0 - 30.0 * torch.rand(R, E, generator=gen(5))
    got = run_route(logits.to(DEV), k, scoring="sigmoid")
    ow, oids = O.moe_route(f64(logits), k, scoring="sigmoid")
    w, ids = f64(got[0]), got[1].cpu().numpy()
    assert np.array_equal(ids, oids)
    chosen = np.take_along_axis(f64(logits), oids, 1)
    exact = np.exp(chosen - chosen.max(1, keepdims=True))
    exact /= exact.sum(1, keepdims=True)
    spacing = 2.0 ** -1074 / np.exp(chosen.max(1, keepdims=True))  # of a score, relative to the largest
    # each score is off by half a spacing at most, the sum by k of them; one rounding to fp32
    assert np.all(np.abs(w - exact) <= (k + 1) * spacing + 2.0 ** -23 * exact + 2.0 ** -126)
    assert np.all(np.abs(ow - exact) <= (k + 1) * spacing + 2.0 ** -40)


@pytest.mark.parametrize("top", [-45.0, -20.0, -1.0, 3.0])
@pytest.mark.parametrize("renormalize", [False, True])
def test_sigmoid_weights_far_below_the_largest(top, renormalize):
    # all experts are chosen; scores down to e^-120 under a largest one of e^-45 or more: ratios
    # that are ordinary fp32 numbers although e^120 and e^-120 are none
    R, E = 60, 8
    logits = top - 85.0 * torch.rand(R, E, generator=gen(int(top) + 99))
    logits[:, 3] = top
    got = run_route(logits.to(DEV), E, scoring="sigmoid", renormalize=renormalize, weight_scale=2.5)
    ow, oids = O.moe_route(f64(logits), E, scoring="sigmoid", renormalize=renormalize, weight_scale=2.5)
    assert np.array_equal(got[1].cpu().numpy(), oids)
    # two exponentials (2 steps each) of arguments off by half a step of at most 130, two
    # divisions, a sum of 8 and the scale; where the weight is subnormal, its spacing
    rel = (40 + 4 * 130) * 2.0 ** -24
    assert np.all(np.abs(f64(got[0]) - ow) <= rel * np.abs(ow) + 2.0 ** -126)
