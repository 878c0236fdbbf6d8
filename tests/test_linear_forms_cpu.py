"""The forms that mhc_linear chooses between, and the tests' products that reach them."""

import ctypes
import math
import random

import pytest

from mhc_residual_stream_b200 import build
from mhc_residual_stream_b200 import mhc as M

from _forms import MORE_FORMS
from test_gpu_sublayer import FORMS


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    M.lib()
    yield


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def test_every_form_has_a_tested_product():
    tested = {(*kind, *M.mhc_debug_linear_form(R, K, N, *kind)[:3]) for kind, v in FORMS.items() for R, K, N in v}
    for kind, v in MORE_FORMS.items():
        for R, K, N, form in v:
            assert M.mhc_debug_linear_form(R, K, N, *kind)[:3] == form, (kind, R, K, N)
            tested.add((*kind, *form))
    rng = random.Random(7)
    for _ in range(60000):
        fp8, gated = rng.random() < 0.5, rng.random() < 0.5
        R, K, N = spread(rng, 1, 4096), spread(rng, 1, 2048) * (32 if fp8 else 8), spread(rng, 1, 20000)
        if fp8 and gated:
            N = -(-N // 128) * 128
        if K > 65536:
            continue
        form = M.mhc_debug_linear_form(R, K, N, fp8, gated)
        assert (fp8, gated, *form[:3]) in tested, (fp8, gated, R, K, N, form)
        assert form[3] % 16 == 0 and 16 <= form[3] <= 256 and (not form[0] or form[1:3] == (1, 1))


def test_form_refusals():
    form = (ctypes.c_int * 4)()
    for a in ((0, 64, 64, 0, 0), (1, 60, 64, 0, 0), (1, 48, 64, 1, 0), (1, 64, 64, 1, 1), (1, 64, 0, 0, 0)):
        assert M.lib().mhc_debug_linear_form(*a, form) == M.UNSUPPORTED_SHAPE, a
    assert M.lib().mhc_debug_linear_form(1, 64, 64, 0, 0, None) == M.INVALID_ARG
    with pytest.raises(M.MhcError):
        M.mhc_debug_linear_form(1, 60, 64)
