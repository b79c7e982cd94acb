"""Every form of the 8-bit products on the GPU against binary64, at sizes that reach it
(tests/test_int8_forms.py holds them to that)."""

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from int8_helpers import DT, codes_in_64, gradient_check, held, rand, values_of
from tests import int8_forms as F

pytestmark = pytest.mark.gpu


def activations(rows, cols, seed, dtype):
    x = rand((rows, cols), seed, 1.0, dtype)
    x[:, ::97] *= 8
    x[rows // 2] = 0
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", sorted(F.FORWARD))
def test_forward(form, dtype):
    """The exact sum, rounded to fp32, and its two scalings are each off by half a step of
    binary32 at most, the result by half a step of its type."""
    M, N, K = F.FORWARD[form]
    x, w = activations(M, K, 5, dtype), rand((N, K), 6, 0.02, dtype)
    y = T.linear_int8(x, held(w))
    (qx, sx), (qw, sw) = codes_in_64(x), codes_in_64(w)
    exact = (qx.double() @ qw.double().t().contiguous()) * sx.double()[:, None] * sw.double()
    fi = torch.finfo(y.dtype)
    tol = exact.abs() * (fi.eps / 2 + 4 * 2.0 ** -24) + fi.smallest_normal * fi.eps
    bad = ~((y.double() - exact).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", sorted(F.GRADS))
def test_dx(form, dtype):
    R, C, S = F.GRADS[form]
    dy, w = rand((R, S), 1, 0.05, dtype), rand((S, C), 2, 0.02, dtype)
    gradient_check(T.gemm_int8_dx(dy, held(w)), dy, values_of(*codes_in_64(w), DT[dtype]))


@pytest.mark.parametrize("dtype,out", [("bf16", "16"), ("f16", "16"), ("f16", "f32"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("form", sorted(F.GRADS))
def test_dw(form, dtype, out):
    R, C, S = F.GRADS[form]
    dy, x = rand((S, R), 3, 0.05, dtype), activations(S, C, 4, dtype)
    dw = T.gemm_int8_dw(dy, held(x), dtype=torch.float32 if out == "f32" else None)
    gradient_check(dw, dy.t(), values_of(*codes_in_64(x), DT[dtype]))
