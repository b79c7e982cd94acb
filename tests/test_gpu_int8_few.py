"""The 8-bit layer for one to four rows (decode)."""

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from int8_helpers import codes_in_64, held, rand
from tests import int8_forms as F

pytestmark = pytest.mark.gpu


def few_check(x, wq, codes, scale, where=""):
    """The layer in its three forms (the codes kept or not, or given) against the exact
    integer sums: the sum, rounded to fp32, and its two scalings are each off by half a
    step of binary32 at most, the result by half a step of its type."""
    (M, K), dtype = x.shape, x.dtype
    qx, sx = codes_in_64(x)
    exact = (qx.double() @ codes.double().t().contiguous()) * sx.double()[:, None] * scale.double()
    fi = torch.finfo(dtype)
    tol = exact.abs() * (fi.eps / 2 + 4 * 2.0 ** -24) + fi.smallest_normal * fi.eps
    saved = T.empty_int8_rows((M, K), dtype)
    y = T.linear_int8(x, wq)
    bad = ~((y.double() - exact).abs() <= tol)
    assert not bad.any(), (where, int(bad.sum()), bad.nonzero()[0].tolist())
    assert torch.equal(T.linear_int8(x, wq, saved=saved), y), where
    assert torch.equal(saved.codes[:, :K].long(), qx) and torch.equal(saved.scale, sx), where
    assert not saved.codes[:, K:].any(), where
    assert torch.equal(T.gemm_int8(saved, wq), y), where


@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K", [(4096, 14336), (2048, 1024), (131072, 16)])
def test_a_weight_that_ends_with_its_pages(M, N, K):
    """Codes of whole 2 MiB; K is no whole number of a wave's 4 KB."""
    torch.cuda.empty_cache()
    wq = held(rand((N, K), 1, 0.02))
    assert wq.codes.untyped_storage().nbytes() % 2**21 == 0
    few_check(rand((M, K), 2), wq, wq.codes[:, :K], wq.scale, (M, N, K))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", [40, 4096, 4100, 9000])
@pytest.mark.parametrize("N", sorted(F.FEW))
@pytest.mark.parametrize("M", [2, 3, 4])
def test_several_rows_of_w_a_wave(M, N, K, dtype):
    """(tests/test_int8_forms.py holds N to its rows a wave.)  One, two and three batches of
    loads a row, so that the two sets of registers change places within rows and between
    them; a last wave whose rows end past N."""
    wq = held(rand((N, K), N + K, 0.02, dtype), spare=16)
    x = rand((M, K), M + K, 1.0, dtype)
    x[:, ::97] *= 8
    few_check(x, wq, wq.codes[:, :K], wq.scale, (M, N, K))
