"""Infinities and NaN in an adapter: its own rows get what the formula gives in
64 bits (the signed infinity, or NaN where 0 x inf or inf - inf stands), whatever
the number of rows and the form of the product; the other rows are unchanged."""

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from tests import rows_forms as F
from tests.rows_helpers import check, device_plan, rand, stack
from tests.test_gpu_adapters import reference

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
BROKEN = F.ADAPTERS_BROKEN
# streaming forms of 16, 32 and 64 places, K in parts and whole; the tiled form
SIZES = [(3, 96, 192), (12, 96, 192), (12, 9001, 192), (12, 17000, 192), (25, 96, 192),
         (25, 17000, 192), (60, 96, 192), (60, 17000, 192), (BROKEN[0], BROKEN[3], BROKEN[4])]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_the_formula_decides(m, n, k, dtype):
    pool, rank = 3, 32
    ids = torch.arange(m) % pool
    q, w = stack(0, n, k, 41, "linear", "nf4", dtype)
    x = rand((m, k), 42, 1.0, dtype)
    a = rand((pool, rank, k), 43, 0.1, dtype)
    b = rand((pool, n, rank), 44, 0.3, dtype)
    # ranks whose X . A^T is a number of few bits, a zero, and infinite
    a[1, 0:3] = 0
    a[1, 0, 0], a[1, 1, 0] = 1.0, -0.5
    a[1, 3, 7] = INF
    x[:, 0] = torch.where(torch.arange(m) % 2 == 0, 2.0, -4.0).to(x)
    x[:, 7] = torch.where(torch.arange(m) % 4 < 2, 1.5, -0.25).to(x)
    # rows of B (output columns): what meets the infinite X . A^T is finite
    # there, of few bits or of many, or zero
    b[1, :, 3] = 0.5
    b[1, 10:20, 3] = rand((10,), 45, 0.3, dtype)
    b[1, 20, 3] = 0
    # an infinite B beside it; by turns of the same and of the other sign
    b[1, 30, 0], b[1, 31, 0] = INF, -INF
    b[1, 32, 2] = INF                                 # meets the zero
    b[1, 33, 5] = -INF                                # meets a number of many bits
    b[1, 34, 3] = -INF                                # meets the infinity
    b[1, 35, 6] = NAN
    # the second adapter has no infinite X . A^T: its other sums stay finite
    a[2, 0] = 0
    a[2, 0, 0] = 1.0
    a[2, 1] = 0
    b[2, 40, 0], b[2, 41, 0] = INF, -INF
    b[2, 42, 1] = INF                                 # meets a zero
    b[2, 43, 4], b[2, 43, 5] = INF, -INF
    b[2, 44, 6] = NAN
    b[2, 45, 7] = INF
    b[2, n - 1, 31] = -INF
    scale = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    print(f"infinite adapters M={m} N={n} K={k} {dtype}", flush=True)
    y = T.linear_adapters(x, q, device_plan(ids, pool), a, b, scale)
    torch.cuda.synchronize()
    exact = formula(x, w, ids, a, b, scale)
    compare(y, exact)
    fine = exact.isfinite().all(1).nonzero().flatten()
    assert fine.tolist() == [i for i in range(m) if i % 3 == 0]
    want, spread = reference(x[fine], w, ids[fine.cpu()], a, b, scale)
    check(y[fine], want, spread, k + rank)


def formula(x, w, ids, a, b, scale):
    """Y in binary64, an infinity or NaN wherever one takes part."""
    y = x.double() @ w.t().contiguous()
    for i, g in enumerate(ids.tolist()):
        low = (x[i].double() * a[g].double()).sum(1) * scale[g].double()
        y[i] += (low * b[g].double()).sum(1)
    return y


def compare(y, exact):
    got = y.double()
    for name, f in (("NaN", torch.isnan), ("+inf", lambda t: t == INF), ("-inf", lambda t: t == -INF)):
        off = (f(got) != f(exact)).nonzero()
        assert off.numel() == 0, (f"{name}: {off.shape[0]} elements differ, first at "
                                  f"{off[0].tolist()}: {got[tuple(off[0])].item()} for "
                                  f"{exact[tuple(off[0])].item()}")


@pytest.mark.parametrize("m,n,k", SIZES)
def test_an_infinite_term_beside_a_sum_past_fp16(m, n, k):
    """The finite part of Y lies beyond fp16's range, the infinite term on the
    other side of zero: the sum is the infinite term's."""
    q, w = stack(0, n, k, 51, "linear", "nf4", "f16")
    x = torch.zeros(m, k, dtype=torch.float16, device="cuda")
    x[:, 0] = 60000.0
    a = torch.zeros(1, 16, k, dtype=torch.float16, device="cuda")
    a[0, 0, 0], a[0, 1, 0] = 1.0, 1.0
    b = torch.zeros(1, n, 16, dtype=torch.float16, device="cuda")
    b[0, :, 0] = 4.0                                  # a term of 240000
    b[0, 5, 1] = -INF
    b[0, 7, 0], b[0, 7, 1] = -4.0, INF
    b[0, 9, 1], b[0, 9, 2] = -INF, INF                # -inf, and 0 x inf
    b[0, 11, 0], b[0, 11, 1] = -INF, INF
    ids = torch.zeros(m, dtype=torch.int32)
    scale = torch.ones(1, device="cuda")
    y = T.linear_adapters(x, q, device_plan(ids, 1), a, b, scale)
    torch.cuda.synchronize()
    exact = formula(x, w, ids, a, b, scale)
    assert (exact[:, 0] > 1e5).all() and exact[0, 5] == -INF and exact[0, 7] == INF
    assert torch.isnan(exact[0, 9]) and torch.isnan(exact[0, 11])
    compare(y, exact.half().double())                 # past fp16: infinite too
