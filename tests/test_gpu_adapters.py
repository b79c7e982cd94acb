"""bnbx_gemm_nf4_adapters (one 4-bit weight beside the adapters of many
requests) against binary64 products, element by element."""

import math

import pytest
import torch

import dequant_gemm_nf4_amd as bnbx
from dequant_gemm_nf4_amd import tensors as T
from tests.rows_helpers import DT, check, device_plan, product, rand, stack

pytestmark = pytest.mark.gpu


def reference(x, w, ids, a, b, scale):
    """Exact Y, and the 2-norm of its products with the adapter's term counted
    through the fp32 sum X . A^T (its error reaches Y times |B|) and that sum's
    16 bits: 2^-17 of it, 2^7 steps of the fp32 unit."""
    y, spread = product(x, w)
    for g in set(i for i in ids.tolist() if 0 <= i < a.shape[0]):
        rows = (ids == g).nonzero().flatten().to(x.device)
        low, low_spread = product(x[rows], a[g])
        up, _ = product(low * scale[g].double(), b[g])
        y[rows] += up
        mag = (low.abs() * 2.0 ** 7 / (16 * math.sqrt(x.shape[1])) + low_spread) \
            * scale[g].double().abs()
        spread[rows] += (mag.square() @ b[g].double().square().t().contiguous()).sqrt()
        spread[rows] += ((low * scale[g].double()).square()
                         @ b[g].double().square().t().contiguous()).sqrt()
    return y, spread


def run_case(ids, adapters, rank, n, k, dq="linear", quant="nf4", dtype="bf16", seed=1):
    ids = torch.as_tensor(ids, dtype=torch.int32)
    m = ids.numel()
    plan = device_plan(ids, adapters)
    q, w = stack(0, n, k, seed, dq, quant, dtype)
    x = rand((m, k), seed + 1, 1.0, dtype)
    a = rand((adapters, rank, k), seed + 2, 1 / math.sqrt(k), dtype)
    b = rand((adapters, n, rank), seed + 3, 0.3, dtype)
    scale = (torch.rand(adapters, generator=torch.Generator().manual_seed(seed)) + 0.5).cuda()
    print(f"adapters M={m} L={adapters} r={rank} N={n} K={k} {dq} {quant} {dtype}", flush=True)
    y = T.linear_adapters(x, q, plan, a, b, scale)
    torch.cuda.synchronize()
    exact, spread = reference(x, w, ids, a, b, scale)
    check(y, exact, spread, k + rank)
    # rows of no adapter get the 4-bit product; the others' term is not lost
    plain, _ = product(x, w)
    own = (ids >= 0) & (ids < adapters)
    if own.any():
        rows = own.nonzero().flatten().cuda()
        assert ((plain - exact)[rows].norm() / exact[rows].norm()) > 0.05


def random_ids(m, adapters, seed, run=1, none=0.2):
    g = torch.Generator().manual_seed(seed)
    which = torch.cumsum((torch.rand(m, generator=g) < 1 / run).int(), 0)
    pick = torch.randint(0, adapters, (m + 1,), generator=g)
    pick[torch.rand(m + 1, generator=g) < none] = -1
    return pick[which]


TYPES = [("linear", "nf4", "bf16"), ("linear", "fp4", "f16"), ("dynamic", "nf4", "f16"),
         (None, "fp4", "bf16"), (None, "nf4", "f16"), ("dynamic", "fp4", "bf16")]


@pytest.mark.parametrize("dq,quant,dtype", TYPES)
@pytest.mark.parametrize("m,adapters,rank,n,k", [
    (1, 1, 16, 16, 64), (1, 5, 64, 100, 320), (4, 4, 32, 65, 128), (16, 20, 48, 130, 1088),
    (17, 3, 80, 64, 576), (40, 9, 256, 200, 192), (70, 2, 16, 33, 4160), (130, 70, 144, 96, 256)])
def test_small(m, adapters, rank, n, k, dq, quant, dtype):
    run_case(random_ids(m, adapters, m + rank, none=0.2 if m > 1 else 0), adapters, rank, n, k,
             dq, quant, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,adapters,rank,n,k,run", [
    (1, 3, 16, 4096, 4096, 1), (16, 16, 64, 4096, 4096, 1), (64, 8, 16, 2048, 4096, 8),
    (333, 12, 48, 1000, 2048, 40), (600, 3, 64, 520, 1024, 100), (1030, 1, 128, 260, 512, 2000),
    (2048, 5, 32, 768, 1024, 500), (300, 40, 256, 300, 11008, 3)])
def test_larger(m, adapters, rank, n, k, run, dtype):
    run_case(random_ids(m, adapters, m + n, run), adapters, rank, n, k, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,rank,n,k", [
    (7, 48, 9000, 320), (7, 48, 15000, 1088), (12, 16, 30000, 256), (12, 80, 60000, 320),
    (25, 48, 5000, 1088), (25, 80, 13000, 576), (25, 48, 25000, 256), (25, 16, 50000, 320),
    (60, 80, 6000, 320), (60, 48, 13000, 576), (60, 48, 30000, 256)])
def test_wide(m, rank, n, k, dtype):
    """Many weight rows: the ranks shared out over one to eight waves."""
    run_case(random_ids(m, 6, m + n), 6, rank, n, k, dtype=dtype)


@pytest.mark.parametrize("m", [3, 50, 700])
def test_one_adapter_for_all_and_none_at_all(m):
    run_case([0] * m, 1, 32, 200, 256)
    run_case([2] * m, 4, 32, 200, 256)
    run_case([-1] * m, 4, 32, 200, 256)


def test_rows_alternate_between_all_adapters():
    run_case([i % 64 for i in range(640)], 64, 16, 300, 512)


def test_most_adapters():
    """1024 adapters, most without a row."""
    run_case(random_ids(300, 1024, 51), 1024, 16, 48, 128)


def test_no_rows():
    q, _ = stack(0, 64, 128, 5)
    y = T.linear_adapters(rand((0, 128), 1), q, device_plan([], 2), rand((2, 16, 128), 2),
                          rand((2, 64, 16), 3), torch.ones(2, device="cuda"))
    assert y.shape == (0, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [9, 60, 600])
def test_a_broken_adapter_stays_its_own(m, dtype):
    """NaN and infinities in one adapter, and in one row of X, do not reach the
    rows of others (in one row tile, in one matrix-core product)."""
    n, k, rank = 96, 192, 32
    ids = torch.arange(m) % 3
    plan = device_plan(ids, 3)
    q, w = stack(0, n, k, 41, "linear", "nf4", dtype)
    x = rand((m, k), 42, 1.0, dtype)
    a = rand((3, rank, k), 43, 0.1, dtype)
    b = rand((3, n, rank), 44, 0.3, dtype)
    a[1, 3, 7] = float("inf")
    b[1, 5, :] = float("nan")
    b[1, 6, 2] = float("-inf")
    x[2, 1] = float("nan")
    scale = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    y = T.linear_adapters(x, q, plan, a, b, scale)
    torch.cuda.synchronize()
    good = torch.tensor([i for i in range(m) if i % 3 != 1 and i != 2])
    exact, spread = reference(x[good.cuda()], w, ids[good], a, b, scale)
    check(y[good.cuda()], exact, spread, k + rank)
    bad = torch.tensor([i for i in range(m) if i % 3 == 1]).cuda()
    assert not torch.isfinite(y[bad]).any()
    assert torch.isnan(y[2]).all()


def test_large_terms_in_fp16_do_not_overflow_on_the_way():
    """X . A^T beyond fp16's range with small B: the term itself fits."""
    m, n, k, rank = 20, 64, 256, 16
    q, w = stack(0, n, k, 51, "linear", "nf4", "f16")
    x = rand((m, k), 52, 100.0, "f16")
    a = rand((1, rank, k), 53, 100.0, "f16")
    b = rand((1, n, rank), 54, 1e-4, "f16")
    scale = torch.ones(1, device="cuda")
    ids = torch.zeros(m, dtype=torch.int32)
    y = T.linear_adapters(x, q, device_plan(ids, 1), a, b, scale)
    torch.cuda.synchronize()
    assert (x.double() @ a[0].double().t().contiguous()).abs().max() > 65504 * 2
    exact, spread = reference(x, w, ids, a, b, scale)
    check(y, exact, spread, k + rank)


def test_strided_pool_of_adapters_and_guards():
    """Adapters inside a wider pool (a slice of slots, padded rows), x and y
    inside wider buffers."""
    m, n, k, rank = 21, 70, 192, 32
    ids = random_ids(m, 3, 61)
    plan = device_plan(ids, 3)
    q, _ = stack(0, n, k, 62)
    nan = float("nan")
    pa = torch.full((5, rank + 16, k + 8), nan, dtype=torch.bfloat16, device="cuda")
    pb = torch.full((5, n + 3, rank + 24), nan, dtype=torch.bfloat16, device="cuda")
    pa[1:4, 16:, :k] = rand((3, rank, k), 63, 0.07)
    pb[1:4, :n, 8:8 + rank] = rand((3, n, rank), 64, 0.3)
    a, b = pa[1:4, 16:, :k], pb[1:4, :n, 8:8 + rank]
    scale = torch.rand(3, device="cuda")
    xbig = torch.full((m, k + 72), nan, dtype=torch.bfloat16, device="cuda")
    xbig[:, 8:8 + k] = rand((m, k), 65)
    ybig = torch.full((m + 4, n + 11), 9.0, dtype=torch.bfloat16, device="cuda")
    T.linear_adapters(xbig[:, 8:8 + k], q, plan, a, b, scale, out=ybig[2:2 + m, 5:5 + n])
    ref = T.linear_adapters(xbig[:, 8:8 + k].contiguous(), q, plan, a.contiguous(), b.contiguous(),
                            scale)
    torch.cuda.synchronize()
    assert torch.equal(ybig[2:2 + m, 5:5 + n], ref)
    ybig[2:2 + m, 5:5 + n] = 9.0
    assert torch.all(ybig == 9.0)


def test_repeats_and_workspace_contents_do_not_matter():
    m, n, k, rank = 100, 300, 1024, 64
    plan = device_plan(random_ids(m, 9, 71), 9)
    q, _ = stack(0, n, k, 72)
    args = (rand((m, k), 73), q, plan, rand((9, rank, k), 74, 0.03), rand((9, n, rank), 75, 0.3),
            torch.rand(9, device="cuda"))
    ws = torch.empty(bnbx.bnbx_gemm_nf4_adapters_workspace_bytes(m, rank), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)
    a = T.linear_adapters(*args, workspace=ws)
    ws.fill_(0x11)
    b = T.linear_adapters(*args, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    with pytest.raises(bnbx.BnbxError) as e:
        T.linear_adapters(*args, workspace=ws[:-16])
    assert e.value.status == bnbx.BNBX_E_WORKSPACE


def test_captured_and_replayed_with_new_requests():
    m, n, k, rank, adapters = 40, 200, 512, 32, 6
    q, w = stack(0, n, k, 81)
    x = rand((m, k), 82)
    a, b = rand((adapters, rank, k), 83, 0.05), rand((adapters, n, rank), 84, 0.3)
    scale = torch.rand(adapters, device="cuda") + 0.5
    ids = torch.zeros(m, dtype=torch.int32, device="cuda")
    plan = T.empty_row_groups(m, adapters)
    y = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(bnbx.bnbx_gemm_nf4_adapters_workspace_bytes(m, rank), dtype=torch.uint8,
                     device="cuda")

    def path():
        T.group_rows(ids, adapters, out=plan)
        T.linear_adapters(x, q, plan, a, b, scale, out=y, workspace=ws)

    path()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        path()
    for rep in range(4):
        new = random_ids(m, adapters, 90 + rep)
        ids.copy_(new)
        ws.fill_(0xFF)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        exact, spread = reference(x, w, new, a, b, scale)
        check(y, exact, spread, k + rank, f"replay {rep}")
        path()
        torch.cuda.synchronize()
