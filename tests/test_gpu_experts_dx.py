"""bnbx_gemm_nf4_experts_dx (the input gradient of the expert-grouped product)
against binary64 products, element by element, and against differences of the
forward."""

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from tests.rows_helpers import DT, check, device_plan, product, rand, stack
from tests.test_gpu_experts import ids_of

pytestmark = pytest.mark.gpu


def run_case(counts, n, k, none=0, mode="scatter", dq="linear", quant="nf4", dtype="bf16", seed=1):
    groups = len(counts)
    plan = device_plan(ids_of(counts, seed, none), groups)
    rows = plan.rows
    q, w = stack(groups, n, k, seed + 1, dq, quant, dtype)
    dy = rand((rows, n), seed + 2, 0.3, dtype)
    out = torch.full((rows, k), 3.5, dtype=DT[dtype], device="cuda")
    print(f"experts_dx {counts} none={none} N={n} K={k} {mode} {dq} {quant} {dtype}", flush=True)
    dx = T.gemm_experts_dx(dy, q, plan, gather=1 if mode == "gather" else 0,
                           scatter=mode == "scatter", out=out)
    torch.cuda.synchronize()
    touched = torch.zeros(rows, dtype=torch.bool, device="cuda")
    off, order = plan.offsets.tolist(), plan.order.long()
    for g in range(groups):
        places = torch.arange(off[g], off[g + 1], device="cuda")
        if places.numel() == 0:
            continue
        yr = order[places] if mode == "gather" else places
        xr = order[places] if mode == "scatter" else places
        exact, spread = product(dy[yr], w[g].t())
        check(dx[xr], exact, spread, n, f"group {g}")
        touched[xr] = True
    assert torch.all(dx[~touched] == 3.5)


TYPES = [("linear", "nf4", "bf16"), ("linear", "fp4", "f16"), ("dynamic", "nf4", "f16"),
         (None, "fp4", "bf16"), (None, "nf4", "f16"), ("dynamic", "fp4", "bf16")]


@pytest.mark.parametrize("dq,quant,dtype", TYPES)
@pytest.mark.parametrize("counts,n,k", [
    ([1], 64, 64), ([1, 0, 1], 64, 128), ([3, 5, 0, 1], 128, 320), ([16, 16], 192, 256),
    ([17, 1, 15, 0, 33], 64, 576), ([64, 1], 320, 4160), ([40, 25], 1024, 192)])
def test_small(counts, n, k, dq, quant, dtype):
    run_case(counts, n, k, none=2, dq=dq, quant=quant, dtype=dtype)


@pytest.mark.parametrize("mode", ["gather", "scatter", "places"])
@pytest.mark.parametrize("counts,n,k,none", [
    ([2, 0, 0, 0, 7], 256, 704, 0), ([0, 0, 130, 0], 64, 192, 5), ([1] * 70, 128, 128, 3),
    ([0] * 199 + [9], 64, 256, 0), ([31, 0, 90, 200], 192, 64, 0), ([100, 3], 2112, 64, 7)])
def test_layouts(mode, counts, n, k, none):
    run_case(counts, n, k, none=none, mode=mode)


@pytest.mark.parametrize("counts,n,k", [
    ([1, 1], 4096, 4096), ([2] * 8, 4096, 1024), ([9] * 4, 1088, 2048), ([20] * 8, 640, 2048),
    ([300, 20, 0, 77], 512, 1024), ([130] * 3, 11008, 320), ([1000, 24], 768, 512),
    ([257, 255, 256], 640, 320)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_larger(counts, n, k, dtype):
    run_case(counts, n, k, none=1, dtype=dtype)


def test_most_groups():
    """1024 groups: tiles found past the first 64 groups, several in some."""
    run_case([2, 0, 0, 1] * 128 + [0] * 500 + [40] * 11 + [3], 64, 128, none=9)


def test_against_differences_of_the_forward():
    """d/dx <dy, f(x)> along single inputs of a row: the forward is linear, so
    the difference of two forwards a unit apart, in binary64 over its 16-bit
    rows, equals the gradient up to the roundings of both."""
    counts, n, k = [5, 0, 12], 128, 192
    plan = device_plan(ids_of(counts, 31), 3)
    q, w = stack(3, n, k, 32, None, "nf4", "f16")
    dy = rand((17, n), 33, 1.0, "f16")
    dx = T.gemm_experts_dx(dy, q, plan)
    for col in (0, 63, 64, k - 1):
        x = torch.zeros(17, k, dtype=torch.float16, device="cuda")
        x[:, col] = 1.0
        up = T.gemm_experts(x, q, plan).double()
        down = T.gemm_experts(-x, q, plan).double()
        torch.cuda.synchronize()
        terms = dy.double() * (up - down) / 2
        diff = terms.sum(1)
        # the forward's rows here are single weights (exact); dx rounds once
        tol = 2.0 ** -11 * diff.abs() * (1 + 2.0 ** -6) + 2.0 ** -20 * terms.square().sum(1).sqrt()
        assert torch.all((dx[:, col].double() - diff).abs() <= tol)


def test_strided_rows_and_guards():
    counts, n, k = [5, 20, 0, 3], 128, 192
    plan = device_plan(ids_of(counts, 3), 4)
    q, _ = stack(4, n, k, 9)
    ybig = torch.full((28, n + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    ybig[:, 8:8 + n] = rand((28, n), 10)
    xbig = torch.full((32, k + 11), 9.0, dtype=torch.bfloat16, device="cuda")
    T.gemm_experts_dx(ybig[:, 8:8 + n], q, plan, scatter=True, out=xbig[2:30, 5:5 + k])
    ref = T.gemm_experts_dx(ybig[:, 8:8 + n].contiguous(), q, plan, scatter=True)
    torch.cuda.synchronize()
    assert torch.equal(xbig[2:30, 5:5 + k], ref)
    xbig[2:30, 5:5 + k] = 9.0
    assert torch.all(xbig == 9.0)


def test_infinite_rows_stay_their_own():
    plan = device_plan([0] * 6 + [1] * 30, 2)
    q, w = stack(2, 64, 192, 12)
    dy = rand((36, 64), 13)
    dy[2, 5] = float("inf")
    dy[3, :] = float("nan")
    dy[20, 63] = float("-inf")
    dx = T.gemm_experts_dx(dy, q, plan)
    torch.cuda.synchronize()
    clean = torch.tensor([i for i in range(36) if i not in (2, 3, 20)], device="cuda")
    for g, lo, hi in ((0, 0, 6), (1, 6, 36)):
        rows = clean[(clean >= lo) & (clean < hi)]
        exact, spread = product(dy[rows], w[g].t())
        check(dx[rows], exact, spread, 64)
    assert torch.isnan(dx[3]).all() and not torch.isfinite(dx[2][w[0][5] != 0]).any()


def test_a_wrong_plan_stays_inside_the_buffers():
    q, w = stack(2, 64, 128, 15)
    dy = rand((5, 64), 16)
    plan = T.RowGroups(2, torch.tensor([-5, 3, 99], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, -7, 2, 2**31 - 1, 3], dtype=torch.int32, device="cuda"))
    big = torch.full((9, 128), 8.0, dtype=torch.bfloat16, device="cuda")
    T.gemm_experts_dx(dy, q, plan, gather=1, scatter=True, out=big[2:7])
    torch.cuda.synchronize()
    for row, g in ((0, 0), (2, 0), (3, 1)):
        exact, spread = product(dy[row:row + 1], w[g].t())
        check(big[2 + row:3 + row], exact, spread, 64)
    assert torch.all(big[[0, 1, 3, 6, 7, 8]] == 8.0)


def test_no_rows_and_rows_of_no_group():
    q, _ = stack(3, 64, 128, 5)
    assert T.gemm_experts_dx(rand((0, 64), 6), q, device_plan([], 3)).shape == (0, 128)
    out = torch.full((3, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    T.gemm_experts_dx(rand((3, 64), 6), q, device_plan([-1, -1, 7], 3), out=out)
    torch.cuda.synchronize()
    assert torch.all(out == 2.0)


def test_captured_and_replayed_with_new_plans():
    groups, rows, n, k = 4, 50, 192, 512
    q, w = stack(groups, n, k, 21)
    dy = rand((rows, n), 22)
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    plan = T.empty_row_groups(rows, groups)
    dx = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    T.group_rows(ids, groups, out=plan)
    T.gemm_experts_dx(dy, q, plan, gather=1, scatter=True, out=dx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        T.group_rows(ids, groups, out=plan)
        T.gemm_experts_dx(dy, q, plan, gather=1, scatter=True, out=dx)
    for rep in range(4):
        g = torch.Generator().manual_seed(rep)
        ids.copy_(torch.randint(-1, groups, (rows,), generator=g, dtype=torch.int32))
        dx.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for e in range(groups):
            sel = ids == e
            if sel.any():
                exact, spread = product(dy[sel], w[e].t())
                check(dx[sel], exact, spread, n, f"replay {rep}")
        assert torch.all(dx[ids < 0] == 1.0)
        T.gemm_experts_dx(dy, q, plan, gather=1)
        torch.cuda.synchronize()
