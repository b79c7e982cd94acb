"""The tiled kernels over grouped rows (many rows and many columns a call):
the products, the input gradient and the adapters against binary64, element by
element.  The sizes are those of tests/rows_forms.py, where a host test holds
that the library takes the tiled form for them."""

import dataclasses

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from tests import rows_forms as F
from tests import test_gpu_adapters as adapters
from tests import test_gpu_experts as experts
from tests import test_gpu_experts_dx as experts_dx
from tests.rows_helpers import check, device_plan, product, rand, stack

pytestmark = pytest.mark.gpu

TYPES = experts.TYPES


@pytest.mark.parametrize("dq,quant,dtype", TYPES)
@pytest.mark.parametrize("counts,n,k", F.EXPERTS)
def test_experts(counts, n, k, dq, quant, dtype):
    experts.run_case(counts, n, k, none=1, dq=dq, quant=quant, dtype=dtype)


@pytest.mark.parametrize("mode,topk", [("gather", 1), ("gather", 3), ("scatter", 1), ("places", 1)])
def test_experts_layouts(mode, topk):
    counts, n, k = F.EXPERTS_LAYOUT
    experts.run_case(counts, n, k, none=6, mode=mode, topk=topk)


@pytest.mark.parametrize("dq,quant,dtype", TYPES)
@pytest.mark.parametrize("counts,n,k", F.DX)
def test_experts_dx(counts, n, k, dq, quant, dtype):
    experts_dx.run_case(counts, n, k, none=1, dq=dq, quant=quant, dtype=dtype)


@pytest.mark.parametrize("mode", ["gather", "scatter", "places"])
def test_experts_dx_layouts(mode):
    counts, n, k = F.DX_LAYOUT
    experts_dx.run_case(counts, n, k, none=6, mode=mode)


@pytest.mark.parametrize("dq,quant,dtype", TYPES)
@pytest.mark.parametrize("m,pool,rank,n,k", F.ADAPTERS)
def test_adapters(m, pool, rank, n, k, dq, quant, dtype):
    ids = adapters.random_ids(m, pool, m + rank, run=1 if pool > 100 else 60)
    adapters.run_case(ids, pool, rank, n, k, dq, quant, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_hundreds_of_adapters_in_one_tile(dtype):
    """All but one of the adapters with a single row."""
    m, pool, rank, n, k = F.ADAPTERS[-1]
    ids = torch.zeros(m, dtype=torch.int64)
    ids[torch.randperm(m, generator=torch.Generator().manual_seed(1))[:pool - 1]] = \
        torch.arange(1, pool)
    adapters.run_case(ids, pool, rank, n, k, dtype=dtype)


@pytest.mark.parametrize("dq", ["linear", "dynamic", None])
def test_block_scales_at_any_address(dq):
    """Block codes and maxima that start at an element's own alignment only."""
    q, _ = stack(2, 9001, 256, 41, dq)
    plan = device_plan(experts.ids_of([600, 1], 42), 2)
    x = rand((601, 256), 43)
    ref = T.gemm_experts(x, q, plan)
    odd = torch.cat((q.absmax[:1], q.absmax))[1:]
    y = T.gemm_experts(x, dataclasses.replace(q, absmax=odd), plan)
    torch.cuda.synchronize()
    assert torch.equal(y, ref)


@pytest.mark.parametrize("fn", ["forward", "dx"])
def test_strided_rows_and_guards(fn):
    counts, n, k = F.EXPERTS_LAYOUT if fn == "forward" else F.DX_LAYOUT
    run, win, wout = ((T.gemm_experts, k, n) if fn == "forward" else (T.gemm_experts_dx, n, k))
    rows = sum(counts)
    plan = device_plan(experts.ids_of(counts, 3), 4)
    q, _ = stack(4, n, k, 9)
    xbig = torch.full((rows, win + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    xbig[:, 8:8 + win] = rand((rows, win), 10)
    ybig = torch.full((rows + 4, wout + 11), 9.0, dtype=torch.bfloat16, device="cuda")
    run(xbig[:, 8:8 + win], q, plan, gather=1, scatter=True, out=ybig[2:2 + rows, 5:5 + wout])
    ref = run(xbig[:, 8:8 + win].contiguous(), q, plan, gather=1, scatter=True)
    torch.cuda.synchronize()
    assert torch.equal(ybig[2:2 + rows, 5:5 + wout], ref)
    ybig[2:2 + rows, 5:5 + wout] = 9.0
    assert torch.all(ybig == 9.0)


@pytest.mark.parametrize("fn", ["forward", "dx"])
def test_infinite_rows_stay_their_own(fn):
    (counts, n, k), run = ((F.EXPERTS_LAYOUT, T.gemm_experts) if fn == "forward" else
                           (F.DX_LAYOUT, T.gemm_experts_dx))
    width = k if fn == "forward" else n
    rows = sum(counts)
    plan = device_plan([g for g, c in enumerate(counts) for _ in range(c)], 4)
    q, w = stack(4, n, k, 12)
    if fn == "dx":
        w = w.transpose(1, 2)
    x = rand((rows, width), 13)
    odd = {2: (5, 1.0), 300: (width - 1, -1.0), 450: (0, 1.0)}
    for i, (col, sign) in odd.items():
        x[i, col] = sign * float("inf")
    x[3, :] = float("nan")
    y = run(x, q, plan)
    torch.cuda.synchronize()
    at = 0
    for g, c in enumerate(counts):
        sel = [i for i in range(at, at + c) if i not in odd and i != 3]
        at += c
        if sel:
            exact, spread = product(x[sel], w[g])
            check(y[sel], exact, spread, width)
    for i, (col, sign) in odd.items():
        g = plan_group(counts, i)
        want = w[g][:, col] * sign
        hit = want != 0
        assert torch.equal(y[i][hit].double(), torch.sign(want[hit]) * float("inf"))
    assert torch.isnan(y[3]).all()


def plan_group(counts, row):
    g = 0
    while row >= counts[g]:
        row -= counts[g]
        g += 1
    return g


@pytest.mark.parametrize("fn", ["forward", "dx"])
def test_a_wrong_plan_stays_inside_the_buffers(fn):
    """Rows outside X or Y are left out; bounds are clamped to the plan."""
    n, k = (9001, 64) if fn == "forward" else (64, 8192)
    run, win, wout = ((T.gemm_experts, k, n) if fn == "forward" else (T.gemm_experts_dx, n, k))
    rows = 700
    q, w = stack(2, n, k, 15)
    x = rand((rows, win), 16)
    order = torch.arange(rows, dtype=torch.int32)
    bad = [1, 77, 300, 511, 699]
    order[bad] = torch.tensor([-7, 2**31 - 1, rows, -2**31, 10**6], dtype=torch.int32)
    plan = T.RowGroups(2, torch.tensor([-5, 350, 10**6], dtype=torch.int32, device="cuda"),
                       order.cuda())
    big = torch.full((rows + 4, wout), 8.0, dtype=torch.bfloat16, device="cuda")
    run(x, q, plan, gather=1, scatter=True, out=big[2:2 + rows])
    torch.cuda.synchronize()
    good = [i for i in range(rows) if i not in bad]
    for g in (0, 1):
        sel = [i for i in good if (i >= 350) == bool(g)]
        exact, spread = product(x[sel], w[g] if fn == "forward" else w[g].t())
        check(big[2:2 + rows][sel], exact, spread, win)
    assert torch.all(big[[0, 1, rows + 2, rows + 3] + [2 + i for i in bad]] == 8.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_broken_adapter_stays_its_own(dtype):
    m, pool, rank, n, k = F.ADAPTERS_BROKEN
    ids = torch.arange(m) % 3
    q, w = stack(0, n, k, 41, "linear", "nf4", dtype)
    x = rand((m, k), 42, 1.0, dtype)
    a = rand((pool, rank, k), 43, 0.1, dtype)
    b = rand((pool, n, rank), 44, 0.3, dtype)
    a[1, 3, 7] = float("inf")
    b[1, 5, :] = float("nan")
    b[1, 6, 2] = float("-inf")
    x[2, 1] = float("nan")
    scale = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    y = T.linear_adapters(x, q, device_plan(ids, pool), a, b, scale)
    torch.cuda.synchronize()
    good = torch.tensor([i for i in range(m) if i % 3 != 1 and i != 2])
    exact, spread = adapters.reference(x[good.cuda()], w, ids[good], a, b, scale)
    check(y[good.cuda()], exact, spread, k + rank)
    assert not torch.isfinite(y[[i for i in range(m) if i % 3 == 1]]).any()
    assert torch.isnan(y[2]).all()


@pytest.mark.parametrize("op", ["experts", "experts_dx", "adapters"])
def test_captured_and_replayed_with_new_plans(op):
    counts, n, k = F.DX_LAYOUT if op == "experts_dx" else F.EXPERTS_LAYOUT
    rows, groups = F.ADAPTERS_BROKEN[0] if op == "adapters" else 700, 3
    q, w = stack(0 if op == "adapters" else groups, n, k, 21)
    width = n if op == "experts_dx" else k
    x = rand((rows, width), 22)
    a, b = rand((groups, 32, k), 23, 0.05), rand((groups, n, 32), 24, 0.3)
    scale = torch.rand(groups, device="cuda") + 0.5
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    plan = T.empty_row_groups(rows, groups)
    y = torch.zeros(rows, k if op == "experts_dx" else n, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(rows * 4 * 32, dtype=torch.uint8, device="cuda")

    def path():
        T.group_rows(ids, groups, out=plan)
        if op == "adapters":
            T.linear_adapters(x, q, plan, a, b, scale, out=y, workspace=ws)
        else:
            fn = T.gemm_experts if op == "experts" else T.gemm_experts_dx
            fn(x, q, plan, gather=1, scatter=True, out=y)

    path()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        path()
    for rep in range(3):
        new = torch.randint(-1, groups, (rows,), generator=torch.Generator().manual_seed(rep),
                            dtype=torch.int32)
        ids.copy_(new)
        y.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        if op == "adapters":
            exact, spread = adapters.reference(x, w, new, a, b, scale)
            check(y, exact, spread, k + 32, f"replay {rep}")
        else:
            for e in range(groups):
                sel = (new == e).cuda()
                exact, spread = product(x[sel], w[e].t() if op == "experts_dx" else w[e])
                check(y[sel], exact, spread, width, f"replay {rep}")
            assert torch.all(y[(new < 0).cuda()] == 1.0)
        path()
        torch.cuda.synchronize()


def test_repeats_bit_for_bit_and_on_a_side_stream():
    counts, n, k = F.EXPERTS_LAYOUT
    plan = device_plan(experts.ids_of(counts, 3), 4)
    q, _ = stack(4, n, k, 19)
    x = rand((sum(counts), k), 20)
    first = T.gemm_experts(x, q, plan, gather=1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = T.gemm_experts(x, q, plan, gather=1)
    s.synchronize()
    assert torch.equal(first, again)
