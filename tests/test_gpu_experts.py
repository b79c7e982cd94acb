"""bnbx_gemm_nf4_experts (4-bit products grouped by expert) against binary64
products on the dequantized weights, element by element."""

import dataclasses

import pytest
import torch

import oracle
import synth
from dequant_gemm_nf4_amd import tensors as T
from tests.gpu_helpers import dev_bf16, upload_state
from tests.rows_helpers import DT, check, device_plan, product, rand, stack

pytestmark = pytest.mark.gpu


def ids_of(counts, seed, none=0):
    """ids with counts[g] rows of group g and `none` of none, shuffled."""
    ids = [g for g, c in enumerate(counts) for _ in range(c)] + [-1] * none
    g = torch.Generator().manual_seed(seed)
    return torch.tensor(ids, dtype=torch.int32)[torch.randperm(len(ids), generator=g)]


def run_case(counts, n, k, none=0, mode="gather", topk=1, dq="linear", quant="nf4", dtype="bf16",
             seed=1):
    groups = len(counts)
    ids = ids_of(counts, seed, none)
    plan = device_plan(ids, groups)
    rows = ids.numel()
    q, w = stack(groups, n, k, seed + 1, dq, quant, dtype)
    gather = topk if mode == "gather" else 0
    x = rand((-(-rows // topk) if gather else rows, k), seed + 2, 1.0, dtype)
    out = torch.full((rows, n), 3.5, dtype=DT[dtype], device="cuda")
    print(f"experts {counts} none={none} N={n} K={k} {mode} topk={topk} {dq} {quant} {dtype}",
          flush=True)
    y = T.gemm_experts(x, q, plan, gather=gather, scatter=mode == "scatter", out=out)
    torch.cuda.synchronize()
    assert y is out
    touched = torch.zeros(rows, dtype=torch.bool, device="cuda")
    off, order = plan.offsets.tolist(), plan.order.long()
    for g in range(groups):
        places = torch.arange(off[g], off[g + 1], device="cuda")
        if places.numel() == 0:
            continue
        xr = order[places] // topk if gather else places
        yr = order[places] if mode == "scatter" else places
        exact, spread = product(x[xr], w[g])
        check(y[yr], exact, spread, k, f"group {g}")
        touched[yr] = True
    assert torch.all(y[~touched] == 3.5)
    return y


TYPES = [("linear", "nf4", "bf16"), ("linear", "fp4", "f16"), ("dynamic", "nf4", "f16"),
         (None, "fp4", "bf16"), (None, "nf4", "f16"), ("dynamic", "fp4", "bf16")]


@pytest.mark.parametrize("dq,quant,dtype", TYPES)
@pytest.mark.parametrize("counts,n,k", [
    ([1], 16, 64), ([1, 0, 1], 17, 128), ([3, 5, 0, 1], 130, 320), ([16, 16], 64, 256),
    ([17, 1, 15, 0, 33], 100, 576), ([64, 1], 129, 4160), ([40, 25], 96, 1024)])
def test_small(counts, n, k, dq, quant, dtype):
    run_case(counts, n, k, none=2, dq=dq, quant=quant, dtype=dtype)


@pytest.mark.parametrize("mode", ["gather", "scatter", "places"])
@pytest.mark.parametrize("counts,n,k,none", [
    ([2, 0, 0, 0, 7], 257, 704, 0), ([0, 0, 130, 0], 63, 192, 5), ([1] * 70, 33, 128, 3),
    ([0] * 199 + [9], 40, 256, 0), ([31, 0, 90, 200], 1, 64, 0), ([100, 3], 3, 2112, 7)])
def test_layouts(mode, counts, n, k, none):
    run_case(counts, n, k, none=none, mode=mode)


@pytest.mark.parametrize("topk", [2, 3, 8])
def test_slots_of_tokens(topk):
    run_case([11, 0, 40, 24, 5], 200, 512, none=4, topk=topk)


@pytest.mark.parametrize("counts,n,k", [
    ([1, 1], 4096, 4096), ([2] * 8, 1000, 4096), ([9] * 4, 2000, 1088), ([20] * 8, 640, 2048),
    ([300, 20, 0, 77], 520, 1024), ([130] * 3, 300, 11008), ([1000, 24], 768, 512),
    ([257, 255, 256], 260, 640)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_larger(counts, n, k, dtype):
    run_case(counts, n, k, none=1, dtype=dtype)


@pytest.mark.parametrize("dq,quant,dtype", TYPES)
@pytest.mark.parametrize("k", [320, 512, 1088])
@pytest.mark.parametrize("counts,n", [
    ([6, 5, 9], 2000), ([6, 5, 9], 4200), ([6, 5, 9], 10000), ([6, 5, 9], 17000),
    ([20, 25], 3000), ([20, 25], 7000), ([20, 25], 14000), ([20, 25], 30000),
    ([50, 40], 3001), ([50, 40], 7000), ([50, 40], 17000)])
def test_wide(counts, n, k, dq, quant, dtype):
    """Few rows a group and many weight rows: every way to share them and K out
    among waves, with row lengths of a multiple of four blocks and others."""
    run_case(counts, n, k, none=1, dq=dq, quant=quant, dtype=dtype)


@pytest.mark.parametrize("dq", ["linear", None])
@pytest.mark.parametrize("rows", [1, 9, 24, 60, 900])
def test_block_scales_at_any_address(rows, dq):
    """Block codes and maxima that start at an element's own alignment only."""
    q, _ = stack(2, 300, 1024, 41, dq)
    plan = device_plan(ids_of([rows, 1], 42), 2)
    x = rand((rows + 1, 1024), 43)
    ref = T.gemm_experts(x, q, plan)
    odd = torch.cat((q.absmax[:1], q.absmax))[1:]
    assert odd.data_ptr() % 16 != 0
    y = T.gemm_experts(x, dataclasses.replace(q, absmax=odd), plan)
    torch.cuda.synchronize()
    assert torch.equal(y, ref)


def test_all_rows_of_no_group_leave_the_output():
    q, _ = stack(3, 64, 128, 5)
    plan = device_plan([-1, -1, 7], 3)
    out = torch.full((3, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    T.gemm_experts(rand((3, 128), 6), q, plan, gather=1, out=out)
    torch.cuda.synchronize()
    assert torch.all(out == 2.0)
    zero = T.gemm_experts(rand((3, 128), 6), q, plan, gather=1)
    assert torch.all(zero == 0)


def test_most_groups():
    """1024 groups: tiles found past the first 64 groups, several in some."""
    run_case([2, 0, 0, 1] * 128 + [0] * 500 + [40] * 11 + [3], 48, 128, none=9)


def test_no_rows():
    q, _ = stack(3, 64, 128, 5)
    plan = device_plan([], 3)
    y = T.gemm_experts(rand((0, 128), 6), q, plan, gather=1)
    assert y.shape == (0, 64)


def test_against_the_oracle():
    """The stack quantized by the oracle (linear map, the groups of 256 scales
    crossing experts), its own dequantized weights."""
    groups, n, k = 3, 40, 320
    bits = synth.normal_bf16((groups * n, k), 0.02, 77)
    ref = oracle.quantize(bits, True)
    q = upload_state(ref, (groups, n, k))
    w = oracle.bf16_bits_to_f32(oracle.dequantize(ref["packed"], ref)).reshape(groups, n, k)
    xb = synth.normal_16((9, k), 1.0, 78, "bf16")
    plan = device_plan([2, 0, 0, 1, -1, 2, 2, 1, 0], groups)
    y = T.gemm_experts(dev_bf16(xb, (9, k)), q, plan, gather=1, scatter=True)
    torch.cuda.synchronize()
    x = torch.from_numpy(oracle.bf16_bits_to_f32(xb).reshape(9, k)).double()
    for i, g in enumerate([2, 0, 0, 1, -1, 2, 2, 1, 0]):
        if g >= 0:
            exact, spread = product(x[i:i + 1], torch.from_numpy(w[g].copy()))
            check(y[i:i + 1].cpu(), exact, spread, k, f"row {i}")
        else:
            assert torch.all(y[i] == 0)


def test_strided_rows_and_guards():
    """Rows inside wider buffers; nothing outside the rows is written."""
    counts, n, k = [5, 20, 0, 3], 70, 192
    plan = device_plan(ids_of(counts, 3), 4)
    q, w = stack(4, n, k, 9)
    xbig = torch.full((28, k + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    xbig[:, 8:8 + k] = rand((28, k), 10)
    ybig = torch.full((32, n + 11), 9.0, dtype=torch.bfloat16, device="cuda")
    T.gemm_experts(xbig[:, 8:8 + k], q, plan, gather=1, scatter=True, out=ybig[2:30, 5:5 + n])
    torch.cuda.synchronize()
    ref = T.gemm_experts(xbig[:, 8:8 + k].contiguous(), q, plan, gather=1, scatter=True)
    assert torch.equal(ybig[2:30, 5:5 + n], ref)
    ybig[2:30, 5:5 + n] = 9.0
    assert torch.all(ybig == 9.0)


def test_infinite_rows_stay_their_own():
    """A row of X with infinities or NaN does not reach other rows, also where
    K ends inside a step."""
    counts, n, k = [6, 30], 48, 192
    plan = device_plan([0] * 6 + [1] * 30, 2)
    q, w = stack(2, n, k, 12)
    x = rand((36, k), 13)
    x[2, 5] = float("inf")
    x[3, :] = float("nan")
    x[20, k - 1] = float("-inf")
    x[7, 0] = float("inf")
    y = T.gemm_experts(x, q, plan)
    torch.cuda.synchronize()
    clean = torch.tensor([i for i in range(36) if i not in (2, 3, 20, 7)], device="cuda")
    for g, lo, hi in ((0, 0, 6), (1, 6, 36)):
        rows = clean[(clean >= lo) & (clean < hi)]
        exact, spread = product(x[rows], w[g])
        check(y[rows], exact, spread, k)
        for i in (2, 20, 7):
            if lo <= i < hi:
                col = {2: 5, 20: k - 1, 7: 0}[i]
                sign = torch.sign(w[g][:, col]) * (-1 if i == 20 else 1)
                hit = sign != 0
                assert torch.equal(y[i][hit].double(), sign[hit] * float("inf"))
    assert torch.isnan(y[3]).all()


def test_a_wrong_plan_stays_inside_the_buffers():
    """Rows outside X or Y are left out; bounds are clamped to the plan."""
    q, w = stack(2, 64, 128, 15)
    x = rand((4, 128), 16)
    plan = T.RowGroups(2, torch.tensor([-5, 3, 99], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, -7, 2, 2**31 - 1, 3], dtype=torch.int32, device="cuda"))
    big = torch.full((5 + 4, 64), 8.0, dtype=torch.bfloat16, device="cuda")
    T.gemm_experts(torch.cat((x, x[:1])), q, plan, gather=1, scatter=True, out=big[2:7])
    torch.cuda.synchronize()
    for row, g in ((0, 0), (2, 0), (3, 1)):
        exact, spread = product(x[row:row + 1], w[g])
        check(big[2 + row:3 + row], exact, spread, 128)
    assert torch.all(big[[0, 1, 3, 6, 7, 8]] == 8.0)


def test_repeats_bit_for_bit_and_on_a_side_stream():
    counts, n, k = [9, 70, 0, 21], 500, 2048
    plan = device_plan(ids_of(counts, 3), 4)
    q, _ = stack(4, n, k, 19)
    x = rand((100, k), 20)
    a = T.gemm_experts(x, q, plan, gather=1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = T.gemm_experts(x, q, plan, gather=1)
    s.synchronize()
    assert torch.equal(a, b)


def test_captured_and_replayed_with_new_plans():
    """The plan is read on the device: a replay follows new ids."""
    groups, rows, n, k = 4, 50, 200, 512
    q, w = stack(groups, n, k, 21)
    x = rand((rows, k), 22)
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    plan = T.empty_row_groups(rows, groups)
    y = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    T.group_rows(ids, groups, out=plan)
    T.gemm_experts(x, q, plan, gather=1, scatter=True, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        T.group_rows(ids, groups, out=plan)
        T.gemm_experts(x, q, plan, gather=1, scatter=True, out=y)
    for rep in range(4):
        g = torch.Generator().manual_seed(rep)
        ids.copy_(torch.randint(-1, groups, (rows,), generator=g, dtype=torch.int32))
        y.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for e in range(groups):
            sel = ids == e
            if sel.any():
                exact, spread = product(x[sel], w[e])
                check(y[sel], exact, spread, k, f"replay {rep}")
        assert torch.all(y[ids < 0] == 1.0)
        T.gemm_experts(x, q, plan, gather=1)
        torch.cuda.synchronize()
