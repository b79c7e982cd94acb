"""bnbx_group_rows (rows to groups) against the plan by its definition, bit for
bit: one workgroup and many, ids of no group, empty groups, one group only."""

import pytest
import torch

import dequant_gemm_nf4_amd as bnbx
from dequant_gemm_nf4_amd import tensors as T
from tests.rows_helpers import plan_of

pytestmark = pytest.mark.gpu


def ids_of(rows, groups, seed, none=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, groups, (rows,), generator=g, dtype=torch.int32)
    ids[torch.rand(rows, generator=g) < none] = -1
    return ids


def assert_plan(plan, ids, groups):
    offsets, order = plan_of(ids, groups)
    assert plan.offsets.tolist() == offsets
    assert plan.order.tolist() == order


@pytest.mark.parametrize("groups", [1, 2, 3, 8, 63, 64, 65, 255, 1024])
@pytest.mark.parametrize("rows", [0, 1, 2, 63, 64, 65, 333, 1024, 1025, 8191, 8192, 8193, 20000])
def test_sizes(rows, groups):
    ids = ids_of(rows, groups, 100 + rows + groups)
    plan = T.group_rows(ids.cuda(), groups)
    torch.cuda.synchronize()
    assert_plan(plan, ids, groups)


@pytest.mark.parametrize("rows,groups", [(131072, 64), (300001, 1024), (262144, 1)])
def test_many_chunks(rows, groups):
    ids = ids_of(rows, groups, 7)
    plan = T.group_rows(ids.cuda(), groups)
    torch.cuda.synchronize()
    assert_plan(plan, ids, groups)


@pytest.mark.parametrize("rows", [200, 30000])
def test_ids_outside_the_groups_go_last(rows):
    """Every id that is not 0 .. groups-1 counts as none, the extremes too."""
    ids = ids_of(rows, 5, 11)
    ids[::3] = torch.tensor([-1, 5, 6, 2**31 - 1, -2**31, 1024, 7]).repeat(rows)[:ids[::3].numel()]
    plan = T.group_rows(ids.cuda(), 5)
    torch.cuda.synchronize()
    assert_plan(plan, ids, 5)


@pytest.mark.parametrize("rows", [100, 50000])
@pytest.mark.parametrize("fill", [-1, 0, 9])
def test_all_rows_alike(rows, fill):
    ids = torch.full((rows,), fill, dtype=torch.int32)
    plan = T.group_rows(ids.cuda(), 10)
    torch.cuda.synchronize()
    assert_plan(plan, ids, 10)


def test_writes_nothing_else_and_repeats():
    """Guard words around the outputs stay; a second call gives the same."""
    rows, groups = 30000, 17
    ids = ids_of(rows, groups, 13).cuda()
    big = torch.full((rows + groups + 1 + 96,), 77, dtype=torch.int32, device="cuda")
    plan = T.RowGroups(groups, big[32:32 + groups + 1], big[64 + groups + 1:64 + groups + 1 + rows])
    T.group_rows(ids, groups, out=plan)
    first = big.clone()
    T.group_rows(ids, groups, out=plan)
    torch.cuda.synchronize()
    assert torch.equal(big, first)
    assert_plan(plan, ids.cpu(), groups)
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[32:32 + groups + 1] = False
    mask[64 + groups + 1:64 + groups + 1 + rows] = False
    assert torch.all(big[mask] == 77)


def test_workspace_too_small_is_refused():
    ids = ids_of(30000, 17, 14).cuda()
    plan = T.empty_row_groups(30000, 17)
    need = bnbx.bnbx_group_rows_workspace_bytes(30000, 17)
    assert need > 0
    with pytest.raises(bnbx.BnbxError) as e:
        T.group_rows(ids, 17, out=plan,
                     workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == bnbx.BNBX_E_WORKSPACE


def test_captured_and_replayed():
    ids = ids_of(30000, 17, 15).cuda()
    small = ids_of(90, 4, 16).cuda()
    p1, p2 = T.empty_row_groups(30000, 17), T.empty_row_groups(90, 4)
    ws = torch.empty(bnbx.bnbx_group_rows_workspace_bytes(30000, 17), dtype=torch.uint8,
                     device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        T.group_rows(ids, 17, out=p1, workspace=ws)
        T.group_rows(small, 4, out=p2)
    for rep in range(4):
        ids.copy_(ids_of(30000, 17, 20 + rep))
        small.copy_(ids_of(90, 4, 30 + rep))
        ws.fill_(0xAB)
        g.replay()
        torch.cuda.synchronize()
        assert_plan(p1, ids.cpu(), 17)
        assert_plan(p2, small.cpu(), 4)
        T.group_rows(ids, 17)
        torch.cuda.synchronize()
