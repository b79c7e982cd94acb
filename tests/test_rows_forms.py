"""The choice of form of the products over grouped rows, on the host: the GPU
tests of the tiled kernels are of sizes that reach them."""

import pytest

from tests import rows_forms as F


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    return F.load(str(tmp_path_factory.mktemp("form")))


def test_the_tiled_tests_reach_the_tiles(rule):
    for counts, n, k in F.EXPERTS + [F.EXPERTS_LAYOUT]:
        for none in (0, 1, 6):
            assert rule.tiles(sum(counts) + none, len(counts), n, k, 0, 0, F.CUS), (counts, n)
    for counts, _, k in F.DX + [F.DX_LAYOUT]:
        for none in (0, 1, 6):
            assert rule.dx_tiles(sum(counts) + none, len(counts), k, F.CUS), (counts, k)
    for rows, groups in F.PLAIN:
        assert rule.tiles(rows, groups, 9001, 64, 0, 0, F.CUS)
        assert rows == 601 or rule.dx_tiles(rows, groups, 8192, F.CUS)
    for rows, pool, rank, n, k in F.ADAPTERS + [F.ADAPTERS_BROKEN]:
        assert rule.tiles(rows, 0, n, k, pool, rank, F.CUS), (rows, pool, rank, n, k)


@pytest.mark.parametrize("rows,groups,cols,tiled,dx_tiled", [
    (512, 8, 4096, 0, 0), (2048, 8, 4096, 1, 1), (400, 8, 4096, 0, 0), (333, 0, 4096, 0, 0),
    (1, 1, 1, 0, 0), (2**31 - 1, 1, 1, 1, 1), (2**31 - 1, 0, 2**31 - 1, 1, 1)])
def test_the_rule_at_measured_sizes(rule, rows, groups, cols, tiled, dx_tiled):
    assert rule.tiles(rows, groups, cols, 4096, 0, 0, F.CUS) == tiled
    assert rule.dx_tiles(rows, groups, cols, F.CUS) == dx_tiled


@pytest.mark.parametrize("rows,adapters,rank,n,k,tiled", [
    (600, 64, 256, 11008, 4096, 0), (600, 64, 64, 11008, 4096, 0), (1024, 64, 256, 8192, 8192, 0),
    (2048, 300, 256, 4096, 4096, 0), (2048, 300, 64, 4096, 4096, 0),
    (2048, 64, 256, 4096, 4096, 0), (2048, 8, 256, 8192, 8192, 1), (2048, 64, 256, 8192, 8192, 1),
    (4096, 256, 64, 11008, 4096, 1), (8192, 64, 64, 4096, 4096, 1)])
def test_the_low_rank_term_counts(rule, rows, adapters, rank, n, k, tiled):
    """The form measured as the faster one, by 10 % to three times."""
    assert rule.tiles(rows, 0, n, k, adapters, rank, F.CUS) == tiled
