"""The choice of form of the 8-bit products, on the host: the GPU tests of every form are
of sizes that reach it."""

import pytest

from tests import int8_forms as F


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    return F.load(str(tmp_path_factory.mktemp("form")))


def test_the_sizes_reach_every_form(rule):
    for table, fn, grad in ((F.FORWARD, rule.forward, 0), (F.GRADS, rule.grad, 1)):
        for (rows, cols, split), sizes in table.items():
            assert grad or sizes[0] > rule.wave_rows()
            got = F.form(fn, *sizes)
            assert (got[0], got[1], got[2] > 1) == (rows, cols, split), (sizes, got)
        assert len({k[:2] for k in table}) == rule.shapes(grad) and len(table) == 2 * len(
            {k[:2] for k in table})


@pytest.mark.parametrize("sizes", [(1, 1, 1), (33, 1, 131071), (2**31 - 512, 16, 32),
                                   (16, 2**31 - 512, 32), (2**31 - 512, 2**31 - 512, 131071),
                                   (33, 4096, 131071), (2**31 - 1, 2**31 - 1, 2**31 - 1),
                                   (64, 64, 2**31 - 1)])
@pytest.mark.parametrize("cus", [1, 80, 256])
def test_a_split_covers_the_summed_axis(rule, sizes, cus):
    for fn, step, most in ((rule.forward, 128, 16), (rule.grad, 64, 32)):
        _, _, splits, per = F.form(fn, *sizes, cus=cus)
        steps = -(-sizes[2] // step)
        assert 1 <= splits <= most and splits * per >= steps and (splits - 1) * per < steps


def test_nothing_summed(rule):
    assert F.form(rule.grad, 300, 4096, 0)[2:] == (1, 0)


def test_rows_of_w_a_wave(rule):
    for n, rows in F.FEW.items():
        assert rule.few_rows(1, n, F.CUS) == 1
        assert [rule.few_rows(m, n, F.CUS) for m in (2, 3, 4)] == [rows] * 3
    assert rule.few_rows(4, 1, F.CUS) == 1 and rule.few_rows(2, 2**31 - 512, F.CUS) == 8
    assert rule.few_rows(2, 33, 1) == 3
