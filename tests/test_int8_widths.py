"""Inputs of another width than the weight's are refused by the 8-bit layer and its ops,
also where its codes hold as many columns."""

import pytest
import torch

from dequant_gemm_nf4_amd.torch_ops import Linear8bit

ops = torch.ops.bnbx


@pytest.mark.parametrize("width", [1, 16, 4090, 4097, 4112])
def test_the_module_takes_its_own_width_only(width):
    m = Linear8bit(4096, 8, device="meta")
    with pytest.raises(ValueError, match="4096"):
        m(torch.empty(3, width, dtype=torch.bfloat16, device="meta"))
    assert m(torch.empty(3, 4096, dtype=torch.bfloat16, device="meta")).shape == (3, 8)


def test_the_module_refuses_widths_of_the_same_padded_row():
    m = Linear8bit(20, 8, device="meta")
    for width in (17, 19, 21, 32):
        with pytest.raises(ValueError, match="20"):
            m(torch.empty(3, width, dtype=torch.bfloat16, device="meta"))


@pytest.mark.parametrize("width", [1, 100, 4080, 4097])
def test_the_ops_take_codes_of_their_own_width_only(width):
    codes, scale = torch.zeros(8, 4096, dtype=torch.int8), torch.zeros(8)
    bf = torch.bfloat16
    with pytest.raises(ValueError, match="columns"):
        ops.linear8bit(torch.zeros(3, width, dtype=bf), codes, scale)
    with pytest.raises(ValueError, match="columns"):
        ops.linear8bit_dx(torch.zeros(3, 8, dtype=bf), codes, scale, width)
    with pytest.raises(ValueError, match="columns"):
        ops.linear8bit_dw(torch.zeros(8, 5, dtype=bf), codes, scale, width, bf)
