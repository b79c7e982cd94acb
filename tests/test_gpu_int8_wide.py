"""The 8-bit forward product of weights whose scales lie past 2^31 bytes.  (Past 2^32 a
result that one launch takes is larger than the card; smaller ones are refused.)"""

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from int8_helpers import DT, codes_in_64, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,dtype", [(65, 2**29 + 320, "bf16"), (129, 2**29 + 77, "f16")])
def test_scales_past_32_bit_offsets(M, N, dtype):
    """Windows of Y around 0 and 2^29 and at the end; one product's sum, rounded to
    fp32, and its two scalings are each off by half a step of binary32 at most, the result
    by half a step of its type."""
    K, wide = 16, 200
    torch.cuda.empty_cache()
    codes = torch.ones(N, K, dtype=torch.int8, device="cuda")
    scale = torch.ones(N, dtype=torch.float32, device="cuda")
    windows = [slice(0, wide), slice(2**29 - wide, 2**29 + 77), slice(N - wide, N)]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    for s in windows:
        n = s.stop - s.start
        codes[s] = torch.randint(-127, 128, (n, K), generator=gen, device="cuda").to(torch.int8)
        scale[s] = torch.rand(n, generator=gen, device="cuda") + 0.5
    x = rand((M, K), 1, 1.0, dtype)
    qx, sx = codes_in_64(x)
    y = T.linear_int8(x, T.Int8Rows((N, K), codes, scale, DT[dtype]))
    fi = torch.finfo(DT[dtype])
    for s in windows:
        exact = (qx.double() @ codes[s].double().t().contiguous()) * sx.double()[:, None] * \
            scale[s].double()
        tol = exact.abs() * (fi.eps / 2 + 4 * 2.0 ** -24) + fi.smallest_normal * fi.eps
        assert ((y[:, s].double() - exact).abs() <= tol).all(), s
    del y, codes, scale
    torch.cuda.empty_cache()
