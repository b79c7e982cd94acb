"""Weights past a launch's output tiles are refused before anything is enqueued."""

import pytest

import dequant_gemm_nf4_amd as bnbx

A, B, C, D, E = (i << 20 for i in range(1, 6))   # fake device addresses


@pytest.mark.parametrize("M,N,dtype", [(65, 2**30 + 321, 0), (33, 2**29 + 320, 1)])
def test_more_output_tiles_than_a_launch_takes(M, N, dtype):
    w = bnbx.Int8RowsDesc(A, B, 16, N, 16, dtype)
    x = bnbx.Int8RowsDesc(C, D, 16, M, 16, dtype)
    for call in (lambda: bnbx.bnbx_linear_int8(C, 16, M, w, None, E, N, D, 1 << 62, 0),
                 lambda: bnbx.bnbx_gemm_int8(x, w, E, N, D, 1 << 62, 0)):
        with pytest.raises(bnbx.BnbxError) as e:
            call()
        assert e.value.status == bnbx.BNBX_E_UNSUPPORTED
