"""Calls of the 8-bit gradients with widths that are no pieces of eight, captured and on
a given stream, and a training step without rows."""

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from dequant_gemm_nf4_amd.torch_ops import Linear8bitTrain
from int8_helpers import codes_in_64, gradient_check, held, rand, values_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 77, 300), (9, 1001, 500), (300, 333, 1000)])
def test_widths_that_are_no_pieces_in_a_graph(M, N, K):
    """dY is copied within the call: every replay, with other gradients and eager calls
    between, gives what eager calls give."""
    w, q = held(rand((N, K), 1, 0.02)), held(rand((M, K), 2))
    dy = rand((M, N), 3, 0.1)

    def call():
        return T.gemm_int8_dx(dy, w), T.gemm_int8_dw(dy, q, dtype=torch.float32)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        dy.copy_(rand((M, N), 20 + i, 0.1))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_widths_that_are_no_pieces_on_a_given_stream():
    """The copy of dY belongs to the stream that runs the call, not to the current one."""
    M, N, K = 130, 333, 700
    w, q, dy = held(rand((N, K), 1, 0.02)), held(rand((M, K), 2)), rand((M, N), 3, 0.1)
    want = T.gemm_int8_dx(dy, w), T.gemm_int8_dw(dy, q)
    side, late = torch.cuda.Stream(), torch.zeros_like(dy)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late.copy_(dy)
    for given in (side, side.cuda_stream):
        got = T.gemm_int8_dx(late, w, stream=given), T.gemm_int8_dw(late, q, stream=given)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("N", [64, 63])
def test_a_training_step_without_rows(N):
    m = Linear8bitTrain(96, N)
    x = torch.empty(3, 0, 96, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    m(x).backward(torch.empty(3, 0, N, dtype=torch.bfloat16, device="cuda"))
    assert x.grad.shape == x.shape
    assert m.weight.grad.shape == (N, 96) and not m.weight.grad.any()


def test_an_update_between_the_passes():
    """The gradients are those of the weight that the forward pass multiplied."""
    m = Linear8bitTrain(200, 120)
    x, g = rand((33, 200), 1).requires_grad_(), rand((33, 120), 2, 0.1)
    codes = codes_in_64(m.weight)
    y = m(x)
    with torch.no_grad():
        m.weight.mul_(3.0)
    y.backward(g)
    gradient_check(x.grad, g, values_of(*codes, torch.bfloat16))
    gradient_check(m.weight.grad, g.t(), values_of(*codes_in_64(x), torch.bfloat16))
