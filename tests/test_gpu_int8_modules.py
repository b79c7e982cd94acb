"""The 8-bit layer as a user has it: ops, modules, autograd, streams and graphs on
the GPU, against the formulas in binary64 and against differences."""

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from dequant_gemm_nf4_amd.torch_ops import Linear8bit, Linear8bitTrain
from int8_helpers import DT, check, codes_in_64, gradient_check, held, rand, values_of

pytestmark = pytest.mark.gpu
ops = torch.ops.bnbx


def forward_check(y, x, w):
    """rnd16 of the exact sums times the scales (fl32 of the sum and of two products)."""
    x2 = x.reshape(-1, x.shape[-1])
    qx, sx = codes_in_64(x2)
    qw, sw = codes_in_64(w)
    exact = (qx.double() @ qw.double().t().contiguous()) * sx.double()[:, None] * sw.double()
    tol = exact.abs() * (torch.finfo(y.dtype).eps / 2 + 4 * 2.0 ** -24) + 2.0 ** -25
    assert ((y.reshape(exact.shape).double() - exact).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lead,K,N", [((), 96, 40), ((1,), 4096, 512), ((2, 3), 200, 77),
                                      ((5, 30), 333, 130), ((4, 0), 64, 16), ((300,), 1024, 600)])
def test_linear8bit(lead, K, N, dtype):
    w = rand((N, K), 1, 0.05, dtype)
    lin = torch.nn.Linear(K, N, bias=False, device="cuda", dtype=DT[dtype])
    with torch.no_grad():
        lin.weight.copy_(w)
    m = Linear8bit.from_linear(lin, compute_dtype=DT[dtype])
    x = rand(lead + (K,), 2, 1.0, dtype).requires_grad_()
    y = m(x)
    assert y.shape == lead + (N,) and y.dtype == DT[dtype]
    forward_check(y, x, w)
    v = values_of(*codes_in_64(w), DT[dtype])
    assert torch.equal(m.dequantize().double(), v)
    g = rand(lead + (N,), 3, 0.1, dtype)
    y.backward(g)
    gradient_check(x.grad.reshape(-1, K), g.reshape(-1, N), v)
    m2 = Linear8bit(K, N, DT[dtype])
    m2.load_state_dict(m.state_dict())
    assert torch.equal(m2(x), y)


def test_linear8bit_takes_any_strides():
    K, N = 200, 50
    w = rand((N, K), 1, 0.05)
    m = Linear8bit(K, N).load_weight(w.float())
    wide = rand((6, 7, 2 * K + 3), 2)
    for x in (wide[..., 1:K + 1], wide[..., ::2][..., :K], wide[:, 3, :K], wide[:1, :1, :K].expand(6, 7, K),
              rand((K, 9), 3).t()):
        y = m(x)
        assert torch.equal(y, m(x.contiguous()))
    one = Linear8bit(1, 5).load_weight(rand((5, 1), 4))
    x = rand((1, 8), 5).t()
    assert torch.equal(one(x), one(x.clone(memory_format=torch.contiguous_format)))


def test_gradient_of_a_broadcast_output():
    """An expanded dY (a sum's gradient) and one with odd columns."""
    for N in (64, 63):
        w = rand((N, 100), 1, 0.05)
        m = Linear8bit(100, N).load_weight(w)
        x = rand((9, 100), 2).requires_grad_()
        m(x).sum().backward()
        ones = torch.ones(9, N, dtype=torch.bfloat16, device="cuda")
        gradient_check(x.grad, ones, values_of(*codes_in_64(w), torch.bfloat16))
        t = Linear8bitTrain(100, N)
        t(x).sum().backward()
        gradient_check(t.weight.grad, ones.t(), values_of(*codes_in_64(x), torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lead,K,N", [((1,), 64, 8), ((3, 5), 100, 72), ((140,), 515, 130),
                                      ((2, 150), 1024, 640)])
def test_linear8bit_train(lead, K, N, dtype):
    m = Linear8bitTrain(K, N, DT[dtype])
    w = m.weight.detach()
    x = rand(lead + (K,), 2, 1.0, dtype).requires_grad_()
    g = rand(lead + (N,), 3, 0.1, dtype)
    y = m(x)
    forward_check(y, x, w)
    y.backward(g)
    gradient_check(x.grad.reshape(-1, K), g.reshape(-1, N), values_of(*codes_in_64(w), DT[dtype]))
    vx = values_of(*codes_in_64(x.reshape(-1, K)), DT[dtype])
    gradient_check(m.weight.grad, g.reshape(-1, N).t(), vx)
    first = m.weight.grad.clone()
    m(x).backward(g)                       # gradients add up
    assert torch.equal(m.weight.grad, first + first)
    assert torch.equal(m.freeze()(x), y)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_against_differences(dtype):
    """Rows of small whole numbers times 2^-5 beside one 127 (whose partners are
    zero): their codes are the numbers, a step of 2^-5 moves one code by one, the
    layer is linear there and every value exact in 16 bits, so that differences
    equal the gradients."""
    dt, M, N, K, h = DT[dtype], 5, 6, 9, 2.0 ** -5
    gen = torch.Generator().manual_seed(1)
    x = torch.randint(-3, 4, (M, K), generator=gen).double()
    w = torch.randint(-3, 4, (N, K), generator=gen).double()
    g = torch.randint(-2, 3, (M, N), generator=gen).double()
    x[:, 0], w[:, 0], x[:, 1], w[:, 1] = 127, 0, 0, 127

    def f(x, w):
        m = Linear8bitTrain(K, N, dt)
        with torch.no_grad():
            m.weight.copy_((w * h).to(dt))
            return float((m((x * h).to(dt).cuda()).double() * g.cuda()).sum())

    m = Linear8bitTrain(K, N, dt)
    with torch.no_grad():
        m.weight.copy_((w * h).to(dt))
    xg = (x * h).to(dt).cuda().requires_grad_()
    m(xg).backward(g.to(dt).cuda())
    for r in range(M):
        for k in range(2, K):
            d = torch.zeros_like(x)
            d[r, k] = 1
            assert (f(x + d, w) - f(x - d, w)) / (2 * h) == float(xg.grad[r, k])
    for r in range(N):
        for k in range(2, K):
            d = torch.zeros_like(w)
            d[r, k] = 1
            assert (f(x, w + d) - f(x, w - d)) / (2 * h) == float(m.weight.grad[r, k])


def test_layers_together():
    """Two trained layers around a nonlinearity, then the frozen ones: every
    gradient is the formula's on what the layer before it gave."""
    a, b = Linear8bitTrain(200, 328), Linear8bitTrain(328, 120)
    x = rand((70, 200), 1).requires_grad_()
    h = a(x)
    s = torch.nn.functional.silu(h)
    y = b(s)
    h.retain_grad()
    s.retain_grad()
    g = rand((70, 120), 2, 0.1)
    y.backward(g)
    bf = torch.bfloat16
    gradient_check(b.weight.grad, g.t(), values_of(*codes_in_64(s), bf))
    gradient_check(s.grad, g, values_of(*codes_in_64(b.weight), bf))
    gradient_check(a.weight.grad, h.grad.t(), values_of(*codes_in_64(x), bf))
    gradient_check(x.grad, h.grad, values_of(*codes_in_64(a.weight), bf))
    fa, fb = a.freeze(), b.freeze()
    assert torch.equal(fb(torch.nn.functional.silu(fa(x))), y)


def test_what_is_kept_for_the_backward_pass():
    m = Linear8bitTrain(512, 256)
    x = rand((64, 512), 1).requires_grad_()
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        m(x)
    assert sorted((t.dtype, tuple(t.shape)) for t in kept if t.dtype == torch.int8) == \
        [(torch.int8, (64, 512)), (torch.int8, (256, 512))]
    assert all(t.dtype in (torch.int8, torch.float32) for t in kept)


def test_compile_full_graph():
    m = Linear8bit(128, 64).load_weight(rand((64, 128), 1, 0.05))
    x = rand((20, 128), 2)
    f = torch.compile(lambda t: torch.relu(m(t)) + 1, fullgraph=True, backend="aot_eager")
    assert torch.equal(f(x), torch.relu(m(x)) + 1)


def adapter_gradient(dy, low, q, scale):
    """dA = s (dY . B)^T . X_hat of an adapter beside a layer whose input was saved."""
    return T.gemm_int8_dw((dy.float() @ low.float() * scale).to(dy.dtype), q, dtype=torch.float32)


def test_adapter_gradient_from_saved_activations():
    M, N, K, r = 300, 96, 1000, 16
    x, dy, b = rand((M, K), 1), rand((M, N), 2, 0.1), rand((N, r), 3, 0.2)
    q = T.quantize_rows(x)
    dA = adapter_gradient(dy, b, q, 2.0)
    g = (dy.float() @ b.float() * 2.0).bfloat16()
    gradient_check(dA, g.t(), values_of(*codes_in_64(x), torch.bfloat16))


CASES = [(1, 512, 1024), (4, 300, 4096), (16, 520, 2048), (50, 264, 1000), (200, 1024, 2048),
         (600, 2048, 512)]


@pytest.mark.parametrize("M,N,K", CASES)
def test_graph_replays(M, N, K):
    """The layer, its gradients and the quantizer in one graph: every replay, with
    other inputs and eager calls between, gives what eager calls give."""
    w = held(rand((N, K), 1, 0.02))
    x, dy = rand((M, K), 2), rand((M, N), 3, 0.1)
    saved = T.empty_int8_rows((M, K))

    def call():
        y = T.linear_int8(x, w, saved=saved)
        return (y, T.gemm_int8_dx(dy, w), T.gemm_int8_dw(dy, saved),
                T.gemm_int8_dw(dy, saved, dtype=torch.float32), T.dequantize_rows(saved))

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        x.copy_(rand((M, K), 10 + i))
        dy.copy_(rand((M, N), 20 + i, 0.1))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_two_graphs_share_a_workspace():
    """One caller's workspace in two captured graphs, replayed in turn."""
    M, N, K = 300, 520, 8192
    w, x, dy = held(rand((N, K), 1, 0.02)), rand((M, K), 2), rand((M, N), 3, 0.1)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    y, dx = T.linear_int8(x, w), T.gemm_int8_dx(dy, w)
    a, b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(a):
        ya = T.linear_int8(x, w, workspace=ws)
    with torch.cuda.graph(b):
        dxb = T.gemm_int8_dx(dy, w, workspace=ws)
    for _ in range(4):
        a.replay()
        b.replay()
        assert torch.equal(ya, y) and torch.equal(dxb, dx)
        ya.zero_(), dxb.zero_()


def test_streams():
    """On a given stream, and on the current one of a `with`: ordered behind that
    stream's work, not the default stream's."""
    M, N, K = 64, 512, 2048
    x, w = rand((M, K), 1), held(rand((N, K), 2, 0.02))
    y = T.linear_int8(x, w)
    side = torch.cuda.Stream()
    buf = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        buf.copy_(x)
        late = T.linear_int8(buf, w)
    given = T.linear_int8(buf, w, stream=side)
    dx = T.gemm_int8_dx(late, w, stream=side)
    side.synchronize()
    assert torch.equal(late, y) and torch.equal(given, y)
    assert torch.equal(dx, T.gemm_int8_dx(y, w))
    with pytest.raises(ValueError):
        T.linear_int8(x.cpu(), w)


def test_two_calls_at_once():
    """Independent calls on two streams do not disturb each other."""
    w = held(rand((1024, 4096), 1, 0.02))
    xs = [rand((m, 4096), m) for m in (3, 40, 300)]
    want = [T.linear_int8(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [T.linear_int8(x, w, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
