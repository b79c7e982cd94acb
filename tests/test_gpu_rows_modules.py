"""The row-grouped layers as a model uses them: a mixture of experts (plan, up
projection, down projection, weighted sum) with its gradient, and a step of many
adapters over several layers, against binary64; compiled, captured, on two
streams."""

import math

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from dequant_gemm_nf4_amd.torch_ops import Experts4bit, Linear4bit, Linear4bitAdapters
from tests.rows_helpers import DT, check, product, rand

pytestmark = pytest.mark.gpu


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def experts(groups, k, n, seed, **kw):
    m = Experts4bit(groups, k, n, **kw)
    m.load_weight(rand((groups, n, k), seed, 1 / math.sqrt(k)))
    return m


class Mixture(torch.nn.Module):
    def __init__(self, groups, d, h, topk, **kw):
        super().__init__()
        self.groups, self.topk = groups, topk
        self.up, self.down = experts(groups, d, h, 1, **kw), experts(groups, h, d, 2, **kw)

    def forward(self, x, ids, weights):
        plan = torch.ops.bnbx.group_rows(ids, self.groups)
        hidden = torch.nn.functional.silu(self.up(x, plan, gather=self.topk))
        out = self.down(hidden, plan, scatter=True)
        return (out.view(x.shape[0], self.topk, -1) * weights[..., None]).sum(1)

    def exact(self, x, ids, weights):
        up, down = T.dequantize(self.up.quantized()), T.dequantize(self.down.quantized())
        y = torch.zeros_like(x)
        for s in range(self.topk):
            for g in range(self.groups):
                sel = ids[:, s] == g
                if sel.any():
                    h = torch.nn.functional.silu(x[sel] @ up[g].double().t().contiguous())
                    z = h @ down[g].double().t().contiguous()
                    y = y.index_add(0, sel.nonzero().flatten(), z * weights[sel, s, None])
        return y


def routing(tokens, groups, topk, seed, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(tokens, groups, generator=g).topk(topk, 1).indices.to(torch.int32)
    ids[torch.rand(tokens, topk, generator=g) < drop] = -1
    return ids.cuda(), torch.rand(tokens, topk, generator=g).cuda()


# roundings on the way (up, silu, down, weighting, sum: at most 6 of half a
# step each), and as many again on the way back
@pytest.mark.parametrize("tokens,groups,d,h,topk", [(1, 4, 128, 192, 2), (33, 5, 256, 320, 3),
                                                    (700, 3, 192, 256, 1), (900, 4, 256, 512, 2)])
@pytest.mark.parametrize("dtype,dq_map", [("bf16", "linear"), ("f16", "dynamic")])
def test_mixture_and_its_gradient(tokens, groups, d, h, topk, dtype, dq_map):
    m = Mixture(groups, d, h, topk, compute_dtype=DT[dtype], dq_map=dq_map)
    ids, weights = routing(tokens, groups, topk, tokens)
    if tokens == 1:
        ids[0, 0] = 2
    x = rand((tokens, d), 5, 1.0, dtype).requires_grad_()
    w = weights.to(DT[dtype])
    print(f"mixture tokens={tokens} groups={groups} d={d} h={h} topk={topk} {dtype}", flush=True)
    y = m(x, ids, w)
    dy = rand((tokens, d), 6, 1.0, dtype)
    (dx,) = torch.autograd.grad(y, x, dy)
    torch.cuda.synchronize()
    x64 = x.detach().double().requires_grad_()
    y64 = m.exact(x64, ids, w.double())
    (dx64,) = torch.autograd.grad(y64, x64, dy.double())
    eps = torch.finfo(DT[dtype]).eps / 2
    assert rel(y, y64.detach()) <= 6 * eps
    assert rel(dx, dx64) <= 12 * eps


def test_token_gradient_is_the_sum_over_its_slots():
    """A broadcast input: every slot of a token reads the same row."""
    groups, d, n, topk, tokens = 4, 128, 64, 3, 20
    m = experts(groups, d, n, 11)
    w = T.dequantize(m.quantized()).double()
    ids, _ = routing(tokens, groups, topk, 12)
    plan = torch.ops.bnbx.group_rows(ids, groups)
    x = rand((tokens, d), 13).requires_grad_()
    y = m(x, plan, gather=topk)
    dy = rand((tokens * topk, n), 14)
    (dx,) = torch.autograd.grad(y, x, dy)
    want = torch.zeros(tokens, d, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    places = {int(s): p for p, s in enumerate(plan[1].tolist())}
    for t in range(tokens):
        for s in range(topk):
            g = int(ids[t, s])
            if g >= 0:
                part = dy[places[t * topk + s]].double() @ w[g]
                want[t] += part
                size[t] += part.abs()
    # half a step per slot, and one for the sum
    assert torch.all((dx.double() - want).abs() <= 2.0 ** -8 * (size + want.abs()) * 1.02 + 1e-9)


def test_expanded_and_unaligned_rows():
    """One row expanded to all places, as input and as the gradient that a sum
    over the rows hands back, and rows that start off 16 bytes."""
    groups, d, n, rows = 3, 128, 192, 21
    m = experts(groups, d, n, 21)
    plan = torch.ops.bnbx.group_rows(torch.arange(rows, dtype=torch.int32, device="cuda") % groups,
                                     groups)
    one = rand((1, d), 22)
    x = one.expand(rows, d)
    assert torch.equal(m(x, plan, gather=1), m(x.contiguous(), plan, gather=1))
    flat = torch.cat((one[0, :1], x.reshape(-1)))[1:].view(rows, d)
    assert flat.data_ptr() % 16 != 0
    assert torch.equal(m(flat, plan, gather=1), m(x.contiguous(), plan, gather=1))
    x = rand((rows, d), 23).requires_grad_()
    y = m(x, plan, gather=1, scatter=True)
    v = rand((n,), 24)
    (dx,) = torch.autograd.grad(y, x, v.expand(rows, n), retain_graph=True)
    (ref,) = torch.autograd.grad(y, x, v.expand(rows, n).contiguous())
    torch.cuda.synchronize()
    assert torch.equal(dx, ref) and dx.abs().max() > 0
    q = Linear4bitAdapters(d, n, 2, device="cuda").load_weight(rand((n, d), 25, 0.05))
    q.load_adapter(1, rand((16, d), 26), rand((n, 16), 27))
    plan = torch.ops.bnbx.group_rows(torch.ones(rows, dtype=torch.int32, device="cuda"), 2)
    x = one.expand(rows, d)
    assert torch.equal(q(x, plan), q(x.contiguous(), plan))


def test_a_given_stream_runs_all_of_a_call():
    """What a call allocates and clears runs on the stream it is given, not on
    the busy current one."""
    m = experts(2, 128, 64, 31)
    q = m.quantized()
    x = rand((40, 128), 32)
    ids = torch.tensor([0, 1, -1, 1] * 10, dtype=torch.int32, device="cuda")
    plan = T.group_rows(ids, 2)
    ref = T.gemm_experts(x, q, plan, gather=1, scatter=True)
    back = T.gemm_experts_dx(ref, q, plan, gather=1, scatter=True)
    w = T.quantize(rand((64, 128), 33, 0.05), True)
    a, b, scale = rand((2, 16, 128), 34), rand((2, 64, 16), 35), torch.ones(2, device="cuda")
    low = T.linear_adapters(x, w, plan, a, b, scale)
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for _ in range(8):
            big = big @ big * 1e-3   # the current stream has work in front
        made = T.group_rows(ids, 2, stream=stream)
        y = T.gemm_experts(x, q, made, gather=1, scatter=True, stream=stream)
        dx = T.gemm_experts_dx(y, q, made, gather=1, scatter=True, stream=stream)
        z = T.linear_adapters(x, w, made, a, b, scale, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(made.order, plan.order)
        assert torch.equal(y, ref) and torch.equal(dx, back) and torch.equal(z, low)


def test_opcheck_and_compiled_equal_eager():
    m = Mixture(4, 128, 192, 2)
    ids, weights = routing(30, 4, 2, 21)
    x = rand((30, 128), 22).requires_grad_()
    w = weights.bfloat16()
    torch.library.opcheck(torch.ops.bnbx.group_rows.default, (ids, 4))
    offsets, order = torch.ops.bnbx.group_rows(ids, 4)
    up = m.up
    args = (up.packed, up.absmax, up.absmax2, up.absmax_mean, offsets, order)
    torch.library.opcheck(torch.ops.bnbx.experts4bit.default, (x, *args, 192, 2, False, "nf4"))
    torch.library.opcheck(torch.ops.bnbx.experts4bit_dx.default,
                          (rand((60, 192), 23), *args, 128, 0, True, "nf4"))
    eager = m(x, ids, w)
    (g1,) = torch.autograd.grad(eager, x, torch.ones_like(eager))
    compiled = torch.compile(m, fullgraph=True, backend="aot_eager")
    y = compiled(x, ids, w)
    (g2,) = torch.autograd.grad(y, x, torch.ones_like(y))
    assert torch.equal(eager, y) and torch.equal(g1, g2)


def adapters_layer(k, n, slots, rank, seed, dtype="bf16", **kw):
    m = Linear4bitAdapters(k, n, slots, rank, compute_dtype=DT[dtype], **kw)
    m.load_weight(rand((n, k), seed, 1 / math.sqrt(k)))
    for s in range(slots):
        r = rank if s % 2 == 0 else rank // 2
        m.load_adapter(s, rand((r, k), seed + 10 + s, 1 / math.sqrt(k)),
                       rand((n, r), seed + 30 + s, 0.3), 0.5 + s)
    return m


def exact_adapters(m, x, slots_of):
    w = T.dequantize(m.quantized())
    y, _ = product(x, w)
    for s in range(m.adapters):
        sel = (slots_of == s).nonzero().flatten()
        if sel.numel():
            low = x[sel].double() @ m.lora_a[s].double().t().contiguous()
            y[sel] += m.scale[s].double() * (low @ m.lora_b[s].double().t().contiguous())
    return y


@pytest.mark.parametrize("rows", [1, 24, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_step_of_many_requests(rows, dtype):
    """One plan for all layers of a batch; adapters of two ranks in one pool;
    batched leading dimensions."""
    slots, k, n = 5, 256, 320
    layers = [adapters_layer(k, n, slots, 32, 100 * i, dtype) for i in (1, 2)]
    g = torch.Generator().manual_seed(rows)
    which = torch.randint(-1, slots, (rows,), generator=g, dtype=torch.int32).cuda()
    plan = torch.ops.bnbx.group_rows(which, slots)
    x = rand((rows, k), 7, 1.0, dtype)
    for m in layers:
        y = m(x, plan)
        assert rel(y, exact_adapters(m, x, which)) <= torch.finfo(DT[dtype]).eps / 2
        if rows == 24:
            assert torch.equal(m(x.view(2, 12, k), plan).view(rows, n), y)
    m = layers[0]
    torch.library.opcheck(torch.ops.bnbx.linear4bit_adapters.default,
                          (x, m.packed, m.absmax, m.absmax2, m.absmax_mean, *plan, m.lora_a,
                           m.lora_b, m.scale, n, "nf4"))
    compiled = torch.compile(m, fullgraph=True, backend="aot_eager")
    assert torch.equal(compiled(x, plan), m(x, plan))


def test_rows_of_no_adapter_equal_the_plain_layer():
    """The 4-bit product alone: the same W_hat and accumulation in fp32 as the
    layer without adapters, so equal up to one rounding and the order of sums
    (compared with the exact product)."""
    m = adapters_layer(256, 320, 2, 16, 300)
    plain = Linear4bit(256, 320)
    plain.load_state_dict({k: v for k, v in m.state_dict().items() if k in plain.state_dict()})
    x = rand((40, 256), 8)
    plan = torch.ops.bnbx.group_rows(torch.full((40,), -1, dtype=torch.int32, device="cuda"), 2)
    exact, spread = product(x, T.dequantize(m.quantized()))
    check(m(x, plan), exact, spread, 256)
    assert rel(plain(x), exact) < 5e-3


def test_two_streams_at_once():
    """Calls that overlap on two streams with their own outputs and
    workspaces do not disturb each other."""
    m = adapters_layer(1024, 1024, 6, 64, 400)
    e = experts(6, 1024, 1024, 401)
    g = torch.Generator().manual_seed(3)
    jobs = []
    for rows in (20, 150):
        which = torch.randint(-1, 6, (rows,), generator=g, dtype=torch.int32).cuda()
        jobs.append((rand((rows, 1024), rows), which))
    def both(x, which):
        plan = torch.ops.bnbx.group_rows(which, 6)
        return m(x, plan), e(x, plan, gather=1, scatter=True)
    want = [both(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = both(*jobs[i])
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_step_replays_with_new_requests():
    """A whole step (plan, mixture, adapter layer) in one HIP graph; every
    replay, with eager work between, equals the eager result."""
    mix = Mixture(4, 256, 320, 2)
    lora = adapters_layer(256, 256, 5, 32, 500)
    tokens = 40
    x = rand((tokens, 256), 31)
    ids, weights = routing(tokens, 4, 2, 32)
    w = weights.bfloat16()
    which = torch.zeros(tokens, dtype=torch.int32, device="cuda")

    @torch.no_grad()
    def step():
        plan = torch.ops.bnbx.group_rows(which, 5)
        return mix(lora(x, plan), ids, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        y = step()
    for rep in range(4):
        new, _ = routing(tokens, 4, 2, 40 + rep)
        ids.copy_(new)
        which.copy_(torch.randint(-1, 5, (tokens,), generator=torch.Generator().manual_seed(rep),
                                  dtype=torch.int32))
        x.copy_(rand((tokens, 256), 50 + rep))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step()), rep
        torch.cuda.synchronize()
