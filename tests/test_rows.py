"""The row-grouped operators without a GPU: the exported symbols, every
refusal on the host before a launch (the pointers are never dereferenced), the
torch-tensor layer's checks, and the ops' and modules' shapes on meta tensors."""

import dataclasses
import os
import re
import subprocess

import pytest
import torch

import dequant_gemm_nf4_amd as bnbx
from dequant_gemm_nf4_amd import tensors as T
from dequant_gemm_nf4_amd import torch_ops  # noqa: F401  (registers the ops)
from dequant_gemm_nf4_amd.torch_ops import Experts4bit, Linear4bitAdapters

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E = (i << 20 for i in range(1, 6))   # fake device addresses


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "bnbx_rows.h")).read()
    declared = sorted(re.findall(r"BNBX_ROWS_API\s+[\w\s\*]*?\b(bnbx_\w+)\s*\(", text))
    assert declared == sorted(bnbx.ROWS_EXPORTED_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", bnbx.rows_library_path()],
                         capture_output=True, text=True, check=True).stdout
    assert sorted(re.findall(r"\sT\s(\w+)$", out, flags=re.M)) == declared
    assert not set(declared) & set(bnbx.EXPORTED_SYMBOLS)


def state(n, dq=1, **kw):
    f = dict(n=n, blocksize=64, double_quant=dq, quant_type=0, compute_dtype=0, absmax=C,
             absmax2=D if dq else None, absmax_mean=D + 4096 if dq else None)
    f.update(kw)
    return bnbx.Nf4State(**f)


def plan(**kw):
    f = dict(offsets=E, order=E + 8192, groups=4, rows=10)
    f.update(kw)
    return bnbx.RowGroupsDesc(**f)


def status_of(fn, *args):
    try:
        fn(*args)
    except bnbx.BnbxError as e:
        return e.status
    raise AssertionError("call was accepted (it would have launched)")


INVAL, ALIGN, UNSUP, WS = (bnbx.BNBX_E_INVAL, bnbx.BNBX_E_ALIGN, bnbx.BNBX_E_UNSUPPORTED,
                           bnbx.BNBX_E_WORKSPACE)


@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), INVAL), (dict(groups=0), INVAL), (dict(groups=-3), INVAL),
    (dict(groups=1025), UNSUP), (dict(ids=None), INVAL), (dict(order=None), INVAL),
    (dict(offsets=None), INVAL), (dict(ids=A + 2), ALIGN), (dict(order=B + 1), ALIGN),
    (dict(offsets=C + 2), ALIGN), (dict(rows=100000), WS),
    (dict(rows=100000, ws=D, nbytes=8), WS), (dict(rows=100000, ws=D + 2, nbytes=1 << 20), ALIGN)])
def test_group_rows_rejects(kw, expect):
    f = dict(ids=A, rows=10, groups=4, offsets=C, order=B, ws=None, nbytes=0)
    f.update(kw)
    assert status_of(bnbx.bnbx_group_rows, f["ids"], f["rows"], f["groups"], f["offsets"],
                     f["order"], f["ws"], f["nbytes"], 0) == expect


def test_workspace_queries():
    assert bnbx.bnbx_group_rows_workspace_bytes(8192, 1024) == 0
    assert bnbx.bnbx_group_rows_workspace_bytes(8193, 1024) > 0
    assert bnbx.bnbx_group_rows_workspace_bytes(2**31 - 1, 1024) <= 128 * 1025 * 4
    assert bnbx.bnbx_group_rows_workspace_bytes(-1, 4) == 0
    assert bnbx.bnbx_group_rows_workspace_bytes(10**6, 1025) == 0
    assert bnbx.bnbx_gemm_nf4_adapters_workspace_bytes(10, 16) == 10 * 2 * 16 * 2
    assert bnbx.bnbx_gemm_nf4_adapters_workspace_bytes(2**31 - 1, 256) == (2**31 - 1) * 1024
    for r in (0, 8, 24, 272):
        assert bnbx.bnbx_gemm_nf4_adapters_workspace_bytes(10, r) == 0


EXPERT_CASES = [
    (dict(x=None), INVAL), (dict(packed=None), INVAL), (dict(y=None), INVAL),
    (dict(x_rows=-1), INVAL), (dict(y_rows=-1), INVAL), (dict(N=0), INVAL), (dict(K=0), INVAL),
    (dict(K=96), INVAL), (dict(gather=-1), INVAL), (dict(scatter=2), INVAL),
    (dict(ldx=64), INVAL), (dict(ldy=64), INVAL), (dict(ldx=132), ALIGN), (dict(x=A + 2), ALIGN),
    (dict(packed=B + 8), ALIGN), (dict(y=D + 1), ALIGN),
    (dict(plan=plan(groups=0)), INVAL), (dict(plan=plan(groups=5)), INVAL),
    (dict(plan=plan(rows=-1)), INVAL), (dict(plan=plan(offsets=None)), INVAL),
    (dict(plan=plan(order=None)), INVAL), (dict(plan=plan(groups=1025)), UNSUP),
    (dict(plan=plan(order=E + 2)), ALIGN), (dict(plan=plan(offsets=E + 1)), ALIGN),
    (dict(st=state(4 * 128 * 128 - 2)), INVAL), (dict(st=state(128 * 128)), INVAL),
    (dict(st=state(4 * 128 * 128, blocksize=128)), UNSUP),
    (dict(st=state(4 * 128 * 128, quant_type=2)), INVAL),
    (dict(st=state(4 * 128 * 128, compute_dtype=2)), INVAL),
    (dict(st=state(4 * 128 * 128, dq=3)), INVAL),
    (dict(st=state(4 * 128 * 128, absmax=None)), INVAL),
    (dict(st=state(4 * 128 * 128, absmax2=None)), INVAL),
    (dict(st=state(4 * 128 * 128, absmax2=D + 2)), ALIGN),
    (dict(st=state(4 * 128 * 128, dq=0, absmax=C + 2)), ALIGN),
    # more tiles than the kernels count, were the groups to overlap
    (dict(plan=plan(rows=2**31 - 1, groups=1024), st=state(1024 * 128 * 128)), UNSUP),
    # a weight past 32-bit offsets
    (dict(N=1 << 16, K=1 << 16, ldx=1 << 16, ldy=1 << 16, st=state(4 << 32)), UNSUP),
]


@pytest.mark.parametrize("fn", ["bnbx_gemm_nf4_experts", "bnbx_gemm_nf4_experts_dx"])
@pytest.mark.parametrize("kw,expect", EXPERT_CASES)
def test_experts_reject(fn, kw, expect):
    f = dict(x=A, ldx=128, x_rows=10, packed=B, st=state(4 * 128 * 128), plan=plan(), N=128, K=128,
             gather=1, scatter=0, y=D + 65536, ldy=128, y_rows=10)
    f.update(kw)
    assert status_of(getattr(bnbx, fn), f["x"], f["ldx"], f["x_rows"], f["packed"], f["st"],
                     f["plan"], f["N"], f["K"], f["gather"], f["scatter"], f["y"], f["ldy"],
                     f["y_rows"], 0) == expect


def test_experts_dx_needs_whole_steps_of_rows():
    st = state(4 * 96 * 128)
    assert status_of(bnbx.bnbx_gemm_nf4_experts_dx, A, 96, 10, B, st, plan(), 96, 128, 0, 0, D,
                     128, 10, 0) == UNSUP


def test_calls_without_rows_do_nothing():
    """No rows in the plan, in X or in Y: accepted without a launch (there is
    no GPU here to launch on)."""
    st = state(4 * 128 * 128)
    empty = plan(rows=0, order=None)
    for fn in (bnbx.bnbx_gemm_nf4_experts, bnbx.bnbx_gemm_nf4_experts_dx):
        fn(A, 128, 10, B, st, empty, 128, 128, 0, 0, D, 128, 10, 0)
        fn(None, 128, 0, B, st, plan(), 128, 128, 0, 0, D, 128, 10, 0)
        fn(A, 128, 10, B, st, plan(), 128, 128, 0, 0, None, 128, 0, 0)
    ad = adapters()
    bnbx.bnbx_gemm_nf4_adapters(None, 128, B, state(128 * 128), empty, 128, 128, ad, None, 128,
                                None, 0, 0)


BIG = dict(lda=64, stride_a=16 * 64, ldb=16, stride_b=4096 * 16)


@pytest.mark.parametrize("rows,groups,n", [
    # a last tile would pass 31 bits: every row in one group, or in two
    (2**31 - 1, 1, 16), (2**31 - 256, 2, 16),
    # more workgroups than a launch counts threads for (2^23 of 512), X past the
    # 32-bit offsets of the tiled form
    (2**24, 1, 4096), (2**24, 3, 8000)])
def test_more_rows_than_a_launch_takes(rows, groups, n):
    st, one = state(groups * n * 64), state(n * 64)
    p = plan(rows=rows, groups=groups)
    assert status_of(bnbx.bnbx_gemm_nf4_experts, A, 64, rows, B, st, p, n, 64, 1, 1, D, n, rows,
                     0) == UNSUP
    n64 = -(-n // 64) * 64
    assert status_of(bnbx.bnbx_gemm_nf4_experts_dx, A, 64, rows, B, state(groups * n64 * 64), p, 64,
                     n64, 1, 1, D, n64, rows, 0) == UNSUP
    assert status_of(bnbx.bnbx_gemm_nf4_adapters, A, 64, B, one, p, n, 64, adapters(**BIG), D, n,
                     E, 2**40, 0) == UNSUP


def adapters(**kw):
    f = dict(lora_a=A + 65536, lora_b=B + 65536, scale=C + 65536, lda=128, stride_a=16 * 128,
             ldb=16, stride_b=128 * 16, r=16)
    f.update(kw)
    return bnbx.AdaptersDesc(**f)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INVAL), (dict(y=None), INVAL), (dict(K=100), INVAL), (dict(ldy=100), INVAL),
    (dict(ldx=130), ALIGN), (dict(st=state(4 * 128 * 128)), INVAL), (dict(ad=None), INVAL),
    (dict(ad=adapters(lora_a=None)), INVAL), (dict(ad=adapters(lora_b=None)), INVAL),
    (dict(ad=adapters(scale=None)), INVAL), (dict(ad=adapters(r=8)), INVAL),
    (dict(ad=adapters(r=24, ldb=24)), INVAL), (dict(ad=adapters(r=272, ldb=272)), INVAL),
    (dict(ad=adapters(lda=64)), INVAL), (dict(ad=adapters(ldb=8)), INVAL),
    (dict(ad=adapters(stride_a=-8)), INVAL), (dict(ad=adapters(stride_b=-8)), INVAL),
    (dict(ad=adapters(lda=132)), ALIGN), (dict(ad=adapters(ldb=20)), ALIGN),
    (dict(ad=adapters(stride_a=4)), ALIGN), (dict(ad=adapters(stride_b=4)), ALIGN),
    (dict(ad=adapters(lora_a=A + 8)), ALIGN), (dict(ad=adapters(lora_b=A + 8)), ALIGN),
    (dict(ad=adapters(scale=C + 2)), ALIGN), (dict(ws=None), WS), (dict(nbytes=639), WS),
    (dict(ws=E + 65544), ALIGN), (dict(plan=plan(groups=0)), INVAL)])
def test_adapters_reject(kw, expect):
    f = dict(x=A, ldx=128, packed=B, st=state(128 * 128), plan=plan(), N=128, K=128, ad=adapters(),
             y=D + 65536, ldy=128, ws=E + 65536, nbytes=640)
    f.update(kw)
    assert status_of(bnbx.bnbx_gemm_nf4_adapters, f["x"], f["ldx"], f["packed"], f["st"],
                     f["plan"], f["N"], f["K"], f["ad"], f["y"], f["ldy"], f["ws"], f["nbytes"],
                     0) == expect


# ---------------------------------------------------------------------------
# the torch-tensor layer
# ---------------------------------------------------------------------------
def cpu_plan(groups=3, rows=6):
    return T.RowGroups(groups, torch.zeros(groups + 1, dtype=torch.int32),
                       torch.zeros(rows, dtype=torch.int32))


def cpu_stack(shape=(3, 64, 128), dtype=torch.bfloat16):
    return T.empty_quantized(shape, True, "cpu", dtype=dtype)


def test_a_plan_checks_its_arrays():
    i32 = dict(dtype=torch.int32)
    for offsets, order in ((torch.zeros(4), torch.zeros(6, **i32)),
                           (torch.zeros(3, **i32), torch.zeros(6, **i32)),
                           (torch.zeros(4, **i32), torch.zeros(2, 3, **i32)),
                           (torch.zeros(4, **i32), torch.zeros(12, **i32)[::2]),
                           (torch.zeros(4, **i32), torch.zeros(6, dtype=torch.int64))):
        with pytest.raises(ValueError):
            T.RowGroups(3, offsets, order)


def test_a_workspace_is_checked():
    device = torch.device("meta")
    assert T._scratch(None, 64, device).numel() == 64
    given = torch.empty(16, device="meta")
    assert T._scratch(given, 64, device) is given
    for bad in (torch.empty(16), torch.empty(8, 8, device="meta")[:, :2]):
        with pytest.raises(ValueError):
            T._scratch(bad, 64, device)


def test_rows_past_31_bits_are_refused():
    with pytest.raises(ValueError):
        T.RowGroups(1, torch.empty(2, dtype=torch.int32, device="meta"),
                    torch.empty(2**31, dtype=torch.int32, device="meta"))
    with pytest.raises(ValueError):
        T.group_rows(torch.empty(2**31, dtype=torch.int32, device="meta"), 1)
    with pytest.raises(ValueError):
        T._check_matrix("x", torch.empty(2**31, 64, dtype=torch.bfloat16, device="meta"), 64,
                        torch.bfloat16, torch.device("meta"))


def test_group_rows_checks():
    with pytest.raises(ValueError):
        T.group_rows(torch.zeros(4, dtype=torch.int64), 3)
    with pytest.raises(ValueError):
        T.group_rows(torch.zeros(2, 2, dtype=torch.int32), 3)
    with pytest.raises(ValueError):
        T.group_rows(torch.zeros(4, dtype=torch.int32), 3, out=cpu_plan(3, 5))
    with pytest.raises(ValueError, match="GPU"):
        T.group_rows(torch.zeros(4, dtype=torch.int32), 3)


@pytest.mark.parametrize("fn,width,out", [(T.gemm_experts, 128, 64), (T.gemm_experts_dx, 64, 128)])
def test_experts_checks(fn, width, out):
    bf = dict(dtype=torch.bfloat16)
    x, q, p = torch.zeros(6, width, **bf), cpu_stack(), cpu_plan()
    with pytest.raises(ValueError):
        fn(x, cpu_stack((64, 128)), p)                    # not a stack
    with pytest.raises(ValueError):
        fn(x, q, cpu_plan(4))                             # other groups
    with pytest.raises(ValueError):
        fn(torch.zeros(6, width + 8, **bf), q, p)
    with pytest.raises(TypeError):
        fn(x.half(), q, p)
    with pytest.raises(ValueError):
        fn(x[:5], q, p)                                   # fewer rows than places
    with pytest.raises(ValueError):
        fn(x[:2], q, p, gather=2)                         # three tokens of two slots
    with pytest.raises(ValueError):
        fn(x, q, p, gather=-1)
    with pytest.raises(ValueError):
        fn(torch.zeros(width, 6, **bf).t(), q, p)         # columns contiguous
    with pytest.raises(ValueError):
        fn(x, q, p, out=torch.zeros(5, out, **bf))
    with pytest.raises(TypeError):
        fn(x, q, p, out=torch.zeros(6, out))
    with pytest.raises(ValueError, match="GPU"):
        fn(x, q, p)


def test_a_weight_holds_what_its_shape_says():
    """The kernels read all of a weight's shape: buffers of fewer elements,
    other types or views are refused."""
    bf = dict(dtype=torch.bfloat16)
    x, p, a, b, s = (torch.zeros(6, 128, **bf), cpu_plan(), torch.zeros(3, 16, 128, **bf),
                     torch.zeros(3, 64, 16, **bf), torch.ones(3))
    for dq, dq_map in ((True, "linear"), (True, "dynamic"), (False, "linear")):
        whole = T.empty_quantized((3, 64, 128), dq, "cpu", dq_map=dq_map)
        one = T.empty_quantized((64, 128), dq, "cpu", dq_map=dq_map)
        for q, call in ((whole, lambda q: T.gemm_experts(x, q, p)),
                        (whole, lambda q: T.gemm_experts_dx(x[:, :64], q, p)),
                        (one, lambda q: T.linear_adapters(x, q, p, a, b, s))):
            with pytest.raises(ValueError, match="GPU"):
                call(q)
            bad = [dict(packed=q.packed[:-1]), dict(packed=q.packed.view(torch.int8)),
                   dict(absmax=q.absmax[:-1]), dict(absmax=q.absmax.to(torch.float64)),
                   dict(packed=torch.zeros(2 * q.packed.numel(), dtype=torch.uint8)[::2])]
            if dq:
                bad += [dict(absmax2=q.absmax2[:0]), dict(absmax2=None), dict(absmax_mean=None),
                        dict(absmax_mean=q.absmax_mean.double()), dict(absmax=q.absmax.float()),
                        dict(absmax2=q.absmax2.to("meta"))]
            for kw in bad:
                with pytest.raises(ValueError, match="the weight's"):
                    call(dataclasses.replace(q, **kw))


def test_rows_wider_than_the_weight_are_refused():
    """The ops take K (N for the gradient) from the rows: a layer given wider ones
    would read past its weight."""
    m, p = Experts4bit(3, 128, 64, device="cpu"), cpu_plan()
    wide = torch.zeros(6, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="the weight's"):
        m(wide, (p.offsets, p.order), gather=1)
    with pytest.raises(ValueError, match="the weight's"):
        torch.ops.bnbx.experts4bit_dx(wide, m.packed, m.absmax, m.absmax2, m.absmax_mean, p.offsets,
                                      p.order, 128, 1, False, "nf4")
    layer = Linear4bitAdapters(128, 64, adapters=3, device="cpu")
    with pytest.raises(ValueError, match="the weight's"):
        layer(wide, (p.offsets, p.order))
    plain = torch_ops.Linear4bit(128, 64, device="cpu")
    with pytest.raises(ValueError, match="the weight's"):
        plain(wide)
    with pytest.raises(ValueError, match="the weight's"):
        torch.ops.bnbx.linear4bit_dx(wide, m.packed, m.absmax, m.absmax2, m.absmax_mean, 128, "nf4")


def test_adapters_checks():
    bf = dict(dtype=torch.bfloat16)
    x, q, p = torch.zeros(6, 128, **bf), cpu_stack((64, 128)), cpu_plan()
    a, b, s = torch.zeros(3, 16, 128, **bf), torch.zeros(3, 64, 16, **bf), torch.ones(3)
    f = T.linear_adapters
    for bad in ((x, cpu_stack(), p, a, b, s), (x[:5], q, p, a, b, s), (x, q, p, a[:2], b, s),
                (x, q, p, a, b[:2], s), (x, q, p, a, b, s[:2]), (x, q, p, a[0], b, s),
                (x, q, p, a, b[:, :, :8], s), (x, q, p, a[:, :, ::1].transpose(1, 2), b, s)):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(TypeError):
        f(x, q, p, a.half(), b, s)
    with pytest.raises(TypeError):
        f(x, q, p, a, b, s.double())
    with pytest.raises(ValueError):
        f(x, q, p, a, b, s, out=torch.zeros(5, 64, **bf))
    with pytest.raises(ValueError, match="GPU"):
        f(x, q, p, a, b, s)


# ---------------------------------------------------------------------------
# the ops and modules, shapes only
# ---------------------------------------------------------------------------
def meta_plan(ids, groups):
    return torch.ops.bnbx.group_rows(ids, groups)


def test_ops_on_meta():
    offsets, order = meta_plan(torch.empty(5, 2, dtype=torch.int32, device="meta"), 4)
    assert offsets.shape == (5,) and order.shape == (10,) and order.dtype == torch.int32
    m = Experts4bit(4, 128, 96, device="meta")
    assert m.packed.shape == (4 * 96 * 128 // 2,) and m.quantized().shape == (4, 96, 128)
    x = torch.empty(5, 128, dtype=torch.bfloat16, device="meta")
    assert m(x, (offsets, order), gather=2).shape == (10, 96)
    assert "experts=4" in repr(m) and "out_features=96" in repr(m)


def test_experts_autograd_shapes_on_meta():
    plan = meta_plan(torch.empty(5, 2, dtype=torch.int32, device="meta"), 4)
    up, down = (Experts4bit(4, 128, 64, device="meta"), Experts4bit(4, 64, 128, device="meta"))
    x = torch.empty(5, 128, dtype=torch.bfloat16, device="meta", requires_grad=True)
    y = down(up(x, plan, gather=2), plan, scatter=True)
    assert y.shape == (10, 128)
    (g,) = torch.autograd.grad(y, x, torch.empty_like(y))
    assert g.shape == x.shape and g.dtype == x.dtype


def test_experts_module_checks():
    with pytest.raises(ValueError):
        Experts4bit(0, 128, 64, device="meta")
    with pytest.raises(ValueError):
        Experts4bit(2, 100, 64, device="meta")
    m = Experts4bit(2, 128, 64, device="meta")
    plan = meta_plan(torch.empty(3, dtype=torch.int32, device="meta"), 2)
    with pytest.raises(TypeError):
        m(torch.empty(3, 128, dtype=torch.float16, device="meta"), plan, gather=1)
    with pytest.raises(ValueError):
        m(torch.empty(3, 128, dtype=torch.bfloat16, device="meta"),
          meta_plan(torch.empty(3, dtype=torch.int32, device="meta"), 3), gather=1)
    with pytest.raises(ValueError):
        m.load_weight(torch.empty(2, 128, 64, dtype=torch.bfloat16, device="meta"))
    with pytest.raises(TypeError):
        Experts4bit.from_linear(torch.nn.Linear(128, 64, bias=False))


def test_adapters_module_on_meta():
    m = Linear4bitAdapters(128, 96, adapters=5, rank=32, device="meta")
    assert m.lora_a.shape == (5, 32, 128) and m.lora_b.shape == (5, 96, 32)
    plan = meta_plan(torch.empty(6, dtype=torch.int32, device="meta"), 5)
    x = torch.empty(2, 3, 128, dtype=torch.bfloat16, device="meta", requires_grad=True)
    y = m(x, plan)
    assert y.shape == (2, 3, 96)
    with pytest.raises(RuntimeError, match="autograd"):
        y.sum().backward()
    with pytest.raises(ValueError):
        m(x, meta_plan(torch.empty(6, dtype=torch.int32, device="meta"), 4))
    with pytest.raises(TypeError):
        m(x.half(), plan)
    assert "adapters=5, rank=32" in repr(m)
    for kw in (dict(rank=8), dict(rank=272), dict(adapters=0)):
        with pytest.raises(ValueError):
            Linear4bitAdapters(128, 96, **{"adapters": 2, "rank": 16, **kw}, device="meta")
    m = Linear4bitAdapters(128, 96, adapters=2, rank=32, device="cpu")
    a, b = torch.ones(16, 128), torch.ones(96, 16)
    for bad in ((2, a, b), (-1, a, b), (0, a[:, :64], b), (0, a, b[:, :8]), (0, a[0], b),
                (0, torch.ones(48, 128), torch.ones(96, 48))):
        with pytest.raises(ValueError):
            m.load_adapter(*bad)
    m.load_adapter(1, a * 3, b * 3, 0.5)
    m.load_adapter(1, a[:8], b[:, :8], 2.0)              # a lower rank leaves no rest
    assert m.lora_a[1].float().sum() == 8 * 128 and m.lora_b[1].float().sum() == 8 * 96
    assert m.scale.tolist() == [0.0, 2.0] and not m.lora_a[0].any()
