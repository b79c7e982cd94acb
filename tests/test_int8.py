"""The 8-bit operators without a GPU: the exported symbols, every refusal on the
host before a launch (the pointers are never dereferenced), the torch-tensor
layer's checks, the ops' and modules' shapes on meta tensors, and the two
constructions of the row format that the GPU tests compare with."""

import dataclasses
import os
import re
import subprocess

import pytest
import torch

import dequant_gemm_nf4_amd as bnbx
from dequant_gemm_nf4_amd import tensors as T
from dequant_gemm_nf4_amd.torch_ops import Linear8bit, Linear8bitTrain
from int8_helpers import codes_by_definition, codes_in_64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F = (i << 20 for i in range(1, 7))   # fake device addresses
INVAL, ALIGN, UNSUP, WS = (bnbx.BNBX_E_INVAL, bnbx.BNBX_E_ALIGN, bnbx.BNBX_E_UNSUPPORTED,
                           bnbx.BNBX_E_WORKSPACE)


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "bnbx_int8.h")).read()
    declared = sorted(re.findall(r"BNBX_INT8_API\s+[\w\s\*]*?\b(bnbx_\w+)\s*\(", text))
    assert declared == sorted(bnbx.INT8_EXPORTED_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", bnbx.int8_library_path()],
                         capture_output=True, text=True, check=True).stdout
    assert sorted(re.findall(r"\sT\s(\w+)$", out, flags=re.M)) == declared
    assert not set(declared) & (set(bnbx.EXPORTED_SYMBOLS) | set(bnbx.ROWS_EXPORTED_SYMBOLS))
    assert int(re.search(r"BNBX_INT8_MAX_COLS (\d+)", text).group(1)) == bnbx.BNBX_INT8_MAX_COLS
    assert int(re.search(r"BNBX_DTYPE_F32 = (\d+)", text).group(1)) == bnbx.BNBX_DTYPE_F32


def rows(codes=A, scale=B, ld=1024, rows=100, cols=1000, dtype=0):
    return bnbx.Int8RowsDesc(codes, scale, ld, rows, cols, dtype)


def status_of(fn, *args):
    try:
        fn(*args)
    except bnbx.BnbxError as e:
        return e.status
    raise AssertionError("call was accepted (it would have launched)")


BAD_ROWS = [
    (dict(rows=-1), INVAL), (dict(cols=0), INVAL), (dict(cols=-5), INVAL), (dict(dtype=2), INVAL),
    (dict(dtype=-1), INVAL), (dict(ld=992), INVAL), (dict(ld=-1024), INVAL),
    (dict(codes=None), INVAL), (dict(scale=None), INVAL), (dict(ld=1032), ALIGN),
    (dict(codes=A + 8), ALIGN), (dict(scale=B + 2), ALIGN), (dict(ld=1 << 23), UNSUP)]


@pytest.mark.parametrize("kw,expect", BAD_ROWS)
def test_rows_are_refused_everywhere(kw, expect):
    bad, good = rows(**kw), rows()
    assert status_of(bnbx.bnbx_quantize_rows_int8, C, 1024, bad, 0) == expect
    assert status_of(bnbx.bnbx_dequantize_rows_int8, bad, C, 1024, 0) == expect
    assert status_of(bnbx.bnbx_gemm_int8, bad, good, C, 100, D, 1 << 30, 0) == expect
    assert status_of(bnbx.bnbx_gemm_int8, good, bad, C, 100, D, 1 << 30, 0) == expect
    assert status_of(bnbx.bnbx_linear_int8, C, 1024, 100, bad, None, D, 100, E, 1 << 30, 0) == expect
    assert status_of(bnbx.bnbx_linear_int8, C, 1024, 100, good, bad, D, 100, E, 1 << 30,
                     0) == expect
    assert status_of(bnbx.bnbx_gemm_int8_dx, C, 104, 100, bad, D, 1000, E, 1 << 30, 0) == expect
    assert status_of(bnbx.bnbx_gemm_int8_dw, C, 104, 100, bad, D, 1000, 0, E, 1 << 30, 0) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INVAL), (dict(ldx=999), INVAL), (dict(x=C + 1), ALIGN)])
def test_quantize_and_dequantize_reject(kw, expect):
    f = dict(x=C, ldx=1000)
    f.update(kw)
    assert status_of(bnbx.bnbx_quantize_rows_int8, f["x"], f["ldx"], rows(), 0) == expect
    assert status_of(bnbx.bnbx_dequantize_rows_int8, rows(), f["x"], f["ldx"], 0) == expect


LONG = dict(cols=20000, ld=20000)


@pytest.mark.parametrize("kw,expect", [
    (dict(y=None), INVAL), (dict(ldy=99), INVAL), (dict(y=C + 1), ALIGN),
    (dict(w=rows(cols=999)), INVAL), (dict(w=rows(**LONG, dtype=1)), INVAL),
    (dict(w=rows(**LONG, rows=0)), INVAL),
    (dict(x=rows(cols=131072, ld=131072), w=rows(cols=131072, ld=131072)), UNSUP),
    (dict(ws=None), WS), (dict(nbytes=16), WS), (dict(ws=D + 8), ALIGN)])
def test_gemm_rejects(kw, expect):
    f = dict(x=rows(**LONG, rows=200), w=rows(**LONG), y=C, ldy=100, ws=D, nbytes=1 << 30)
    f.update(kw)
    assert bnbx.bnbx_gemm_int8_workspace_bytes(200, 100, 20000) > 16
    assert status_of(bnbx.bnbx_gemm_int8, f["x"], f["w"], f["y"], f["ldy"], f["ws"], f["nbytes"],
                     0) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INVAL), (dict(x=None), INVAL), (dict(ldx=999), INVAL), (dict(x=C + 1), ALIGN),
    (dict(y=None), INVAL), (dict(ldy=99), INVAL), (dict(y=D + 1), ALIGN),
    (dict(saved=rows(rows=199)), INVAL), (dict(saved=rows(rows=200, cols=999)), INVAL),
    (dict(saved=rows(rows=200, dtype=1)), INVAL), (dict(w=rows(rows=0)), INVAL),
    (dict(w=rows(cols=131072, ld=131072), ldx=131072), UNSUP),
    (dict(ws=None), WS), (dict(nbytes=199 * 1008), WS), (dict(ws=E + 8), ALIGN)])
def test_linear_rejects(kw, expect):
    f = dict(x=C, ldx=1000, M=200, w=rows(), saved=None, y=D, ldy=100, ws=E, nbytes=1 << 30)
    f.update(kw)
    assert status_of(bnbx.bnbx_linear_int8, f["x"], f["ldx"], f["M"], f["w"], f["saved"], f["y"],
                     f["ldy"], f["ws"], f["nbytes"], 0) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), INVAL), (dict(dy=None), INVAL), (dict(lddy=96), INVAL), (dict(dy=C + 8), ALIGN),
    (dict(lddy=100), ALIGN), (dict(lddy=1 << 22), UNSUP), (dict(dx=None), INVAL),
    (dict(lddx=999), INVAL), (dict(dx=D + 1), ALIGN), (dict(w=rows(rows=0)), INVAL),
    (dict(w=rows(rows=4000), lddy=4000, M=100, ws=None), WS),
    (dict(w=rows(rows=4000), lddy=4000, M=100, nbytes=16), WS)])
def test_dx_rejects(kw, expect):
    f = dict(dy=C, lddy=104, M=200, w=rows(), dx=D, lddx=1000, ws=E, nbytes=1 << 30)
    f.update(kw)
    assert bnbx.bnbx_gemm_int8_dx_workspace_bytes(100, 4000, 1000) > 16
    assert status_of(bnbx.bnbx_gemm_int8_dx, f["dy"], f["lddy"], f["M"], f["w"], f["dx"], f["lddx"],
                     f["ws"], f["nbytes"], 0) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(N=0), INVAL), (dict(N=-1), INVAL), (dict(dy=None), INVAL), (dict(lddy=96), INVAL),
    (dict(dy=C + 8), ALIGN), (dict(lddy=100), ALIGN), (dict(lddy=1 << 22), UNSUP),
    (dict(dw=None), INVAL), (dict(lddw=999), INVAL), (dict(dw=D + 1), ALIGN),
    (dict(dw=D + 2, out=2), ALIGN), (dict(out=1), INVAL), (dict(out=3), INVAL),
    (dict(x=rows(rows=4000), ws=None), WS), (dict(x=rows(rows=4000), nbytes=16), WS)])
def test_dw_rejects(kw, expect):
    f = dict(dy=C, lddy=104, N=100, x=rows(), dw=D, lddw=1000, out=0, ws=E, nbytes=1 << 30)
    f.update(kw)
    assert bnbx.bnbx_gemm_int8_dw_workspace_bytes(4000, 100, 1000) > 16
    assert status_of(bnbx.bnbx_gemm_int8_dw, f["dy"], f["lddy"], f["N"], f["x"], f["dw"], f["lddw"],
                     f["out"], f["ws"], f["nbytes"], 0) == expect


def test_sizes_past_a_launch_are_refused_before_anything_is_enqueued():
    most = 2**31 - 512
    big = dict(ws=E, nbytes=1 << 62)
    for M, N in ((most + 1, 16), (16, most + 1), (20, most), (100, most)):
        x, w = rows(rows=M, cols=32, ld=32), rows(rows=N, cols=32, ld=32)
        assert status_of(bnbx.bnbx_gemm_int8, x, w, C, N, big["ws"], big["nbytes"], 0) == UNSUP
        assert status_of(bnbx.bnbx_linear_int8, C, 32, M, w, None, D, N, big["ws"], big["nbytes"],
                         0) == UNSUP
    w = rows(rows=16, cols=32, ld=32)
    assert status_of(bnbx.bnbx_gemm_int8_dx, C, 16, most + 1, w, D, 32, E, 1 << 62, 0) == UNSUP
    assert status_of(bnbx.bnbx_gemm_int8_dw, C, 16, 16, rows(rows=most + 1, cols=32, ld=32), D, 32,
                     0, E, 1 << 62, 0) == UNSUP


def test_calls_without_rows_do_nothing():
    none = rows(codes=None, scale=None, rows=0)
    bnbx.bnbx_quantize_rows_int8(None, 1000, none, 0)
    bnbx.bnbx_dequantize_rows_int8(none, None, 1000, 0)
    bnbx.bnbx_gemm_int8(none, rows(), None, 100, None, 0, 0)
    bnbx.bnbx_linear_int8(None, 1000, 0, rows(), None, None, 100, None, 0, 0)
    bnbx.bnbx_linear_int8(None, 1000, 0, rows(), none, None, 100, None, 0, 0)
    bnbx.bnbx_gemm_int8_dx(None, 104, 0, rows(), None, 1000, None, 0, 0)


def test_workspace_queries():
    for fn in (bnbx.bnbx_gemm_int8_workspace_bytes, bnbx.bnbx_linear_int8_workspace_bytes,
               bnbx.bnbx_gemm_int8_dx_workspace_bytes):
        for bad in ((0, 5, 5), (-1, 5, 5), (5, 0, 5), (5, 5, 0), (5, 5, -1)):
            assert fn(*bad) == 0
    assert bnbx.bnbx_gemm_int8_dw_workspace_bytes(-1, 5, 5) == 0
    assert bnbx.bnbx_gemm_int8_dw_workspace_bytes(0, 5, 5) == 0
    assert bnbx.bnbx_gemm_int8_workspace_bytes(100, 100, 131072) == 0
    # codes of X: whole rows of 16 bytes, then the scales, in pieces of 256
    n = bnbx.bnbx_linear_int8_workspace_bytes(2048, 8192, 8190)
    assert n == 2048 * 8192 + 2048 * 4
    assert bnbx.bnbx_linear_int8_workspace_bytes(2048, 8192, 8190, 1) == 0
    # one token: everything in one launch
    assert bnbx.bnbx_linear_int8_workspace_bytes(1, 4096, 4096) == 0
    # sums too large for a weight's 32 bits are counted in 64
    assert bnbx.bnbx_linear_int8_workspace_bytes(2**31 - 1, 16, 131071) >= (2**31 - 1) * 131072


def cpu_rows(r, c, dtype=torch.bfloat16, **kw):
    q = T.empty_int8_rows((r, c), dtype, "cpu")
    return dataclasses.replace(q, **kw) if kw else q


def test_rows_check_their_tensors():
    good = cpu_rows(3, 20)
    assert good.codes.shape == (3, 32) and good.desc.ld == 32 and good.desc.cols == 20
    assert cpu_rows(1, 20, codes=torch.empty(1, 48, dtype=torch.int8)).desc.ld == 32
    for bad in (dict(shape=(3, 20, 1)), dict(shape=(3, 0)), dict(shape=(4, 20)),
                dict(shape=(3, 33)), dict(codes=torch.empty(3, 64, dtype=torch.int8)[:, ::2]),
                dict(codes=torch.empty(32, 3, dtype=torch.int8).t()),
                dict(scale=torch.empty(4)), dict(scale=torch.empty(6)[::2])):
        with pytest.raises(ValueError):
            dataclasses.replace(good, **bad)
    for bad in (dict(codes=torch.empty(3, 32, dtype=torch.uint8)), dict(dtype=torch.float32),
                dict(scale=torch.empty(3, dtype=torch.float64))):
        with pytest.raises(TypeError):
            dataclasses.replace(good, **bad)


def test_tensor_layer_refuses():
    x, w = torch.zeros(4, 20, dtype=torch.bfloat16), cpu_rows(6, 20)
    dy = torch.zeros(4, 6, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        T.quantize_rows(x)                              # not on a GPU
    with pytest.raises(TypeError):
        T.quantize_rows(x.float())
    with pytest.raises(ValueError):
        T.quantize_rows(x[0])
    with pytest.raises(ValueError):
        T.quantize_rows(x, out=cpu_rows(4, 21))
    with pytest.raises(ValueError):
        T.quantize_rows(x, out=cpu_rows(4, 20, torch.float16))
    with pytest.raises(ValueError):
        T.quantize_rows(x.t())                          # rows not contiguous
    with pytest.raises(ValueError):
        T.dequantize_rows(w, out=torch.zeros(5, 20, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        T.dequantize_rows(w, out=torch.zeros(6, 20))
    with pytest.raises(ValueError):
        T.linear_int8(torch.zeros(4, 21, dtype=torch.bfloat16), w)
    with pytest.raises(TypeError):
        T.linear_int8(x.half(), w)
    with pytest.raises(ValueError):
        T.linear_int8(x, w, saved=cpu_rows(3, 20))
    with pytest.raises(ValueError):
        T.linear_int8(x, w, out=torch.zeros(4, 5, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        T.gemm_int8(cpu_rows(4, 21), w)
    with pytest.raises(ValueError):
        T.gemm_int8(cpu_rows(4, 20, torch.float16), w)
    with pytest.raises(ValueError):
        T.gemm_int8_dx(torch.zeros(4, 7, dtype=torch.bfloat16), w)
    with pytest.raises(TypeError):
        T.gemm_int8_dx(dy.half(), w)
    with pytest.raises(ValueError):
        T.gemm_int8_dw(torch.zeros(5, 6, dtype=torch.bfloat16), cpu_rows(4, 20))
    with pytest.raises(TypeError):
        T.gemm_int8_dw(dy, cpu_rows(4, 20), dtype=torch.float16)
    with pytest.raises(TypeError):
        T.gemm_int8_dw(dy, cpu_rows(4, 20), out=torch.zeros(6, 20), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        T.gemm_int8_dw(dy, cpu_rows(4, 20), out=torch.zeros(7, 20))


def test_gradient_pieces_are_copied_where_they_must_be():
    whole = torch.zeros(5, 16, dtype=torch.bfloat16)
    assert T._pieces(whole, True) is whole
    ragged = torch.arange(35, dtype=torch.float32).reshape(5, 7).bfloat16()
    copy = T._pieces(ragged, True)
    assert copy.stride(0) == 8 and torch.equal(copy, ragged)
    assert not copy.as_strided((5, 8), (8, 1))[:, 7].any()
    wide = torch.zeros(5, 16, dtype=torch.bfloat16)[:, :7]
    assert T._pieces(wide, False) is wide and T._pieces(wide, True) is not wide
    # the last row's piece would end behind the storage
    short = torch.zeros(4 * 16 + 7, dtype=torch.bfloat16).as_strided((5, 7), (16, 1))
    assert T._pieces(short, False) is not short
    one = torch.zeros(1, 7, dtype=torch.bfloat16).expand(5, 7)
    assert T._pieces(one, False).stride(0) == 8


def test_ops_on_meta_tensors():
    ops = torch.ops.bnbx
    x = torch.empty(2, 3, 20, dtype=torch.bfloat16, device="meta", requires_grad=True)
    codes = torch.empty(8, 32, dtype=torch.int8, device="meta")
    scale = torch.empty(8, device="meta")
    y = ops.linear8bit(x, codes, scale)
    assert y.shape == (2, 3, 8) and y.dtype == torch.bfloat16
    y.sum().backward()
    assert x.grad.shape == x.shape
    q, s = ops.quantize_rows8(x.detach())
    assert q.shape == (6, 32) and q.dtype == torch.int8 and s.shape == (6,)
    assert ops.linear8bit_dw(y.detach(), q, s, 20, torch.float32).shape == (8, 20)
    w = torch.empty(8, 20, dtype=torch.bfloat16, device="meta", requires_grad=True)
    out = ops.linear8bit_train(x, w)
    assert [tuple(o.shape) for o in out] == [(2, 3, 8), (6, 32), (6,), (8, 32), (8,)]
    assert [o.requires_grad for o in out] == [True, False, False, False, False]
    out[0].sum().backward()
    assert w.grad.shape == w.shape and w.grad.dtype == torch.bfloat16


def test_modules_refuse():
    with pytest.raises(ValueError):
        Linear8bit(16, 16, torch.float32, device="meta")
    with pytest.raises(ValueError):
        Linear8bit(0, 16, device="meta")
    with pytest.raises(ValueError):
        Linear8bitTrain(16, 16, torch.float32, device="meta")
    m = Linear8bit(20, 8, device="meta")
    with pytest.raises(ValueError):
        m.load_weight(torch.zeros(20, 8))
    with pytest.raises(TypeError):
        m(torch.zeros(2, 20, device="meta"))
    with pytest.raises(TypeError):
        Linear8bitTrain(20, 8, device="meta")(torch.zeros(2, 20, device="meta"))
    biased = torch.nn.Linear(4, 4, device="meta")
    for cls in (Linear8bit, Linear8bitTrain):
        with pytest.raises(ValueError):
            cls.from_linear(biased)
    assert m(torch.zeros(5, 20, device="meta", dtype=torch.bfloat16)).shape == (5, 8)
    assert sorted(m.state_dict()) == ["codes", "scale"]


def test_the_two_constructions_of_the_codes_agree():
    g = torch.Generator().manual_seed(3)
    for dtype in (torch.bfloat16, torch.float16):
        x = torch.randn(40, 50, generator=g).to(dtype)
        x[3] = 0
        x[5, 7] = float("inf")
        x[6] = x[6] * 1e-6
        a, s = codes_by_definition(x)
        b, t = codes_in_64(x)
        assert torch.equal(a, b)
        assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(t, nan=-1.0))
