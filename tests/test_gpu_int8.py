"""The 8-bit operators on the GPU against their definitions in binary64: the row
format, the products over codes, and both gradients, at sizes around their tiles,
pieces and splits."""

import math

import pytest
import torch

from dequant_gemm_nf4_amd import tensors as T
from int8_helpers import (DT, check, codes_by_definition, codes_in_64, gradient_check, held, rand,
                          values_of)

pytestmark = pytest.mark.gpu


def activations(rows, cols, seed, dtype="bf16"):
    """Normal rows with a few large columns, one row of zeros."""
    x = rand((rows, cols), seed, 1.0, dtype)
    x[:, ::97] *= 8
    if rows > 2:
        x[rows // 2] = 0
    return x


# ---------------------------------------------------------------------------
# rows -> codes -> values
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 16), (2, 17), (7, 512), (4, 520),
                                       (6, 2049), (3, 4096), (2, 8200), (2, 16400), (3, 32769),
                                       (1, 40000)])
def test_quantize_is_the_definition(rows, cols, dtype):
    x = activations(rows, cols, rows * 131 + cols, dtype)
    q = T.quantize_rows(x)
    codes, scale = codes_in_64(x)
    assert torch.equal(q.codes[:, :cols].long(), codes)
    assert torch.equal(q.scale, scale)
    assert not q.codes[:, cols:].any()
    if rows * cols <= 4000:
        by_def, s = codes_by_definition(x)
        assert torch.equal(codes.cpu(), by_def) and torch.equal(scale.cpu(), s)
    v = T.dequantize_rows(q)
    assert torch.equal(v.double(), values_of(codes, scale, DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1500, 300), (1100, 2000), (1030, 4096), (1025, 8192),
                                       (1024, 11008)])
def test_quantize_many_rows(rows, cols, dtype):
    x = activations(rows, cols, rows + cols, dtype)
    q = T.quantize_rows(x)
    codes, scale = codes_in_64(x)
    assert torch.equal(q.codes[:, :cols].long(), codes)
    assert torch.equal(q.scale, scale)
    assert torch.equal(T.dequantize_rows(q).double(), values_of(codes, scale, DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_ties_go_to_even(dtype):
    """a = 127 2^k makes a code of every x / 2^k: halves are ties."""
    row = torch.arange(-254, 255, dtype=torch.float32) / 2
    x = torch.stack([row.clamp(-127, 127) * 2.0 ** k for k in (-8, -1, 0, 3)]).to(DT[dtype])
    x = x.cuda()
    codes, scale = codes_by_definition(x)
    q = T.quantize_rows(x)
    assert torch.equal(q.codes[:, :x.shape[1]].long().cpu(), codes)
    assert torch.equal(q.scale.cpu(), scale)
    assert bool((codes[0].float() == torch.round(row.clamp(-127, 127))).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_pair_of_significands(dtype):
    """Rows whose maximum takes every significand of the type (binary16: every
    eighth), each with all values of two exponents below it."""
    bits = 7 if dtype == "bf16" else 10
    one = 127 << 7 if dtype == "bf16" else 15 << 10
    tops = range(0, 1 << bits, 1 if dtype == "bf16" else 8)
    row = torch.arange(one - (2 << bits) - 1, one + (1 << bits))
    x = torch.stack([torch.where(row <= one + t, row, torch.zeros_like(row)) for t in tops])
    x = x.to(torch.int16).view(DT[dtype]).cuda()
    q = T.quantize_rows(x)
    codes, scale = codes_in_64(x)
    assert torch.equal(q.codes[:, :x.shape[1]].long(), codes)
    assert torch.equal(q.scale, scale)
    pick = x[::32]
    by_def, _ = codes_by_definition(pick)
    assert torch.equal(codes[::32].cpu(), by_def)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_ends_of_the_range(dtype):
    """The largest and smallest magnitudes of the type, subnormals among them."""
    fi = torch.finfo(DT[dtype])
    small = fi.smallest_normal * fi.eps
    tops = [fi.max, fi.max / 2, fi.smallest_normal, fi.smallest_normal / 2, small, 3 * small, 1.0]
    x = torch.tensor([[t, -t, t / 2, t / 3, 0.0, -t / 127, t / 1000] for t in tops],
                     dtype=torch.float64).to(DT[dtype]).cuda()
    codes, scale = codes_by_definition(x)
    q = T.quantize_rows(x)
    assert torch.equal(q.codes[:, :7].long().cpu(), codes)
    assert torch.equal(q.scale.cpu(), scale)
    v = T.dequantize_rows(q).double().cpu()
    assert torch.equal(v, values_of(codes, scale, DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_quantize_rows_that_are_not_finite(bad, dtype):
    x = activations(5, 700, 3, dtype)
    x[1, 699] = bad
    x[3, 0] = bad
    q = T.quantize_rows(x)
    codes, scale = codes_in_64(x)
    assert torch.equal(q.codes[:, :700].long(), codes)
    assert torch.isnan(q.scale[[1, 3]]).all()
    assert torch.equal(q.scale[[0, 2, 4]], scale[[0, 2, 4]])
    v = T.dequantize_rows(q)
    assert torch.isnan(v[[1, 3]]).all() and torch.isfinite(v[[0, 2, 4]]).all()


@pytest.mark.parametrize("cols,pad,shift", [(64, 8, 0), (64, 3, 0), (61, 0, 0), (64, 8, 1),
                                            (4100, 1, 5), (300, 0, 8)])
def test_quantize_and_dequantize_strides(cols, pad, shift):
    wide = rand((9, cols + pad + shift), cols, 1.0)
    x = wide[:, shift:shift + cols]
    q = T.quantize_rows(x)
    codes, scale = codes_in_64(x)
    assert torch.equal(q.codes[:, :cols].long(), codes) and torch.equal(q.scale, scale)
    out = torch.full_like(wide, 3.0)
    T.dequantize_rows(q, out=out[:, shift:shift + cols])
    want = torch.full_like(wide, 3.0)
    want[:, shift:shift + cols] = values_of(codes, scale, torch.bfloat16).bfloat16()
    assert torch.equal(out, want)


def test_quantize_leaves_what_lies_behind():
    """Rows of a longer pitch: 16-byte pieces behind the padded row stay."""
    x = rand((6, 40), 1)
    buf = torch.full((7, 96), 55, dtype=torch.int8, device="cuda")
    scale = torch.full((7,), 9.0, device="cuda")
    T.quantize_rows(x, out=T.Int8Rows((6, 40), buf[:6], scale[:6]))
    assert (buf[:6, 48:] == 55).all() and (buf[6] == 55).all() and scale[6] == 9.0
    assert not buf[:6, 40:48].any()


# ---------------------------------------------------------------------------
# products over codes
# ---------------------------------------------------------------------------
def product_check(y, x, w, where=""):
    """y[m, n] = rnd16(fl32(fl32(S) sx) sw) with the exact integer S: fl32(S) and two
    products are each off by half a step of binary32 at most."""
    qx, sx = codes_in_64(x)
    qw, sw = codes_in_64(w)
    exact = (qx.double() @ qw.double().t().contiguous()) * sx.double()[:, None] * sw.double()
    fi = torch.finfo(y.dtype)
    tol = exact.abs() * (fi.eps / 2 + 4 * 2.0 ** -24) + fi.smallest_normal * fi.eps
    off = (y.double() - exact).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (where, int(bad.sum()), bad.nonzero()[0].tolist())


SIZES = [(1, 1, 1), (1, 17, 33), (2, 64, 128), (5, 100, 1000), (16, 256, 512), (17, 65, 2050),
         (33, 129, 4096), (64, 64, 64), (65, 63, 16), (100, 1000, 77), (128, 130, 640),
         (300, 700, 1030), (513, 515, 144), (1, 5000, 4096), (16, 4096, 11008), (40, 48, 20000)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_is_the_product_of_the_codes(M, N, K, dtype):
    x, w = activations(M, K, M + K, dtype), rand((N, K), N + K, 0.02, dtype)
    wq = held(w)
    y = T.linear_int8(x, wq)
    product_check(y, x, w, (M, N, K))
    saved = T.empty_int8_rows((M, K), DT[dtype])
    y2 = T.linear_int8(x, wq, saved=saved)
    assert torch.equal(y, y2)
    codes, scale = codes_in_64(x)
    assert torch.equal(saved.codes[:, :K].long(), codes) and torch.equal(saved.scale, scale)
    assert not saved.codes[:, K:].any()
    assert torch.equal(T.gemm_int8(saved, wq), y)


@pytest.mark.parametrize("M,N,K,dtype", [
    (2048, 6100, 512, "bf16"), (1000, 8192, 272, "f16"), (4097, 4096, 96, "bf16"),
    (2000, 8100, 2000, "bf16"), (2047, 4090, 1040, "f16"), (1000, 4090, 1500, "bf16"),
    (290, 4090, 1300, "f16"), (130, 4096, 4096, "bf16"), (70, 300, 20000, "f16"),
    (300, 2000, 16000, "bf16"), (600, 1000, 12000, "f16"), (1, 40, 65536, "bf16"),
    (2, 300, 32768, "f16"), (3, 100, 21824, "bf16"), (4, 50, 16384, "f16"),
    (4, 50, 16400, "bf16"), (64, 130, 131071, "f16")])
def test_linear_large_tiles(M, N, K, dtype):
    x, w = activations(M, K, 5, dtype), rand((N, K), 6, 0.02, dtype)
    product_check(T.linear_int8(x, held(w)), x, w, (M, N, K))


def test_linear_largest_sums():
    """Codes of +-127 and -128 throughout, the longest K: |sum| up to 2^31 - 2^14."""
    K = 131071
    ld = -(-K // 16) * 16
    codes = torch.zeros(3, ld, dtype=torch.int8, device="cuda")
    codes[0, :K] = -128
    codes[1, :K] = 127
    codes[2, :K:2] = -128
    one = torch.ones(3, device="cuda")
    q = T.Int8Rows((3, K), codes, one)
    y = T.gemm_int8(q, q).double()
    c = codes[:, :K].double()
    want = (c @ c.t().contiguous()).float().bfloat16().double()
    assert torch.equal(y, want)


def test_linear_rows_that_are_not_finite_stay_alone():
    x, w = activations(40, 600, 1), rand((70, 600), 2, 0.02)
    clean = T.linear_int8(x, held(w))
    x[7, 3] = math.inf
    w[11, 599] = math.nan
    y = T.linear_int8(x, held(w))
    assert torch.isnan(y[7]).all() and torch.isnan(y[:, 11]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[7] = False
    keep[:, 11] = False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M,N,K", [(3, 100, 130), (70, 250, 600), (300, 300, 300)])
def test_linear_strides_and_what_lies_around(M, N, K):
    wide = activations(M, K + 24, 8)
    x, w = wide[:, 5:5 + K], rand((N, K), 9, 0.02)
    wq = held(w, spare=32)
    for pad in (0, 1, 8):
        out = torch.full((M + 1, N + pad), 3.0, dtype=torch.bfloat16, device="cuda")
        T.linear_int8(x, wq, out=out[:M, :N])
        product_check(out[:M, :N], x, w)
        assert (out[M] == 3).all() and (out[:, N:] == 3).all()


@pytest.mark.parametrize("M", [1, 4, 20, 70, 300])
@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_outputs_at_any_address(M, shift):
    """Outputs that start `shift` values into a buffer (2-byte aligned only)."""
    N, K = 200, 264
    x, w, dy = activations(M, K, 1), held(rand((N, K), 2, 0.02)), rand((M, N), 3, 0.05)
    y = T.linear_int8(x, w)
    buf = torch.zeros(M * 512 + 64, dtype=torch.bfloat16, device="cuda")
    out = buf[shift:shift + M * 512].view(M, 512)[:, :N]
    assert torch.equal(T.linear_int8(x, w, out=out), y)
    out = buf[shift:shift + M * 512].view(M, 512)[:, :K]
    assert torch.equal(T.gemm_int8_dx(dy, w, out=out), T.gemm_int8_dx(dy, w))
    saved = T.quantize_rows(x)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.zeros(N * 512 + 64, dtype=dt, device="cuda")
        out = buf[shift:shift + N * 512].view(N, 512)[:, :K]
        assert torch.equal(T.gemm_int8_dw(dy, saved, out=out),
                           T.gemm_int8_dw(dy, saved, dtype=dt))


@pytest.mark.parametrize("M", [2, 20, 70])
def test_codes_past_32_bit_offsets(M):
    """A weight, and saved activations, of more than 2^32 bytes: the last rows."""
    R, K, last = 525_000, 8192, 120
    codes = torch.randint(-127, 128, (R, K), dtype=torch.int8, device="cuda")
    scale = torch.rand(R, device="cuda") + 0.5
    q = T.Int8Rows((R, K), codes, scale)
    x = activations(M, K, 1)
    y = T.linear_int8(x, q)
    qx, sx = codes_in_64(x)
    tail = codes[-last:].double()
    exact = (qx.double() @ tail.t().contiguous()) * sx.double()[:, None] * scale[-last:].double()
    assert ((y[:, -last:].double() - exact).abs() <= exact.abs() * 2.0 ** -8 * 1.001).all()
    dy = torch.zeros(M, R, dtype=torch.bfloat16, device="cuda")
    dy[:, -last:] = rand((M, last), 2, 0.05)
    v = values_of(codes[-last:].long(), scale[-last:], torch.bfloat16)
    gradient_check(T.gemm_int8_dx(dy, q), dy[:, -last:], v, "dx")
    dy = torch.zeros(R, 8, dtype=torch.bfloat16, device="cuda")
    dy[-last:] = rand((last, 8), 3, 0.05)
    gradient_check(T.gemm_int8_dw(dy, q), dy[-last:].t(), v, "dw")
    assert torch.equal(T.dequantize_rows(q)[-last:].double(), v)


def test_outputs_past_32_bit_offsets():
    M, N, K = 300_001, 8200, 48
    x, w = rand((M, K), 1), rand((N, K), 2, 0.02)
    wq, last = held(w), 90
    y = T.linear_int8(x, wq)
    product_check(y[-last:], x[-last:], w)
    dy = rand((M, 16), 3, 0.05)
    v = rand((16, N), 4, 0.02)
    gradient_check(T.gemm_int8_dx(dy, held(v), out=y)[-last:], dy[-last:],
                   values_of(*codes_in_64(v), torch.bfloat16))


def test_linear_no_rows():
    w = held(rand((20, 32), 1))
    assert T.linear_int8(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 20)
    assert T.gemm_int8_dx(torch.empty(0, 20, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 32)
    x = T.empty_int8_rows((0, 32))
    assert T.quantize_rows(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), out=x) is x
    assert T.dequantize_rows(x).shape == (0, 32)
    assert T.gemm_int8(x, w).shape == (0, 20)
    dw = T.gemm_int8_dw(torch.empty(0, 24, dtype=torch.bfloat16, device="cuda"), x,
                        out=torch.full((24, 32), 7.0, device="cuda"))
    assert not dw.any()


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
GRADS = [(1, 8, 1), (1, 16, 16), (3, 64, 100), (33, 40, 130), (64, 128, 256), (65, 200, 129),
         (130, 72, 1000), (257, 1000, 300), (20, 4096, 500), (7, 2048, 4100), (300, 8, 260)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", GRADS)
def test_dx(M, N, K, dtype):
    dy, w = rand((M, N), M + N, 0.05, dtype), rand((N, K), N + K, 0.02, dtype)
    q = held(w, spare=16)
    v = values_of(*codes_in_64(w), DT[dtype])
    gradient_check(T.gemm_int8_dx(dy, q), dy, v, (M, N, K))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["16", "f32"])
@pytest.mark.parametrize("M,N,K", GRADS)
def test_dw(M, N, K, out, dtype):
    dy, x = rand((M, N), M + N, 0.05, dtype), activations(M, K, M + K, dtype)
    q = held(x, spare=16)
    v = values_of(*codes_in_64(x), DT[dtype])
    dw = T.gemm_int8_dw(dy, q, dtype=torch.float32 if out == "f32" else None)
    assert dw.dtype == (torch.float32 if out == "f32" else DT[dtype])
    gradient_check(dw, dy.t(), v, (M, N, K))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_large_tiles(dtype):
    M, N, K = 3500, 200, 4100
    dy, w = rand((M, N), 1, 0.05, dtype), rand((N, K), 2, 0.02, dtype)
    gradient_check(T.gemm_int8_dx(dy, held(w)), dy, values_of(*codes_in_64(w), DT[dtype]), "dx")
    M, N, K = 200, 3500, 4100
    dy, x = rand((M, N), 3, 0.05, dtype), activations(M, K, 4, dtype)
    v = values_of(*codes_in_64(x), DT[dtype])
    gradient_check(T.gemm_int8_dw(dy, held(x)), dy.t(), v, "dw")
    gradient_check(T.gemm_int8_dw(dy, held(x), dtype=torch.float32), dy.t(), v, "dw f32")


@pytest.mark.parametrize("R,C,T_", [(200, 4096, 4096), (1000, 4100, 1000), (1001, 4100, 777),
                                    (64, 4090, 4096), (2048, 6100, 320), (40, 130, 9000),
                                    (2000, 2000, 130), (700, 700, 5000)])
def test_gradients_of_every_form(R, C, T_):
    dy, w = rand((R, T_ // 8 * 8), 1, 0.05), rand((T_ // 8 * 8, C), 2, 0.02)
    gradient_check(T.gemm_int8_dx(dy, held(w)), dy, values_of(*codes_in_64(w), torch.bfloat16),
                   "dx")
    dy, x = rand((T_, R), 3, 0.05, "f16"), activations(T_, C, 4, "f16")
    v = values_of(*codes_in_64(x), torch.float16)
    gradient_check(T.gemm_int8_dw(dy, held(x)), dy.t(), v, "dw")
    gradient_check(T.gemm_int8_dw(dy, held(x), dtype=torch.float32), dy.t(), v, "dw f32")


@pytest.mark.parametrize("N", [1, 5, 15, 100, 333])
@pytest.mark.parametrize("M,K", [(1, 20), (70, 300), (700, 64)])
def test_gradients_of_widths_that_are_no_pieces(M, N, K):
    dy = rand((M, N), M + N, 0.05)
    w, x = rand((N, K), 1, 0.02), activations(M, K, 2)
    gradient_check(T.gemm_int8_dx(dy, held(w)), dy, values_of(*codes_in_64(w), torch.bfloat16))
    v = values_of(*codes_in_64(x), torch.bfloat16)
    gradient_check(T.gemm_int8_dw(dy, held(x)), dy.t(), v)
    # behind the rows lies NaN: it must not reach a result
    wide = torch.full((M, -(-N // 8) * 8 + 8), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, :N] = dy
    gradient_check(T.gemm_int8_dx(wide[:, :N], held(w)), dy,
                   values_of(*codes_in_64(w), torch.bfloat16))
    gradient_check(T.gemm_int8_dw(wide[:, :N], held(x)), dy.t(), v)


@pytest.mark.parametrize("M,N,K", [(70, 250, 600), (300, 304, 300)])
def test_gradients_leave_what_lies_around(M, N, K):
    dy, w, x = rand((M, N), 1, 0.05), rand((N, K), 2, 0.02), activations(M, K, 3)
    for pad in (0, 1, 4, 8):
        out = torch.full((M + 1, K + pad), 3.0, dtype=torch.bfloat16, device="cuda")
        T.gemm_int8_dx(dy, held(w), out=out[:M, :K])
        gradient_check(out[:M, :K], dy, values_of(*codes_in_64(w), torch.bfloat16))
        assert (out[M] == 3).all() and (out[:, K:] == 3).all()
        for dt in (torch.bfloat16, torch.float32):
            out = torch.full((N + 1, K + pad), 3.0, dtype=dt, device="cuda")
            T.gemm_int8_dw(dy, held(x), out=out[:N, :K])
            gradient_check(out[:N, :K], dy.t(), values_of(*codes_in_64(x), torch.bfloat16))
            assert (out[N] == 3).all() and (out[:, K:] == 3).all()


def test_gradients_take_the_values_of_the_codes():
    """One-hot gradients return the values bit for bit."""
    for dtype in ("bf16", "f16"):
        w = rand((200, 300), 1, 0.02, dtype)
        q = held(w)
        v = T.dequantize_rows(q)
        eye = torch.eye(200, dtype=DT[dtype], device="cuda")
        assert torch.equal(T.gemm_int8_dx(eye, q), v)
        assert torch.equal(T.gemm_int8_dw(eye, q), v)
        assert torch.equal(T.gemm_int8_dw(eye, q, dtype=torch.float32), v.float())


def test_dx_rows_that_are_not_finite():
    dy, w = rand((50, 96), 1, 0.05), rand((96, 200), 2, 0.02)
    clean = T.gemm_int8_dx(dy, held(w))
    dy[4, 95] = math.nan
    y = T.gemm_int8_dx(dy, held(w))
    assert torch.isnan(y[4]).all()
    rest = [i for i in range(50) if i != 4]
    assert torch.equal(y[rest], clean[rest])
    w[5, 0] = math.inf
    assert torch.isnan(T.gemm_int8_dx(dy, held(w))).all()


def test_results_repeat():
    for M, N, K in ((1, 4096, 4096), (16, 1000, 4096), (301, 1024, 4100), (2048, 4096, 512)):
        x, w, dy = activations(M, K, 1), held(rand((N, K), 2, 0.02)), rand((M, N), 3, 0.05)
        saved = T.empty_int8_rows((M, K))
        a = (T.linear_int8(x, w, saved=saved), T.gemm_int8_dx(dy, w), T.gemm_int8_dw(dy, saved))
        for _ in range(20):
            b = (T.linear_int8(x, w), T.gemm_int8_dx(dy, w), T.gemm_int8_dw(dy, saved))
            assert all(torch.equal(p, q) for p, q in zip(a, b)), (M, N, K)
