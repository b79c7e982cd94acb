"""Helpers for the tests of the 8-bit operators: rows of codes by their
definition, products in binary64, and elementwise error bounds."""

from __future__ import annotations

import math

import torch

from dequant_gemm_nf4_amd import tensors as T
from rows_helpers import DT, check, rand  # noqa: F401


def codes_by_definition(x: torch.Tensor):
    """(codes int64 [rows, K], scale float32 [rows]) of a 16-bit matrix, on the CPU:
    a = max |x|, q the integer nearest to the exact quotient 127 x / a, ties to
    even, scale = fl32(a / 127); a row that is not finite: scale NaN, codes 0.

    binary64 holds 254 x exactly; q = floor((254 x + a) / 2a) and the tie are found
    with integer arithmetic on the common exponent (Python integers)."""
    v = x.detach().cpu().double()
    rows, cols = v.shape
    codes = torch.zeros(rows, cols, dtype=torch.int64)
    scale = torch.zeros(rows, dtype=torch.float32)
    for r in range(rows):
        row = v[r]
        if not bool(torch.isfinite(row).all()):
            scale[r] = math.nan
            continue
        a = float(row.abs().max())
        if a == 0.0:
            continue
        # binary64 a / 127 rounded to binary32: 127 is odd, so the quotient of a 16-bit a
        # is never within 2^-29 of a midpoint of binary32 unless it is exact
        scale[r] = torch.tensor(a / 127.0, dtype=torch.float64).float()
        an, ad = a.as_integer_ratio()
        for k, e in enumerate(row.tolist()):
            n, d = e.as_integer_ratio()
            num, den = 127 * n * ad, d * an            # 127 e / a as a fraction
            q, rest = divmod(num, den)
            if 2 * rest > den or (2 * rest == den and q % 2 == 1):
                q += 1
            codes[r, k] = q
    return codes, scale


def codes_in_64(x: torch.Tensor):
    """The same in binary64 (round of the binary64 quotient; a 16-bit quotient that
    is no half-integer is 2^-20 away from one, so this rounds as the exact one)."""
    v = x.detach().double()
    a = v.abs().amax(1)
    ok = torch.isfinite(v).all(1)
    safe = torch.where(ok & (a > 0), a, torch.ones_like(a))
    q = torch.round(torch.where(ok[:, None], v, torch.zeros_like(v)) * 127.0 / safe[:, None])
    scale = torch.where(ok, (a / 127.0), torch.full_like(a, math.nan)).float()
    return q.long(), scale


def values_of(codes, scale, dtype):
    """v = rnd16(fl32(code * scale)) in binary64, from the format's definition."""
    return (codes.float() * scale[:, None]).to(dtype).double()


def held(x: torch.Tensor, spare: int = 0) -> T.Int8Rows:
    """The codes of x as a descriptor of device buffers, without the library;
    rows `spare` bytes longer than they must be, those bytes not zero."""
    rows, cols = x.shape
    codes, scale = codes_in_64(x)
    ld = -(-cols // 16) * 16
    buf = torch.full((max(rows, 1), ld + spare), 77, dtype=torch.int8, device=x.device)
    buf[:, :ld] = 0
    buf[:rows, :cols] = codes.to(torch.int8)
    return T.Int8Rows((rows, cols), buf[:rows], scale.contiguous(), x.dtype)


def gradient_check(y, a, v, where=""):
    """y against a . v (binary64), fp32 accumulation and one rounding."""
    a, v = a.double().contiguous(), v.contiguous()
    spread = (a.square() @ v.square()).sqrt()
    check(y, a @ v, spread, a.shape[1], where)
