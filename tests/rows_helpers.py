"""Helpers for the tests of the row-grouped operators: plans, stacks of 4-bit
weights, and products in binary64 with an elementwise error bound."""

from __future__ import annotations

import math

import torch

from dequant_gemm_nf4_amd import tensors as T

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def plan_of(ids: torch.Tensor, groups: int):
    """(offsets, order) of a plan by its definition, in Python integers."""
    lists = [[] for _ in range(groups + 1)]
    for i, g in enumerate(ids.tolist()):
        lists[g if 0 <= g < groups else groups].append(i)
    offsets = [0]
    for rows in lists[:-1]:
        offsets.append(offsets[-1] + len(rows))
    return offsets, [i for rows in lists for i in rows]


def device_plan(ids, groups: int) -> T.RowGroups:
    """The same plan as device arrays, without the library."""
    offsets, order = plan_of(torch.as_tensor(ids), groups)
    return T.RowGroups(groups, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                       torch.tensor(order, dtype=torch.int32, device="cuda"))


def rand(shape, seed, std=1.0, dtype="bf16"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(DT[dtype]).cuda()


def stack(groups, n, k, seed, dq="linear", quant="nf4", dtype="bf16"):
    """A quantized stack [groups, n, k] and its dequantized values (float64),
    as bnbx_dequantize_nf4 gives them (bit-exact against the oracle in its
    own tests)."""
    shape = (groups, n, k) if groups else (n, k)
    w = rand(shape, seed, 0.05)
    q = T.quantize(w, dq is not None, quant_type=quant, dtype=DT[dtype], dq_map=dq or "linear")
    return q, T.dequantize(q).double()


def check(y, exact, spread, terms, where=""):
    """Every element of y within one rounding of the output type and the fp32
    accumulation's error of the exact value.

    Output rounding: half a step, eps / 2 relative to the value (plus half
    the smallest subnormal).  Accumulation: `terms` fp32 additions of products
    whose 2-norm is `spread`; each rounds a partial sum of at most a few times
    that norm by 2^-24 of it, and the roundings add up like a random walk:
    sqrt(terms) 2^-24 spread, times 16 for partial sums of three norms at
    five standard deviations."""
    fi = torch.finfo(y.dtype)
    got = y.double()
    tol = (fi.eps / 2) * exact.abs() * (1 + 2.0 ** -6) + fi.smallest_normal * fi.eps \
        + 16 * math.sqrt(terms) * 2.0 ** -24 * spread
    bad = ~((got - exact).abs() <= tol)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{where}: {int(bad.sum())} of {bad.numel()} elements off, first at "
                             f"{i}: {got[tuple(i)].item()} for {exact[tuple(i)].item()} "
                             f"(tolerance {tol[tuple(i)].item()})")


def product(x, w):
    """X . W^T in binary64 and the 2-norm of every element's products."""
    x, w = x.double(), w.double()
    return x @ w.t().contiguous(), (x.square() @ w.square().t().contiguous()).sqrt()
