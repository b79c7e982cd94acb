"""Torch-tensor convenience layer over the C ABI: allocates device buffers
with PyTorch (plumbing only) and calls the bnbx_* entry points.  Nothing is
computed here."""

from __future__ import annotations

import contextlib
import dataclasses
import math

import torch

from . import (AdaptersDesc, Nf4State, RowGroupsDesc, bnbx_dequantize_nf4, bnbx_gemm_nf4_experts,
               bnbx_gemm_nf4_adapters, bnbx_gemm_nf4_adapters_workspace_bytes,
               bnbx_gemm_nf4_experts_dx,
               bnbx_group_rows, bnbx_group_rows_workspace_bytes,
               bnbx_gemm_nf4, bnbx_gemm_nf4_dx, bnbx_gemm_nf4_lora,
               bnbx_gemm_nf4_workspace_bytes, bnbx_gemv_nf4, bnbx_gemv_nf4_grouped, bnbx_lora_down,
               bnbx_quantize_nf4, bnbx_quantize_nf4_grouped,
               bnbx_quantize_nf4_grouped_workspace_bytes, bnbx_quantize_nf4_workspace_bytes)

BLOCKSIZE = 64
GROUP = 256
QUANT_TYPES = {"nf4": 0, "fp4": 1}
# second-level maps of the block scales (bnbx_nf4_state.double_quant)
DQ_MAPS = {"linear": 1, "dynamic": 2}
DTYPES = {torch.bfloat16: 0, torch.float16: 1}


@dataclasses.dataclass
class QuantizedWeight:
    """Device buffers of one 4-bit tensor plus its C descriptor.  ``dtype``
    is the compute dtype (bf16 or fp16) of its dequantized values and of the
    activations it multiplies; ``dq_map`` the second-level map of the block
    scales with double quant ("linear": int8 codes, "dynamic": uint8 codes
    into the dynamic 8-bit map)."""

    n: int
    shape: tuple
    double_quant: bool
    packed: torch.Tensor          # uint8 [n/2]
    absmax: torch.Tensor          # float32 [nb] or int8 [nb]
    absmax2: torch.Tensor | None  # float32 [ng]
    absmax_mean: torch.Tensor | None  # float32 [1]
    quant_type: str = "nf4"
    dtype: torch.dtype = torch.bfloat16
    dq_map: str = "linear"

    def __post_init__(self):
        # the kernels read all that the shape says
        n, device = math.prod(self.shape), self.packed.device
        blocks = -(-n // BLOCKSIZE)
        if n != self.n:
            raise ValueError(f"the weight's n is {self.n}, its shape {self.shape}")
        scales = (torch.float32 if not self.double_quant else
                  torch.uint8 if self.dq_map == "dynamic" else torch.int8)
        parts = [("packed", self.packed, torch.uint8, n // 2), ("absmax", self.absmax, scales, blocks)]
        if self.double_quant:
            parts += [("absmax2", self.absmax2, torch.float32, -(-blocks // GROUP)),
                      ("absmax_mean", self.absmax_mean, torch.float32, 1)]
        for name, t, dtype, count in parts:
            if (t is None or t.dtype is not dtype or t.numel() < count or t.device != device
                    or not t.is_contiguous()):
                raise ValueError(f"the weight's {name} must be {count} contiguous {dtype} on "
                                 f"{device} for its shape {self.shape}")

    @property
    def state(self) -> Nf4State:
        return Nf4State(
            n=self.n, blocksize=BLOCKSIZE,
            double_quant=DQ_MAPS[self.dq_map] if self.double_quant else 0,
            quant_type=QUANT_TYPES[self.quant_type], compute_dtype=DTYPES[self.dtype],
            absmax=self.absmax.data_ptr(),
            absmax2=self.absmax2.data_ptr() if self.absmax2 is not None else None,
            absmax_mean=self.absmax_mean.data_ptr() if self.absmax_mean is not None else None)


def empty_quantized(shape, double_quant: bool, device="cuda", quant_type: str = "nf4",
                    dtype: torch.dtype = torch.bfloat16, dq_map: str = "linear") -> QuantizedWeight:
    n = 1
    for s in shape:
        n *= int(s)
    nb = -(-n // BLOCKSIZE)
    ng = -(-nb // GROUP)
    packed = torch.empty(n // 2, dtype=torch.uint8, device=device)
    if double_quant:
        absmax = torch.empty(nb, dtype=torch.uint8 if dq_map == "dynamic" else torch.int8,
                             device=device)
        absmax2 = torch.empty(ng, dtype=torch.float32, device=device)
        mean = torch.empty(1, dtype=torch.float32, device=device)
    else:
        absmax = torch.empty(nb, dtype=torch.float32, device=device)
        absmax2 = mean = None
    if dq_map not in DQ_MAPS:
        raise ValueError(f"unknown second-level map {dq_map!r}")
    return QuantizedWeight(n, tuple(shape), double_quant, packed, absmax, absmax2, mean,
                           quant_type, dtype, dq_map)


def workspace_for(n: int, double_quant: bool, device="cuda") -> torch.Tensor | None:
    nbytes = bnbx_quantize_nf4_workspace_bytes(n, BLOCKSIZE, int(double_quant))
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def quantize(w: torch.Tensor, double_quant: bool, out: QuantizedWeight | None = None,
             workspace: torch.Tensor | None = None, stream=None, quant_type: str = "nf4",
             dtype: torch.dtype = torch.bfloat16, dq_map: str = "linear") -> QuantizedWeight:
    """bnbx_quantize_nf4 on a bf16 tensor (any shape, contiguous); ``dtype``
    is the compute dtype recorded for later dequantize / matmul calls,
    ``dq_map`` the second-level map with double quant (ignored with ``out``,
    which carries its own)."""
    assert w.dtype == torch.bfloat16 and w.is_contiguous()
    q = out if out is not None else empty_quantized(w.shape, double_quant, w.device, quant_type,
                                                    dtype, dq_map)
    ws = workspace if workspace is not None else workspace_for(q.n, double_quant, w.device)
    bnbx_quantize_nf4(w, q.packed, q.state, ws, 0 if ws is None else ws.numel(), stream)
    return q


def grouped_workspace_for(ns, double_quant: bool, device="cuda") -> torch.Tensor | None:
    nbytes = bnbx_quantize_nf4_grouped_workspace_bytes(ns, BLOCKSIZE, int(double_quant))
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def quantize_grouped(ws: list, double_quant: bool, outs: list | None = None,
                     workspace: torch.Tensor | None = None, stream=None, quant_type: str = "nf4",
                     dtype: torch.dtype = torch.bfloat16,
                     dq_map: str = "linear") -> list:
    """bnbx_quantize_nf4_grouped on up to eight bf16 tensors (a layer's
    weights) in one call; each result equals quantize() on that tensor."""
    assert all(w.dtype == torch.bfloat16 and w.is_contiguous() for w in ws)
    qs = outs if outs is not None else [
        empty_quantized(w.shape, double_quant, w.device, quant_type, dtype, dq_map) for w in ws]
    wsp = workspace if workspace is not None else grouped_workspace_for(
        [q.n for q in qs], double_quant, ws[0].device)
    bnbx_quantize_nf4_grouped([(w, q.packed, q.state) for w, q in zip(ws, qs)], wsp,
                              0 if wsp is None else wsp.numel(), stream)
    return qs


def dequantize(q: QuantizedWeight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    o = out if out is not None else torch.empty(q.shape, dtype=q.dtype, device=q.packed.device)
    assert o.dtype == q.dtype
    bnbx_dequantize_nf4(q.packed, q.state, o, stream)
    return o


def gemv(x: torch.Tensor, q: QuantizedWeight, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Y = X . W_hat^T for X [M, K] (M <= 16), W [N, K]."""
    M, K = x.shape
    N = q.shape[0]
    assert x.dtype == q.dtype
    y = out if out is not None else torch.empty(M, N, dtype=q.dtype, device=x.device)
    bnbx_gemv_nf4(x, x.stride(0), q.packed, q.state, M, N, K, y, y.stride(0), stream)
    return y


def gemv_grouped(x: torch.Tensor, qs: list, outs: list | None = None, stream=None) -> list:
    """Y_i = X . W_hat_i^T for up to four weights sharing X [M, K] (M <= 16),
    in one call (bnbx_gemv_nf4_grouped)."""
    M, K = x.shape
    ys = outs if outs is not None else [
        torch.empty(M, q.shape[0], dtype=q.dtype, device=x.device) for q in qs]
    for q in qs:
        assert x.dtype == q.dtype and q.shape[1] == K
    bnbx_gemv_nf4_grouped(x, x.stride(0),
                          [(q.packed, q.state, q.shape[0], y, y.stride(0)) for q, y in zip(qs, ys)],
                          M, K, stream)
    return ys


def gemm(x: torch.Tensor, q: QuantizedWeight, out: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Y = X . W_hat^T for X [M, K], W [N, K], any M."""
    M, K = x.shape
    N = q.shape[0]
    assert x.dtype == q.dtype
    y = out if out is not None else torch.empty(M, N, dtype=q.dtype, device=x.device)
    nbytes = bnbx_gemm_nf4_workspace_bytes(M, N, K)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    bnbx_gemm_nf4(x, x.stride(0), q.packed, q.state, M, N, K, y, y.stride(0), ws, nbytes, stream)
    return y


def gemm_dx(dy: torch.Tensor, q: QuantizedWeight, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """dX = dY . W_hat for dY [M, N], W [N, K] (the input gradient of gemm)."""
    M, N = dy.shape
    K = q.shape[1]
    assert dy.dtype == q.dtype and N == q.shape[0]
    dx = out if out is not None else torch.empty(M, K, dtype=q.dtype, device=dy.device)
    bnbx_gemm_nf4_dx(dy, dy.stride(0), q.packed, q.state, M, N, K, dx, dx.stride(0), stream)
    return dx


def gemm_lora(x: torch.Tensor, q: QuantizedWeight, xa: torch.Tensor, lora_b: torch.Tensor,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X . W_hat^T + XA . B^T for X [M, K], XA [M, r] (= s X A^T), B [N, r]."""
    M, K = x.shape
    N = q.shape[0]
    r = xa.shape[1]
    assert x.dtype == q.dtype == xa.dtype == lora_b.dtype and lora_b.shape == (N, r)
    y = out if out is not None else torch.empty(M, N, dtype=q.dtype, device=x.device)
    bnbx_gemm_nf4_lora(x, x.stride(0), q.packed, q.state, M, N, K, xa, xa.stride(0), lora_b,
                       lora_b.stride(0), r, y, y.stride(0), stream)
    return y


def lora_down(x: torch.Tensor, lora_a: torch.Tensor, scale: float,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """XA = s . X . A^T for X [M, K] and the adapter weight A [r, K]."""
    M, K = x.shape
    r = lora_a.shape[0]
    assert x.dtype == lora_a.dtype and lora_a.shape[1] == K
    xa = out if out is not None else torch.empty(M, r, dtype=x.dtype, device=x.device)
    bnbx_lora_down(x, x.stride(0), lora_a, lora_a.stride(0), M, K, r, scale, DTYPES[x.dtype], xa,
                   xa.stride(0), stream)
    return xa


def linear_lora(x: torch.Tensor, q: QuantizedWeight, lora_a: torch.Tensor, lora_b: torch.Tensor,
                scale: float, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X . W_hat^T + s . (X . A^T) . B^T: the down-projection, then the GEMM
    with the low-rank term fused in (both in the library)."""
    xa = lora_down(x, lora_a, scale, stream=stream)
    return gemm_lora(x, q, xa, lora_b, out=out, stream=stream)



# --------------------------------------------------------------------------
# rows that belong to groups (include/bnbx_rows.h)
# --------------------------------------------------------------------------
@dataclasses.dataclass(frozen=True)
class RowGroups:
    """A plan of bnbx_group_rows: the rows 0 .. rows-1 in group order.  Group
    g holds the places offsets[g] .. offsets[g+1]-1 of ``order``; places
    behind offsets[groups] are rows of no group."""

    groups: int
    offsets: torch.Tensor   # int32 [groups + 1]
    order: torch.Tensor     # int32 [rows]

    def __post_init__(self):
        for name, t, n in (("offsets", self.offsets, self.groups + 1),
                           ("order", self.order, self.order.numel())):
            if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous():
                raise ValueError(f"plan: {name} must be a contiguous int32 vector of {n}")
        if self.order.numel() >= 2 ** 31:
            raise ValueError("plan: rows are numbered in 31 bits")
        if self.offsets.device != self.order.device:
            raise ValueError("plan: offsets and order are on different devices")

    @property
    def rows(self) -> int:
        return self.order.shape[0]

    @property
    def desc(self) -> RowGroupsDesc:
        return RowGroupsDesc(self.offsets.data_ptr(), self.order.data_ptr(), self.groups,
                             self.order.shape[0])


def _check_matrix(name: str, t: torch.Tensor, cols: int, dtype, device) -> None:
    if t.dim() != 2 or t.shape[1] != cols:
        raise ValueError(f"{name} must be [rows, {cols}], not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.stride(1) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must have contiguous rows")
    if t.shape[0] >= 2 ** 31:
        raise ValueError(f"{name}: rows are numbered in 31 bits")


def _ld(t: torch.Tensor) -> int:
    """Row stride; of a matrix of at most one row (whose stride torch leaves
    open) its width, rounded up to the ABI's 8."""
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """The device of the data as the current one, for the launch, and a given
    stream as its current stream: what is allocated or cleared for the call then
    belongs to the stream that runs it."""
    if device.type != "cuda":
        raise ValueError(f"the data must be on a GPU, not on {device}")
    if stream is None:
        return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device) if stream
                  else torch.cuda.default_stream(device))
    if stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the data on {device}")
    return torch.cuda.stream(stream)


def _scratch(workspace: torch.Tensor | None, nbytes: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be contiguous and on {device}")
    return workspace


def empty_row_groups(rows: int, groups: int, device="cuda") -> RowGroups:
    return RowGroups(groups, torch.empty(groups + 1, dtype=torch.int32, device=device),
                     torch.empty(rows, dtype=torch.int32, device=device))


def group_rows(ids: torch.Tensor, groups: int, out: RowGroups | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> RowGroups:
    """bnbx_group_rows: the plan of an int32 vector of group ids (any id
    outside 0 .. groups-1: no group), on the device, stable."""
    rows = ids.numel()
    if ids.dtype != torch.int32 or ids.shape != (rows,) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 vector")
    device = ids.device
    if rows >= 2 ** 31:
        raise ValueError("ids: rows are numbered in 31 bits")
    if out is not None and (out.groups != groups or out.rows != rows
                            or out.order.device != device):
        raise ValueError("out: a plan of other sizes, or on another device")
    with _on(device, stream):
        plan = out if out is not None else empty_row_groups(rows, groups, device)
        nbytes = bnbx_group_rows_workspace_bytes(rows, groups)
        ws = _scratch(workspace, nbytes, device) if nbytes else None
        bnbx_group_rows(ids, rows, groups, plan.offsets, plan.order, ws,
                        ws.numel() * ws.element_size() if nbytes else 0, stream)
    return plan


def _check_plan(rows: RowGroups, device) -> None:
    if rows.order.device != device:
        raise ValueError(f"the plan is on {rows.order.device}, the data on {device}")


def _check_stack(q: QuantizedWeight, rows: RowGroups) -> None:
    if len(q.shape) != 3 or q.shape[0] != rows.groups:
        raise ValueError(f"the weight must be a stack [{rows.groups}, N, K], not {q.shape}")


def _rows_product(call, name: str, t: torch.Tensor, q: QuantizedWeight, rows: RowGroups,
                  cin: int, cout: int, gather: int, scatter: bool, out, stream) -> torch.Tensor:
    device = q.packed.device
    _check_matrix(name, t, cin, q.dtype, device)
    _check_plan(rows, device)
    if out is not None:
        _check_matrix("out", out, cout, q.dtype, device)
    if gather < 0:
        raise ValueError("gather must be 0 or the slots per row")
    if t.shape[0] * max(gather, 1) < rows.rows or (out is not None and out.shape[0] < rows.rows):
        raise ValueError("fewer rows than the plan has places")
    with _on(device, stream):
        y = out if out is not None else torch.zeros(rows.rows, cout, dtype=q.dtype, device=device)
        call(t, _ld(t), t.shape[0], q.packed, q.state, rows.desc, q.shape[1], q.shape[2], gather,
             int(scatter), y, _ld(y), y.shape[0], stream)
    return y


def gemm_experts(x: torch.Tensor, q: QuantizedWeight, rows: RowGroups, gather: int = 0,
                 scatter: bool = False, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Y_i = X_i . W_hat_g^T for the places i of every group g of the plan
    (bnbx_gemm_nf4_experts), W_hat [groups, N, K].  ``gather`` >= 1 reads row
    order[i] // gather of x (top_k for tokens with top_k slots), 0 row i;
    ``scatter`` writes row order[i] of the result, else row i.  Rows without a
    group keep what ``out`` holds (zero if it is allocated here)."""
    _check_stack(q, rows)
    return _rows_product(bnbx_gemm_nf4_experts, "x", x, q, rows, q.shape[2], q.shape[1], gather,
                         scatter, out, stream)


def gemm_experts_dx(dy: torch.Tensor, q: QuantizedWeight, rows: RowGroups, gather: int = 0,
                    scatter: bool = False, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """dX_i = dY_i . W_hat_g (bnbx_gemm_nf4_experts_dx, the input gradient of
    gemm_experts; N a multiple of 64): dY [.., N], the result [.., K]; rows are
    read and written as in gemm_experts."""
    _check_stack(q, rows)
    return _rows_product(bnbx_gemm_nf4_experts_dx, "dy", dy, q, rows, q.shape[1], q.shape[2],
                         gather, scatter, out, stream)


def linear_adapters(x: torch.Tensor, q: QuantizedWeight, rows: RowGroups, lora_a: torch.Tensor,
                    lora_b: torch.Tensor, scale: torch.Tensor, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X . W_hat^T + s_g . (X . A_g^T) . B_g^T with the adapter of each
    row's group (bnbx_gemm_nf4_adapters): A [groups, r, K], B [groups, N, r] (any
    strides of whole rows), scale float32 [groups]; rows of no group get the
    4-bit product alone."""
    if len(q.shape) != 2:
        raise ValueError(f"the weight must be [N, K], not {q.shape}")
    N, K = q.shape
    device, groups = q.packed.device, rows.groups
    _check_matrix("x", x, K, q.dtype, device)
    _check_plan(rows, device)
    if x.shape[0] != rows.rows:
        raise ValueError(f"x has {x.shape[0]} rows, the plan {rows.rows}")
    r = lora_a.shape[1] if lora_a.dim() == 3 else 0
    if lora_a.shape != (groups, r, K) or lora_b.shape != (groups, N, r) or scale.shape != (groups,):
        raise ValueError(f"the adapters must be A [{groups}, r, {K}], B [{groups}, {N}, r] and "
                         f"scale [{groups}], not {tuple(lora_a.shape)}, {tuple(lora_b.shape)} and "
                         f"{tuple(scale.shape)}")
    if lora_a.dtype != q.dtype or lora_b.dtype != q.dtype or scale.dtype != torch.float32:
        raise TypeError(f"the adapters must be {q.dtype}, their scales float32")
    if lora_a.device != device or lora_b.device != device or scale.device != device:
        raise ValueError(f"the adapters must be on {device}")
    if lora_a.stride(2) != 1 or lora_b.stride(2) != 1 or (groups > 1 and scale.stride(0) != 1):
        raise ValueError("the adapters must have contiguous rows")
    if out is not None:
        _check_matrix("out", out, N, q.dtype, device)
        if out.shape[0] != rows.rows:
            raise ValueError(f"out has {out.shape[0]} rows, the plan {rows.rows}")
    desc = AdaptersDesc(lora_a.data_ptr(), lora_b.data_ptr(), scale.data_ptr(), _row(lora_a),
                        lora_a.stride(0) if groups > 1 else 0, _row(lora_b),
                        lora_b.stride(0) if groups > 1 else 0, r)
    with _on(device, stream):
        y = out if out is not None else torch.empty(rows.rows, N, dtype=q.dtype, device=device)
        workspace = _scratch(workspace, bnbx_gemm_nf4_adapters_workspace_bytes(rows.rows, r),
                             device)
        bnbx_gemm_nf4_adapters(x, _ld(x), q.packed, q.state, rows.desc, N, K, desc, y, _ld(y),
                               workspace, workspace.numel() * workspace.element_size(), stream)
    return y


def _row(t: torch.Tensor) -> int:
    """Row stride of a stack of matrices."""
    return t.stride(1) if t.shape[1] > 1 else t.shape[2]
