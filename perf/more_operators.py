"""The 8-bit operators of the library, as they are measured.

A row x of K values is held as int8 codes and one scale: a = max |x_k|, s = a / 127,
q_k = round_half_even(127 x_k / a); the value of a code is rnd16(fl32(q_k * s)), in the
rows' own 16-bit type, as the 4-bit format's values are. Four operators work on such rows:

* ``checkpoint``: rows of activations -> codes and scales, and back to 16 bits;
* ``linear``: Y = X . W^T over 8-bit integers, X quantized per row (token) within the
  call, W held per row (channel): Y[m, n] = rnd16(sum_k qx[m, k] qw[n, k] * sx[m] * sw[n]);
* ``dx``: the input gradient dX = dY . W_hat, W_hat the values of the weight's codes;
* ``dw``: the weight's gradient dW = dY^T . X_hat from activations saved in 8 bits (with
  few columns of dY: the gradient of a low-rank adapter's down-projection).

Each has a plain form here (``own`` false): elementary torch operations in 32 bits, rounded
once at the end. ``exact`` gives the same from the definitions in 64 bits.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _checkpoint(name, rows, k, dt="bf16", pad=0):
    return {"name": name, "op": "checkpoint", "rows": rows, "K": k, "dtype": dt, "pad": pad}


def _linear(name, rows, n, k, dt="bf16", pad=0):
    return {"name": name, "op": "linear", "rows": rows, "N": n, "K": k, "dtype": dt, "pad": pad}


def _dx(name, rows, n, k, dt="bf16", pad=0):
    return {"name": name, "op": "dx", "rows": rows, "N": n, "K": k, "dtype": dt, "pad": pad}


def _dw(name, rows, n, k, dt="bf16", out="bf16", pad=0):
    return {"name": name, "op": "dw", "rows": rows, "N": n, "K": k, "dtype": dt, "out": out,
            "pad": pad}


def listed():
    return [
        # a decode batch's activations: latency
        _checkpoint("checkpoint_decode_batch", 16, 4096),
        # a ragged fine-tuning batch, its rows part of wider ones
        _checkpoint("checkpoint_ragged", 1237, 11008, "f16", pad=64),
        # the widest activations of a training step
        _checkpoint("checkpoint_train", 8192, 14336),
        # one token through a square layer: the latency of a decode step
        _linear("linear_one_token", 1, 4096, 4096),
        # a decode batch through an up projection: bound by streaming the weight
        _linear("linear_decode_batch", 16, 11008, 4096),
        # a short ragged prompt through a down projection
        _linear("linear_ragged_down", 301, 4096, 11008, "f16", pad=8),
        # a long prefill
        _linear("linear_prefill", 2048, 8192, 8192),
        # the backward of a small fine-tuning batch
        _dx("dx_small", 200, 4096, 4096, "f16"),
        # the backward of a training step
        _dx("dx_train", 4096, 11008, 4096),
        # an adapter's gradient over a training batch, for a float32 optimizer
        _dw("dw_adapter", 4096, 64, 4096, "bf16", "f32"),
        # odd sizes: a small layer, a ragged batch
        _dw("dw_odd", 777, 1001, 4100, "f16", "f16", pad=7),
        # the weight's gradient of a training step
        _dw("dw_train", 4096, 11008, 4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["checkpoint", "linear", "linear", "dx", "dw"])
    dt = rng.choice(["bf16", "f16"])
    rows, k = _log_int(rng, 1, 8192), _log_int(rng, 16, 14336)
    if rng.random() < 0.5:
        k = -(-k // 16) * 16
    if op == "checkpoint":
        c = _checkpoint("", rows, k, dt, rng.choice([0, 0, 8, 64]))
    else:
        n = _log_int(rng, 16, 14336)
        rows = max(1, min(rows, 4096 * 11008 * 4096 // (n * k)))
        if op == "linear":
            c = _linear("", rows, n, k, dt, rng.choice([0, 0, 8, 64]))
        elif op == "dx":
            # rows of dY are whole 16-byte pieces
            c = _dx("", rows, -(-n // 8) * 8, k, dt, rng.choice([0, 0, 8, 64]))
        else:
            c = _dw("", rows, n, k, dt, rng.choice([dt, dt, "f32"]), -n % 8)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pitch(k):
    """Bytes of a row of codes: whole 16-byte pieces, zero behind the row."""
    return -(-k // 16) * 16


def _quantize(x):
    """16-bit [rows, K] -> (int8 [rows, pitch], float32 [rows])."""
    rows, k = x.shape
    v = x.float()
    amax = v.abs().amax(1)
    q = torch.round(v * 127.0 / torch.where(amax > 0, amax, torch.ones_like(amax))[:, None])
    codes = torch.zeros(rows, _pitch(k), dtype=torch.int8, device=x.device)
    codes[:, :k] = q
    return codes, amax / 127.0


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, m, k = _DT[case["dtype"]], case["rows"], case["K"]

    def rows_of(rows, width, std, features=False):
        """Rows of width + pad columns, the pad cut off."""
        v = torch.randn(rows, width + case["pad"], generator=gen, device="cuda") * std
        if features:                                   # a few features are larger everywhere
            big = torch.rand(width + case["pad"], generator=gen, device="cuda") < 0.002
            v = torch.where(big, v * 8.0, v)
        return v.to(dt)[:, :width]

    def held(rows, std, features=False):
        v = torch.randn(rows, k, generator=gen, device="cuda") * std
        if features:
            big = torch.rand(k, generator=gen, device="cuda") < 0.002
            v = torch.where(big, v * 8.0, v)
        return _quantize(v.to(dt))

    d = {}
    if case["op"] in ("checkpoint", "linear"):
        d["x"] = rows_of(m, k, 1.0, True)
    else:
        d["dy"] = rows_of(m, case["N"], 0.05)
    if case["op"] in ("linear", "dx"):
        d["codes"], d["scale"] = held(case["N"], 0.02)
    elif case["op"] == "dw":
        d["codes"], d["scale"] = held(m, 1.0, True)
    return d


def prepare(case, seed):
    st = dict(_inputs(case, seed), case=case)
    dt, m, k, op = _DT[case["dtype"]], case["rows"], case["K"], case["op"]
    # the caller's output buffer
    if op == "dw":
        st["out"] = torch.empty(case["N"], k, dtype=_DT[case["out"]], device="cuda")
    else:
        width = case["N"] if op == "linear" else k
        st["out"] = torch.empty(m, width, dtype=dt, device="cuda")
    if own:
        from dequant_gemm_nf4_amd import tensors
        st["lib"] = tensors
        if op == "checkpoint":
            st["saved"] = tensors.empty_int8_rows((m, k), dt)
        else:
            rows = m if op == "dw" else case["N"]
            st["q"] = tensors.Int8Rows((rows, k), st["codes"], st["scale"], dt)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _values(codes, scale, k, dt):
    return (codes[:, :k].float() * scale[:, None]).to(dt)


def run(st):
    case, out = st["case"], st["out"]
    op, k, dt = case["op"], case["K"], _DT[case["dtype"]]
    if own:
        lib = st["lib"]
        if op == "checkpoint":
            q = lib.quantize_rows(st["x"], out=st["saved"])
            return lib.dequantize_rows(q, out=out), q.scale
        if op == "linear":
            return lib.linear_int8(st["x"], st["q"], out=out)
        if op == "dx":
            return lib.gemm_int8_dx(st["dy"], st["q"], out=out)
        return lib.gemm_int8_dw(st["dy"], st["q"], out=out)
    if op == "checkpoint":
        codes, scale = _quantize(st["x"])
        return out.copy_(_values(codes, scale, k, dt)), scale
    if op == "linear":
        codes, scale = _quantize(st["x"])
        acc = codes[:, :k].float() @ st["codes"][:, :k].float().t()
        return out.copy_(acc * scale[:, None] * st["scale"])
    held = _values(st["codes"], st["scale"], k, dt).float()
    if op == "dx":
        return out.copy_(st["dy"].float() @ held)
    return out.copy_(st["dy"].float().t() @ held)


def _exact_rows(x):
    """Codes and scales of rows in float64: q the nearest integer to 127 x / a, ties even."""
    v = x.double()
    a = v.abs().max(dim=1).values
    safe = torch.where(a == 0, torch.ones_like(a), a)
    t = torch.div(v * 127.0, safe.unsqueeze(1))
    low = torch.floor(t)
    rest = t - low
    up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(low, 2.0) == 1.0))
    return low + up.double(), a / 127.0


def exact(case, seed):
    d = _inputs(case, seed)
    k = case["K"]
    if case["op"] == "checkpoint":
        q, s = _exact_rows(d["x"])
        return q * s.unsqueeze(1), s
    if case["op"] == "linear":
        q, s = _exact_rows(d["x"])
        w = d["codes"].narrow(1, 0, k).double() * d["scale"].double().unsqueeze(1)
        return torch.matmul(q * s.unsqueeze(1), w.t())
    # the format's value of a code: the binary32 product, then the 16-bit type
    wide = d["codes"].narrow(1, 0, k).double() * d["scale"].double().unsqueeze(1)
    held = wide.float().to(_DT[case["dtype"]]).double()
    dy = d["dy"].double()
    return torch.matmul(dy if case["op"] == "dx" else dy.t(), held)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    m, k = case["rows"], case["K"]
    if case["op"] == "checkpoint":
        # 16 bits in, 8 written and read again, 16 out
        return {"bytes": 6 * m * k + 8 * m, "flops": 0}
    n = case["N"]
    if case["op"] == "linear":
        moved = 2 * m * k + n * k + 4 * n + 2 * m * n
    elif case["op"] == "dx":
        moved = 2 * m * n + n * k + 4 * n + 2 * m * k
    else:
        moved = 2 * m * n + m * k + 4 * m + (4 if case["out"] == "f32" else 2) * n * k
    return {"bytes": moved, "flops": 2 * m * n * k}
