"""The row-grouped operators of the 4-bit library, as they are measured.

Three operators work on rows that belong to groups (the experts of a mixture,
the adapters of a batch of requests):

* ``group_rows``: the group of every row -> the rows in group order and each
  group's bounds (the plan the other two take);
* ``experts``: Y_i = X_i . W_hat_g^T with the 4-bit weight of the row's expert
  (``experts_dx``: the input gradient dX_i = dY_i . W_hat_g);
* ``adapters``: Y = X . W_hat^T + s_g . (X . A_g^T) . B_g^T, one shared 4-bit
  weight beside the low-rank adapter of each row's request.

Each has a plain form here (``own`` false): elementary torch operations in 32
bits, rounded once at the end.  ``exact`` gives the same from the definitions in
64 bits.  The dequantized weight is W_hat = rnd16(fl32(L[code] * scale)) by
definition of the stored format, in every form.
"""

import math
import statistics

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _experts(name, tokens, topk, experts, n, k, qt="nf4", dt="bf16", dq=True, dropped=0.0,
             skew=0.5, layout="gather"):
    return {"name": name, "op": "experts", "tokens": tokens, "topk": topk, "experts": experts,
            "N": n, "K": k, "quant": qt, "dtype": dt, "dq": dq, "dropped": dropped, "skew": skew,
            "layout": layout}


def _experts_dx(name, tokens, topk, experts, n, k, qt="nf4", dt="bf16", dq=True, skew=0.5):
    c = _experts(name, tokens, topk, experts, n, k, qt, dt, dq, 0.0, skew, "scatter")
    c["op"] = "experts_dx"
    return c


def _adapters(name, rows, adapters, rank, n, k, qt="nf4", dt="bf16", dq=True, none=0.2, run=1):
    return {"name": name, "op": "adapters", "rows": rows, "adapters": adapters, "rank": rank,
            "N": n, "K": k, "quant": qt, "dtype": dt, "dq": dq, "none": none, "run": run}


def listed():
    return [
        # the plan of one small decode step: 16 tokens, two experts each
        {"name": "plan_decode", "op": "group_rows", "rows": 32, "groups": 8, "dropped": 0.0},
        # the plan of a long prefill over many experts, some slots over capacity
        {"name": "plan_prefill", "op": "group_rows", "rows": 131072, "groups": 64,
         "dropped": 0.05},
        # one token of one user: two experts of eight, the latency of a decode step
        _experts("experts_one_token", 1, 2, 8, 4096, 4096, skew=0.0),
        # a decode batch over every expert: bound by streaming the 4-bit weights
        _experts("experts_decode_batch", 16, 2, 8, 14336, 4096, skew=0.0),
        # the down projection of a short ragged prompt, slots dropped by a
        # capacity limit, results returned in slot order
        _experts("experts_ragged_down", 301, 2, 16, 4096, 11008, "fp4", "f16", dropped=0.06,
                 skew=1.0, layout="scatter"),
        # a long prefill through the up projection
        _experts("experts_prefill", 4096, 2, 8, 14336, 4096),
        # the backward of a small fine-tuning batch, scales without a second level
        _experts_dx("experts_dx_small", 200, 2, 8, 4096, 4096, "nf4", "f16", False),
        # the backward of a training step
        _experts_dx("experts_dx_train", 4096, 2, 8, 11008, 4096),
        # one token with its own adapter: the latency of a decode step
        _adapters("adapters_one_token", 1, 4, 16, 4096, 4096, none=0.0),
        # a decode batch in which nearly every request brings another adapter
        _adapters("adapters_decode_batch", 16, 32, 64, 11008, 4096, none=0.1),
        # a mixed step: a few prompts' chunks and single tokens together
        _adapters("adapters_mixed_step", 333, 12, 48, 4096, 11008, "fp4", "f16", run=40),
        # the prompts of several requests in one prefill
        _adapters("adapters_prefill", 2048, 8, 64, 8192, 8192, run=400),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["group_rows", "experts", "experts", "experts_dx", "adapters", "adapters"])
    if op == "group_rows":
        return {"op": op, "rows": _log_int(rng, 1, 131072), "groups": _log_int(rng, 1, 256),
                "dropped": rng.choice([0.0, 0.1])}
    quant, dt = rng.choice(["nf4", "fp4"]), rng.choice(["bf16", "f16"])
    dq = rng.random() < 0.75
    k = 64 * _log_int(rng, 4, 172)
    if op == "adapters":
        rows = _log_int(rng, 1, 2048)
        n = _log_int(rng, 200, 12000)
        c = _adapters("", rows, _log_int(rng, 1, 64), 16 * rng.randint(1, 16), n, k, quant, dt, dq,
                      rng.choice([0.0, 0.2, 0.6]), rng.choice([1, 30, 300]))
    else:
        experts = _log_int(rng, 2, 64)
        topk = rng.randint(1, min(4, experts))
        rows = _log_int(rng, 1, 8192)
        n = _log_int(rng, 200, 14336)
        n = min(n, 8 * 14336 * 4096 // (experts * k))
        if op == "experts":
            c = _experts("", max(1, rows // topk), topk, experts, max(n, 17), k, quant, dt, dq,
                         rng.choice([0.0, 0.1]), rng.uniform(0.0, 1.5),
                         rng.choice(["gather", "scatter"]))
        else:
            # the input gradient takes whole blocks of 64 output features
            c = _experts_dx("", max(1, rows // topk), topk, experts, max(n // 64 * 64, 64), k,
                            quant, dt, dq, rng.uniform(0.0, 1.5))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# the stored 4-bit format, in plain torch
# ---------------------------------------------------------------------------
def _levels(quant):
    """The 16 levels by code: NF4 (normal quantiles scaled to +-1) or FP4 (E2M1 / 6)."""
    if quant == "fp4":
        mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        return [m / 6.0 for m in mags] + [-m / 6.0 for m in mags]
    q = statistics.NormalDist().inv_cdf
    d = 1.0 - (1.0 / 30.0 + 1.0 / 32.0) / 2.0
    pos = [q(d + (0.5 - d) * i / 8.0) for i in range(8)]
    neg = [-q(d + (0.5 - d) * i / 7.0) for i in range(7)]
    return [v / pos[0] for v in sorted(neg + [0.0] + pos)]


def _quantize(w, quant):
    """bf16 [N, K] -> (packed bytes, fp32 block maxima): nearest level per block of 64."""
    lv = torch.tensor(_levels(quant), dtype=torch.float64, device=w.device)
    blocks = w.float().reshape(-1, 64)
    amax = blocks.abs().amax(1)
    x = blocks / torch.where(amax > 0, amax, torch.ones_like(amax))[:, None]
    asc, order = torch.sort(lv, stable=True)
    keep = torch.cat((torch.ones_like(asc[:1], dtype=torch.bool), asc[1:] != asc[:-1]))
    asc, order = asc[keep], order[keep]                # FP4 holds zero twice: one code of it
    mid = ((asc[1:] + asc[:-1]) / 2).float()
    codes = order[torch.bucketize(x, mid)].to(torch.uint8).reshape(-1)
    return (codes[0::2] << 4) | codes[1::2], amax


def _double_quant(amax):
    mean = amax.double().mean().float()
    c = amax - mean
    nb = amax.numel()
    ng = -(-nb // 256)
    pad = torch.zeros(ng * 256, dtype=torch.float32, device=amax.device)
    pad[:nb] = c
    s = pad.reshape(ng, 256).abs().amax(1)
    q = torch.round(pad.reshape(ng, 256) / torch.where(s > 0, s, torch.ones_like(s))[:, None] * 127)
    return q.reshape(-1)[:nb].to(torch.int8), s, mean.reshape(1)


def _weight(gen, shape, quant, dq):
    """A quantized stack of normal weights [G, N, K]: packed, absmax, absmax2, mean."""
    g, n, k = shape
    packed = torch.empty(g * n * k // 2, dtype=torch.uint8, device="cuda")
    amax = torch.empty(g * n * k // 64, dtype=torch.float32, device="cuda")
    for i in range(g):
        w = torch.randn(n, k, generator=gen, device="cuda", dtype=torch.float32) * 0.02
        p, a = _quantize(w.bfloat16(), quant)
        packed[i * n * k // 2:(i + 1) * n * k // 2] = p
        amax[i * n * k // 64:(i + 1) * n * k // 64] = a
    if not dq:
        return packed, amax, None, None
    q, s, mean = _double_quant(amax)
    return packed, q, s, mean


def _plain_weight(st, i):
    """W_hat of stack entry i as fp32 [N, K]: rnd16(fl32(L[code] * scale))."""
    c = st["case"]
    n, k = c["N"], c["K"]
    lv = st["levels"]
    p = st["packed"][i * n * k // 2:(i + 1) * n * k // 2]
    vals = torch.stack((lv[(p >> 4).int()], lv[(p & 15).int()]), 1).reshape(-1, 64)
    b0, b1 = i * n * k // 64, (i + 1) * n * k // 64
    a = st["absmax"][b0:b1]
    if c["dq"]:
        group = torch.arange(b0, b1, device=a.device) // 256
        a = a.float() * (st["absmax2"][group] / 127.0) + st["mean"]
    return (vals * a[:, None]).to(_DT[c["dtype"]]).float().reshape(n, k)


def _exact_weight(c, weight, i):
    """W_hat of stack entry i in float64, written from the format's definition.  The
    scale and the product are binary32 by that definition; numpy forms each level."""
    packed, absmax, s, mean = weight
    n, k = c["N"], c["K"]
    lv = torch.from_numpy(np.asarray(_levels(c["quant"]), dtype=np.float32)).cuda()
    lo, hi = i * n * k, (i + 1) * n * k
    byte = packed[lo // 2:hi // 2].long()
    code = torch.empty(hi - lo, dtype=torch.long, device=byte.device)
    code[0::2], code[1::2] = torch.div(byte, 16, rounding_mode="floor"), byte % 16
    block = torch.arange(lo // 64, hi // 64, device=byte.device)
    if c["dq"]:
        step = (s.double() / 127.0).float()            # correctly rounded quotient
        prod = (absmax[block].double() * step[block // 256].double()).float()
        scale = (prod.double() + mean.double()).float()
    else:
        scale = absmax[block]
    w = (lv[code].double() * scale.double().repeat_interleave(64)).float()
    return w.to(_DT[c["dtype"]]).double().reshape(n, k)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _route(case, gen):
    """ids [tokens * topk]: distinct experts per token by noisy scores, -1 where dropped."""
    e, t, k = case["experts"], case["tokens"], case["topk"]
    bias = torch.randn(e, generator=gen, device="cuda") * case["skew"]
    noise = -torch.log(-torch.log(torch.rand(t, e, generator=gen, device="cuda") * 0.9998 + 1e-4))
    ids = (bias + noise).topk(k, dim=1).indices.to(torch.int32).reshape(-1)
    if case["dropped"]:
        gone = torch.rand(t * k, generator=gen, device="cuda") < case["dropped"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous()


def _requests(case, gen):
    """ids [rows]: runs of rows of one request, each with an adapter or none (-1)."""
    m, run = case["rows"], case["run"]
    cut = torch.rand(m, generator=gen, device="cuda") < 1.0 / run
    which = torch.cumsum(cut.int(), 0)
    pick = torch.randint(0, case["adapters"], (m + 1,), generator=gen, device="cuda")
    none = torch.rand(m + 1, generator=gen, device="cuda") < case["none"]
    pick = torch.where(none, torch.full_like(pick, -1), pick)
    return pick[which].to(torch.int32).contiguous()


def _plan(ids, groups):
    """(offsets [groups + 1], order): rows by group, in their own order; ungrouped rows last."""
    key = torch.where((ids >= 0) & (ids < groups), ids, torch.full_like(ids, groups)).long()
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, order


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] == "group_rows":
        ids = torch.randint(0, case["groups"], (case["rows"],), generator=gen, device="cuda")
        if case["dropped"]:
            gone = torch.rand(case["rows"], generator=gen, device="cuda") < case["dropped"]
            ids = torch.where(gone, torch.full_like(ids, -1), ids)
        return {"ids": ids.to(torch.int32)}
    dt = _DT[case["dtype"]]
    n, k = case["N"], case["K"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    d = {}
    if case["op"] == "adapters":
        g, r = case["adapters"], case["rank"]
        d["ids"] = _requests(case, gen)
        d["x"] = normal(case["rows"], k)
        d["a"] = normal(g, r, k, std=1.0 / math.sqrt(k))
        d["b"] = normal(g, n, r, std=0.3)
        d["scale"] = torch.rand(g, generator=gen, device="cuda") * 1.5 + 0.5
        stack = 1
    else:
        d["ids"] = _route(case, gen)
        rows = case["tokens"] * case["topk"]
        if case["op"] == "experts_dx":
            d["x"] = normal(rows, n, std=0.05)         # dY, in group order
        else:
            d["x"] = normal(case["tokens"] if case["layout"] == "gather" else rows, k)
        stack = case["experts"]
    d["weight"] = _weight(gen, (stack, n, k), case["quant"], case["dq"])
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    st = {"case": case, "ids": d["ids"]}
    if case["op"] == "group_rows":
        if own:
            from dequant_gemm_nf4_amd import tensors
            st["lib"] = tensors
            st["plan"] = tensors.empty_row_groups(case["rows"], case["groups"])
        return st
    groups = case["adapters"] if case["op"] == "adapters" else case["experts"]
    st["offsets"], st["order"] = _plan(d["ids"], groups)
    st["bounds"] = st["offsets"].tolist()
    st["levels"] = torch.tensor(_levels(case["quant"]), dtype=torch.float32, device="cuda")
    st["packed"], st["absmax"], st["absmax2"], st["mean"] = d["weight"]
    for key in ("x", "a", "b", "scale"):
        if key in d:
            st[key] = d[key]
    # the caller's output buffer: rows without an expert stay as they are, zero
    width = case["K"] if case["op"] == "experts_dx" else case["N"]
    st["y"] = torch.zeros(d["ids"].numel(), width, dtype=_DT[case["dtype"]], device="cuda")
    if own:
        from dequant_gemm_nf4_amd import tensors
        st["lib"] = tensors
        shape = (case["N"], case["K"]) if case["op"] == "adapters" else \
            (case["experts"], case["N"], case["K"])
        n = math.prod(shape)
        st["q"] = tensors.QuantizedWeight(n, shape, case["dq"], st["packed"], st["absmax"],
                                          st["absmax2"], st["mean"], case["quant"],
                                          _DT[case["dtype"]], "linear")
        st["rows"] = tensors.RowGroups(groups, st["offsets"], st["order"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        lib = st["lib"]
        if op == "group_rows":
            plan = lib.group_rows(st["ids"], case["groups"], out=st["plan"])
            return plan.offsets, plan.order
        if op == "adapters":
            return lib.linear_adapters(st["x"], st["q"], st["rows"], st["a"], st["b"],
                                       st["scale"], out=st["y"])
        if op == "experts_dx":
            return lib.gemm_experts_dx(st["x"], st["q"], st["rows"], scatter=True, out=st["y"])
        if case["layout"] == "gather":
            return lib.gemm_experts(st["x"], st["q"], st["rows"], gather=case["topk"],
                                    out=st["y"])
        return lib.gemm_experts(st["x"], st["q"], st["rows"], scatter=True, out=st["y"])
    if op == "group_rows":
        return _plan(st["ids"], case["groups"])
    x, y, order, bounds = st["x"], st["y"], st["order"].long(), st["bounds"]
    if op == "adapters":
        acc = x.float() @ _plain_weight(st, 0).t()
        for g in range(case["adapters"]):
            rows = order[bounds[g]:bounds[g + 1]]
            if rows.numel():
                low = (x[rows].float() @ st["a"][g].float().t()) * st["scale"][g]
                acc[rows] += low @ st["b"][g].float().t()
        return y.copy_(acc)
    for e in range(case["experts"]):
        i0, i1 = bounds[e], bounds[e + 1]
        if i1 == i0:
            continue
        w = _plain_weight(st, e)
        if op == "experts_dx":
            y[order[i0:i1]] = (x[i0:i1].float() @ w).to(y.dtype)
        elif case["layout"] == "gather":
            y[i0:i1] = (x[order[i0:i1] // case["topk"]].float() @ w.t()).to(y.dtype)
        else:
            y[order[i0:i1]] = (x[i0:i1].float() @ w.t()).to(y.dtype)
    return y


def exact(case, seed):
    d = _inputs(case, seed)
    ids = d["ids"].cpu().numpy()
    if case["op"] == "group_rows":
        lists = [np.flatnonzero(ids == g) for g in range(case["groups"])]
        lists.append(np.flatnonzero((ids < 0) | (ids >= case["groups"])))
        offsets = np.concatenate(([0], np.cumsum([len(v) for v in lists[:-1]])))
        return (torch.from_numpy(offsets.astype(np.int32)),
                torch.from_numpy(np.concatenate(lists).astype(np.int32)))
    x = d["x"].double()
    if case["op"] == "adapters":
        y = torch.matmul(x, _exact_weight(case, d["weight"], 0).t())
        for g in np.unique(ids[ids >= 0]):
            rows = torch.from_numpy(np.flatnonzero(ids == g)).cuda()
            up = d["b"][g].double() * d["scale"][g].double()
            y[rows] = y[rows] + torch.matmul(torch.matmul(x[rows], d["a"][g].double().t()), up.t())
        return y
    width = case["K"] if case["op"] == "experts_dx" else case["N"]
    y = torch.zeros(len(ids), width, dtype=torch.float64, device="cuda")
    at = 0
    for e in range(case["experts"]):
        slots = np.flatnonzero(ids == e)
        if len(slots) == 0:
            continue
        w = _exact_weight(case, d["weight"], e)
        grouped = torch.arange(at, at + len(slots), device="cuda")
        slot = torch.from_numpy(slots).cuda()
        at += len(slots)
        if case["op"] == "experts_dx":
            y[slot] = torch.matmul(x[grouped], w)
        elif case["layout"] == "gather":
            y[grouped] = torch.matmul(x[slot // case["topk"]], w.t())
        else:
            y[slot] = torch.matmul(x[grouped], w.t())
    return y


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _weight_bytes(stack, n, k, dq):
    per = n * k / 2 + n * k / 64 * (1 if dq else 4) + (n * k / 64 / 256 * 4 if dq else 0)
    return stack * per


def work(case):
    if case["op"] == "group_rows":
        return {"bytes": 4 * (2 * case["rows"] + case["groups"] + 1), "flops": 0}
    n, k = case["N"], case["K"]
    if case["op"] == "adapters":
        m, r = case["rows"], case["rank"]
        with_one = m * (1.0 - case["none"])
        requests = max(1.0, with_one / case["run"])
        used = case["adapters"] * (1.0 - (1.0 - 1.0 / case["adapters"]) ** requests)
        return {"bytes": int(_weight_bytes(1, n, k, case["dq"]) + 2 * m * (n + k)
                             + 2 * used * r * (n + k) + 8 * m),
                "flops": int(2 * m * n * k + 2 * with_one * r * (n + k))}
    rows = case["tokens"] * case["topk"] * (1.0 - case["dropped"])
    used = case["experts"] * (1.0 - (1.0 - case["topk"] / case["experts"]) ** case["tokens"])
    read = rows if case["layout"] == "scatter" else case["tokens"]
    wide = (n, k) if case["op"] == "experts_dx" else (k, n)
    return {"bytes": int(_weight_bytes(used, n, k, case["dq"]) + 2 * read * wide[0]
                         + 2 * rows * wide[1] + 4 * rows),
            "flops": int(2 * rows * n * k)}
