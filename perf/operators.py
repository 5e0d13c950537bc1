"""The operators of a mixture-of-experts layer with 4-bit weights, as cases to measure.

``route``         scores, groups, top-k and weights of a router, and the expert-sorted order of the rows
``route_bwd``     the gradient of its weights with respect to the logits
``mx_linear``     rows quantised to MXFP4 times MXFP4 weights
``mx_experts``    the same over the experts' rows, gathered through the router's order
``combine``       the experts' rows back to the tokens, weighted
``combine_bwd``   its gradients: the experts' rows' and the weights'

``run`` computes them in elementary torch operations, or, with ``own`` true, by the calls of this
repository's package.  ``exact`` gives the same answers from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32              # elements of one MXFP4 scale
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # a decoding step's router: a few sequences, one token each
        {"name": "route-decode", "op": "route", "tokens": 16, "experts": 64, "top_k": 2, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "group_top": 1, "renorm": True, "scale": 1.0, "dtype": "f32"},
        # one training step's router: the package's 64-expert top-2 layer over 16384 tokens
        {"name": "route-train", "op": "route", "tokens": 16384, "experts": 64, "top_k": 2, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "group_top": 1, "renorm": True, "scale": 1.0, "dtype": "bf16"},
        # many small experts in groups, balanced by a bias on sigmoid scores
        {"name": "route-groups", "op": "route", "tokens": 65536, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "keep": 4, "group_top": 2, "renorm": True, "scale": 1.5, "dtype": "f32"},
        # gradient of softmax weights that are not renormalised: every expert's logit takes part
        {"name": "route-bwd", "op": "route_bwd", "tokens": 16384, "experts": 64, "top_k": 2, "score": "softmax",
         "renorm": False, "scale": 1.0, "dtype": "bf16"},
        # gradient of the grouped sigmoid router, an odd number of tokens
        {"name": "route-bwd-sigmoid", "op": "route_bwd", "tokens": 40001, "experts": 160, "top_k": 6,
         "score": "sigmoid", "renorm": True, "scale": 1.5, "dtype": "f32"},
        # one token through the up projection of the package's FFN block: the weights' bytes are all that counts
        {"name": "mx-decode", "op": "mx_linear", "rows": 1, "n": 14336, "k": 4096, "dtype": "bf16", "out": "bf16"},
        # a ragged chunk of a prompt, sizes that fill no tile and no scale block
        {"name": "mx-ragged", "op": "mx_linear", "rows": 333, "n": 1411, "k": 2024, "dtype": "f32", "out": "f32"},
        # a training batch through the up projection of the package's FFN block
        {"name": "mx-train", "op": "mx_linear", "rows": 8192, "n": 14336, "k": 4096, "dtype": "bf16", "out": "bf16"},
        # 16 decoded tokens through the package's 64 experts, most of them with no row or one
        {"name": "experts-decode", "op": "mx_experts", "tokens": 16, "experts": 64, "top_k": 2, "n": 1408, "k": 2048,
         "dtype": "bf16", "out": "bf16"},
        # a training batch through the same experts, the rows' sizes uneven as a router leaves them
        {"name": "experts-train", "op": "mx_experts", "tokens": 16384, "experts": 64, "top_k": 2, "n": 1408, "k": 2048,
         "dtype": "bf16", "out": "bf16"},
        # that batch's expert outputs back to the tokens
        {"name": "combine-train", "op": "combine", "tokens": 16384, "experts": 64, "top_k": 2, "width": 2048,
         "dtype": "bf16"},
        # and its gradients
        {"name": "combine-bwd", "op": "combine_bwd", "tokens": 16384, "experts": 64, "top_k": 2, "width": 2048,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "mx_linear", "mx_experts", "combine", "combine_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        experts = groups * max(2, _log_int(rng, 4, 256) // groups)
        tokens = _log_int(rng, 1, 65536)
        keep = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, experts // groups * keep))
        case = {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k,
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 1.5]), "dtype": dtype}
        if op == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, keep=keep, group_top=rng.choice([1, 2]))
        return case
    if op == "mx_linear":
        return {"op": op, "rows": _log_int(rng, 1, 8192), "n": _log_int(rng, 100, 8192), "k": _log_int(rng, 100, 8192),
                "dtype": dtype, "out": rng.choice(["f32", "bf16"])}
    if op == "mx_experts":
        experts = _log_int(rng, 4, 64)
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "experts": experts, "top_k": rng.randint(1, min(4, experts)),
                "n": _log_int(rng, 100, 2048), "k": _log_int(rng, 100, 2048), "dtype": dtype,
                "out": rng.choice(["f32", "bf16"])}
    experts, tokens, top_k = _log_int(rng, 8, 64), _log_int(rng, 1, 16384), rng.randint(1, 8)
    widest = min(4096, (1 << (26 if dtype == "bf16" else 25)) // (tokens * top_k))      # as many bytes as the largest
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "width": _log_int(rng, 64, widest),
            "dtype": dtype}


def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    s = size[case["dtype"]]
    if op in ("route", "route_bwd"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        if op == "route":
            # logits in; ids, weights, both maps and the offsets out
            return {"bytes": T * E * s + T * k * 16 + 8 * (E + 1) + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
        # the other experts' logits are needed only by a softmax that is not renormalised
        full = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": (T * E if full else T * k) * s + T * k * 8 + T * E * s, "flops": (4 * T * E if full else 8 * T * k)}
    if op == "mx_linear":
        M, N, K = case["rows"], case["n"], case["k"]
        return {"bytes": M * K * s + N * (K // 2 + -(-K // BLOCK)) + M * N * size[case["out"]], "flops": 2 * M * N * K}
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    R = T * k
    if op == "mx_experts":
        N, K = case["n"], case["k"]
        hit = max(1, int(E * (1.0 - (1.0 - 1.0 / E) ** R)))     # experts that have a row, about
        return {"bytes": T * K * s + R * 4 + hit * N * (K // 2 + -(-K // BLOCK)) + R * N * size[case["out"]],
                "flops": 2 * R * N * K}
    D = case["width"]
    if op == "combine":
        return {"bytes": (R + T) * D * s + R * 8, "flops": 2 * R * D}
    return {"bytes": (2 * R + T) * D * s + R * 12, "flops": 3 * R * D}


# ------------------------------------------------------------------ inputs ----

def _logits(g, T, E, dtype):
    """Router logits: a token's own preferences and an expert's popularity."""
    popular = torch.randn(E, generator=g, device="cuda") * 0.5
    return (torch.randn(T, E, generator=g, device="cuda") * 1.5 + popular).to(dtype)


def _choices(g, T, E, k):
    """k different experts of every token, skewed as a router's: [T, k] int64."""
    x = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda") * 0.7
    return x.argsort(dim=1, descending=True)[:, :k].contiguous()


def _order(ids, E):
    """(offsets int64 [E + 1], slot_row, row_slot int32) of the slots sorted by expert, in slot order within one."""
    flat = ids.reshape(-1).long()
    by = torch.argsort(flat, stable=True)
    slot_row = torch.empty_like(by)
    slot_row[by] = torch.arange(by.numel(), device=by.device)
    offsets = torch.searchsorted(flat[by], torch.arange(E + 1, device=by.device))
    return offsets, slot_row.to(torch.int32).reshape(ids.shape), by.to(torch.int32)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "route":
        T, E = case["tokens"], case["experts"]
        s["logits"] = _logits(g, T, E, dt)
        s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if case["bias"] else None
    elif op == "route_bwd":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        s["logits"] = _logits(g, T, E, dt)
        s["ids"] = s["logits"].double().argsort(dim=1, descending=True, stable=True)[:, :k].to(torch.int32).contiguous()
        s["dweights"] = torch.randn(T, k, generator=g, device="cuda") * 1e-3
    elif op == "mx_linear":
        M, N, K = case["rows"], case["n"], case["k"]
        s["x"] = torch.randn(M, K, generator=g, device="cuda").to(dt)
        s["W"] = (torch.randn(1, N, K, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    elif op == "mx_experts":
        T, E, k, N, K = case["tokens"], case["experts"], case["top_k"], case["n"], case["k"]
        s["x"] = torch.randn(T, K, generator=g, device="cuda").to(dt)
        s["offsets"], s["slot_row"], s["row_slot"] = _order(_choices(g, T, E, k), E)
        s["bounds"] = s["offsets"].tolist()
        s["W"] = (torch.randn(E, N, K, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    else:
        T, E, k, D = case["tokens"], case["experts"], case["top_k"], case["width"]
        s["slot_row"] = _order(_choices(g, T, E, k), E)[1]
        w = torch.rand(T, k, generator=g, device="cuda") + 0.05
        s["weights"] = w / w.sum(dim=1, keepdim=True)
        s["rows"] = torch.randn(T * k, D, generator=g, device="cuda").to(dt)
        if op == "combine_bwd":
            s["dy"] = (torch.randn(T, D, generator=g, device="cuda") * 1e-2).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _handles(s)
    elif "W" in s:
        s["w"] = torch.stack([_mx_values(w) for w in s["W"]])       # the values that 4-bit weights stand for
    return s


def _handles(s):
    """Descriptors, outputs and workspaces that a program keeps between its calls."""
    from stochastic_rounding_quantization_amd import s3r
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op in ("route", "route_bwd"):
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        s["desc"] = s3r.route_desc(T, E, k, score=s3r.SIGMOID if c["score"] == "sigmoid" else s3r.SOFTMAX,
                                   groups=c.get("groups", 1), keep=c.get("keep", 1), group_top=c.get("group_top", 1),
                                   renorm=c["renorm"], scale=c["scale"])
        if op == "route":
            s["routed"] = s3r.routed_buffers(s["desc"], "cuda")
        else:
            s["dlogits"] = torch.empty(T, E, dtype=dt, device="cuda")
    elif op in ("mx_linear", "mx_experts"):
        R = c["rows"] if op == "mx_linear" else c["tokens"] * c["top_k"]
        s["out"] = torch.empty(R, c["n"], dtype=DTYPES[c["out"]], device="cuda")
        s["w"] = s3r.mx_rows(s["W"])                                 # 4-bit weights, laid out once
        s["ws"] = s3r.mx_linear_buffer(R, c["k"], "cuda")
    elif op == "combine":
        s["y"] = torch.empty(c["tokens"], c["width"], dtype=dt, device="cuda")
    else:
        s["drows"] = torch.empty_like(s["rows"])
        s["dw"] = torch.empty_like(s["weights"])


# --------------------------------------------------------------- one pass ----

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from stochastic_rounding_quantization_amd import s3r
    op = s["case"]["op"]
    if op == "route":
        r = s["routed"]
        s3r.s3r_route(s["desc"], s["logits"], s["bias"], r.ids, r.weights, r.offsets, r.slot_row, r.row_slot, r.ws)
        return r.ids, r.weights, r.offsets, r.slot_row, r.row_slot
    if op == "route_bwd":
        s3r.s3r_route_backward(s["desc"], s["logits"], s["ids"], s["dweights"], s["dlogits"])
        return s["dlogits"]
    if op == "mx_linear":
        s3r.s3r_mx_linear(s["x"], s["w"], s["out"], ws=s["ws"])
        return s["out"]
    if op == "mx_experts":
        s3r.s3r_mx_linear(s["x"], s["w"], s["out"], offsets=s["offsets"], index=s["row_slot"],
                          index_div=s["case"]["top_k"], ws=s["ws"])
        return s["out"]
    if op == "combine":
        s3r.s3r_combine(s["rows"], s["slot_row"], s["weights"], s["y"])
        return s["y"]
    s3r.s3r_combine_backward(s["dy"], s["rows"], s["slot_row"], s["weights"], s["drows"], s["dw"])
    return s["drows"], s["dw"]


# -------------------------------------------------------------- plain forms ----

def _scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(s):
    c, x = s["case"], s["logits"]
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    # keys in 64 bits: two experts may be closer than 32 bits tell apart; without a bias the logits have
    # the scores' order
    if s["bias"] is None and (c["groups"] == 1 or c["group_top"] == 1):
        key = x.double()
    else:
        key = _scores(x.double(), c["score"])
        if s["bias"] is not None:
            key = key + s["bias"].double()
    if c["groups"] > 1:
        per = E // c["groups"]
        inside = key.reshape(T, c["groups"], per).sort(dim=2, descending=True).values
        of_group = inside[:, :, :c["group_top"]].sum(dim=2)
        best = of_group.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(T, c["groups"], dtype=torch.bool, device=x.device).scatter(1, best, True)
        key = torch.where(kept.repeat_interleave(per, dim=1), key, float("-inf"))
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = _scores(x.float(), c["score"]).gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * c["scale"]
    offsets, slot_row, row_slot = _order(ids, E)
    return ids.to(torch.int32), w, offsets, slot_row, row_slot


def _plain_route_bwd(s):
    c, x = s["case"], s["logits"]
    ids, g = s["ids"].long(), s["dweights"] * c["scale"]
    sc = _scores(x.float(), c["score"])
    mine = sc.gather(1, ids)
    if c["renorm"]:
        total = mine.sum(dim=1, keepdim=True)
        g = (g - (g * mine).sum(dim=1, keepdim=True) / total) / total     # gradient of the chosen scores
    if c["score"] == "sigmoid":
        out = torch.zeros_like(sc).scatter(1, ids, g * mine * (1.0 - mine))
    elif c["renorm"]:
        out = torch.zeros_like(sc).scatter(1, ids, g * mine)              # the rest of the row cancels
    else:
        out = sc * (torch.zeros_like(sc).scatter(1, ids, g) - (g * mine).sum(dim=1, keepdim=True))
    return out.to(x.dtype)


def _two_to(k):
    """2^k as float64, exact."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _mx_values(x):
    """The values that MXFP4 leaves of x [R, K]: a block of 32 along K has the scale 2^k with the smallest k
    such that its largest magnitude is at most 6 * 2^k (k >= -127); E2M1 values, ties to even."""
    R, K = x.shape
    pad = -K % BLOCK
    v = torch.nn.functional.pad(x.double(), (0, pad)).reshape(R, -1, BLOCK)
    top = v.abs().amax(dim=2, keepdim=True)
    m, e = torch.frexp(top)
    k = torch.where(top > 0, torch.where(m <= 0.75, e - 3, e - 2), -127).clamp(-127, 127)
    scale = _two_to(k)
    y = v / scale
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    q = step * torch.round(y / step) * scale
    q = torch.where(torch.isfinite(top), q, float("nan"))
    return q.reshape(R, -1)[:, :K].float()


def _plain_linear(s):
    return torch.matmul(_mx_values(s["x"]), s["w"][0].t()).to(DTYPES[s["case"]["out"]])


def _plain_experts(s):
    c = s["case"]
    x = _mx_values(s["x"])[s["row_slot"].long() // c["top_k"]]
    out = torch.empty(x.shape[0], c["n"], dtype=DTYPES[c["out"]], device=x.device)
    for e in range(c["experts"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if b > a:
            out[a:b] = torch.matmul(x[a:b], s["w"][e].t())
    return out


def _plain_combine(s):
    c = s["case"]
    y = torch.zeros(c["tokens"], c["width"], device="cuda")
    for j in range(c["top_k"]):
        y = y + s["weights"][:, j:j + 1] * s["rows"][s["slot_row"][:, j].long()].float()
    return y.to(DTYPES[c["dtype"]])


def _plain_combine_bwd(s):
    c = s["case"]
    dy = s["dy"].float()
    drows = torch.empty_like(s["rows"])
    dw = torch.empty_like(s["weights"])
    for j in range(c["top_k"]):
        r = s["slot_row"][:, j].long()
        drows[r] = (s["weights"][:, j:j + 1] * dy).to(drows.dtype)
        dw[:, j] = (dy * s["rows"][r].float()).sum(dim=1)
    return drows, dw


_PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "mx_linear": _plain_linear,
          "mx_experts": _plain_experts, "combine": _plain_combine, "combine_bwd": _plain_combine_bwd}


# --------------------------------------------- the definitions in 64 bits ----

def exact(case, seed):
    return _EXACT[case["op"]](case, _inputs(case, seed))


def _softmax64(x):
    z = np.exp(x - x.max(axis=1, keepdims=True))
    return z / z.sum(axis=1, keepdims=True)


def _exact_route(c, s):
    x = s["logits"].double().cpu().numpy()
    T, E, k, G = c["tokens"], c["experts"], c["top_k"], c["groups"]
    score = np.exp(-np.logaddexp(0.0, -x)) if c["score"] == "sigmoid" else _softmax64(x)
    key = score + s["bias"].double().cpu().numpy() if s["bias"] is not None else score
    if s["bias"] is None and (G == 1 or c["group_top"] == 1):
        key = x                                      # the same order
    if G > 1:
        parts = key.reshape(T, G, E // G)
        high = -np.partition(-parts, c["group_top"] - 1, axis=2)[:, :, :c["group_top"]].sum(axis=2)
        rank = np.argsort(np.argsort(-high, axis=1, kind="stable"), axis=1)
        key = np.where((rank < c["keep"])[:, :, None], parts, -np.inf).reshape(T, E)
    ids = np.empty((T, k), dtype=np.int64)
    left = key.copy()
    for j in range(k):                               # the largest that is left; argmax takes the lowest index
        ids[:, j] = left.argmax(axis=1)
        np.put_along_axis(left, ids[:, j:j + 1], -np.inf, axis=1)
    w = np.take_along_axis(score, ids, axis=1)
    w = c["scale"] * (w / w.sum(axis=1, keepdims=True) if c["renorm"] else w)
    flat = ids.reshape(-1)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    row_slot = np.lexsort((np.arange(flat.size), flat))
    slot_row = np.empty(flat.size, dtype=np.int64)
    slot_row[row_slot] = np.arange(flat.size)
    return (ids.astype(np.int32), w, offsets.astype(np.int64), slot_row.reshape(T, k).astype(np.int32),
            row_slot.astype(np.int32))


def _exact_route_bwd(c, s):
    x = s["logits"].double().cpu().numpy()
    ids, g = s["ids"].cpu().numpy().astype(np.int64), s["dweights"].double().cpu().numpy() * c["scale"]
    if c["score"] == "sigmoid":
        log_s = -np.logaddexp(0.0, -np.take_along_axis(x, ids, axis=1))
        other = np.exp(-np.logaddexp(0.0, np.take_along_axis(x, ids, axis=1)))     # 1 - s
        p = _softmax64(log_s) if c["renorm"] else np.exp(log_s)
        chosen = p * (g - (p * g).sum(axis=1, keepdims=True)) * other if c["renorm"] else g * p * other
    elif c["renorm"]:
        p = _softmax64(np.take_along_axis(x, ids, axis=1))
        chosen = p * (g - (p * g).sum(axis=1, keepdims=True))
    else:
        p = _softmax64(x)
        spread = np.zeros_like(x)
        np.put_along_axis(spread, ids, g, axis=1)
        return p * (spread - (p * spread).sum(axis=1, keepdims=True))
    out = np.zeros_like(x)
    np.put_along_axis(out, ids, chosen, axis=1)
    return out


def _exact_values(x):
    """E2M1 by its table of values: the nearest, a tie to the even place of the table."""
    R, K = x.shape
    v = torch.zeros(R, -(-K // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :K] = x
    v = v.reshape(R, -1, BLOCK)
    top = v.abs().amax(dim=2)
    k = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -300) / 6.0)).to(torch.int64) - 1
    for _ in range(3):
        k = torch.where(6.0 * _two_to(k) < top, k + 1, k)
    unit = _two_to(k.clamp(-127, 127))[:, :, None]
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    mid = (table[1:] + table[:-1]) / 2
    y = v.abs() / unit
    lower = torch.bucketize(y, mid, right=False)      # a tie stays on the lower side
    upper = torch.bucketize(y, mid, right=True)
    at = torch.where(lower % 2 == 0, lower, upper)
    return (torch.sign(v) * table[at] * unit).reshape(R, -1)[:, :K]


def _exact_linear(c, s):
    return torch.matmul(_exact_values(s["x"].double()), _exact_values(s["W"][0].double()).t())


def _exact_experts(c, s):
    x = _exact_values(s["x"].double())[s["row_slot"].long() // c["top_k"]]
    parts = [torch.matmul(x[a:b], _exact_values(s["W"][e].double()).t())
             for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])) if b > a]
    return torch.cat(parts)


def _exact_combine(c, s):
    rows = s["rows"].double()[s["slot_row"].long()]                 # [T, k, D]
    return (rows * s["weights"].double()[:, :, None]).sum(dim=1)


def _exact_combine_bwd(c, s):
    at = s["slot_row"].long()
    dy, w = s["dy"].double(), s["weights"].double()
    drows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=dy.device)
    dw = torch.zeros_like(w)
    for t0 in range(0, at.shape[0], 2048):
        t = slice(t0, t0 + 2048)
        drows[at[t].reshape(-1)] = (w[t][:, :, None] * dy[t][:, None, :]).reshape(-1, dy.shape[1])
        dw[t] = (s["rows"][at[t].reshape(-1)].double().reshape(*at[t].shape, -1) * dy[t][:, None, :]).sum(dim=2)
    return drows, dw


_EXACT = {"route": _exact_route, "route_bwd": _exact_route_bwd, "mx_linear": _exact_linear,
          "mx_experts": _exact_experts, "combine": _exact_combine, "combine_bwd": _exact_combine_bwd}
