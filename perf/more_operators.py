"""Cases of the operators of a mixture-of-experts layer around and with its 8-bit
expert products: RMS norm with the residual's addition and quantised output,
routing to experts, experts in FP8 with a scale for each block of 128, SwiGLU
with quantised output, and the weighted sum of the experts' outputs.

`run` computes a case in elementary torch operations (`own` false) or with the
library's entry points (`own` true); `exact` computes it in 64 bits.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the norm of a decode step's few tokens, in front of FP8 experts
        {"name": "norm_decode", "op": "norm", "rows": 5, "width": 7168, "dtype": "bf16", "weight": "bf16", "out": "fp8", "scales": "block",
         "residual": True, "wide": False},
        # the norm of a prompt, in front of a tokenwise FP8 projection
        {"name": "norm_prompt", "op": "norm", "rows": 8191, "width": 7168, "dtype": "bf16", "weight": "bf16", "out": "fp8", "scales": "token",
         "residual": True, "wide": False},
        # routing of a decode step: sigmoid scores with a bias for balance, 4 of 8 groups
        {"name": "route_decode", "op": "route", "tokens": 5, "experts": 256, "top_k": 8, "dtype": "fp32", "scoring": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_best": 2, "renorm": True},
        # the same of a prompt batch
        {"name": "route_prompt", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8, "dtype": "fp32", "scoring": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_best": 2, "renorm": True},
        # a softmax router of few experts, 16-bit logits, ragged counts
        {"name": "route_softmax", "op": "route", "tokens": 4097, "experts": 60, "top_k": 4, "dtype": "bf16", "scoring": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_best": 1, "renorm": False},
        # gate and up of a few decoding users: each expert has a row or two, the weights' stream
        {"name": "experts_decode", "op": "experts", "tokens": 4, "experts": 256, "top_k": 8, "N": 4096, "K": 7168, "mode": "indexed"},
        # down projection of a decode batch, rows sorted by expert: a few rows for each of 256 experts
        {"name": "experts_batch", "op": "experts", "tokens": 251, "experts": 256, "top_k": 8, "N": 7168, "K": 2048, "mode": "grouped"},
        # a prompt over the experts of one rank: the compute-bound end
        {"name": "experts_prompt", "op": "experts", "tokens": 4095, "experts": 32, "top_k": 8, "N": 4096, "K": 7168, "mode": "indexed"},
        # between the two expert products of a few tokens, in front of a tokenwise FP8 projection
        {"name": "silu_decode", "op": "silu", "rows": 37, "width": 2048, "dtype": "fp16", "out": "fp8", "scales": "token"},
        # the same of a prompt, in front of FP8 experts
        {"name": "silu_prompt", "op": "silu", "rows": 16376, "width": 2048, "dtype": "bf16", "out": "fp8", "scales": "block"},
        # the sum over each token's experts, a decode step and a prompt with the residual
        {"name": "combine_decode", "op": "combine", "tokens": 5, "top_k": 8, "width": 7168, "dtype": "bf16", "order": "pairs", "add": True},
        {"name": "combine_prompt", "op": "combine", "tokens": 4095, "top_k": 8, "width": 7168, "dtype": "bf16", "order": "sorted", "add": True},
    ]


MOST_FLOPS, MOST_WEIGHTS = 1.5e12, 2e9  # of a drawn case: below the largest listed one's


def spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "route", "experts", "experts", "experts", "silu", "combine"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("norm", "silu"):
        out, scales = rng.choice([(dtype, "none"), ("fp8", "token"), ("fp8", "block"), ("fp8", "block"), ("int8", "token")])
        if op == "silu" and out == dtype:
            out, scales = "fp8", "token"
        rows = spread(rng, 1, 8192)
        width = 128 * spread(rng, 1, 64) if scales == "block" else 8 * spread(rng, 16, 1024) if op == "silu" or rng.random() < 0.7 else spread(rng, 100, 9000)
        case = {"op": op, "rows": rows, "width": width, "dtype": dtype, "out": out, "scales": scales}
        if op == "norm":
            case |= {"weight": rng.choice([dtype, dtype, "fp32"]), "residual": rng.random() < 0.75, "wide": rng.random() < 0.25}
        return case
    if op == "route":
        experts, groups = rng.choice([(8, 1), (16, 1), (60, 1), (64, 1), (64, 8), (128, 1), (128, 4), (160, 8), (256, 1), (256, 8), (384, 1), (512, 8)])
        top_groups = rng.randint(max(1, groups // 4), max(1, groups // 2))
        return {"op": op, "tokens": spread(rng, 1, 16384), "experts": experts, "top_k": rng.randint(1, min(10, experts // groups * top_groups)),
                "dtype": rng.choice(["fp32", "fp32", dtype]), "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": groups, "top_groups": top_groups, "group_best": rng.choice([1, 2]), "renorm": rng.random() < 0.6}
    if op == "combine":
        return {"op": op, "tokens": spread(rng, 1, 4096), "top_k": rng.randint(1, 10), "width": rng.choice([512, 1000, 1024, 1777, 2048, 4096, 5120, 7168]),
                "dtype": dtype, "order": rng.choice(["pairs", "sorted"]), "add": rng.random() < 0.6}
    while True:
        experts = spread(rng, 2, 256)
        case = {"op": op, "tokens": spread(rng, 1, 4096), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                "N": rng.choice([256, 1000, 1024, 1536, 2048, 4096, 5000, 7168]), "K": 128 * spread(rng, 2, 56), "mode": rng.choice(["indexed", "grouped"])}
        if work(case)["flops"] < MOST_FLOPS and experts * case["N"] * case["K"] < MOST_WEIGHTS:
            return case


def held(case):
    """How many experts have rows, for routes as prepare() makes them: the mean."""
    p = popularity(case["experts"])
    return sum(1 - (1 - min(1.0, x * case["top_k"])) ** case["tokens"] for x in p)


def popularity(experts):
    """Experts are not equally liked: a gentle slope, the most liked three times as often as the least."""
    w = [3.0 ** (-e / max(1, experts - 1)) for e in range(experts)]
    return [x / sum(w) for x in w]


def scale_bytes(case):
    return 4 * case["rows"] * {"none": 0, "token": 1, "block": case["width"] // 128}[case["scales"]]


def work(case):
    op = case["op"]
    if op in ("norm", "silu"):
        n, size = case["rows"] * case["width"], 2 if case["scales"] == "none" else 1
        if op == "silu":
            return {"bytes": n * (4 + size) + scale_bytes(case), "flops": 8 * n}
        return {"bytes": n * (2 + (4 if case["residual"] else 0) + size) + scale_bytes(case) + case["width"] * (4 if case["weight"] == "fp32" else 2), "flops": 7 * n}
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * (e * (4 if case["dtype"] == "fp32" else 2) + 8 * k) + (4 * e if case["bias"] else 0), "flops": t * e * 8}
    if op == "combine":
        t, k, n = case["tokens"], case["top_k"], case["width"]
        return {"bytes": 2 * t * n * (k + 1 + (1 if case["add"] else 0)) + t * k * (4 if case["order"] == "pairs" else 8), "flops": 2 * t * k * n}
    t, k, n, depth = case["tokens"], case["top_k"], case["N"], case["K"]
    rows = t if case["mode"] == "indexed" else t * k
    weights = held(case) * (n * depth + 4 * (depth // 128) * -(-n // 128))
    return {"bytes": int(weights) + rows * (depth + depth // 32) + 2 * t * k * n, "flops": 2 * t * k * n * depth}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def routes(case, gen):
    """top_k different experts for each token, the liked ones more often (their weights drawn with exponentials)."""
    p = torch.tensor(popularity(case["experts"]), device="cuda")
    draws = torch.empty(case["tokens"], case["experts"], device="cuda").exponential_(generator=gen) / p
    return draws.argsort(1)[:, :case["top_k"]].to(torch.int32).contiguous()


def by_expert(ids, experts):
    """The pairs' numbers sorted by expert, and where each expert's begin."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    start = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    start[1:] = torch.bincount(flat, minlength=experts).cumsum(0)
    return order.to(torch.int32), start


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op == "norm":
        m, k, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
        # a residual stream has a few wide channels; `wide`: the rows are a slice of wider ones
        channel = torch.exp(0.6 * normal(k)) * 2.0
        x = (normal(m, k + 64 if case["wide"] else k)).to(dt)
        s |= {"x": x[:, :k], "r": (normal(m, k) * channel).to(dt) if case["residual"] else None, "sum": torch.empty(m, k, dtype=dt, device="cuda"),
              "w": (1.0 + 0.2 * normal(k)).to(DTYPES[case["weight"]])}
    elif op == "silu":
        s |= {"gate_up": (1.5 * normal(case["rows"], 2 * case["width"])).to(DTYPES[case["dtype"]])}
    elif op == "route":
        t, e = case["tokens"], case["experts"]
        s |= {"logits": (1.3 * normal(t, e) + 0.5 * normal(e)).to(DTYPES[case["dtype"]]), "bias": 0.1 * normal(e) if case["bias"] else None,
              "ids": torch.empty(t, case["top_k"], dtype=torch.int32, device="cuda"), "weights": torch.empty(t, case["top_k"], device="cuda"),
              "scale": 1.0 + random.Random(seed).random()}
    elif op == "combine":
        t, k, n, dt = case["tokens"], case["top_k"], case["width"], DTYPES[case["dtype"]]
        w = torch.rand(t, k, device="cuda", generator=gen) + 0.05
        s |= {"y": normal(t * k, n).to(dt), "w": w / w.sum(1, keepdim=True), "add": (2.0 * normal(t, n)).to(dt) if case["add"] else None,
              "order": by_expert(torch.randint(0, 64, (t, k), device="cuda", generator=gen), 64)[0] if case["order"] == "sorted" else None,
              "out": torch.empty(t, n, dtype=dt, device="cuda"), "work": torch.empty(t * k + 4, dtype=torch.int32, device="cuda")}
    else:
        t, e, k, n, depth = case["tokens"], case["experts"], case["top_k"], case["N"], case["K"]
        blocks, cols, padded = depth // 128, -(-n // 128), -(-n // 16) * 16
        ids = routes(case, gen)
        order, start = by_expert(ids, e)
        rows = t if case["mode"] == "indexed" else t * k
        a = (60.0 * normal(rows, depth)).clamp(-448, 448).to(torch.float8_e4m3fn)
        w = torch.empty(e, depth, n, dtype=torch.float8_e4m3fn, device="cuda")
        packed = torch.zeros(e, padded // 16, depth // 64, 64, 16, dtype=torch.uint8, device="cuda")
        for i in range(e):
            w[i] = (60.0 * normal(depth, n)).clamp(-448, 448).to(torch.float8_e4m3fn)
            # the packed layout: strips of 16 columns, 64 of K; lane l holds column l % 16 and the 16 of K from 16 (l / 16)
            full = torch.zeros(depth, padded, dtype=torch.uint8, device="cuda")
            full[:, :n] = w[i].view(torch.uint8)
            packed[i] = full.view(depth // 64, 4, 16, padded // 16, 16).permute(3, 0, 1, 4, 2).reshape(padded // 16, depth // 64, 64, 16)
        s |= {"a": a, "sa": torch.exp(0.5 * normal(rows, blocks)) / 60.0, "w": w, "packed": packed,
              "sw": torch.exp(0.3 * normal(e, blocks, cols)) / (60.0 * depth ** 0.5), "ids": ids, "order": order, "start": start,
              "out": torch.empty(t * k, n, dtype=torch.bfloat16, device="cuda")}
    return s


# ---------------------------------------------------------------------------
# plain forms: elementary operations in 32 bits (scores that are ranked: 64)
# ---------------------------------------------------------------------------

def quantised(y, case):
    """y as codes and scales: [codes, scales], or the rounded values themselves."""
    if case["scales"] == "none":
        return [y.to(DTYPES[case["out"]])]
    top = 448.0 if case["out"] == "fp8" else 127.0
    parts = y.view(y.shape[0], -1, 128 if case["scales"] == "block" else y.shape[1])
    amax = parts.abs().amax(2, keepdim=True)
    scale = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    codes = (parts / scale).clamp(-top, top)
    return values(codes.to(torch.float8_e4m3fn) if case["out"] == "fp8" else codes.round().to(torch.int8), scale.squeeze(2), case)


def values(codes, scale, case):
    """What the codes stand for, and the scales: FP8 codes are values themselves, integers times their row's scale."""
    scale = scale.view(case["rows"], -1)
    codes = codes.reshape(case["rows"], -1)
    return [codes if codes.dtype == torch.float8_e4m3fn else (codes.float() * scale).to(DTYPES[case["dtype"]]), scale]


def plain_norm(s):
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
        s["sum"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * s["w"].float()
    return quantised(y, s["case"]) + ([s["sum"]] if s["r"] is not None else [])


def plain_silu(s):
    gate, up = s["gate_up"].float().chunk(2, 1)
    return quantised(gate / (1.0 + torch.exp(-gate)) * up, s["case"])


def best(x, k):
    """The places of the k largest of each row, ties to the lowest."""
    return torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]


def plain_route(s):
    case = s["case"]
    x = s["logits"].double()
    if case["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    rank = score if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        t, e = x.shape
        members = rank.view(t, case["groups"], -1)
        of_group = torch.sort(members, dim=2, descending=True).values[:, :, :case["group_best"]].sum(2)
        stay = torch.zeros(t, case["groups"], dtype=torch.bool, device="cuda").scatter_(1, best(of_group, case["top_groups"]), True)
        rank = torch.where(stay[:, :, None], members, -math.inf).view(t, e)
    ids = best(rank, case["top_k"])
    weights = score.gather(1, ids)
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    s["ids"].copy_(ids)
    s["weights"].copy_(weights * s["scale"])
    return [s["ids"], s["weights"]]


def plain_combine(s):
    case = s["case"]
    y, t, k = s["y"], case["tokens"], case["top_k"]
    if s["order"] is not None:  # row i holds the pair order[i]
        at = torch.empty_like(s["order"])
        at[s["order"].long()] = torch.arange(t * k, dtype=torch.int32, device="cuda")
        y = y[at.long()]
    total = (y.float().view(t, k, -1) * s["w"][:, :, None]).sum(1)
    s["out"].copy_(total if s["add"] is None else total + s["add"].float())
    return [s["out"]]


def by_blocks(codes, scale, n, dtype):
    """Weights [K][N] times the scale of each block of 128 x 128."""
    k = codes.shape[0]
    wide = scale.to(dtype).repeat_interleave(128, 1)[:, :n]
    return (codes.to(dtype).view(k // 128, 128, n) * wide[:, None]).view(k, n)


def plain_experts(s):
    case = s["case"]
    a = s["a"].float().view(s["a"].shape[0], -1, 128) * s["sa"][:, :, None]
    a = a.view(s["a"].shape)
    start = s["start"].tolist()
    for e in range(case["experts"]):
        lo, hi = start[e], start[e + 1]
        if lo == hi:
            continue
        w = by_blocks(s["w"][e], s["sw"][e], case["N"], torch.float32)
        if case["mode"] == "grouped":
            s["out"][lo:hi] = (a[lo:hi] @ w).to(torch.bfloat16)
        else:
            pairs = s["order"][lo:hi].long()
            s["out"][pairs] = (a[pairs // case["top_k"]] @ w).to(torch.bfloat16)
    return [s["out"]]


PLAIN = {"norm": plain_norm, "silu": plain_silu, "route": plain_route, "combine": plain_combine, "experts": plain_experts}


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------

def own_scales(case, hq):
    """Descriptor constants of the case's output and its empty codes and scales."""
    m, k = case["rows"], case["width"]
    kind, each = {"none": (hq.HQ_ASCALE_NONE, 0), "token": (hq.HQ_ASCALE_PER_TOKEN_F32, 1), "block": (hq.HQ_ASCALE_PER_BLOCK128_F32, k // 128)}[case["scales"]]
    return (CODES(hq)[case["out"]], kind, torch.empty(m, k, dtype=DTYPES[case["out"]], device="cuda"),
            torch.empty(m, each, device="cuda") if each else None)


def CODES(hq):
    return {"bf16": hq.HQ_DT_BF16, "fp16": hq.HQ_DT_FP16, "fp32": hq.HQ_DT_FP32, "fp8": hq.HQ_DT_FP8_E4M3, "int8": hq.HQ_DT_INT8}


def own_norm(s, hq):
    case = s["case"]
    k = case["width"]
    if "own" not in s:
        code, kind, out, scale = own_scales(case, hq)
        desc = hq.norm_desc(CODES(hq)[case["dtype"]], code, kind, eps=1e-6, weight_dtype=CODES(hq)[case["weight"]])
        s["own"] = desc, out, scale
    desc, out, scale = s["own"]
    hq.hq_rmsnorm(desc, case["rows"], k, s["x"], s["x"].stride(0), s["w"], out, scale, residual=s["r"], residual_stride=k,
                  sum_out=s["sum"] if s["r"] is not None else None, sum_stride=k)
    return (values(out, scale, case) if scale is not None else [out]) + ([s["sum"]] if s["r"] is not None else [])


def own_silu(s, hq):
    case = s["case"]
    if "own" not in s:
        s["own"] = own_scales(case, hq)
    code, kind, out, scale = s["own"]
    hq.hq_silu_mul_quant(CODES(hq)[case["dtype"]], code, kind, case["rows"], case["width"], s["gate_up"], out, scale)
    return values(out, scale, case) if scale is not None else [out]


def own_route(s, hq):
    case = s["case"]
    if "own" not in s:
        s["own"] = hq.route_desc(CODES(hq)[case["dtype"]], case["experts"], case["top_k"], sigmoid=case["scoring"] == "sigmoid",
                                 renormalize=case["renorm"], groups=case["groups"], top_groups=case["top_groups"],
                                 group_best=case["group_best"], scale=s["scale"])
    hq.hq_moe_route(s["own"], case["tokens"], s["logits"], case["experts"], s["bias"], s["ids"], s["weights"])
    return [s["ids"], s["weights"]]


def own_combine(s, hq):
    case = s["case"]
    hq.hq_moe_combine(CODES(hq)[case["dtype"]], case["tokens"], case["top_k"], case["width"], s["y"], s["w"], s["out"], add=s["add"],
                      sorted_pairs=s["order"], workspace=s["work"], ws_bytes=4 * s["work"].numel())
    return [s["out"]]


def own_experts(s, hq):
    case = s["case"]
    t, k = case["tokens"], case["top_k"]
    if "own" not in s:
        desc = hq.desc_moe_fp8_blockwise(case["experts"], case["N"], case["K"])
        nbytes = hq.hq_workspace_bytes(desc, t, k)
        s["own"] = desc, torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda"), nbytes
    desc, work_space, nbytes = s["own"]
    indexed = case["mode"] == "indexed"
    hq.hq_moe_gemm(desc, hq.HQ_MOE_INDEXED if indexed else hq.HQ_MOE_GROUPED, t, k, s["a"], s["sa"], s["ids"] if indexed else None,
                   None if indexed else s["start"], s["packed"], s["sw"], None, s["out"], work_space, nbytes)
    return [s["out"]]


OWN = {"norm": own_norm, "silu": own_silu, "route": own_route, "combine": own_combine, "experts": own_experts}


def run(state):
    if own:
        from bit_quantized_gemm_w4a16_amd import hq
        return OWN[state["case"]["op"]](state, hq)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact_codes(y, case):
    """Codes and scales of y in 64 bits: scales of the exact maxima, values rounded by the grid of their type."""
    if case["scales"] == "none":
        return [y]
    m, k = y.shape
    step = 128 if case["scales"] == "block" else k
    peak = np.abs(y).reshape(m, k // step, step).max(2)
    top = 448.0 if case["out"] == "fp8" else 127.0
    scale = np.where(peak > 0, peak / top, 1.0)
    ratio = y / np.repeat(scale, step, 1)
    if case["out"] == "int8":
        return [np.rint(ratio) * np.repeat(scale, step, 1), scale]
    # E4M3: steps of 2^(e-3) for 2^e <= |v| < 2^(e+1), not below 2^-9
    grid = np.exp2(np.maximum(np.frexp(ratio)[1] - 1, -6) - 3.0)
    return [np.rint(ratio / grid) * grid, scale]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    if op == "norm":
        h = host(s["x"]) + (host(s["r"]) if s["r"] is not None else 0.0)
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * host(s["w"])
        return exact_codes(y, case) + ([h] if s["r"] is not None else [])
    if op == "silu":
        both = host(s["gate_up"])
        g, u = both[:, :case["width"]], both[:, case["width"]:]
        t = np.exp(-np.abs(g))
        return exact_codes(np.where(g >= 0, g, g * t) / (1.0 + t) * u, case)
    if op == "route":
        x = host(s["logits"])
        if case["scoring"] == "sigmoid":
            score = 0.5 * (1.0 + np.tanh(0.5 * x))
        else:
            score = np.exp(x - np.logaddexp.reduce(x, axis=1, keepdims=True))
        # ranking by logits where there is no bias: the scores grow with them
        rank = x.copy() if s["bias"] is None else score + host(s["bias"])
        t, e, g = case["tokens"], case["experts"], case["groups"]
        rows = np.arange(t)
        if g > 1:
            value = (score if s["bias"] is None else rank).reshape(t, g, e // g)
            value = -np.partition(-value, case["group_best"] - 1, axis=2)[:, :, :case["group_best"]].sum(2)
            out_of = np.argsort(-value, axis=1, kind="stable")[:, case["top_groups"]:]
            parts = rank.reshape(t, g, e // g)
            parts[rows[:, None], out_of] = -np.inf
        ids = np.argsort(-rank, axis=1, kind="stable")[:, :case["top_k"]]
        w = score[rows[:, None], ids]
        if case["renorm"]:
            w = w / w.sum(1, keepdims=True)
        return [ids.astype(np.int32), w * s["scale"]]
    if op == "combine":
        t, k = case["tokens"], case["top_k"]
        y = s["y"].double()
        out = torch.zeros(t, case["width"], dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
        pair = torch.arange(t * k, device="cuda") if s["order"] is None else s["order"].long()
        return [out.index_add_(0, pair // k, y * s["w"].double().reshape(-1)[pair][:, None])]
    ids = s["ids"].long().reshape(-1)
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():
        pairs = torch.nonzero(ids == e)[:, 0]
        at = pairs if case["mode"] == "indexed" else torch.arange(int(s["start"][e]), int(s["start"][e + 1]), device="cuda")
        rows = at // case["top_k"] if case["mode"] == "indexed" else at
        a = s["a"][rows].double() * s["sa"][rows].double().repeat_interleave(128, 1)
        scale = s["sw"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:, :case["N"]]
        out[at] = a @ (s["w"][e].double() * scale)
    return [out]
