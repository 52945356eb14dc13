"""Cases of the operators around the experts' products: inputs, plain forms,
exact values and the work that each cannot do without.

Four operators (`op` of a case):

  router   scores of T tokens for E experts to the k experts of each token and
           their combine weights: softmax or sigmoid scores, a bias that takes
           part in the choice alone, groups of experts, renormalised weights;
           with `train` the gradient of the logits as well;
  swiglu   h = silu(g) * u of the gate and up halves of one matrix; with
           `train` the gradient as well, taken from an MXFP8 copy of the input
           that the forward pass keeps;
  combine  the weighted sum over a token's experts; with `train` the gradients
           of the experts' rows and of the weights as well;
  experts  the same activation between the two MXFP8 products of routed
           experts, whose rows are grouped by expert and padded: h in 32-blocks
           along its columns, as the down product reads it; with `train` h times
           its row's combine weight in 32-blocks along the rows as well (the
           down weights' gradient reads it), and of the gradient of h the
           gradient of the gate and up values in both block directions and that
           of the combine weights, from an MXFP8 copy of the input.

MX encoding: 32 values along the contraction share one power-of-two scale
2^(byte - 127), byte = clamp(floor(log2 amax) - 8, -127, 127) + 127 (0 for a
block of zeros); elements are the scaled values rounded to nearest even as
E4M3 and saturated (448).
"""

import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _router(T, E, k, score="softmax", bias=False, groups=1, topk_groups=1, group_score="max", renormalize=True,
            scale=1.0, dtype="fp32", masked=False, train=False):
    return {"op": "router", "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "topk_groups": topk_groups, "group_score": group_score, "renormalize": renormalize, "scale": scale,
            "dtype": dtype, "masked": masked, "train": train}


def listed():
    return [
        # decoding one sequence: latency
        {"name": "router-1-token", **_router(1, 16, 1, "sigmoid", renormalize=False, dtype="bf16")},
        # a micro-batch over fine-grained experts in groups, balanced by a bias; some experts and tokens masked
        {"name": "router-4096x256-groups", **_router(4096, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5, "fp32", True, True)},
        # a large micro-batch, softmax over all experts, weights as they are
        {"name": "router-65600x32", **_router(65600, 32, 8, renormalize=False, dtype="bf16", train=True)},
        # decoding 7 sequences through a dense layer's activation: latency
        {"name": "swiglu-7x8192", "op": "swiglu", "M": 7, "N": 8192, "train": False},
        # a shared expert's micro-batch, an odd number of tokens
        {"name": "swiglu-4099x2048", "op": "swiglu", "M": 4099, "N": 2048, "train": True},
        # the dense activation of a whole sequence batch: bandwidth
        {"name": "swiglu-16384x8192", "op": "swiglu", "M": 16384, "N": 8192, "train": True},
        # one token's eight experts: latency
        {"name": "combine-1x8x7168", "op": "combine", "T": 1, "k": 8, "N": 7168, "dtype": "bf16", "masked": False, "train": False},
        # a micro-batch whose padding tokens were not routed, fp32 rows
        {"name": "combine-2047x4x5120", "op": "combine", "T": 2047, "k": 4, "N": 5120, "dtype": "fp32", "masked": True, "train": True},
        # a large micro-batch: bandwidth
        {"name": "combine-8192x8x7168", "op": "combine", "T": 8192, "k": 8, "N": 7168, "dtype": "bf16", "masked": False, "train": True},
        # the tiny workload's sizes: launches
        {"name": "experts-tiny", "op": "experts", "T": 128, "k": 2, "E": 2, "N": 512, "train": True},
        # fine-grained experts
        {"name": "experts-deepseek", "op": "experts", "T": 4096, "k": 8, "E": 32, "N": 2048, "train": True},
        # a few wide experts, one for each token
        {"name": "experts-llama4", "op": "experts", "T": 16384, "k": 1, "E": 16, "N": 8192, "train": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(max(round(v / step), -(-lo // step)), hi // step) * step)


def draw(rng):
    op = rng.choice(["router", "router", "swiglu", "combine", "experts"])
    if op == "router":
        groups = rng.choice([1, 1, 2, 4, 8])
        each = _log(rng, 2, 1024 // groups if groups > 1 else 640)
        kept = rng.randint(1, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return _router(_log(rng, 1, 16384), groups * each, rng.randint(1, min(16, kept * each)), score,
                       rng.random() < 0.5, groups, kept, rng.choice(["max", "top2"]), rng.random() < 0.6,
                       rng.choice([1.0, 2.5]), rng.choice(["fp32", "bf16"]), rng.random() < 0.4, rng.random() < 0.7)
    if op == "swiglu":
        return {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 32, 8192, 32), "train": rng.random() < 0.7}
    if op == "combine":
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "N": _log(rng, 8, 7168, 8),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "masked": rng.random() < 0.4, "train": rng.random() < 0.7}
    E, k, N = rng.randint(1, 64), rng.randint(1, 8), _log(rng, 128, 8192, 128)
    k = min(k, E)
    return {"op": op, "T": _log(rng, 1, min(16384, (1 << 27) // (k * N) - 31 * E // k)), "k": k, "E": E, "N": N,
            "train": rng.random() < 0.7}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _randn(gen, shape, std=1.0, outliers=False, dtype="bf16"):
    """N(0, std); with outliers one value in a thousand is 50 times as large."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std)
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device=DEV) < 1e-3, x * 50.0, x)
    return x.to(_TYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        logits = _randn(gen, (T, E), 1.5, dtype=case["dtype"])
        if case["masked"]:
            # one expert in twenty out of use, three tokens in a hundred padding
            off = (torch.rand(E, generator=gen, device=DEV) < 0.05) | (torch.rand((T, 1), generator=gen, device=DEV) < 0.03)
            logits = logits.masked_fill(off, -math.inf)
        bias = _randn(gen, (E,), 0.05, dtype="fp32") if case["bias"] else None
        dw = _randn(gen, (T, k), 1e-3, dtype="fp32") if case["train"] else None
        return {"case": dict(case), "logits": logits.requires_grad_(case["train"]), "bias": bias, "dw": dw}
    if op == "swiglu":
        M, N = case["M"], case["N"]
        return {"case": dict(case), "gu": _randn(gen, (M, 2 * N), 1.0, True).requires_grad_(case["train"]),
                "dh": _randn(gen, (M, N), 1e-3) if case["train"] else None}
    if op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        y = _randn(gen, (T, k, N), 1.0, False, case["dtype"])
        combine = torch.softmax(_randn(gen, (T, k), dtype="fp32"), -1)
        pos = None
        if case["masked"]:
            # rows of items that were not routed hold anything
            off = torch.rand((T, 1), generator=gen, device=DEV).expand(T, k) < 0.1
            y = y.masked_fill(off.unsqueeze(2), math.nan)
            pos = torch.where(off.reshape(-1), -1, torch.arange(T * k, device=DEV)).int()
        return {"case": dict(case), "y": y.requires_grad_(case["train"]), "combine": combine.requires_grad_(case["train"]),
                "pos": pos, "dout": _randn(gen, (T, N), 1e-3) if case["train"] else None}
    T, k, E, N = (case[v] for v in ("T", "k", "E", "N"))
    # the grouping that the layer's first product leaves: each expert's items in their order, then
    # rows of zeros up to a multiple of 32; the rows behind the last group hold anything
    ids = torch.sort(torch.randn((T, E), generator=gen, device=DEV), dim=1, descending=True).indices[:, :k].reshape(-1)
    order = torch.argsort(ids, stable=True)
    counts = (ids.unsqueeze(1) == torch.arange(E, device=DEV)).sum(0)
    padded = (counts + 31) // 32 * 32
    pos = torch.empty(T * k, dtype=torch.int64, device=DEV)
    pos[order] = torch.arange(T * k, device=DEV) + (padded.cumsum(0) - padded - counts.cumsum(0) + counts)[ids[order]]
    M = (T * k + 31 * E + 127) // 128 * 128
    rows = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    rows[pos] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    r = torch.arange(M, device=DEV).unsqueeze(1)
    behind, real = r >= padded.sum(), (rows >= 0).unsqueeze(1)

    def grouped(cols, std, outliers):
        return (_randn(gen, (M, cols), std, outliers) * real).masked_fill(behind, math.nan)

    return {"case": dict(case), "gu": grouped(2 * N, 1.0, True), "dh": grouped(N, 1e-3, False) if case["train"] else None,
            "combine": torch.softmax(_randn(gen, (T, k), dtype="fp32"), -1), "rows": rows, "pos": pos.int()}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _scores(l, masked, score):
    """Scores of logits l (the masked ones 0; all 0 where a row has no other)."""
    if score == "sigmoid":
        return torch.where(masked, 0.0, 1 / (1 + torch.exp(-l)))
    top = torch.where(masked, -math.inf, l).amax(-1, keepdim=True)
    e = torch.where(masked, 0.0, torch.exp(l - torch.where(top > -math.inf, top, 0.0)))
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def _choose(logits, bias, r):
    """The experts of each token, int64 [T, k]: by the scores in 64 bits where
    they are added to something, else by the logits, which order them alike."""
    E, G = r["E"], r["groups"]
    masked = logits <= torch.finfo(logits.dtype).min
    if bias is None and (G == 1 or r["group_score"] == "max"):
        c = logits.double()
    else:
        c = _scores(logits.double(), masked, r["score"])
        if bias is not None:
            c = c + bias.double()
    lowest = torch.finfo(torch.float64).min
    if G > 1:
        cg = torch.where(masked, -math.inf, c).unflatten(1, (G, E // G))
        if r["group_score"] == "max":
            value = cg.amax(2)
        else:
            two = torch.sort(cg, dim=2, descending=True).values[..., :2]
            value = torch.where(two[..., 0] == -math.inf, -math.inf, torch.where(two == -math.inf, 0.0, two).sum(2))
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, : r["topk_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True).repeat_interleave(E // G, 1)
    else:
        kept = torch.ones_like(masked)
    c = torch.where(kept, torch.where(masked, lowest, c), -math.inf)
    return torch.sort(c, dim=1, descending=True, stable=True).indices[:, : r["k"]]


def _weights(logits, ids, r):
    """Combine weights fp32 [T, k], with what their gradient needs."""
    masked = logits <= torch.finfo(logits.dtype).min
    s = _scores(logits.float(), masked, r["score"])
    sel = s.gather(1, ids)
    if r["renormalize"]:
        total = sel.sum(1, keepdim=True)
        sel = torch.where(total > 0, sel / total, 0.0)
    return sel * r["scale"], s, sel


def _router_grad(s, sel, ids, dw, r):
    """dlogits fp32 [T, E] of the weights' gradient dw [T, k]; sel: the weights over the scale."""
    g = dw * r["scale"]
    out = torch.zeros_like(s)
    if r["score"] == "softmax" and not r["renormalize"]:
        full = out.scatter(1, ids, g)
        return s * (full - (g * sel).sum(1, keepdim=True))
    if r["renormalize"]:
        d = sel * (g - (g * sel).sum(1, keepdim=True))
        if r["score"] == "sigmoid":
            d = d * (1 - s.gather(1, ids))
    else:
        d = g * sel * (1 - sel)
    return out.scatter(1, ids, d)


def _pow2(e):
    """2^e as fp32 for int32 e in [-127, 127], from its bits: exact, so that values halfway between two codes stay there."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).view(torch.float32)


def _mx(x):
    """fp32 [..., C] after its MXFP8 quantization along the last axis, as fp32."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    byte = torch.where(amax > 0, (torch.frexp(amax).exponent - 1 - 8).clamp(-127, 127) + 127, 0).int()
    v = (b * _pow2(127 - byte).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (v * _pow2(byte - 127).unsqueeze(-1)).flatten(-2)


def _mx_t(x):
    """[..., R, C] after its MXFP8 quantization along R, transposed: [..., C, R]."""
    return _mx(x.transpose(-2, -1).contiguous())


def _swiglu(gu):
    g, u = gu.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _swiglu_grad(dh, gu):
    """Gradient of gu [..., 2N] at the values gu."""
    g, u = gu.chunk(2, -1)
    s = 1 / (1 + torch.exp(-g))
    return torch.cat((dh * u * s * (1 + g * (1 - s)), dh * g * s), -1)


def _plain_experts(st):
    case = st["case"]
    rows = st["rows"].long()
    real = (rows >= 0).unsqueeze(1)
    w = st["combine"].reshape(-1)[rows.clamp(min=0)].unsqueeze(1)
    gu = torch.where(real, st["gu"].float(), 0.0)
    h = _swiglu(gu)
    got = {"h": _mx(h).bfloat16()}
    if case["train"]:
        dh, kept = torch.where(real, st["dh"].float(), 0.0), _mx(gu)
        dgu = _swiglu_grad(w * dh, kept)
        got.update(wh_t=_mx_t(w * h).bfloat16(), dgu=_mx(dgu).bfloat16(), dgu_t=_mx_t(dgu).bfloat16(),
                   dcombine=(dh * _swiglu(kept)).sum(1)[st["pos"].long()].view(case["T"], case["k"]))
    return got


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "router":
        logits = st["logits"].detach()
        ids = _choose(logits, st["bias"], case)
        w, s, sel = _weights(logits, ids, case)
        got = {"ids": ids.int(), "combine": w}
        if case["train"]:
            got["dlogits"] = _router_grad(s, sel, ids, st["dw"], case).to(logits.dtype)
        return got
    if op == "swiglu":
        gu = st["gu"].detach().float()
        got = {"h": _swiglu(gu).bfloat16()}
        if case["train"]:
            got["dgu"] = _swiglu_grad(st["dh"].float(), _mx(gu)).bfloat16()
        return got
    if op == "combine":
        y, w, pos = st["y"].detach(), st["combine"].detach(), st["pos"]
        yf = y.float()
        if pos is not None:
            off = (pos < 0).view(w.shape)
            yf, w = yf.masked_fill(off.unsqueeze(2), 0.0), w.masked_fill(off, 0.0)
        got = {"out": (w.unsqueeze(2) * yf).sum(1).bfloat16()}
        if case["train"]:
            d = st["dout"].float().unsqueeze(1)
            got.update(dy=(w.unsqueeze(2) * d).to(y.dtype), dcombine=(yf * d).sum(2))
        return got
    return _plain_experts(st)


def run(st):
    if not own:
        with torch.no_grad():
            return _plain(st)
    import mxfp8_block_scaled_06_amd as mx
    case = st["case"]
    op = case["op"]
    if op == "router":
        ids, w = mx.mx_topk_router(st["logits"], case["k"], score=case["score"], bias=st["bias"], groups=case["groups"],
                                   topk_groups=case["topk_groups"], group_score=case["group_score"],
                                   renormalize=case["renormalize"], scale=case["scale"])
        got = {"ids": ids, "combine": w.detach()}
        if case["train"]:
            got["dlogits"], = torch.autograd.grad(w, st["logits"], st["dw"])
        return got
    if op == "experts":
        if not case["train"]:
            return {"h": mx.mx_dequantize(*mx.mx_swiglu_quantize(st["gu"], st["rows"]), scale_layout="gemm")}
        q, s, q_t, s_t, kept, kept_s = mx.mx_swiglu_quantize_fwd(st["gu"], st["rows"], st["combine"])
        dq, ds, dq_t, ds_t, dcombine = mx.mx_swiglu_quantize_bwd(st["dh"], kept, kept_s, st["rows"], st["pos"], st["combine"])
        return {"h": mx.mx_dequantize(q, s, scale_layout="gemm"), "wh_t": mx.mx_dequantize(q_t, s_t, scale_layout="gemm"),
                "dgu": mx.mx_dequantize(dq, ds, scale_layout="gemm"), "dgu_t": mx.mx_dequantize(dq_t, ds_t, scale_layout="gemm"),
                "dcombine": dcombine}
    if op == "swiglu":
        h = mx.mx_swiglu(st["gu"])
        got = {"h": h.detach()}
        if case["train"]:
            got["dgu"], = torch.autograd.grad(h, st["gu"], st["dh"])
        return got
    out = mx.mx_topk_combine(st["y"], st["combine"], pos=st["pos"])
    got = {"out": out.detach()}
    if case["train"]:
        got["dy"], got["dcombine"] = torch.autograd.grad(out, (st["y"], st["combine"]), st["dout"])
    return got


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, train = case["op"], case.get("train")
    if op == "router":
        T, E, k, size = case["T"], case["E"], case["k"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * E * size * (2 if train else 1) + T * k * (12 if train else 8) + (4 * E if case["bias"] else 0),
                "flops": T * E * (16 if train else 8)}
    if op == "swiglu":
        n = case["M"] * case["N"]
        return {"bytes": n * (12 if train else 6), "flops": n * (20 if train else 6)}
    if op == "combine":
        T, k, N, size = case["T"], case["k"], case["N"], 2 if case["dtype"] == "bf16" else 4
        n = T * k * N
        return {"bytes": n * size * (2 if train else 1) + T * N * (4 if train else 2) + T * k * (8 if train else 4),
                "flops": n * (5 if train else 2)}
    T, k, N = case["T"], case["k"], case["N"]
    n = T * k * N                                   # padding rows are no work; what is held in 8 bits comes back as bf16
    return {"bytes": n * (18 if train else 6) + T * k * (16 if train else 4), "flops": n * (40 if train else 10)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


_GRID = [m * 2.0 ** -9 if not x else (1 + m / 8) * 2.0 ** (x - 7) for x, m in ((v >> 3, v & 7) for v in range(127))]


def _exact_mx(x):
    """float64 [..., C] -> the values that its MXFP8 codes along the last axis stand for."""
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    mids = (grid[1:] + grid[:-1]) / 2
    parts = []
    for p in x.reshape(-1, 32).split(1 << 22):       # blocks, in pieces that fit beside the rest
        top = p.abs().amax(1, keepdim=True)
        e = (torch.frexp(top).exponent - 9).clamp(-127, 127)
        e = torch.where(top > 0, e, -127)
        a = p.abs() * _exact_pow2(-e)
        at = torch.bucketize(a, mids)
        at = torch.where((at % 2 == 1) & (a == mids[at.clamp(max=125)]), at + 1, at)     # a value halfway goes to the even code
        parts.append(torch.copysign(grid[at], p) * _exact_pow2(e))
    return torch.cat(parts).view(x.shape) if parts else x.clone()


def _exact_router(logits, bias, r, dw=None):
    """ids, weights and, given dw, dlogits by the Jacobian of the weights, token by token in pieces."""
    l = logits.detach().double()
    on = logits.detach() > torch.finfo(logits.dtype).min
    some = on.any(1, keepdim=True)
    if r["score"] == "softmax":
        s = torch.softmax(torch.where(on, l, -math.inf), 1)
        s = torch.where(some, s, 0.0)
    else:
        s = torch.where(on, torch.sigmoid(l), 0.0)
    ids = _exact_ids(l, s, on, bias, r)
    w = s.gather(1, ids)
    total = w.sum(1, keepdim=True) if r["renormalize"] else torch.ones_like(w[:, :1])
    w = torch.where(total > 0, w / total, 0.0) * r["scale"]
    if dw is None:
        return ids, w, None
    # through the renormalisation to the chosen scores, then through the scores to the logits
    g = dw.double() * r["scale"]
    if r["renormalize"]:
        g = torch.where(total > 0, (g - (g * w).sum(1, keepdim=True) / r["scale"]) / total, 0.0)
    ds = torch.zeros_like(s).scatter(1, ids, g)
    if r["score"] == "softmax":
        return ids, w, s * ds - s * (s * ds).sum(1, keepdim=True)
    return ids, w, ds * s * (1 - s)


def _exact_ids(l, s, on, bias, r):
    """The choice by repeated arg-max: of groups, then of experts; ties to the lowest index."""
    T, E = l.shape
    G, n = r["groups"], E // r["groups"]
    by_logit = bias is None and (G == 1 or r["group_score"] == "max")
    c = torch.where(on, l if by_logit else s if bias is None else s + bias.double(), -math.inf)
    rows, index = torch.arange(T, device=l.device), torch.arange(E, device=l.device)

    def first_largest(v, free):
        """Index of the largest free value in each row, the lowest one among equals."""
        top = torch.where(free, v, -math.inf).amax(1, keepdim=True)
        return torch.where(free & (v == top), torch.arange(v.shape[1], device=v.device), v.shape[1]).amin(1)

    free = torch.ones_like(on)
    if G > 1:
        cg = c.view(T, G, n)
        value = cg.amax(2)
        if r["group_score"] == "top2":
            lead = first_largest(cg.reshape(T * G, n), torch.ones((T * G, n), dtype=torch.bool, device=l.device)).view(T, G, 1)
            second = cg.scatter(2, lead, -math.inf).amax(2)
            value = torch.where(second > -math.inf, value + second, value)
        open_, kept = torch.ones_like(value, dtype=torch.bool), torch.zeros_like(value, dtype=torch.bool)
        for _ in range(r["topk_groups"]):
            g = first_largest(value, open_)
            kept[rows, g], open_[rows, g] = True, False
        free = kept[:, index // n].clone()
    ids = []
    for _ in range(r["k"]):
        ids.append(first_largest(c, free))
        free[rows, ids[-1]] = False
    return torch.stack(ids, 1)


def _exact_swiglu(gu):
    n = gu.shape[-1] // 2
    g, u = gu[..., :n], gu[..., n:]
    return g * torch.sigmoid(g) * u


def _exact_swiglu_grad(dh, gu):
    n = gu.shape[-1] // 2
    g, u = gu[..., :n], gu[..., n:]
    s = torch.sigmoid(g)
    return torch.cat((dh * u * (s + g * s * (1 - s)), dh * g * s), -1)


def _exact_experts(case, st):
    k, N = case["k"], case["N"]
    pos = st["pos"].long()
    item = torch.arange(pos.numel(), device=DEV)
    gu = torch.zeros(st["gu"].shape, dtype=torch.float64, device=DEV)
    gu[pos] = st["gu"][pos].double()
    h = _exact_swiglu(gu)
    got = {"h": _exact_mx(h)}
    if not case["train"]:
        return got
    c = torch.zeros((gu.shape[0], 1), dtype=torch.float64, device=DEV)
    c[pos, 0] = st["combine"].double()[item // k, item % k]
    got["wh_t"] = _exact_mx((c * h).T.contiguous())
    del h
    dh, kept = torch.zeros((gu.shape[0], N), dtype=torch.float64, device=DEV), _exact_mx(gu)
    del gu
    dh[pos] = st["dh"][pos].double()
    got["dcombine"] = (dh * _exact_swiglu(kept)).sum(1)[pos].view(-1, k)
    dgu = _exact_swiglu_grad(c * dh, kept)
    return dict(got, dgu=_exact_mx(dgu), dgu_t=_exact_mx(dgu.T.contiguous()))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "router":
        _, w, dl = _exact_router(st["logits"], st["bias"], case, st["dw"])
        return {"ids": None, "combine": w, "dlogits": dl} if case["train"] else {"ids": None, "combine": w}
    if op == "swiglu":
        gu = st["gu"].detach().double()
        got = {"h": _exact_swiglu(gu)}
        if case["train"]:
            got["dgu"] = _exact_swiglu_grad(st["dh"].double(), _exact_mx(gu))
        return got
    if op == "combine":
        y, c = st["y"].detach().double(), st["combine"].detach().double()
        on = torch.ones_like(c, dtype=torch.bool) if st["pos"] is None else (st["pos"] >= 0).view(c.shape)
        y = torch.where(on.unsqueeze(2), y, 0.0)
        got = {"out": torch.zeros((case["T"], case["N"]), dtype=torch.float64, device=DEV)}
        for j in range(case["k"]):
            got["out"] += torch.where(on[:, j], c[:, j], 0.0).unsqueeze(1) * y[:, j]
        if case["train"]:
            d = st["dout"].double()
            got["dy"] = torch.where(on, c, 0.0).unsqueeze(2) * d.unsqueeze(1)
            got["dcombine"] = torch.stack([(y[:, j] * d).sum(1) for j in range(case["k"])], 1)
        return got
    return _exact_experts(case, st)
