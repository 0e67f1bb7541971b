"""The FP8 layer operators on their own: the norm that feeds the FP8 products,
grouped expert routing, the block-scaled FP8 product and the routed experts.

Each operator has a plain form (elementary torch operations in 32 or 64 bits)
and, where `own` is true, the call that a user makes of the package.  Sizes
are those of the package's workloads (hidden 2048 / 4096, 128 to 512 experts,
8 per row, intermediates 512 to 1536) over the row counts of serving: one
token, a few drafted or batched ones, a prompt of thousands.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128           # inputs (and outputs) that share a scale
E4M3_MAX = 448.0      # largest finite e4m3 value
TINY = 1e-30          # least magnitude a scale is made of
F8 = torch.float8_e4m3fn
WIDTHS = [256, 384, 512, 640, 896, 1024, 1152, 1280, 1536, 1664, 1792, 2048, 2176, 2432, 2560, 2816, 3200, 3456, 3584, 3840, 4096]
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded token between two layers: latency only
        dict(name="norm_1", op="norm", rows=1, hidden=4096, dtype="bf16", residual=True, quantize=True),
        # a ragged prompt
        dict(name="norm_1021", op="norm", rows=1021, hidden=2048, dtype="fp16", residual=True, quantize=True),
        # the final norm of a batch of long prompts
        dict(name="norm_8192", op="norm", rows=8192, hidden=4096, dtype="bf16", residual=True, quantize=True),
        # one decoded token, grouped sigmoid routing with a balance bias
        dict(name="route_1", op="route", rows=1, experts=256, top_k=8, scoring="sigmoid", bias=True, groups=8,
             group_limit=4, group_score="top2", renorm=True, scale=2.5, dtype="fp32", masked=False),
        # a ragged prompt, plain softmax over a width that is no power of two, some experts taken out
        dict(name="route_777", op="route", rows=777, experts=160, top_k=8, scoring="softmax", bias=False, groups=1,
             group_limit=1, group_score="max", renorm=True, scale=1.0, dtype="bf16", masked=True),
        # a batch of long prompts
        dict(name="route_16384", op="route", rows=16384, experts=256, top_k=8, scoring="sigmoid", bias=True, groups=8,
             group_limit=4, group_score="top2", renorm=True, scale=2.5, dtype="fp32", masked=False),
        # a dense projection for one token: the weights' bytes
        dict(name="matmul_1", op="matmul", rows=1, n=4096, k=4096, out="bf16"),
        # a ragged prompt, an output width that ends inside a block
        dict(name="matmul_333", op="matmul", rows=333, n=1000, k=2048, out="fp32"),
        # a batch of long prompts: the tensor cores' rate
        dict(name="matmul_8192", op="matmul", rows=8192, n=4096, k=4096, out="bf16"),
        # one decoded token through its 8 experts
        dict(name="experts_1", op="experts", rows=1, hidden=2048, experts=128, top_k=8, inter=768, dropped=False),
        # a batch of decoded tokens that touches nearly every expert of a wide layer: the weights' bytes
        dict(name="experts_61", op="experts", rows=61, hidden=4096, experts=160, top_k=8, inter=1536, dropped=True),
        # a batch of prompts
        dict(name="experts_4096", op="experts", rows=4096, hidden=2048, experts=128, top_k=8, inter=768, dropped=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng, op):
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 8192), hidden=rng.choice([rng.choice(WIDTHS), 2 * rng.randint(100, 2047) + 1]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), residual=rng.random() < 0.7, quantize=rng.random() < 0.7)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.randint(max(1, 16 // groups), 512 // groups)
        limit = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, limit * (experts // groups)))
        return dict(op=op, rows=_log(rng, 1, 16384), experts=experts, top_k=top_k, scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, group_limit=limit,
                    group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "bf16", "fp16"]), masked=rng.random() < 0.3)
    if op == "matmul":
        return dict(op=op, rows=_log(rng, 1, 8192), n=rng.choice([rng.choice(WIDTHS), 2 * rng.randint(50, 3000) + 1]),
                    k=rng.choice([rng.choice(WIDTHS), 16 * (2 * rng.randint(8, 190) + 1)]), out=rng.choice(["bf16", "fp16", "fp32"]))
    return dict(op=op, rows=_log(rng, 1, 4096), hidden=rng.choice(WIDTHS), experts=rng.choice([8, 37, 128, 160, 256]),
                top_k=rng.randint(1, 8), inter=BLOCK * rng.randint(1, 12), dropped=rng.random() < 0.3)


def draw(rng):
    op = rng.choice(["norm", "route", "matmul", "matmul", "experts", "experts"])
    largest = [work(c) for c in listed() if c["op"] == op]
    while True:
        case = _draw(rng, op)
        w = work(case)
        if all(w[m] <= max(x[m] for x in largest) for m in w):
            return case


def work(case):
    c = case
    if c["op"] == "norm":
        e = TYPES[c["dtype"]].itemsize
        n = c["rows"] * c["hidden"]
        out = n * e + (n * e if c["residual"] else 0)
        if c["quantize"]:
            out += n + 4 * c["rows"] * -(-c["hidden"] // BLOCK)
        return {"bytes": n * e * (2 if c["residual"] else 1) + c["hidden"] * e + out, "flops": 6 * n}
    if c["op"] == "route":
        n = c["rows"] * c["experts"]
        return {"bytes": n * TYPES[c["dtype"]].itemsize + (4 * c["experts"] if c["bias"] else 0) + 8 * c["rows"] * c["top_k"],
                "flops": 8 * n}
    if c["op"] == "matmul":
        m, n, k = c["rows"], c["n"], c["k"]
        kb = -(-k // BLOCK)
        return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // BLOCK)) + m * n * TYPES[c["out"]].itemsize, "flops": 2 * m * n * k}
    t, h, e, k, i = c["rows"], c["hidden"], c["experts"], c["top_k"], c["inter"]
    k = min(k, e)
    used = e * (1.0 - (1.0 - k / e) ** t)     # experts that some row chooses, rows being alike
    return {"bytes": int(used * 3 * h * i * (1 + 4 / BLOCK ** 2)) + t * h + 4 * t * h // BLOCK + 8 * t * k + 2 * t * h,
            "flops": 6 * t * k * h * i}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows_to_fp8(x):
    """x [.., K] in fp32 -> e4m3 codes and one scale per row and 128 inputs."""
    k = x.shape[-1]
    kb = -(-k // BLOCK)
    pad = torch.nn.functional.pad(x, (0, kb * BLOCK - k)).unflatten(-1, (kb, BLOCK))
    scale = pad.abs().amax(-1).clamp(min=TINY) / E4M3_MAX
    q = (pad / scale.unsqueeze(-1)).flatten(-2)[..., :k].to(F8).contiguous()
    return q, scale


def _weights_to_fp8(w):
    """w [.., N, K] in fp32 -> e4m3 codes and one scale per 128 x 128 block."""
    n, k = w.shape[-2:]
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    pad = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n))
    pad = pad.unflatten(-1, (kb, BLOCK)).unflatten(-3, (nb, BLOCK))          # [.., nb, 128, kb, 128]
    scale = pad.abs().amax((-1, -3)).clamp(min=TINY) / E4M3_MAX             # [.., nb, kb]
    q = (pad / scale.unsqueeze(-2).unsqueeze(-1)).flatten(-2).flatten(-3, -2)[..., :n, :k].to(F8).contiguous()
    return q, scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    s = {"case": dict(c)}
    if c["op"] == "norm":
        t = TYPES[c["dtype"]]
        channel = torch.exp(normal(c["hidden"], std=0.5))       # some channels are larger, as in trained layers
        s["x"] = (normal(c["rows"], c["hidden"]) * channel).to(t)
        s["residual"] = (normal(c["rows"], c["hidden"], std=3.0) * channel).to(t) if c["residual"] else None
        s["weight"] = (1.0 + normal(c["hidden"], std=0.1)).to(t)
    elif c["op"] == "route":
        s["logits"] = normal(c["rows"], c["experts"], std=1.5)
        if c["masked"] and c["rows"] > 1:
            s["logits"][torch.rand(c["rows"], c["experts"], generator=g, device="cuda") < 0.2] = -math.inf
            s["logits"][c["rows"] // 2] = -math.inf            # a padding row: nothing is left
        s["logits"] = s["logits"].to(TYPES[c["dtype"]])
        s["bias"] = torch.rand(c["experts"], generator=g, device="cuda") * 0.2 - 0.1 if c["bias"] else None
    elif c["op"] == "matmul":
        s["a"], s["a_scales"] = _rows_to_fp8(normal(c["rows"], c["k"]))
        s["b"], s["b_scales"] = _weights_to_fp8(normal(c["n"], c["k"], std=0.02))
    else:
        t, h, e, i = c["rows"], c["hidden"], c["experts"], c["inter"]
        k = min(c["top_k"], e)
        s["q"], s["scales"] = _rows_to_fp8(normal(t, h))
        p = torch.sigmoid(normal(t, e, std=1.5) + normal(e, std=0.3))       # some experts are asked more often
        w, ids = p.topk(k, dim=1)
        s["wts"] = (2.5 * w / w.sum(1, keepdim=True)).contiguous()
        s["ids"] = ids.to(torch.int32)
        if c["dropped"] and t > 1:                                         # slots without an expert, one row with none
            s["ids"][torch.rand(t, k, generator=g, device="cuda") < 0.1] = -1
            s["ids"][t // 2] = -1
        for name, (n, m) in (("gate", (i, h)), ("up", (i, h)), ("down", (h, i))):
            q = torch.empty(e, n, m, dtype=F8, device="cuda")
            sc = torch.empty(e, -(-n // BLOCK), -(-m // BLOCK), device="cuda")
            for lo in range(0, e, 32):
                hi = min(e, lo + 32)
                q[lo:hi], sc[lo:hi] = _weights_to_fp8(normal(hi - lo, n, m, std=0.02))
            s[name], s[name + "_scales"] = q, sc
        if own:
            from routed_moe_decode_router_gb300 import ops
            s["ws"] = ops.ExpertsWorkspace(t, k, h, i, e)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        from routed_moe_decode_router_gb300 import ops
        if c["op"] == "norm":
            r = ops.rms_norm(s["x"], s["weight"], eps=1e-6, residual=s["residual"], quantize=c["quantize"])
            return {"y": r.y, "residual": r.residual, "q": r.q, "scales": r.scales}
        if c["op"] == "route":
            ids, wts = ops.route_topk(s["logits"], c["top_k"], scoring=c["scoring"], bias=s["bias"], groups=c["groups"],
                                      group_limit=c["group_limit"], group_score=c["group_score"],
                                      norm_topk_prob=c["renorm"], routed_scaling_factor=c["scale"])
            return {"ids": ids, "wts": wts}
        if c["op"] == "matmul":
            return {"out": ops.matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], out_dtype=TYPES[c["out"]])}
        return {"out": ops.experts_fp8(s["q"], s["scales"], s["ids"], s["wts"], s["gate"], s["gate_scales"], s["up"],
                                       s["up_scales"], s["down"], s["down_scales"], ws=s["ws"])}
    return {"norm": _plain_norm, "route": _plain_route, "matmul": _plain_matmul, "experts": _plain_experts}[c["op"]](s, c)


def _plain_norm(s, c):
    x = s["x"].float()
    total = x + s["residual"].float() if c["residual"] else x
    y = total * torch.rsqrt(total.square().mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    q, scales = _rows_to_fp8(y) if c["quantize"] else (None, None)
    return {"y": y.to(s["x"].dtype), "residual": total.to(s["x"].dtype) if c["residual"] else None, "q": q, "scales": scales}


def _plain_route(s, c):
    # 64 bits: which of two experts comes first is decided by values next to each other
    x = s["logits"].double()
    dead = x.isnan() | (x == -math.inf)
    x = x.masked_fill(dead, -math.inf)
    if c["scoring"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = (p / p.sum(1, keepdim=True)).masked_fill(dead, 0.0)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    biased = p + s["bias"].double() if c["bias"] else p
    key = (biased if c["bias"] else x).masked_fill(dead, -math.inf)
    if c["groups"] > 1:
        member = biased.masked_fill(dead, -math.inf).unflatten(1, (c["groups"], -1)).sort(dim=2, descending=True).values
        score = member[..., 0]
        if c["group_score"] == "top2" and member.shape[2] > 1:
            score = score + torch.where(member[..., 1] == -math.inf, 0.0, member[..., 1])
        order = score.sort(dim=1, descending=True, stable=True).indices
        chosen = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order[:, :c["group_limit"]], True)
        key = key.masked_fill(~chosen.repeat_interleave(c["experts"] // c["groups"], 1), -math.inf)
    value, ids = key.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :c["top_k"]], ids[:, :c["top_k"]]
    none = value == -math.inf
    w = p.gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": ids.masked_fill(none, -1).to(torch.int32), "wts": (w * c["scale"]).float()}


def _rows_from_fp8(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _weights_from_fp8(q, scale):
    n, k = q.shape[-2:]
    return q.float() * scale.repeat_interleave(BLOCK, -1)[..., :k].repeat_interleave(BLOCK, -2)[..., :n, :]


def _plain_matmul(s, c):
    return {"out": (_rows_from_fp8(s["a"], s["a_scales"]) @ _weights_from_fp8(s["b"], s["b_scales"]).t()).to(TYPES[c["out"]])}


def _plain_experts(s, c):
    # the pairs (row, slot) of each chosen expert, padded to the longest list
    t, k = s["ids"].shape
    flat = s["ids"].flatten().long()
    pairs = (flat >= 0).nonzero().flatten()
    if not len(pairs):
        return {"out": torch.zeros(t, c["hidden"], dtype=torch.bfloat16, device=flat.device)}
    used, which, count = torch.unique(flat[pairs], return_inverse=True, return_counts=True)
    order = which.argsort(stable=True)
    place = torch.arange(len(pairs), device=flat.device) - (count.cumsum(0) - count)[which[order]]
    table = torch.full((len(used), int(count.max())), t * k, device=flat.device)
    table[which[order], place] = pairs[order]
    x = _rows_from_fp8(s["q"], s["scales"])
    x = torch.cat([x, x.new_zeros(1, c["hidden"])])[table // k]             # [experts, pairs, hidden]
    g = x @ _weights_from_fp8(s["gate"][used], s["gate_scales"][used]).mT
    u = x @ _weights_from_fp8(s["up"][used], s["up_scales"][used]).mT
    h = _rows_from_fp8(*_rows_to_fp8(g * torch.sigmoid(g) * u))
    y = h @ _weights_from_fp8(s["down"][used], s["down_scales"][used]).mT
    each = x.new_zeros(t * k + 1, c["hidden"]).index_copy(0, table.flatten(), y.flatten(0, 1))[:t * k]
    each = each * (s["ids"] >= 0).flatten().unsqueeze(1)
    return {"out": (each.unflatten(0, (t, k)) * s["wts"].unsqueeze(2)).sum(1).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _wide(q, scale, rows_too):
    """Codes times their scales, in 64 bits, by the index of each one's block."""
    dev = q.device
    col = torch.arange(q.shape[-1], device=dev) // BLOCK
    if not rows_too:
        return q.double() * scale.double()[..., col]
    row = torch.arange(q.shape[-2], device=dev) // BLOCK
    return q.double() * scale.double()[..., row[:, None], col[None, :]]


def _exact_scales(y):
    """One scale per row and 128 inputs of y (64 bits)."""
    k = y.shape[-1]
    return torch.stack([y[..., b:min(b + BLOCK, k)].abs().amax(-1).clamp(min=TINY) for b in range(0, k, BLOCK)], -1) / E4M3_MAX


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        total = s["x"].double() + (s["residual"].double() if c["residual"] else 0.0)
        y = total / (total.pow(2).sum(1) / c["hidden"] + 1e-6).sqrt()[:, None] * s["weight"].double()
        out = {"y": y, "residual": total if c["residual"] else None, "q": None, "scales": None}
        if c["quantize"]:                # the codes: what is rounded to them
            out["scales"] = _exact_scales(y)
            out["q"] = y / out["scales"][:, torch.arange(c["hidden"], device=y.device) // BLOCK]
        return out
    if c["op"] == "route":
        return _exact_route(s, c)
    if c["op"] == "matmul":
        return {"out": _wide(s["a"], s["a_scales"], False) @ _wide(s["b"], s["b_scales"], True).T}
    t, k = s["ids"].shape
    x = _wide(s["q"], s["scales"], False)
    out = torch.zeros(t, c["hidden"], dtype=torch.float64, device=x.device)
    for e in range(c["experts"]):
        row, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if len(row):
            g, u = (x[row] @ _wide(s[n][e], s[n + "_scales"][e], True).T for n in ("gate", "up"))
            h = g / (1.0 + torch.exp(-g)) * u
            sc = _exact_scales(h)[:, torch.arange(c["inter"], device=x.device) // BLOCK]
            h = (h / sc).to(F8).double() * sc                    # held in 8 bits by definition
            y = h @ _wide(s["down"][e], s["down_scales"][e], True).T
            out.index_add_(0, row, y * s["wts"][row, slot].double()[:, None])
    return {"out": out}


def _exact_route(s, c):
    x = s["logits"].double().cpu().numpy()
    t, e, k = c["rows"], c["experts"], c["top_k"]
    live = np.isfinite(x)
    x = np.where(live, x, -np.inf)
    with np.errstate(all="ignore"):
        if c["scoring"] == "softmax":
            p = np.exp(x - x.max(1, keepdims=True))
            p = p / p.sum(1, keepdims=True)
        else:
            p = np.exp(-np.logaddexp(0.0, -x))
    p = np.where(live, p, 0.0)
    score = p + (s["bias"].double().cpu().numpy() if c["bias"] else 0.0)
    key = np.where(live, score if c["bias"] else x, -np.inf)
    if c["groups"] > 1:
        m = np.where(live, score, -np.inf).reshape(t, c["groups"], -1)
        best = m.max(2)
        if c["group_score"] == "top2" and m.shape[2] > 1:
            second = np.partition(m, -2, axis=2)[:, :, -2]
            best = best + np.where(np.isinf(second), 0.0, second)
        rank = np.argsort(-best, axis=1, kind="stable").argsort(1, kind="stable")
        key = np.where(np.repeat(rank < c["group_limit"], e // c["groups"], axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    got = np.isfinite(np.take_along_axis(key, ids, 1))
    w = np.where(got, np.take_along_axis(p, ids, 1), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"ids": np.where(got, ids, -1).astype(np.int32), "wts": w * c["scale"]}
