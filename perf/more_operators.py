"""The operators of a decoding step beside the MoE layer's, on their own: the
paged cache of keys and values (written, in 8 bits or as it is, and read back),
attention of new tokens over it, and the verification of drafted tokens.

Each operator has a plain form (elementary torch operations in 32 or 64 bits)
and, where `own` is true, the call that a user makes of the package.  Sizes are
generic ones of decoding: one sequence to a batch of them, one new token or the
few of a verify step, caches of a few tokens to 131072.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0      # largest finite e4m3 value
TINY = 1e-30          # least magnitude a scale is made of
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": F8}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of one conversation: latency only
        dict(name="attend_1", op="attend", batch=1, rows=1, longest=901, heads=32, kv_heads=8, dim=128, page=64,
             cache="e4m3", dtype="bf16", window=0),
        # a verify step of a few conversations, the drafted tokens behind the last one's
        dict(name="attend_verify", op="attend", batch=9, rows=4, longest=6007, heads=64, kv_heads=8, dim=128, page=16,
             cache="bf16", dtype="bf16", window=0),
        # a layer with a sliding window, its cache kept whole; groups of five heads
        dict(name="attend_window", op="attend", batch=33, rows=3, longest=9001, heads=20, kv_heads=4, dim=64, page=48,
             cache="bf16", dtype="bf16", window=1024),
        # one very long document, few and wide heads
        dict(name="attend_long", op="attend", batch=1, rows=1, longest=131071, heads=16, kv_heads=2, dim=256, page=128,
             cache="fp16", dtype="fp16", window=0),
        # a full batch of long conversations
        dict(name="attend_96", op="attend", batch=96, rows=1, longest=16384, heads=64, kv_heads=8, dim=128, page=64,
             cache="e4m3", dtype="bf16", window=0),
        # the new tokens of a decoded batch
        dict(name="write_61", op="write", tokens=61, kv_heads=8, dim=128, page=64, cache="e4m3", dtype="bf16"),
        # a batch of prompts
        dict(name="write_16383", op="write", tokens=16383, kv_heads=8, dim=128, page=64, cache="e4m3", dtype="bf16"),
        # the start that a new prompt shares with an earlier one
        dict(name="read_777", op="read", tokens=777, kv_heads=4, dim=64, page=16, cache="e4m3", dtype="fp16"),
        # a long document's cache, for the next part of its prompt
        dict(name="read_65536", op="read", tokens=65536, kv_heads=8, dim=128, page=64, cache="e4m3", dtype="bf16"),
        # one conversation
        dict(name="verify_1", op="verify", batch=1, drafts=3, vocab=32768, probs=True, kept=0),
        # drafts looked up in the text (no probabilities of their own), a target cut to its best tokens, an odd vocabulary
        dict(name="verify_13", op="verify", batch=13, drafts=4, vocab=50001, probs=False, kept=50),
        # a full batch
        dict(name="verify_64", op="verify", batch=64, drafts=5, vocab=131072, probs=True, kept=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng, op):
    dim, page, kv = rng.choice([64, 128, 256]), rng.choice([16, 32, 48, 64, 128]), rng.choice([1, 2, 4, 8])
    if op == "attend":
        cache = rng.choice(["e4m3", "e4m3", "bf16", "fp16"])
        longest = _log(rng, 1, 131072)
        return dict(op=op, batch=_log(rng, 1, 256), rows=rng.choice([1, 1, 1, 2, 3, 4, 5, 8]), longest=longest,
                    heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), kv_heads=kv, dim=dim, page=page, cache=cache,
                    dtype=rng.choice(["bf16", "fp16"]) if cache == "e4m3" else cache,
                    window=rng.choice([0, 0, 0, rng.randint(1, 4096)]))
    if op in ("write", "read"):
        cache = rng.choice(["e4m3", "e4m3", "bf16", "fp16"])
        types = ["bf16", "fp16", "fp32"] if cache == "e4m3" else [cache]
        return dict(op=op, tokens=_log(rng, 1, 65536), kv_heads=kv, dim=dim, page=page, cache=cache, dtype=rng.choice(types))
    return dict(op=op, batch=_log(rng, 1, 64), drafts=rng.randint(1, 8), vocab=rng.choice([_log(rng, 16, 200000),
                2 * rng.randint(5000, 70000) + 1]), probs=rng.random() < 0.6, kept=rng.choice([0, 0, 20, 200]))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "read", "verify"])
    largest = [work(c) for c in listed() if c["op"] == op]
    while True:
        case = _draw(rng, op)
        w = work(case)
        if all(w[m] <= max(x[m] for x in largest) for m in w):
            return case


def _lengths(c):
    """The batch's lengths (their order is the inputs'): spread from the longest
    down; from four sequences on, one place of the batch is free."""
    n = [max(1, math.ceil(c["longest"] * (1.0 - i * 0.6180339887498949 % 1.0))) for i in range(c["batch"])]
    if c["batch"] >= 4:
        n[-1] = 0
    return n


def _seen(c, length):
    """Tokens that some row of a sequence sees."""
    first = max(0, length - c["rows"])
    return length - (max(0, first - c["window"] + 1) if c["window"] else 0)


def work(case):
    c = case
    if c["op"] == "attend":
        e, tokens = TYPES[c["cache"]].itemsize, sum(_seen(c, n) for n in _lengths(c))
        per = 2 * c["kv_heads"] * (c["dim"] * e + (4 if c["cache"] == "e4m3" else 0))
        q = c["batch"] * c["rows"] * c["heads"] * c["dim"]
        return {"bytes": tokens * per + 4 * q + 4 * c["batch"], "flops": 4 * tokens * c["rows"] * c["heads"] * c["dim"]}
    if c["op"] in ("write", "read"):
        n = 2 * c["tokens"] * c["kv_heads"]
        held = c["dim"] * TYPES[c["cache"]].itemsize + (4 if c["cache"] == "e4m3" else 0)
        return {"bytes": n * (held + c["dim"] * TYPES[c["dtype"]].itemsize) + 4 * c["tokens"], "flops": 3 * n * c["dim"]}
    rows = c["batch"] * (2 if c["probs"] else 1)      # the rows of the one token that is drawn
    return {"bytes": 4 * rows * c["vocab"] + c["batch"] * (16 * c["drafts"] + 12), "flops": 2 * rows * c["vocab"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _to_8_bits(x):
    """x [.., D] in fp32 -> e4m3 codes and one scale per row."""
    scale = x.abs().amax(-1).clamp(min=TINY) / E4M3_MAX
    return (x / scale.unsqueeze(-1)).to(F8), scale


def _made_cache(c, pages, normal):
    """A cache full of keys and values [pages, heads, page, dim]."""
    made = []
    for channels in (torch.exp(normal(c["kv_heads"], 1, c["dim"], std=0.5)), 1.0):      # keys have larger channels
        t = torch.empty(pages, c["kv_heads"], c["page"], c["dim"], dtype=TYPES[c["cache"]], device="cuda")
        scales = torch.empty(pages, c["kv_heads"], c["page"], device="cuda") if c["cache"] == "e4m3" else None
        step = max(1, (1 << 26) // t[0].numel())
        for lo in range(0, pages, step):
            x = normal(*t[lo:lo + step].shape) * channels
            if scales is None:
                t[lo:lo + step] = x.to(t.dtype)
            else:
                t[lo:lo + step], scales[lo:lo + step] = _to_8_bits(x)
        made += [t, scales]
    return {"k": made[0], "v": made[2], "k_scales": made[1], "v_scales": made[3]}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": dict(c)}
    if c["op"] == "attend":
        order = torch.randperm(c["batch"], generator=g, device="cuda").tolist()
        lengths = [_lengths(c)[i] for i in order]
        counts = [-(-n // c["page"]) for n in lengths]
        pages = sum(counts) + 3
        s.update(_made_cache(c, pages, normal))
        ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((c["batch"], max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(counts):
            table[b, :n] = ids[at:at + n]
            at += n
        s["table"] = table
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        s["q"] = normal(c["batch"], c["rows"], c["heads"], c["dim"]).to(TYPES[c["dtype"]])
    elif c["op"] in ("write", "read"):
        pages = -(-c["tokens"] // c["page"]) * 9 // 8 + 2
        s.update(_made_cache(c, pages, normal))
        slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * c["page"] + torch.arange(c["page"], device="cuda")
        s["slots"] = slots.flatten()[:c["tokens"]].to(torch.int32)
        if c["tokens"] > 8:
            s["slots"][c["tokens"] // 2] = -1        # a place of the batch without a token
        if c["op"] == "write":       # the keys and values lie in the rows of the product that made them
            rows = normal(c["tokens"], 2, c["kv_heads"], c["dim"]).to(TYPES[c["dtype"]])
            s["new_k"], s["new_v"] = rows[:, 0], rows[:, 1]
    else:
        b, n, v = c["batch"], c["drafts"], c["vocab"]
        logits = normal(b, n + 1, v, std=2.5)
        drafted = torch.softmax(logits[:, :n] + normal(b, n, v, std=0.7), -1)
        if c["kept"] and c["kept"] < v:
            logits = logits.masked_fill(logits < logits.topk(c["kept"]).values[..., -1:], -math.inf)
        s["target"] = torch.softmax(logits, -1)
        s["draft"] = torch.multinomial(drafted.flatten(0, 1), 1, generator=g).view(b, n).to(torch.int32)
        if not c["probs"]:       # what is looked up is often what the target wants most
            s["draft"] = torch.where(uniform(b, n) < 0.6, s["target"][:, :n].argmax(-1).to(torch.int32), s["draft"])
        if b > 2:
            s["draft"][b // 2, n // 2:] = -1         # fewer drafts than the others
        s["draft_probs"] = drafted if c["probs"] else None
        s["accept_u"], s["sample_u"] = uniform(b, n), uniform(b)
    if own:
        from routed_moe_decode_router_gb300 import ops
        if "k" in s:
            s["cache"] = ops.KvCache(s["k"], s["v"], s["k_scales"], s["v_scales"])
        if c["op"] == "attend":
            s["ws"] = ops.AttendWorkspace(c["batch"], c["rows"], c["heads"], c["kv_heads"], c["dim"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if own:
        from routed_moe_decode_router_gb300 import ops
        if c["op"] == "attend":
            return {"out": ops.attend_paged(s["q"], s["cache"], s["table"], s["lengths"], window=c["window"], ws=s["ws"])}
        if c["op"] == "write":
            ops.kv_write(s["cache"], s["new_k"], s["new_v"], s["slots"])
            return {n: s[n] for n in ("k", "v", "k_scales", "v_scales")}
        if c["op"] == "read":
            k, v = ops.kv_read(s["cache"], s["slots"], dtype=TYPES[c["dtype"]])
            return {"k": k, "v": v}
        r = ops.verify_draft(s["draft"], s["target"], s["accept_u"], s["sample_u"], draft_probs=s["draft_probs"])
        return {"tokens": r.tokens, "accepted": r.accepted}
    return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read, "verify": _plain_verify}[c["op"]](s, c)


def _plain_attend(s, c):
    b, r, hk, d, page = c["batch"], c["rows"], c["kv_heads"], c["dim"], c["page"]
    tok = torch.arange(s["table"].shape[1] * page, device="cuda")
    pages = s["table"].long()[:, tok // page]                                 # [B, L]
    here = (tok < s["lengths"][:, None]) & (pages >= 0)
    at = (pages.clamp(min=0), slice(None), tok % page)
    k, v = s["k"][at].float(), s["v"][at].float()                            # [B, L, Hkv, D]
    if c["cache"] == "e4m3":
        k, v = k * s["k_scales"][at].unsqueeze(-1), v * s["v_scales"][at].unsqueeze(-1)
    v = v.masked_fill(~here[:, :, None, None], 0.0)
    q = s["q"].float().view(b, r, hk, -1, d).permute(0, 2, 1, 3, 4).flatten(2, 3)    # [B, Hkv, R G, D]
    score = (q @ k.permute(0, 2, 3, 1) * d ** -0.5).unflatten(2, (r, -1))    # [B, Hkv, R, G, L]
    pos = s["lengths"][:, None] - r + torch.arange(r, device="cuda")         # [B, R]
    see = here[:, None] & (tok <= pos[..., None])
    if c["window"]:
        see &= tok > pos[..., None] - c["window"]
    see = see[:, None, :, None]                                               # [B, 1, R, 1, L]
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    out = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (r, -1))    # [B, Hkv, R, G, D]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(b, r, -1, d).to(s["q"].dtype)}


def _plain_write(s, c):
    put = (s["slots"] >= 0).nonzero().flatten()
    slot = s["slots"][put].long()
    at = (slot // c["page"], slice(None), slot % c["page"])
    for n in ("k", "v"):
        x = s["new_" + n][put]
        if c["cache"] == "e4m3":
            codes, scales = _to_8_bits(x.float())
            s[n].view(torch.uint8)[at] = codes.view(torch.uint8)
            s[n + "_scales"][at] = scales
        else:
            s[n][at] = x
    return {n: s[n] for n in ("k", "v", "k_scales", "v_scales")}


def _plain_read(s, c):
    slot = s["slots"].clamp(min=0).long()
    at = (slot // c["page"], slice(None), slot % c["page"])
    out = {}
    for n in ("k", "v"):
        x = s[n][at].float()
        if c["cache"] == "e4m3":
            x = x * s[n + "_scales"][at].unsqueeze(-1)
        out[n] = x.masked_fill((s["slots"] < 0)[:, None, None], 0.0).to(TYPES[c["dtype"]])
    return out


def _plain_verify(s, c):
    # 64 bits: which token a number falls to is decided by sums next to each other
    b, n, v = c["batch"], c["drafts"], c["vocab"]
    x = s["draft"].clamp(min=0).long().unsqueeze(-1)
    there = s["draft"] >= 0
    p = s["target"][:, :n].gather(2, x).squeeze(-1).double()
    q = s["draft_probs"].gather(2, x).squeeze(-1).double() if c["probs"] else torch.ones_like(p)
    good = there & (s["accept_u"].double() * q < p)
    accepted = good.long().cumprod(1).sum(1)                                  # [B]
    every = torch.arange(b, device="cuda")
    row = s["target"][every, accepted].double()
    at = accepted.clamp(max=n - 1)
    refused = (accepted < n) & there[every, at]
    if c["probs"]:
        less = s["draft_probs"][every, at].double()
    else:
        less = torch.zeros_like(row).scatter_(1, x[every, at], 1.0)
    rest = (row - less).clamp(min=0.0)
    rest = torch.where((refused & (rest.sum(1) > 0))[:, None], rest, row)
    sums = rest.cumsum(1)
    token = (sums <= s["sample_u"].double()[:, None] * sums[:, -1:]).sum(1)
    token = torch.where(sums[:, -1] > 0, token.clamp(max=v - 1), -1)
    place = torch.arange(n + 1, device="cuda")
    tokens = torch.cat([s["draft"], s["draft"].new_full((b, 1), -1)], 1).long()
    tokens = torch.where(place < accepted[:, None], tokens, -1)
    tokens = torch.where(place == accepted[:, None], token[:, None], tokens)
    return {"tokens": tokens.to(torch.int32), "accepted": accepted.to(torch.int32)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    return {"attend": _exact_attend, "write": _exact_write, "read": _exact_read, "verify": _exact_verify}[c["op"]](s, c)


def _wide(s, c, name, slots):
    """Rows of the cache [n, heads, dim] in 64 bits, by their slots."""
    x = s[name].transpose(1, 2).flatten(0, 1)[slots].double()
    return x * s[name + "_scales"].transpose(1, 2).flatten(0, 1)[slots].double()[..., None] if c["cache"] == "e4m3" else x


def _exact_attend(s, c):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lengths, group = s["lengths"].tolist(), c["heads"] // c["kv_heads"]
    for b, n in enumerate(lengths):
        lo = n - _seen(c, n)
        places = torch.arange(lo, n, device="cuda")
        slots = s["table"][b].long()[places // c["page"]] * c["page"] + places % c["page"]
        k, v = _wide(s, c, "k", slots), _wide(s, c, "v", slots)
        for r in range(c["rows"]):
            last = n - c["rows"] + r
            first = max(0, last - c["window"] + 1) if c["window"] else 0
            if last < 0:
                continue
            kk, vv = k[first - lo:last + 1 - lo], v[first - lo:last + 1 - lo]
            q = s["q"][b, r].double().unflatten(0, (-1, group))
            w = torch.softmax(torch.einsum("hgd,nhd->hgn", q, kk) / math.sqrt(c["dim"]), -1)
            out[b, r] = torch.einsum("hgn,nhd->hgd", w, vv).flatten(0, 1)
    return {"out": out}


def _exact_write(s, c):
    out = {}
    slots = s["slots"].tolist()
    rows = [t for t, slot in enumerate(slots) if slot >= 0]
    where = torch.tensor([slots[t] for t in rows], device="cuda")
    rows = torch.tensor(rows, device="cuda")
    for n in ("k", "v"):
        held = s[n].double().transpose(1, 2).flatten(0, 1)                     # [slots, heads, dim]
        scales = s[n + "_scales"]
        new = s["new_" + n].double()[rows]
        if scales is not None:               # the codes: what is rounded to them
            scales = scales.double().transpose(1, 2).flatten(0, 1)
            size = torch.maximum(new.abs().max(-1).values, torch.tensor(TINY, dtype=torch.float64, device="cuda")) / E4M3_MAX
            scales[where] = size
            new = new / size[..., None]
            scales = scales.unflatten(0, (-1, c["page"])).transpose(1, 2)
        held[where] = new
        out[n], out[n + "_scales"] = held.unflatten(0, (-1, c["page"])).transpose(1, 2), scales
    return {n: out[n] for n in ("k", "v", "k_scales", "v_scales")}


def _exact_read(s, c):
    live = s["slots"] >= 0
    out = {}
    for n in ("k", "v"):
        out[n] = torch.zeros(c["tokens"], c["kv_heads"], c["dim"], dtype=torch.float64, device="cuda")
        out[n][live] = _wide(s, c, n, s["slots"][live].long())
    return out


def _exact_verify(s, c):
    b, n = c["batch"], c["drafts"]
    draft, accept, sample = (s[x].cpu().numpy() for x in ("draft", "accept_u", "sample_u"))
    tokens, accepted = np.full((b, n + 1), -1, np.int32), np.zeros(b, np.int32)
    for i in range(b):
        j, weights = 0, None
        while j < n and draft[i, j] >= 0:
            p = s["target"][i, j].cpu().numpy().astype(np.float64)
            q = s["draft_probs"][i, j].cpu().numpy().astype(np.float64) if c["probs"] else np.eye(1, c["vocab"], draft[i, j])[0]
            if float(accept[i, j]) * q[draft[i, j]] >= p[draft[i, j]]:
                weights = np.maximum(p - q, 0.0)
                weights = weights if weights.any() else p
                break
            tokens[i, j] = draft[i, j]
            j += 1
        if weights is None:
            weights = s["target"][i, j].cpu().numpy().astype(np.float64)
        sums = np.cumsum(weights)
        if sums[-1] > 0:
            tokens[i, j] = min(int(np.searchsorted(sums, float(sample[i]) * sums[-1], side="right")), c["vocab"] - 1)
        accepted[i] = j
    return {"tokens": tokens, "accepted": accepted}
