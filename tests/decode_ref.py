"""Plain 64-bit definitions of the decoding step's operators (cache write and
read, attention over a paged cache, verification of drafts) and the error bound of
the attention (CPU or GPU tensors alike)."""
import math

import numpy as np
import torch

from tests.ops_ref import F8, half_step, tiny_step


def kv_codes(x):
    """x [..., D] -> (codes, scales): one scale per row."""
    scales = x.double().abs().amax(-1).clamp(min=1e-30).float() / 448.0
    return (x.double() / scales.double().unsqueeze(-1)).clamp(-448, 448).float().to(F8), scales


def wide(cache, name):
    """The cache's keys or values [slots, heads, dim] in 64 bits."""
    x = getattr(cache, name).transpose(1, 2).flatten(0, 1).double()
    s = getattr(cache, name + "_scales")
    return x if s is None else x * s.transpose(1, 2).flatten(0, 1).double().unsqueeze(-1)


def attend(q, cache, table, lengths, scale=None, window=0):
    """(out, bound) of q [B, R, Hq, D]: the definition, and how far fp32 sums of the
    given types may be from it."""
    b, r, hq, d = q.shape
    hk, page, pages = cache.k.shape[1], cache.k.shape[2], cache.k.shape[0]
    g = hq // hk
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    kw, vw = wide(cache, "k"), wide(cache, "v")
    for i in range(b):
        n = min(max(int(lengths[i]), 0), table.shape[1] * page)
        tok = torch.arange(n, device=q.device)
        ids = table[i].long()[tok // page]
        there = (ids >= 0) & (ids < pages)
        slots = (ids * page + tok % page)[there]
        tok = tok[there]
        for row in range(r):
            last = n - r + row
            see = tok <= last
            if window:
                see &= tok > last - window
            at = slots[see]
            if not len(at):
                continue
            k, v = kw[at], vw[at]
            x = q[i, row].double().view(hk, g, d)
            s = torch.einsum("hgd,nhd->hgn", x, k) * scale
            size = torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()).amax(2) * abs(scale)   # [hk, g]
            w = torch.exp(s - s.amax(2, keepdim=True))
            w = w / w.sum(2, keepdim=True)
            out[i, row] = torch.einsum("hgn,nhd->hgd", w, v).reshape(hq, d)
            mean = torch.einsum("hgn,nhd->hgd", w, v.abs())
            # scores: d products and additions and some 16 other steps of fp32, each
            # relative to the sum of magnitudes (the exponent's own rounding among
            # them); exp2 2^-22; both in numerator and denominator
            off = (2 * d + 32) * 2.0 ** -23 * size
            if cache.k_scales is not None:
                # q in e4m3 numbers, the last of which counts in steps of 2^-9 of 2^-5
                # where the row's largest is 2^7: half a step is 2^-22 of that
                off = off + 2.0 ** -22 * abs(scale) * x.abs().amax(2) * \
                    k.abs().sum(2).amax(0).unsqueeze(1)
            rel = 2 * (torch.exp(off) - 1 + 2.0 ** -21)
            # weights as two 16-bit numbers; additions of the tokens and the joins
            rel = rel + (2.0 ** -16 if q.dtype == torch.bfloat16 and cache.k_scales is None
                         else 2.0 ** -21) + (len(at) + 64) * 2.0 ** -22
            # f16 weights below its normal numbers: 2^-25 of the largest contribution's scale
            top = 1.0 if cache.k_scales is None else 448.0
            vmax = v.abs().amax(2).T.unsqueeze(1) if cache.k_scales is None else \
                cache.v_scales.transpose(1, 2).flatten(0, 1)[at].double().T.unsqueeze(1)
            small = len(at) * 2.0 ** -24 * (w * vmax).amax(2) * top
            if cache.k_scales is None:       # the weights alone are held, whatever the values
                small = len(at) * 2.0 ** -24 * w.amax(2) * v.abs().amax()
            o = out[i, row].abs().view(hk, g, d)
            bound[i, row] = (mean * rel.unsqueeze(-1) + small.unsqueeze(-1) +
                             o * half_step(q.dtype) * 1.01 + tiny_step(q.dtype)).view(hq, d)
    return out, bound


def verify(draft, target, accept_u, sample_u, draft_probs=None):
    """(tokens, accepted) by the definition, weights counted in steps of 2^-44 as
    Python's whole numbers."""
    b, n = draft.shape
    v = target.shape[2]
    draft, accept_u, sample_u = (t.cpu().numpy() for t in (draft, accept_u, sample_u))
    tokens, accepted = np.full((b, n + 1), -1, np.int64), np.zeros(b, np.int64)

    def steps(row):
        p = row.cpu().numpy().astype(np.float64)
        p = np.clip(np.where(np.isnan(p), 0.0, p), 0.0, 1.0)
        return np.rint(p * 2.0 ** 44).astype(np.int64)

    for i in range(b):
        j, w = 0, None
        while j < n and draft[i, j] >= 0:
            x = int(draft[i, j])
            p = float(target[i, j, x]) if x < v else 0.0
            q = 1.0 if draft_probs is None else float(draft_probs[i, j, x]) if x < v else 0.0
            if x < v and float(accept_u[i, j]) * q < p:
                tokens[i, j] = x
                j += 1
                continue
            full = steps(target[i, j])
            if draft_probs is None:
                w = full.copy()
                if x < v:
                    w[x] = 0
            else:
                w = np.maximum(full - steps(draft_probs[i, j]), 0)
            if not w.any():
                w = full
            break
        if w is None:
            w = steps(target[i, j])
        sums = np.cumsum(w)
        total = int(sums[-1])
        u = float(sample_u[i])
        u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1 - 2.0 ** -24)
        num, den = u.as_integer_ratio()
        if total:
            tokens[i, j] = int(np.searchsorted(sums, num * total // den, side="right"))
        accepted[i] = j
    return torch.from_numpy(tokens).int(), torch.from_numpy(accepted).int()
