"""Plain 64-bit definitions of the FP8 layer operators and the error bounds
their tests use (CPU or GPU tensors alike)."""
import math

import torch

F8 = torch.float8_e4m3fn
U = 2.0 ** -24        # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny_step(dtype):
    """Half a step of the type's subnormals."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def expand_rows(s, k):
    return s.double().repeat_interleave(128, -1)[..., :k]


def rows_fp8(x):
    """x [T, K] -> (codes, scales) as the FP8 rows are defined."""
    t, k = x.shape
    kb = -(-k // 128)
    pad = torch.zeros(t, kb * 128, dtype=torch.float64, device=x.device)
    pad[:, :k] = x.double()
    scales = pad.view(t, kb, 128).abs().amax(2).clamp(min=1e-30).float() / 448.0
    q = (pad / expand_rows(scales, kb * 128))[:, :k].clamp(-448, 448).float().to(F8)
    return q.contiguous(), scales


def weights_fp8(w):
    """w [N, K] -> (codes, scales) with one scale per 128 x 128 block."""
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    pad = torch.zeros(nb * 128, kb * 128, dtype=torch.float64, device=w.device)
    pad[:n, :k] = w.double()
    scales = pad.view(nb, 128, kb, 128).abs().amax((1, 3)).clamp(min=1e-30).float() / 448.0
    full = scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    q = (pad / full)[:n, :k].clamp(-448, 448).float().to(F8)
    return q.contiguous(), scales


def wide_rows(q, s):
    return q.double() * expand_rows(s, q.shape[-1])


def wide_weights(q, s):
    n, k = q.shape
    return q.double() * s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def norm(x, weight, eps, residual=None):
    s = x.double() + (residual.double() if residual is not None else 0.0)
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * weight.double()
    return s, y


def product(a, sa, b, sb):
    """(A B^T, the bound's scale |A| |B|^T) in 64 bits."""
    x, w = wide_rows(a, sa), wide_weights(b, sb)
    return x @ w.T, x.abs() @ w.abs().T


def product_bound(k):
    """Relative to |A| |B|^T: each of the 128 products of a block is added with
    at most one truncated fp32 step (2 U), then a scale (2 U) and one addition
    per block (U)."""
    return (2 * 128 + 4 + -(-k // 128)) * U


def route(logits, top_k, scoring="softmax", bias=None, groups=1, group_limit=1,
          group_score="max", norm_topk_prob=True, routed_scaling_factor=1.0):
    """Row by row, by the definition."""
    ids_out, wts_out = [], []
    for row in logits.double().cpu().tolist():
        live = [not math.isnan(v) and v != -math.inf for v in row]
        e = len(row)
        if scoring == "softmax":
            m = max([v for v, ok in zip(row, live) if ok], default=0.0)
            ex = [math.exp(v - m) if ok else 0.0 for v, ok in zip(row, live)]
            tot = math.fsum(ex)
            p = [v / tot if tot else 0.0 for v in ex]
        else:
            p = [0.0 if not ok else (1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0)
                 for v, ok in zip(row, live)]
        b = bias.double().cpu().tolist() if bias is not None else [0.0] * e
        score = [p[i] + b[i] for i in range(e)]
        key = score if bias is not None else row
        size = e // groups
        gs = []
        for g in range(groups):
            v = sorted((score[i] for i in range(g * size, (g + 1) * size) if live[i]),
                       reverse=True)
            gs.append(-math.inf if not v else v[0] + (v[1] if group_score == "top2" and
                                                      len(v) > 1 else 0.0))
        taken = set(sorted(range(groups), key=lambda g: (-gs[g], g))[:group_limit])
        cand = [i for i in range(e) if live[i] and (groups == 1 or i // size in taken)]
        ids = sorted(cand, key=lambda i: (-key[i], i))[:top_k]
        w = [p[i] for i in ids]
        if norm_topk_prob:
            tot = math.fsum(w)
            w = [v / tot if tot else 0.0 for v in w]
        w = [v * routed_scaling_factor for v in w]
        ids_out.append(ids + [-1] * (top_k - len(ids)))
        wts_out.append(w + [0.0] * (top_k - len(w)))
    return torch.tensor(ids_out, dtype=torch.int32), torch.tensor(wts_out, dtype=torch.float64)


def experts(q, s, ids, wts, gate, gs, up, us, down, ds, addend=None):
    """(out, bound) in 64 bits.  h is rounded to e4m3 by definition; where its
    fp32 value may fall on the other side of a rounding border, the bound
    takes the whole step in.  y is held in bf16, out rounded to bf16."""
    t, k = ids.shape
    hdim, e = q.shape[1], gate.shape[0]
    out = torch.zeros(t, hdim, dtype=torch.float64, device=q.device)
    err = torch.zeros_like(out)
    if addend is not None:
        out += addend.double()
    kb, ib = hdim // 128, gate.shape[1] // 128
    for x in range(e):
        row, slot = (ids == x).nonzero(as_tuple=True)
        if not len(row):
            continue
        g, ga = product(q[row], s[row], gate[x], gs[x])
        u, ua = product(q[row], s[row], up[x], us[x])
        pb = product_bound(hdim)
        silu = g / (1 + torch.exp(-g))
        h = silu * u
        # |d silu| <= 1.1; __expf: 2 + |x| steps, the divide 2
        eh = 1.1 * ga * pb * u.abs() + silu.abs() * ua * pb + h.abs() * (8 + g.abs()) * 2 * U
        sc = h.view(len(row), ib, 128).abs().amax(2).clamp(min=1e-30) / 448.0
        se = eh.view(len(row), ib, 128).amax(2) / 448.0      # the scale moves as its largest h
        scx, sex = expand_rows(sc, h.shape[1]), expand_rows(se, h.shape[1])

        def code(v):
            return v.clamp(-448, 448).float().to(F8).double()
        z = h / scx
        ez = (eh + z.abs() * sex) / scx + z.abs() * 4 * U
        hq = code(z)
        far = torch.maximum((code(z + ez) - hq).abs(), (code(z - ez) - hq).abs()) * scx
        far = far + hq.abs() * sex + hq.abs() * scx * 2 * U
        hv = hq * scx
        w = wide_weights(down[x], ds[x])
        y = hv @ w.T
        ye = far @ w.abs().T + hv.abs() @ w.abs().T * product_bound(h.shape[1])
        ye = ye + (y.abs() + ye) * half_step(torch.bfloat16)
        f = wts[row, slot].double()[:, None]
        out.index_put_((row,), y * f, accumulate=True)
        err.index_put_((row,), ye * f.abs() + (y * f).abs() * 2 * (k + 1) * U, accumulate=True)
    err = err + (out.abs() + err) * half_step(torch.bfloat16)
    return out, err + 1e-30
