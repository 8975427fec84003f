"""Plain fp64 definitions of the operators around the decode step (torch, CPU),
row by row, and the error bounds of their bf16 results.

Bounds. A result rounded to bf16 is off by at most 2^-8 of its value (half a
step). Attention also rounds each weight p_j to bf16 before the product with
the values, 2^-8 of it at most, which moves the output by at most
2^-8 * sum_j p_j |v_j|; the fp32 arithmetic before it (dot products of d <= 128
exact bf16 products, exponentials, sums) stays below 2^-12 of the same sum for
logits of N(0, 1) inputs: an error e of a logit scales its weight by about
1 + e, and with sum |q_i k_i| * scale <= 32 the accumulation's bound
d * 2^-24 * 32 is 2^-12.
"""
import math

import torch

HALF = 2.0 ** -8
F64 = torch.float64


def attend(q, k, v, scale):
    """(output, sum_j p_j |v_j|, log-sum-exp) of one row over its visible keys."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape, dtype=F64)
        return z, z, -math.inf
    s = (k @ q) * scale
    m = s.max()
    e = torch.exp(s - m)
    p = e / e.sum()
    return p @ v, p @ v.abs(), float(m + torch.log(e.sum()))


def window_rows(q, kc, vc, starts, lens, window, sinks, scale):
    """Reference outputs and bounds [T, Hq, d]; rows outside the sequences are NaN."""
    q, kc, vc = q.cpu().to(F64), kc.cpu().to(F64), vc.cpu().to(F64)
    T, Hq, d = q.shape
    g = Hq // kc.shape[1]
    ref = torch.full((T, Hq, d), math.nan, dtype=F64)
    tol = torch.zeros((T, Hq, d), dtype=F64)
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            pos = lens[b] - n + i
            j = torch.arange(pos + 1)
            if window:
                j = j[(pos - j < window) | (j < sinks)]
            for h in range(Hq):
                o, a, _ = attend(q[starts[b] + i, h], kc[b, h // g][j], vc[b, h // g][j], scale)
                ref[starts[b] + i, h] = o
                tol[starts[b] + i, h] = (HALF + 2.0 ** -12) * a + HALF * o.abs()
    return ref, tol


def rope(x, w, freq, pos, eps, interleaved):
    """[T, H, d] heads normed (w or None) and rotated."""
    x = x.cpu().to(F64)
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.cpu().to(F64)
    freq = freq.cpu().to(F64)
    r = freq.numel()
    y = x.clone()
    for i in range(r):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        ang = pos.cpu().to(F64) * freq[i]
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rope_bound(y):
    """One rounding to bf16, and 2^-18 of the head's largest pair for the fp32 arithmetic:
    some ten roundings of 2^-24 and an angle reduced to 2^-23 of a turn."""
    return HALF * y.abs() + 2.0 ** -18 * math.sqrt(2) * y.abs().amax(-1, keepdim=True)


def prefix_step(q, kc, vc, mask, nk, nv, ws, kp, vp, starts, plen, W, scale, ageing=True):
    """One decode step over prefix and slots: dict of out, tol, scores, and the
    caches and mask after the write."""
    q, kc, vc, nk, nv, kp, vp = (t.cpu().to(F64) for t in (q, kc, vc, nk, nv, kp, vp))
    mask, ws = mask.cpu().clone(), ws.cpu()
    kc, vc = kc.clone(), vc.clone()
    B, Hq, d = q.shape
    Hkv, S = kc.shape[1:3]
    g = Hq // Hkv
    out = torch.zeros((B, Hq, d), dtype=F64)
    tol = torch.zeros_like(out)
    scores = torch.full((B, Hkv, S), math.inf, dtype=F64)
    for b in range(B):
        n = next((i for i in range(len(plen)) if starts[i] <= b < starts[i + 1]), None)
        for u in range(Hkv):
            w = int(ws[b, u])
            if w >= 0:
                kc[b, u, w], vc[b, u, w] = nk[b, u], nv[b, u]
                if ageing:
                    mask[b, u] = torch.where(mask[b, u] >= 0, mask[b, u] + 1, mask[b, u])
                    mask[b, u, w] = 0
                elif mask[b, u, w] < 0:
                    mask[b, u, w] = 0
            live = torch.nonzero(mask[b, u] >= 0)[:, 0]
            P = plen[n] if n is not None else 0
            k = torch.cat([kp[n, u, :P], kc[b, u, live]]) if P else kc[b, u, live]
            v = torch.cat([vp[n, u, :P], vc[b, u, live]]) if P else vc[b, u, live]
            I = torch.zeros(len(live), dtype=F64)
            for h in range(u * g, u * g + g):
                o, a, lse = attend(q[b, h], k, v, scale)
                out[b, h] = o
                tol[b, h] = (HALF + 2.0 ** -12) * a + HALF * o.abs()
                p = torch.exp(k[P:] @ q[b, h] * scale - lse) if len(live) else I
                I = I + p * vc[b, u, live].abs().sum(-1)
            scores[b, u, live] = I
    return {"out": out, "tol": tol, "scores": scores, "k": kc, "v": vc, "mask": mask}
