"""Plain fp64 definitions of the rotation with axes, of eviction by accumulated
weight and of the 4-bit cache (torch, CPU), row by row, and the error bounds of
the library's results.

Bounds. Logits, exponentials and sums are fp32: as in _plain, an error of a logit
below 2^-13 scales its weight by less than 1 + 2^-12. An accumulated weight is off
by that much of the step's own weights, and by the fp32 rounding of the product
and the sum that take it in (2^-23 of the result). In 4 bits a weight times its
scale is rounded to 11 bits, which moves the output by at most 2^-11 of
sum_j p_j |v_j|; the products add codes of up to 15 and take 8 off, so fp32
accumulation over a chain of 48 additions (at most 2^-23 each, the tensor cores
truncate) is off by 48 * 23 * 2^-23 < 2^-12 of sum_j p_j s_j; the logits' own
chain is bounded like that of _plain: 16 products of codes and q per step, 2^-23
of sum |q| 23 s * scale < 2^9, well below 2^-13 a logit for inputs of N(0, 1).
"""
import math

import torch

from _plain import F64, HALF, attend

GROUP = 32


def axes_rope(x, w, freq, pos, axis, eps, interleaved):
    """[T, H, d] heads normed (w or None) and rotated by positions [axes, T]."""
    x = x.cpu().to(F64)
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.cpu().to(F64)
    freq, pos = freq.cpu().to(F64), pos.cpu().to(F64)
    r = freq.numel()
    y = x.clone()
    for i in range(r):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        ang = pos[axis[i]] * freq[i]
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def weights_step(q, kc, vc, mask, weights, nk, nv, ws, W, scale, decay, k, fill=False, evict=False):
    """One decode step that accumulates weights: out and its bound, weights and
    theirs, the state after it. (The choice is a function of the weights: `chosen`.)"""
    q, kc, vc, nk, nv = (t.cpu().to(F64) for t in (q, kc, vc, nk, nv))
    total, mask, ws = weights.cpu().to(F64).clone(), mask.cpu().clone(), ws.cpu()
    # The argument is an fp32 number: 0.97 is off by up to 2^-25 of itself, which is not the
    # kernel's rounding (2^-23 of the result covers the product's and the sum's, 2^-24 each).
    decay = float(torch.tensor(decay, dtype=torch.float32))
    kc, vc = kc.clone(), vc.clone()
    B, Hq, d = q.shape
    Hkv, S = kc.shape[1:3]
    g = Hq // Hkv
    out, tol = torch.zeros((B, Hq, d), dtype=F64), torch.zeros((B, Hq, d), dtype=F64)
    wtol = torch.zeros_like(total)
    for b in range(B):
        for u in range(Hkv):
            w = int(ws[b, u])
            if 0 <= w < S:
                kc[b, u, w], vc[b, u, w] = nk[b, u], nv[b, u]
                mask[b, u] += (mask[b, u] >= 0).int()
                mask[b, u, w] = 0
                total[b, u, w] = 0
            live = torch.nonzero(mask[b, u] >= 0)[:, 0]
            new = torch.zeros(len(live), dtype=F64)
            for h in range(u * g, u * g + g):
                o, a, lse = attend(q[b, h], kc[b, u, live], vc[b, u, live], scale)
                out[b, h], tol[b, h] = o, (HALF + 2.0 ** -12) * a + HALF * o.abs()
                if len(live):
                    new += torch.exp(kc[b, u, live] @ q[b, h] * scale - lse)
            total[b, u, live] = (total[b, u, live] * decay if decay else 0) + new
            wtol[b, u, live] = 2.0 ** -12 * new + 2.0 ** -23 * total[b, u, live].abs()
    return {"out": out, "tol": tol, "weights": total, "wtol": wtol, "k": kc, "v": vc, "mask": mask}


def chosen(weights, mask, W, k, fill):
    """The k slots with the least (weight, slot) per unit, from fp32 weights as stored."""
    B, Hkv, S = mask.shape
    got = torch.full((B, Hkv, k), -1, dtype=torch.int32)
    for b in range(B):
        for u in range(Hkv):
            a = mask[b, u]
            old = torch.nonzero((a >= 0) & (a >= W) & ~torch.isnan(weights[b, u]))[:, 0]
            order = old[torch.sort(weights[b, u, old], stable=True)[1]]
            if fill:
                order = torch.cat([torch.nonzero(a < 0)[:, 0], order])
            got[b, u, :min(k, len(order))] = order[:k].int()
    return got


def prompt_weights(q, kc, starts, lens, weights, rows, scale):
    """Weights [B, Hkv, S] after the call, and their bounds."""
    q, kc, w = q.cpu().to(F64), kc.cpu().to(F64), weights.cpu().to(F64).clone()
    tol = torch.zeros_like(w)
    g = q.shape[1] // kc.shape[1]
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        past = lens[b] - n
        w[b, :, past:lens[b]] = 0
        for i in range(max(0, n - rows) if rows else 0, n):
            for h in range(q.shape[1]):
                s = kc[b, h // g, :past + i + 1] @ q[starts[b] + i, h] * scale
                p = torch.softmax(s, 0)
                w[b, h // g, :past + i + 1] += p
                tol[b, h // g, :past + i + 1] += 2.0 ** -12 * p
    return w, tol + 2.0 ** -20 * w.abs()


def quantise(x):
    """(codes, scales, values) of rows of bf16, in 64 bits; a group that is not finite is NaN."""
    x = x.cpu().to(F64).unflatten(-1, (-1, GROUP))
    top = x.abs().amax(-1)
    s = (top / 7).to(torch.bfloat16).to(F64)
    s = torch.where(torch.isfinite(top), s, math.nan)
    step = x / torch.where(s == 0, 1.0, s)[..., None]
    code = torch.round(step).clamp(-7, 7)  # (ties to even)
    code = torch.where((s == 0)[..., None] | torch.isnan(s)[..., None], 0.0, code)
    return code.flatten(-2), s, (code * s[..., None]).flatten(-2)


def lay(code, piece):
    """Bytes of rows of codes, value by value."""
    d = code.shape[-1]
    out = torch.zeros(code.shape[:-1] + (d // 2,), dtype=torch.int32)
    for c in range(d):
        g, r = c // GROUP, c % GROUP
        at = (r // piece * (d // GROUP) + g) * piece + r % piece
        out[..., at // 2] |= (code[..., c].int() + 8) << (4 * (at % 2))
    return out.to(torch.uint8)


def stand_for(byte, scale, piece):
    """Values of rows of bytes and scales, in 64 bits."""
    byte, scale = byte.cpu().int(), scale.cpu().to(F64)
    d = 2 * byte.shape[-1]
    out = torch.zeros(byte.shape[:-1] + (d,), dtype=F64)
    for c in range(d):
        g, r = c // GROUP, c % GROUP
        at = (r // piece * (d // GROUP) + g) * piece + r % piece
        out[..., c] = (((byte[..., at // 2] >> (4 * (at % 2))) & 15) - 8).double() * scale[..., g]
    return out


def kv4_attention(q, k, v, ks, vs, mask, scale):
    """Outputs and bounds over caches of values [B, Hkv, S, d]; vs their scales [B, Hkv, S, d/32]."""
    q, mask, vs = q.cpu().to(F64), mask.cpu(), vs.cpu().to(F64)
    B, Hq, d = q.shape
    g = Hq // k.shape[1]
    out, tol = torch.zeros((B, Hq, d), dtype=F64), torch.zeros((B, Hq, d), dtype=F64)
    for b in range(B):
        for h in range(Hq):
            u = h // g
            live = torch.nonzero(mask[b, u] >= 0)[:, 0]
            if not len(live):
                continue
            o, a, lse = attend(q[b, h], k[b, u, live], v[b, u, live], scale)
            p = torch.exp(k[b, u, live] @ q[b, h] * scale - lse)
            unit = (p[:, None] * vs[b, u, live]).sum(0).repeat_interleave(GROUP)
            out[b, h] = o
            tol[b, h] = (2.0 ** -11 + 2.0 ** -12) * a + 2.0 ** -12 * unit + HALF * o.abs()
    return out, tol
