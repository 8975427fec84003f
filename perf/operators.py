"""Measured cases of the operators around the decode step.

Three operators that a decode loop needs next to the fused step:

* norms of queries and keys per head with the position rotation, for single
  tokens ("norm_rope") and for prompts that go into the cache ("append");
* attention over an in-order cache with a sliding window and visible first
  tokens ("window"): prompts, chunks of prompts, single tokens;
* decode attention for batches whose sequences share long prefixes ("prefix").

``run`` computes them in plain torch operations, in 32 bits, or (``own``)
through the library. ``exact`` evaluates the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
ROPE_BASE = 1e6
EPS = 1e-6


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One token of one sequence, 32 query and 8 KV heads: the latency of a decode layer's first call.
        dict(name="norm_rope_b1", kind="norm_rope", T=1, Hq=32, Hkv=8, d=128, rot=128, inter=False,
             norm=True, far=16384),
        # The same for a decode batch of 128 at far positions.
        dict(name="norm_rope_b128", kind="norm_rope", T=128, Hq=32, Hkv=8, d=128, rot=128,
             inter=False, norm=True, far=1000000),
        # Ragged prompts of a batch of 32 into caches of 2400 slots.
        dict(name="append_b32_s2400", kind="append", B=32, Hq=32, Hkv=8, d=128, S=2400, rot=128,
             inter=False, norm=True, q_lo=100, q_hi=1300, past=0, offset=0, lens=1),
        # The next chunk of five prompts, partial interleaved rotation, no norm weights,
        # positions that continue a prefix.
        dict(name="append_chunk_d64", kind="append", B=5, Hq=16, Hkv=2, d=64, S=1001, rot=32,
             inter=True, norm=False, q_lo=1, q_hi=333, past=600, offset=5003, lens=2),
        # One sequence's next token over a long cache: latency.
        dict(name="window_decode_b1", kind="window", B=1, Hq=32, Hkv=8, d=128, S=16384, q_lo=1,
             q_hi=1, kv_lo=16384, kv_hi=16384, window=4096, sinks=4, lens=3),
        # A decode batch at ragged lengths: memory bound.
        dict(name="window_decode_b128", kind="window", B=128, Hq=32, Hkv=8, d=128, S=3200, q_lo=1,
             q_hi=1, kv_lo=600, kv_hi=3200, window=1024, sinks=16, lens=4),
        # Whole prompts of up to 2400 tokens through a windowed layer.
        dict(name="window_prefill_b8", kind="window", B=8, Hq=32, Hkv=8, d=128, S=2400, q_lo=1200,
             q_hi=2400, kv_lo=0, kv_hi=0, window=1024, sinks=4, lens=5),
        # One long prompt through a layer without a window: compute bound, the largest.
        dict(name="causal_prefill_16k", kind="window", B=1, Hq=32, Hkv=8, d=128, S=16384,
             q_lo=16384, q_hi=16384, kv_lo=0, kv_hi=0, window=0, sinks=0, lens=6),
        # Mixed chunks and single tokens, head dim 64, odd window and lengths.
        dict(name="window_mixed_d64", kind="window", B=7, Hq=8, Hkv=4, d=64, S=1501, q_lo=1,
             q_hi=300, kv_lo=300, kv_hi=1501, window=333, sinks=5, lens=7),
        # Four samples of one prompt on a small model, with the slot write.
        dict(name="prefix_b4", kind="prefix", B=4, N=1, Hq=4, Hkv=2, d=64, S=256, P=1000,
             p_lo=1000, p_hi=1000, live_lo=1, live_hi=240, write=True, lens=8),
        # 128 samples of one long prompt over full 2400-slot caches.
        dict(name="prefix_b128_p16384", kind="prefix", B=128, N=1, Hq=32, Hkv=8, d=128, S=2400,
             P=16384, p_lo=16384, p_hi=16384, live_lo=2400, live_hi=2400, write=False, lens=9),
        # Nine prompts of odd lengths with a few samples each, ragged caches, groups of 8 heads.
        dict(name="prefix_groups_b67", kind="prefix", B=67, N=9, Hq=32, Hkv=4, d=128, S=2400,
             P=5003, p_lo=0, p_hi=5003, live_lo=0, live_hi=2400, write=False, lens=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    return hkv * rng.choice([1, 2, 4, 8]), hkv, rng.choice([64, 128])


def draw(rng: random.Random):
    kind = rng.choice(["norm_rope", "append", "window", "window", "prefix", "prefix"])
    Hq, Hkv, d = _heads(rng)
    seed = rng.randrange(1 << 30)
    if kind == "norm_rope":
        return dict(kind=kind, T=_log(rng, 1, 4096), Hq=Hq, Hkv=Hkv, d=d,
                    rot=16 * rng.randint(1, d // 16), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.7, far=_log(rng, 100, 1000000))
    if kind == "append":
        S = _log(rng, 64, 8192)
        past = rng.choice([0, rng.randint(0, S // 2)])
        hi = rng.randint(1, S - past)
        B = _log(rng, 1, max(1, min(64, 65536 // S)))
        return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, S=S, rot=16 * rng.randint(1, d // 16),
                    inter=rng.random() < 0.5, norm=rng.random() < 0.7, q_lo=rng.randint(0, hi),
                    q_hi=hi, past=past, offset=rng.choice([0, 7001]), lens=seed)
    if kind == "window":
        S = _log(rng, 64, int(16384 * min(1.0, math.sqrt(32 / Hq))))
        window = rng.choice([0, _log(rng, 1, S), _log(rng, 16, 4096)])
        sinks = rng.choice([0, rng.randint(1, 200)])
        form = rng.choice(["one", "prompt", "mixed"])
        if form == "one":
            B = _log(rng, 1, max(1, min(256, 300000 // S)))
            q_lo = q_hi = 1
            kv_lo, kv_hi = rng.randint(1, S), S
        elif form == "prompt":
            B = _log(rng, 1, max(1, min(32, 16384 // S)))
            q_lo, q_hi = rng.randint(0, S), S
            kv_lo = kv_hi = 0
        else:
            B = _log(rng, 1, max(1, min(32, 32768 // S)))
            q_lo, q_hi = 0, rng.randint(1, max(1, S // 4))
            kv_lo, kv_hi = q_hi, S
        return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, S=S, q_lo=q_lo, q_hi=q_hi, kv_lo=kv_lo,
                    kv_hi=kv_hi, window=window, sinks=sinks, lens=seed)
    S = _log(rng, 64, 8192)
    B = _log(rng, 1, max(1, min(256, 250000 // S)))
    P = _log(rng, 64, 16384)
    N = rng.randint(1, min(B, 12, max(1, 32768 // P)))
    live = rng.randint(0, S)
    return dict(kind=kind, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, S=S, P=P, p_lo=rng.randint(0, P), p_hi=P,
                live_lo=live, live_hi=rng.randint(live, S), write=B * S * Hkv * d < (1 << 24),
                lens=seed)


# ----------------------------------------------------------- ragged lengths --

def _layout(case):
    """Host-side lengths of a ragged case; the same for every input seed."""
    rng = random.Random(case["lens"])
    B = case["B"]
    if case["kind"] == "append":
        n = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(B)]
        past = [rng.randint(0, case["past"]) for _ in range(B)]
        return dict(nq=n, kv=[a + b for a, b in zip(n, past)])
    if case["kind"] == "window":
        n = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(B)]
        kv = list(n) if case["kv_hi"] == 0 else [
            max(a, rng.randint(case["kv_lo"], case["kv_hi"])) for a in n]
        return dict(nq=n, kv=kv)
    N = case["N"]
    cuts = sorted(rng.sample(range(1, B), N - 1)) if N > 1 else []
    start = [0] + cuts + [B]
    plen = [rng.randint(case["p_lo"], case["p_hi"]) for _ in range(N)]
    live = [rng.randint(case["live_lo"], case["live_hi"]) for _ in range(B)]
    return dict(start=start, plen=plen, live=live)


def _starts(n):
    s = [0]
    for x in n:
        s.append(s[-1] + x)
    return s


def _pairs(nq, kv, window, sinks):
    """(visible query-key pairs, cache rows some query sees) of one sequence."""
    pairs = 0
    for p in range(kv - nq, kv):
        if window == 0 or p + 1 <= window:
            pairs += p + 1
        else:
            pairs += window + min(sinks, p + 1 - window)
    if nq == 0:
        return 0, 0
    lo = 0 if window == 0 else max(0, kv - nq - window + 1)
    return pairs, kv - lo + min(sinks, lo)


def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["kind"] == "norm_rope":
        n = case["T"] * (Hq + 2 * Hkv) * d
        return {"bytes": 4 * n + 4 * case["T"], "flops": 8 * n}
    lay = _layout(case)
    if case["kind"] == "append":
        n = sum(lay["nq"]) * (Hq + 2 * Hkv) * d
        return {"bytes": 4 * n + 4 * Hkv * sum(lay["kv"]), "flops": 8 * n}
    if case["kind"] == "window":
        got = [_pairs(a, b, case["window"], case["sinks"]) for a, b in zip(lay["nq"], lay["kv"])]
        return {"bytes": 4 * sum(lay["nq"]) * Hq * d + 4 * Hkv * d * sum(x[1] for x in got),
                "flops": 4 * d * Hq * sum(x[0] for x in got)}
    keys = sum(lay["live"])
    seen = 0
    for i, p in enumerate(lay["plen"]):
        keys += p * (lay["start"][i + 1] - lay["start"][i])
        seen += p
    return {"bytes": 4 * Hkv * d * (seen + sum(lay["live"])) + 4 * case["B"] * Hq * d
            + 4 * case["B"] * Hkv * case["S"], "flops": 4 * d * Hq * keys}


# ------------------------------------------------------------------ inputs --

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(BF)


def _keys(gen, *shape):
    """K rows with lognormal(0, 0.5) norms, as attention sees them: some keys stand out."""
    out = torch.empty(shape, dtype=BF, device=DEV)
    for i in range(shape[0]):
        x = torch.randn(shape[1:], generator=gen, device=DEV)
        f = torch.randn(shape[1:-1] + (1,), generator=gen, device=DEV)
        out[i] = (x * torch.exp(0.5 * f)).to(BF)
    return out


def _int(x):
    return torch.tensor(x, dtype=torch.int32).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    st = {"case": case}
    if case["kind"] in ("norm_rope", "append"):
        rot = case["rot"]
        lay = None if case["kind"] == "norm_rope" else _layout(case)
        T = case["T"] if lay is None else sum(lay["nq"])
        st["qkv"] = _normal(gen, T, Hq + 2 * Hkv, d)
        w = lambda: (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(BF) if case["norm"] else None
        st["wq"], st["wk"] = w(), w()
        e = torch.arange(rot // 2, dtype=torch.float64) * (-2.0 / rot)
        st["freq"] = (ROPE_BASE ** e).float().to(DEV)
        st["q"] = torch.zeros((T, Hq, d), dtype=BF, device=DEV)
        if lay is None:
            st["pos"] = torch.randint(0, case["far"], (T,), generator=gen, device=DEV,
                                      dtype=torch.int32)
            st["k"] = torch.zeros((T, Hkv, d), dtype=BF, device=DEV)
            st["v"] = torch.zeros((T, Hkv, d), dtype=BF, device=DEV)
            return st
        B, S = case["B"], case["S"]
        st["lay"] = lay
        st["start"], st["kv"] = _int(_starts(lay["nq"])), _int(lay["kv"])
        st["offset"] = _int([case["offset"]] * B) if case["offset"] else None
        st["k"] = _normal(gen, B, Hkv, S, d)
        st["v"] = _normal(gen, B, Hkv, S, d)
        st["mask"] = torch.full((B, Hkv, S), -1, dtype=torch.int32, device=DEV)
        for b in range(B):
            past = lay["kv"][b] - lay["nq"][b]
            st["mask"][b, :, :past] = torch.arange(past - 1, -1, -1, dtype=torch.int32, device=DEV)
        return st
    lay = st["lay"] = _layout(case)
    B, S = case["B"], case["S"]
    st["scale"] = 1.0 / math.sqrt(d)
    st["k"] = _keys(gen, B, Hkv, S, d)
    st["v"] = torch.empty_like(st["k"])
    for b in range(B):
        st["v"][b] = _normal(gen, Hkv, S, d)
    if case["kind"] == "window":
        T = sum(lay["nq"])
        st["q"] = _normal(gen, T, Hq, d)
        st["start"], st["kv"] = _int(_starts(lay["nq"])), _int(lay["kv"])
        st["out"] = torch.zeros((T, Hq, d), dtype=BF, device=DEV)
        return st
    N, P = case["N"], case["P"]
    st["q"] = _normal(gen, B, Hq, d)
    st["kp"], st["vp"] = _keys(gen, N, Hkv, P, d), _normal(gen, N, Hkv, P, d)
    st["start"], st["plen"] = _int(lay["start"]), _int(lay["plen"])
    # Ages of an in-order fill, with a few slots emptied by an earlier eviction.
    j = torch.arange(S, device=DEV, dtype=torch.int32)
    live = _int(lay["live"])[:, None, None]
    mask = torch.where(j < live, live - 1 - j, -1).expand(B, Hkv, S).clone()
    holes = torch.rand((B, Hkv, S), generator=gen, device=DEV) < 0.02
    st["mask"] = torch.where(holes, -1, mask).to(torch.int32).contiguous()
    st["nk"], st["nv"] = _normal(gen, B, Hkv, d), _normal(gen, B, Hkv, d)
    ws = torch.randint(0, S, (B, Hkv), generator=gen, device=DEV, dtype=torch.int32)
    st["ws"] = ws if case["write"] else torch.full_like(ws, -1)
    st["out"] = torch.zeros((B, Hq, d), dtype=BF, device=DEV)
    return st


# --------------------------------------------------------------------- run --

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import decode_kv_cache_step_gb300 as lf

    case = st["case"]
    if case["kind"] == "norm_rope":
        lf.qk_norm_rope(st["qkv"], st["wq"], st["wk"], st["freq"], st["pos"], st["q"], st["k"],
                        st["v"], EPS, interleaved=case["inter"])
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    if case["kind"] == "append":
        lf.prefill_append(st["qkv"], st["wq"], st["wk"], st["freq"], st["start"], st["kv"], st["q"],
                          st["k"], st["v"], st["mask"], EPS, interleaved=case["inter"],
                          pos_offset=st["offset"])
        return {"q": st["q"], "k": st["k"], "v": st["v"], "mask": st["mask"]}
    if case["kind"] == "window":
        lf.window_attention(st["q"], st["k"], st["v"], st["start"], st["kv"], st["out"],
                            case["window"], case["sinks"], st["scale"])
        return st["out"]
    lf.decode_attention_prefix(st["q"], st["k"], st["v"], st["mask"], st["nk"], st["nv"], st["ws"],
                               st["kp"], st["vp"], st["start"], st["plen"], st["out"], st["scale"])
    return _prefix_result(st)


def _prefix_result(st):
    if st["case"]["write"]:
        return {"out": st["out"], "k": st["k"], "v": st["v"], "mask": st["mask"]}
    return st["out"]


def _norm_rotate(x, w, freq, pos, inter):
    """[T, H, d] heads, normalised and rotated, in 32 bits (angles in 64)."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a = pos.double()[:, None] * freq.double()
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    r = freq.numel()
    y = x.clone()
    if inter:
        x1, x2 = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        y[..., 0:2 * r:2] = x1 * cos - x2 * sin
        y[..., 1:2 * r:2] = x2 * cos + x1 * sin
    else:
        x1, x2 = x[..., :r], x[..., r:2 * r]
        y[..., :r] = x1 * cos - x2 * sin
        y[..., r:2 * r] = x2 * cos + x1 * sin
    return y.to(BF)


def _run_plain(st):
    case = st["case"]
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    g = Hq // Hkv
    if case["kind"] == "norm_rope":
        x = st["qkv"]
        st["q"].copy_(_norm_rotate(x[:, :Hq], st["wq"], st["freq"], st["pos"], case["inter"]))
        st["k"].copy_(_norm_rotate(x[:, Hq:Hq + Hkv], st["wk"], st["freq"], st["pos"], case["inter"]))
        st["v"].copy_(x[:, Hq + Hkv:])
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    lay = st["lay"]
    if case["kind"] == "append":
        at = _starts(lay["nq"])
        for b in range(case["B"]):
            n, kv = lay["nq"][b], lay["kv"][b]
            x = st["qkv"][at[b]:at[b + 1]]
            pos = torch.arange(kv - n, kv, device=DEV) + case["offset"]
            st["q"][at[b]:at[b + 1]] = _norm_rotate(x[:, :Hq], st["wq"], st["freq"], pos, case["inter"])
            k = _norm_rotate(x[:, Hq:Hq + Hkv], st["wk"], st["freq"], pos, case["inter"])
            st["k"][b, :, kv - n:kv] = k.transpose(0, 1)
            st["v"][b, :, kv - n:kv] = x[:, Hq + Hkv:].transpose(0, 1)
            st["mask"][b, :, :kv] = torch.arange(kv - 1, -1, -1, device=DEV, dtype=torch.int32)
        return {"q": st["q"], "k": st["k"], "v": st["v"], "mask": st["mask"]}
    if case["kind"] == "window":
        at = _starts(lay["nq"])
        w, sinks = case["window"], case["sinks"]
        for b in range(case["B"]):
            n, kv = lay["nq"][b], lay["kv"][b]
            step = max(1, (1 << 28) // max(1, Hq * kv))
            for i in range(0, n, step):
                m = min(step, n - i)
                first, end = kv - n + i, kv - n + i + m
                lo = 0 if w == 0 else max(0, first - w + 1)
                pre = min(sinks, lo)
                kk = torch.cat([st["k"][b, :, :pre], st["k"][b, :, lo:end]], 1).float()
                vv = torch.cat([st["v"][b, :, :pre], st["v"][b, :, lo:end]], 1).float()
                j = torch.cat([torch.arange(pre, device=DEV), torch.arange(lo, end, device=DEV)])
                pos = torch.arange(first, end, device=DEV)[:, None]
                see = j <= pos
                if w:
                    see &= (pos - j < w) | (j < sinks)
                q = st["q"][at[b] + i:at[b] + i + m].float().view(m, Hkv, g, d)
                q = q.permute(1, 2, 0, 3).reshape(Hkv, g * m, d)
                s = (q @ kk.transpose(1, 2) * st["scale"]).view(Hkv, g, m, -1)
                s.masked_fill_(~see, -math.inf)
                p = torch.exp(s - s.amax(-1, keepdim=True))
                o = (p.view(Hkv, g * m, -1) @ vv).view(Hkv, g, m, d) / p.sum(-1, keepdim=True)
                st["out"][at[b] + i:at[b] + i + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, d).to(BF)
        return st["out"]
    S = case["S"]
    if case["write"]:
        at = st["ws"].long()[..., None]
        row = at[..., None].expand(-1, -1, 1, d)
        st["k"].scatter_(2, row, st["nk"][:, :, None])
        st["v"].scatter_(2, row, st["nv"][:, :, None])
        age = st["mask"].gather(2, at)
        st["mask"].scatter_(2, at, age.clamp(min=0))
    for n in range(case["N"]):
        P = lay["plen"][n]
        kp, vp = st["kp"][n, :, :P].float(), st["vp"][n, :, :P].float()
        step = max(1, (1 << 28) // (Hkv * S * d + Hq * P))
        for b0 in range(lay["start"][n], lay["start"][n + 1], step):
            b1 = min(b0 + step, lay["start"][n + 1])
            m = b1 - b0
            q = st["q"][b0:b1].float().view(m, Hkv, g, d)
            own_s = q @ st["k"][b0:b1].float().transpose(2, 3) * st["scale"]
            own_s.masked_fill_(st["mask"][b0:b1, :, None] < 0, -math.inf)
            qp = q.transpose(0, 1).reshape(Hkv, m * g, d)
            pre_s = (qp @ kp.transpose(1, 2) * st["scale"]).view(Hkv, m, g, P).transpose(0, 1)
            s = torch.cat([pre_s, own_s], -1)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            l = p.sum(-1, keepdim=True)
            pp = p[..., :P].transpose(0, 1).reshape(Hkv, m * g, P)
            o = (pp @ vp).view(Hkv, m, g, d).transpose(0, 1)
            v = torch.where(st["mask"][b0:b1, :, :, None] < 0, 0.0, st["v"][b0:b1].float())
            o = (o + p[..., P:] @ v) / torch.where(l == 0, 1.0, l)
            st["out"][b0:b1] = o.reshape(m, Hq, d).to(BF)
    return _prefix_result(st)


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The definitions in 64 bits, on the inputs of ``prepare(case, seed)``."""
    st = prepare(case, seed)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    g = Hq // Hkv
    f64 = torch.float64

    def turn(x, w, pos):
        x = x.to(f64)
        if w is not None:
            x = x * w.to(f64) / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + EPS)
        r = case["rot"] // 2
        first = torch.arange(r, device=DEV) * (2 if case["inter"] else 1)
        second = first + (1 if case["inter"] else r)
        unit = torch.polar(torch.ones((), dtype=f64, device=DEV),
                           torch.outer(pos.to(f64), st["freq"].to(f64)))
        z = torch.complex(x[..., first], x[..., second]) * unit[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    if case["kind"] == "norm_rope":
        q, k, v = st["qkv"].split([Hq, Hkv, Hkv], 1)
        return {"q": turn(q, st["wq"], st["pos"]), "k": turn(k, st["wk"], st["pos"]), "v": v.to(f64)}
    lay = st["lay"]
    if case["kind"] == "append":
        kc, vc, mask = st["k"].to(f64), st["v"].to(f64), st["mask"].clone()
        pos = torch.cat([torch.arange(c - n, c, device=DEV) for n, c in zip(lay["nq"], lay["kv"])])
        q, k, v = st["qkv"].split([Hq, Hkv, Hkv], 1)
        k = turn(k, st["wk"], pos + case["offset"])
        t = 0
        for b, (n, c) in enumerate(zip(lay["nq"], lay["kv"])):
            for h in range(Hkv):
                kc[b, h, c - n:c] = k[t:t + n, h]
                vc[b, h, c - n:c] = v[t:t + n, h].to(f64)
                mask[b, h, :c] = c - 1 - torch.arange(c, device=DEV, dtype=torch.int32)
            t += n
        return {"q": turn(q, st["wq"], pos + case["offset"]), "k": kc, "v": vc, "mask": mask}
    if case["kind"] == "window":
        out = torch.zeros(st["out"].shape, dtype=f64, device=DEV)
        t = 0
        w, sinks = case["window"], case["sinks"]
        for n, kv, b in zip(lay["nq"], lay["kv"], range(case["B"])):
            step = max(1, (1 << 27) // max(1, g * kv))
            for i in range(0, n, step):
                m = min(step, n - i)
                end = kv - n + i + m
                lo = max(0, end - m - w + 1) if w else 0
                keep = torch.arange(end, device=DEV)
                keep = keep[(keep >= lo) | (keep < sinks)]
                p = torch.arange(end - m, end, device=DEV)[:, None]
                hide = keep > p
                if w:
                    hide |= (keep <= p - w) & (keep >= sinks)
                for h in range(Hkv):
                    k, v = st["k"][b, h, keep].to(f64), st["v"][b, h, keep].to(f64)
                    for e in range(h * g, h * g + g):
                        s = st["scale"] * (st["q"][t + i:t + i + m, e].to(f64) @ k.T)
                        s[hide] = -math.inf
                        out[t + i:t + i + m, e] = torch.softmax(s, -1) @ v
            t += n
        return out
    kc, vc, mask = st["k"], st["v"], st["mask"]
    out = torch.zeros(st["out"].shape, dtype=f64, device=DEV)
    ws = st["ws"].tolist()
    for n in range(case["N"]):
        P = lay["plen"][n]
        for b in range(lay["start"][n], lay["start"][n + 1]):
            for h in range(Hkv):
                if ws[b][h] >= 0:
                    kc[b, h, ws[b][h]], vc[b, h, ws[b][h]] = st["nk"][b, h], st["nv"][b, h]
                    if mask[b, h, ws[b][h]] < 0:
                        mask[b, h, ws[b][h]] = 0
                live = mask[b, h] >= 0
                k = torch.cat([st["kp"][n, h, :P], kc[b, h][live]]).to(f64)
                v = torch.cat([st["vp"][n, h, :P], vc[b, h][live]]).to(f64)
                if k.shape[0]:
                    s = st["scale"] * (st["q"][b, h * g:h * g + g].to(f64) @ k.T)
                    out[b, h * g:h * g + g] = torch.softmax(s, -1) @ v
    if not case["write"]:
        return out
    return {"out": out, "k": kc.to(f64), "v": vc.to(f64), "mask": mask}
