"""Measured cases of what a long prompt brings to the decode step.

Three operators, each for prompts and for single tokens:

* head norms with a rotation whose positions have several axes ("axes"):
  tokens of images and video, single and into the caches;
* eviction by accumulated attention weight: the weights that a prompt's last
  rows give its keys ("prompt_weights") and the decode step that adds the
  current token's weights and returns the slots with the least ("weights");
* a cache held in 4 bits: a prompt's keys and values into it and back
  ("kv4_prompt"), and decode attention over it ("kv4_decode").

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
GROUP = 32      # values of a row that share a scale in 4 bits
K_PIECE = 8     # consecutive values of a group that lie together in a row of 4-bit keys
V_PIECE = 4     # and of values


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One text token behind an image, 32 query and 8 KV heads: the latency of a decode layer's first call.
        dict(name="axes_b1", kind="axes", T=1, Hq=32, Hkv=8, d=128, rot=128, inter=False, norm=True,
             far=16384, n_h=24, n_w=24, turn=False),
        # Image and text prompts of a batch of 32 into caches of 2400 slots, the axes taking turns over the pairs.
        dict(name="axes_append_b32", kind="axes_append", B=32, Hq=32, Hkv=8, d=128, S=2400, rot=128,
             inter=False, norm=True, far=2400, n_h=20, n_w=20, turn=True, q_lo=100, q_hi=1300,
             past=200, lens=1),
        # One sequence of a small model with a full 2400-slot cache: latency.
        dict(name="weights_b1_s2400", kind="weights", B=1, Hq=32, Hkv=8, d=128, S=2400, live_lo=2400,
             live_hi=2400, W=32, decay=1.0, k=1, fill=False, write=True, lens=2),
        # A decode batch of 128 over full caches of 3200 slots: memory bound, the largest cache.
        dict(name="weights_b128_s3200", kind="weights", B=128, Hq=32, Hkv=8, d=128, S=3200,
             live_lo=3200, live_hi=3200, W=32, decay=1.0, k=1, fill=False, write=False, lens=3),
        # Ragged long caches, groups of 8 heads, fading weights, four slots at once.
        dict(name="weights_b9_s9001", kind="weights", B=9, Hq=16, Hkv=2, d=64, S=9001, live_lo=1000,
             live_hi=9001, W=64, decay=0.97, k=4, fill=False, write=False, lens=4),
        # The last 32 rows of a batch of long prompts: which keys a budget keeps.
        dict(name="prompt_weights_last32", kind="prompt_weights", B=8, Hq=32, Hkv=8, d=128, S=8192,
             q_lo=2000, q_hi=8192, past=0, rows=32, lens=5),
        # Every row of one prompt of 8192 tokens: compute bound, the largest.
        dict(name="prompt_weights_8k", kind="prompt_weights", B=1, Hq=32, Hkv=8, d=128, S=8192,
             q_lo=8192, q_hi=8192, past=0, rows=0, lens=6),
        # Ragged prompts of a batch of 32 into the 4-bit cache and back for the next chunk's attention.
        dict(name="kv4_prompt_b32_s2400", kind="kv4_prompt", B=32, Hkv=8, d=128, P=2400, S=2400,
             lo=0, hi=2400, lens=7),
        # The newest chunk of five prompts, odd buffers, head dim 64.
        dict(name="kv4_prompt_chunk_d64", kind="kv4_prompt", B=5, Hkv=2, d=64, P=1001, S=1501,
             lo=600, hi=1001, lens=8),
        # One sequence's next token over 16384 keys in 4 bits: latency.
        dict(name="kv4_decode_b1_s16384", kind="kv4_decode", B=1, Hq=32, Hkv=8, d=128, S=16384,
             live_lo=16384, live_hi=16384, write=False, lens=9),
        # The token's write too, into the small cache of a small model, read back as a whole.
        dict(name="kv4_decode_write_d64", kind="kv4_decode", B=4, Hq=4, Hkv=2, d=64, S=256,
             live_lo=1, live_hi=240, write=True, lens=10),
        # A ragged decode batch over long caches, memory bound.
        dict(name="kv4_decode_b64_s16384", kind="kv4_decode", B=64, Hq=32, Hkv=8, d=128, S=16384,
             live_lo=4096, live_hi=16384, write=False, lens=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    kind = rng.choice(["axes", "axes_append", "weights", "weights", "prompt_weights",
                       "prompt_weights", "kv4_prompt", "kv4_decode", "kv4_decode"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq, d = Hkv * rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    lens = rng.randrange(1 << 30)
    if kind in ("axes", "axes_append"):
        rot = 16 * rng.randint(1, d // 16)
        n_h = rng.randint(0, rot // 6)
        c = dict(kind=kind, Hq=Hq, Hkv=Hkv, d=d, rot=rot, inter=rng.random() < 0.5,
                 norm=rng.random() < 0.7, far=_log(rng, 100, 1000000), n_h=n_h,
                 n_w=rng.randint(0, n_h) if rng.random() < 0.5 else n_h, turn=rng.random() < 0.5)
        if kind == "axes":
            return dict(c, T=_log(rng, 1, 4096))
        S = _log(rng, 64, 8192)
        past = rng.choice([0, rng.randint(0, S // 2)])
        hi = rng.randint(1, S - past)
        return dict(c, B=_log(rng, 1, max(1, min(64, 65536 // S))), S=S, q_lo=rng.randint(0, hi),
                    q_hi=hi, past=past, lens=lens)
    if kind == "weights":
        S = _log(rng, 64, 16384)
        live = rng.randint(0, S)
        B = _log(rng, 1, max(1, min(128, 200000 // S)))
        return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, S=S, live_lo=live, live_hi=rng.randint(live, S),
                    W=rng.choice([0, 1, 32, rng.randint(0, S)]), decay=rng.choice([1.0, 1.0, 0.9, 0.0]),
                    k=rng.choice([1, 1, 1, rng.randint(2, 16)]), fill=rng.random() < 0.3,
                    write=B * S * Hkv * d < (1 << 24), lens=lens)
    if kind == "prompt_weights":
        S = _log(rng, 16, 8192)
        past = rng.choice([0, rng.randint(0, S // 2)])
        hi = rng.randint(1, S - past)
        rows = rng.choice([0, 0, rng.randint(1, 128), 32])
        most = (1 << 31) // (Hq * S * (min(rows, hi) if rows else hi))
        return dict(kind=kind, B=_log(rng, 1, max(1, min(64, most))), Hq=Hq, Hkv=Hkv, d=d, S=S,
                    q_lo=rng.randint(0, hi), q_hi=hi, past=past, rows=rows, lens=lens)
    if kind == "kv4_prompt":
        P = _log(rng, 64, 16384)
        lo = rng.randint(0, P)
        return dict(kind=kind, B=_log(rng, 1, max(1, min(64, 76800 // P))), Hkv=Hkv, d=d, P=P,
                    S=P + rng.choice([0, rng.randint(0, 1000)]), lo=lo, hi=rng.randint(lo, P), lens=lens)
    S = _log(rng, 64, 65536)
    B = _log(rng, 1, max(1, min(128, 1000000 // S)))
    live = rng.randint(0, S)
    return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, d=d, S=S, live_lo=live, live_hi=rng.randint(live, S),
                write=B * S * Hkv * d < (1 << 22), lens=lens)


# ----------------------------------------------------------- ragged lengths --

def _layout(case):
    """Host-side lengths of a ragged case; the same for every input seed."""
    rng = random.Random(case["lens"])
    B = case["B"]
    if case["kind"] in ("axes_append", "prompt_weights"):
        nq = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(B)]
        past = [rng.randint(0, case["past"]) for _ in range(B)]
        return dict(nq=nq, kv=[a + b for a, b in zip(nq, past)])
    if case["kind"] == "kv4_prompt":
        first = [rng.randint(0, case["lo"]) for _ in range(B)]
        return dict(first=first, kv=[rng.randint(max(a, case["lo"]), case["hi"]) for a in first])
    return dict(live=[rng.randint(case["live_lo"], case["live_hi"]) for _ in range(B)])


def _pair_axis(case):
    """The axis (0 time, 1 height, 2 width) of each rotated pair: in sections, or taking turns
    from the first pairs on while an axis has any left."""
    half, n_h, n_w = case["rot"] // 2, case["n_h"], case["n_w"]
    if case["turn"]:
        return [1 if i % 3 == 1 and i < 3 * n_h else 2 if i % 3 == 2 and i < 3 * n_w else 0
                for i in range(half)]
    return [0] * (half - n_h - n_w) + [1] * n_h + [2] * n_w


def _rows(case, n):
    return min(n, case["rows"]) if case["rows"] else n


def work(case):
    kind, Hkv, d = case["kind"], case["Hkv"], case["d"]
    if kind == "axes":
        n = case["T"] * (case["Hq"] + 2 * Hkv) * d
        return {"bytes": 4 * n + 12 * case["T"], "flops": 8 * n}
    lay = _layout(case)
    if kind == "axes_append":
        n = sum(lay["nq"]) * (case["Hq"] + 2 * Hkv) * d
        return {"bytes": 4 * n + 12 * sum(lay["nq"]) + 4 * Hkv * sum(lay["kv"]), "flops": 8 * n}
    if kind == "prompt_weights":
        rows = [_rows(case, n) for n in lay["nq"]]
        pairs = sum(r * kv - r * (r - 1) // 2 for r, kv in zip(rows, lay["kv"]))
        old = sum(kv - n for n, kv in zip(lay["nq"], lay["kv"]))
        return {"bytes": 2 * d * case["Hq"] * sum(rows) + Hkv * (2 * d * sum(lay["kv"])
                + 4 * sum(lay["kv"]) + 4 * old), "flops": 2 * d * case["Hq"] * pairs}
    if kind == "kv4_prompt":
        n = Hkv * sum(b - a for a, b in zip(lay["first"], lay["kv"]))
        four = d + d // GROUP * 4  # codes and scales of a key and its value
        return {"bytes": n * (8 * d + 2 * four) + 4 * Hkv * sum(lay["kv"]), "flops": 6 * n * d}
    live, slots = Hkv * sum(lay["live"]), case["B"] * Hkv * case["S"]
    qo = 4 * case["B"] * case["Hq"] * d
    flops = 4 * d * case["Hq"] * sum(lay["live"])
    if kind == "weights":
        return {"bytes": live * (4 * d + 8) + slots * (8 if case["write"] else 4) + qo, "flops": flops}
    n = live * (d + d // GROUP * 4) + 4 * slots + qo
    if case["write"]:  # the cache read back
        n += slots * (d + d // GROUP * 4 + 4 * d)
    return {"bytes": n, "flops": flops}


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


def _values(gen, *shape):
    out = torch.empty(shape, dtype=BF, device=DEV)
    for i in range(shape[0]):
        out[i] = _normal(gen, *shape[1:])
    return out


def _int(x):
    return torch.tensor(x, dtype=torch.int32).to(DEV)


def _ages(gen, case, lay):
    """Ages of an in-order fill, with a few slots emptied by an earlier eviction."""
    B, Hkv, S = case["B"], case["Hkv"], case["S"]
    j = torch.arange(S, device=DEV, dtype=torch.int32)
    live = _int(lay["live"])[:, None, None]
    mask = torch.where(j < live, live - 1 - j, -1).expand(B, Hkv, S)
    holes = torch.rand((B, Hkv, S), generator=gen, device=DEV) < 0.02
    return torch.where(holes, -1, mask).to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    kind, Hkv, d = case["kind"], case["Hkv"], case["d"]
    Hq = case.get("Hq", Hkv)
    st = {"case": case, "scale": 1.0 / math.sqrt(d)}
    lay = st["lay"] = None if kind == "axes" else _layout(case)
    if kind in ("axes", "axes_append"):
        rot = case["rot"]
        T = case["T"] if lay is None else sum(lay["nq"])
        st["qkv"] = _normal(gen, T, Hq + 2 * Hkv, d)
        w = lambda: (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(BF) if case["norm"] else None
        st["wq"], st["wk"] = w(), w()
        e = torch.arange(rot // 2, dtype=torch.float64) * (-2.0 / rot)
        st["freq"] = (ROPE_BASE ** e).float().to(DEV)
        st["axis"] = _pair_axis(case)
        # Text runs on all axes alike; an image's patches spread over height and width.
        st["pos"] = torch.randint(0, case["far"], (3, T), generator=gen, device=DEV, dtype=torch.int32)
        st["q"] = torch.zeros((T, Hq, d), dtype=BF, device=DEV)
        if lay is None:
            st["k"] = torch.zeros((T, Hkv, d), dtype=BF, device=DEV)
            st["v"] = torch.zeros((T, Hkv, d), dtype=BF, device=DEV)
            return st
        B, S = case["B"], case["S"]
        st["k"], st["v"] = _values(gen, B, Hkv, S, d), _values(gen, B, Hkv, S, d)
        j = torch.arange(S, device=DEV, dtype=torch.int32)
        past = _int([b - a for a, b in zip(lay["nq"], lay["kv"])])[:, None, None]
        st["mask"] = torch.where(j < past, past - 1 - j, -1).expand(B, Hkv, S).to(torch.int32).contiguous()
    if kind in ("axes_append", "prompt_weights"):
        st["start"] = _int([sum(lay["nq"][:b]) for b in range(case["B"] + 1)])
        st["kv"] = _int(lay["kv"])
    if kind == "prompt_weights":
        B, S = case["B"], case["S"]
        st["q"] = _normal(gen, sum(lay["nq"]) or 1, Hq, d)
        st["k"] = _keys(gen, B, Hkv, S, d)
        st["weights"] = torch.rand((B, Hkv, S), generator=gen, device=DEV)
    if kind == "kv4_prompt":
        B, P, S = case["B"], case["P"], case["S"]
        st["k"], st["v"] = _keys(gen, B, Hkv, P, d), _values(gen, B, Hkv, P, d)
        st["first"], st["kv"] = _int(lay["first"]), _int(lay["kv"])
        st["k4"], st["ks"] = _empty4(B, Hkv, S, d)
        st["v4"], st["vs"] = _empty4(B, Hkv, S, d)
        st["mask"] = torch.full((B, Hkv, S), -1, dtype=torch.int32, device=DEV)
        st["k2"], st["v2"] = torch.zeros_like(st["k"]), torch.zeros_like(st["v"])
    if kind in ("weights", "kv4_decode"):
        B, S = case["B"], case["S"]
        k, v = _keys(gen, B, Hkv, S, d), _values(gen, B, Hkv, S, d)
        st["q"] = _normal(gen, B, Hq, d)
        st["mask"] = _ages(gen, case, lay)
        st["nk"], st["nv"] = _normal(gen, B, Hkv, d), _normal(gen, B, Hkv, d)
        ws = torch.randint(0, S, (B, Hkv), generator=gen, device=DEV, dtype=torch.int32)
        st["ws"] = ws if case["write"] else torch.full_like(ws, -1)
        st["out"] = torch.zeros((B, Hq, d), dtype=BF, device=DEV)
        if kind == "weights":
            st["k"], st["v"] = k, v
            # What some hundreds of tokens have left: a few keys hold most of the weight.
            st["weights"] = 0.2 * torch.exp(torch.randn((B, Hkv, S), generator=gen, device=DEV))
            st["next"] = torch.zeros((B, Hkv, case["k"]), dtype=torch.int32, device=DEV)
        else:
            st["k4"], st["ks"] = _empty4(B, Hkv, S, d)
            st["v4"], st["vs"] = _empty4(B, Hkv, S, d)
            for b in range(B):
                code, st["ks"][b] = _quantise(k[b])
                st["k4"][b] = _lay(code, K_PIECE)
                code, st["vs"][b] = _quantise(v[b])
                st["v4"][b] = _lay(code, V_PIECE)
            if case["write"]:
                st["k2"], st["v2"] = torch.zeros_like(k), torch.zeros_like(v)
                st["zero"], st["all"] = _int([0] * B), _int([S] * B)
    return st


# --------------------------------------------------------------------- run --

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import decode_kv_cache_step_gb300 as lf

    case = st["case"]
    if case["kind"] == "axes":
        lf.qk_norm_rope_axes(st["qkv"], st["wq"], st["wk"], st["freq"], st["pos"], st["axis"],
                             st["q"], st["k"], st["v"], EPS, interleaved=case["inter"])
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    if case["kind"] == "axes_append":
        lf.prefill_append_axes(st["qkv"], st["wq"], st["wk"], st["freq"], st["start"], st["kv"],
                               st["pos"], st["axis"], st["q"], st["k"], st["v"], st["mask"], EPS,
                               interleaved=case["inter"])
        return {"q": st["q"], "k": st["k"], "v": st["v"], "mask": st["mask"]}
    if case["kind"] == "prompt_weights":
        lf.prompt_weights(st["q"], st["k"], st["start"], st["kv"], st["weights"], st["scale"],
                          rows=case["rows"])
        return st["weights"]
    if case["kind"] == "weights":
        lf.decode_step_weights(st["q"], st["k"], st["v"], st["mask"], st["weights"], st["nk"],
                               st["nv"], st["ws"], st["out"], st["next"], case["W"], st["scale"],
                               decay=case["decay"], k=case["k"],
                               flags=lf.LF_STEP_FILL_EMPTY_FIRST if case["fill"] else 0)
        return _weights_result(st)
    if case["kind"] == "kv4_prompt":
        lf.kv4_pack(st["k"], st["v"], st["first"], st["kv"], st["k4"], st["ks"], st["v4"], st["vs"],
                    st["mask"])
        lf.kv4_unpack(st["k4"], st["ks"], st["v4"], st["vs"], st["first"], st["kv"], st["k2"], st["v2"])
        return {"k": st["k2"], "v": st["v2"], "mask": st["mask"]}
    lf.decode_attention_kv4(st["q"], st["k4"], st["ks"], st["v4"], st["vs"], st["mask"], st["nk"],
                            st["nv"], st["ws"], st["out"], st["scale"])
    if not case["write"]:
        return st["out"]
    lf.kv4_unpack(st["k4"], st["ks"], st["v4"], st["vs"], st["zero"], st["all"], st["k2"], st["v2"])
    return {"out": st["out"], "k": st["k2"], "v": st["v2"], "mask": st["mask"]}


def _weights_result(st):
    got = {"out": st["out"], "weights": st["weights"], "next": st["next"]}
    if st["case"]["write"]:
        got.update(k=st["k"], v=st["v"], mask=st["mask"])
    return got


def _norm_rotate(x, w, freq, pos, axis, inter):
    """[T, H, d] heads, normalised and rotated, in 32 bits (angles in 64)."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    a = pos[axis].double().T * freq.double()
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


def _empty4(B, Hkv, S, d):
    return (torch.zeros((B, Hkv, S, d // 2), dtype=torch.uint8, device=DEV),
            torch.zeros((B, Hkv, S, d // GROUP), dtype=BF, device=DEV))


def _quantise(x):
    """Codes (-7 .. 7) and scales of rows of bf16: a scale is the group's largest magnitude over 7."""
    x = x.float()
    g = x.view(x.shape[:-1] + (-1, GROUP))
    s = (g.abs().amax(-1) / 7).to(BF)
    code = torch.round(g / s.float()[..., None]).clamp(-7, 7)
    return torch.where(s[..., None] == 0, 0.0, code).view(x.shape), s


def _lay(code, piece):
    """The bytes of rows of codes: pieces of the groups in turn, two codes (plus 8) a byte."""
    d = code.shape[-1]
    u = (code + 8).to(torch.uint8).view(code.shape[:-1] + (d // GROUP, GROUP // piece, piece))
    u = u.transpose(-3, -2).reshape(code.shape)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _stand_for(byte, scale, piece):
    """The values of rows of bytes and scales, in 32 bits."""
    u = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).float() - 8
    d = u.shape[-1]
    u = u.view(u.shape[:-1] + (GROUP // piece, d // GROUP, piece)).transpose(-3, -2)
    return (u.reshape(byte.shape[:-1] + (d // GROUP, GROUP)) * scale.float()[..., None]).flatten(-2)


def _attend(q, k, v, live, scale):
    """Outputs and weights of queries [B, Hkv, g, d] over the live keys, in 32 bits."""
    s = (q @ k.transpose(2, 3) * scale).masked_fill(~live[:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l == 0, 1.0, l)
    return p @ v, p


def _run_plain(st):
    case = st["case"]
    kind, Hkv, d = case["kind"], case["Hkv"], case["d"]
    if kind in ("axes", "axes_append"):
        Hq, x = case["Hq"], st["qkv"]
        st["q"].copy_(_norm_rotate(x[:, :Hq], st["wq"], st["freq"], st["pos"], st["axis"], case["inter"]))
        k = _norm_rotate(x[:, Hq:Hq + Hkv], st["wk"], st["freq"], st["pos"], st["axis"], case["inter"])
        if kind == "axes":
            st["k"].copy_(k)
            st["v"].copy_(x[:, Hq + Hkv:])
            return {"q": st["q"], "k": st["k"], "v": st["v"]}
        t = torch.arange(x.shape[0], device=DEV)
        b = torch.searchsorted(st["start"], t, right=True) - 1
        slot = (st["kv"][b] - st["start"][b + 1]).long() + t
        st["k"][b, :, slot] = k
        st["v"][b, :, slot] = x[:, Hq + Hkv:]
        age = st["kv"][:, None, None] - 1 - torch.arange(case["S"], device=DEV, dtype=torch.int32)
        st["mask"].copy_(torch.where(age >= 0, age, st["mask"]))
        return {"q": st["q"], "k": st["k"], "v": st["v"], "mask": st["mask"]}
    if kind == "prompt_weights":
        B, Hq, S = case["B"], case["Hq"], case["S"]
        n = st["start"].diff()
        R = max(_rows(case, x) for x in st["lay"]["nq"]) or 1
        i = torch.arange(R, device=DEV)
        row = st["start"][1:, None] - 1 - i
        there = i < n[:, None]
        q = st["q"][row.clamp(min=0)].float().view(B, R, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
        s = q.reshape(B, Hkv, -1, d) @ st["k"].float().transpose(2, 3) * st["scale"]
        s = s.view(B, Hkv, -1, R, S)
        j = torch.arange(S, device=DEV)
        see = (j <= (st["kv"][:, None] - 1 - i)[..., None]) & there[..., None]
        s.masked_fill_(~see[:, None, None], -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
        l = p.sum(-1, keepdim=True)
        w = (p / torch.where(l == 0, 1.0, l)).sum((2, 3))
        old = torch.where(j < (st["kv"] - n)[:, None, None], st["weights"], 0.0)
        st["weights"].copy_(torch.where(j < st["kv"][:, None, None], old + w, st["weights"]))
        return st["weights"]
    if kind == "kv4_prompt":
        P = case["P"]
        j = torch.arange(P, device=DEV)
        inside = ((j >= st["first"][:, None]) & (j < st["kv"][:, None]))[:, None, :, None]
        (k, ks), (v, vs) = _quantise(st["k"]), _quantise(st["v"])
        k = k.view(k.shape[:-1] + (-1, GROUP)) * ks.float()[..., None]
        v = v.view(v.shape[:-1] + (-1, GROUP)) * vs.float()[..., None]
        st["k2"].copy_(torch.where(inside, k.flatten(-2).to(BF), st["k2"]))
        st["v2"].copy_(torch.where(inside, v.flatten(-2).to(BF), st["v2"]))
        age = st["kv"][:, None, None] - 1 - torch.arange(case["S"], device=DEV, dtype=torch.int32)
        st["mask"].copy_(torch.where(age >= 0, age, st["mask"]))
        return {"k": st["k2"], "v": st["v2"], "mask": st["mask"]}
    B, Hq, S = case["B"], case["Hq"], case["S"]
    ws = st["ws"].long()[..., None]
    here = torch.arange(S, device=DEV) == ws           # the written slot
    q = st["q"].float().view(B, Hkv, Hq // Hkv, d)
    if kind == "weights":
        at, write = ws.clamp(min=0)[..., None].expand(-1, -1, 1, d), (ws >= 0)[..., None]
        st["k"].scatter_(2, at, torch.where(write, st["nk"][:, :, None], st["k"].gather(2, at)))
        st["v"].scatter_(2, at, torch.where(write, st["nv"][:, :, None], st["v"].gather(2, at)))
        age = st["mask"] + ((st["mask"] >= 0) & (ws >= 0)).int()
        st["mask"].copy_(torch.where(here, 0, age))
        live = st["mask"] >= 0
        o, p = _attend(q, st["k"].float(), st["v"].float(), live, st["scale"])
        st["out"].copy_(o.view(B, Hq, d))
        w = torch.where(here, 0.0, st["weights"]) * case["decay"] + p.sum(2)
        st["weights"].copy_(torch.where(live, w, st["weights"]))
        key = torch.where(live & (st["mask"] >= case["W"]), st["weights"], math.inf)
        if case["fill"]:
            key = torch.where(live, key, -math.inf)
        key, slot = torch.sort(key, dim=-1, stable=True)
        st["next"].copy_(torch.where(key == math.inf, -1, slot)[..., :case["k"]])
        return _weights_result(st)
    st["mask"].copy_(torch.where(here & (st["mask"] < 0), 0, st["mask"]))
    k, v = _stand_for(st["k4"], st["ks"], K_PIECE), _stand_for(st["v4"], st["vs"], V_PIECE)
    if case["write"]:
        (nk, ks), (nv, vs) = _quantise(st["nk"]), _quantise(st["nv"])
        here = here[..., None]
        st["k4"].copy_(torch.where(here, _lay(nk, K_PIECE)[:, :, None], st["k4"]))
        st["v4"].copy_(torch.where(here, _lay(nv, V_PIECE)[:, :, None], st["v4"]))
        st["ks"].copy_(torch.where(here, ks[:, :, None], st["ks"]))
        st["vs"].copy_(torch.where(here, vs[:, :, None], st["vs"]))
        k, v = _stand_for(st["k4"], st["ks"], K_PIECE), _stand_for(st["v4"], st["vs"], V_PIECE)
    st["out"].copy_(_attend(q, k, v, st["mask"] >= 0, st["scale"])[0].view(B, Hq, d))
    if not case["write"]:
        return st["out"]
    st["k2"].copy_(k)
    st["v2"].copy_(v)
    return {"out": st["out"], "k": st["k2"], "v": st["v2"], "mask": st["mask"]}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    """The definitions in 64 bits, on the inputs of ``prepare(case, seed)``."""
    st = prepare(case, seed)
    kind, Hkv, d = case["kind"], case["Hkv"], case["d"]
    f64 = torch.float64

    def turn(x, w):
        x = x.to(f64)
        if w is not None:
            x = x * w.to(f64) / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + EPS)
        r = case["rot"] // 2
        first = torch.arange(r, device=DEV) * (2 if case["inter"] else 1)
        second = first + (1 if case["inter"] else r)
        angle = torch.stack([st["pos"][a].to(f64) * st["freq"][i].to(f64)
                             for i, a in enumerate(_pair_axis(case))], 1)
        z = torch.complex(x[..., first], x[..., second])
        z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
        return x

    def fours(x):
        """What rows stand for once they are in 4 bits: the nearest of 15 multiples of the scale."""
        x = x.to(f64).unflatten(-1, (-1, GROUP))
        s = (x.abs().amax(-1, keepdim=True) / 7).to(BF).to(f64)
        step = x / torch.where(s == 0, 1.0, s)
        low = torch.floor(step)
        up = (step - low > 0.5) | ((step - low == 0.5) & (low.remainder(2) == 1))
        return ((low + up).clamp(-7, 7) * s).flatten(-2)

    if kind in ("axes", "axes_append"):
        q, k, v = st["qkv"].split([case["Hq"], Hkv, Hkv], 1)
        q, k = turn(q, st["wq"]), turn(k, st["wk"])
        if kind == "axes":
            return {"q": q, "k": k, "v": v.to(f64)}
        kc, vc, mask = st["k"].to(f64), st["v"].to(f64), st["mask"].clone()
        t = 0
        for b, (n, c) in enumerate(zip(st["lay"]["nq"], st["lay"]["kv"])):
            kc[b, :, c - n:c] = k[t:t + n].transpose(0, 1)
            vc[b, :, c - n:c] = v[t:t + n].transpose(0, 1).to(f64)
            mask[b, :, :c] = torch.arange(c - 1, -1, -1, device=DEV, dtype=torch.int32)
            t += n
        return {"q": q, "k": kc, "v": vc, "mask": mask}
    if kind == "prompt_weights":
        w = st["weights"].to(f64)
        g, t = case["Hq"] // Hkv, 0
        for b, (n, c) in enumerate(zip(st["lay"]["nq"], st["lay"]["kv"])):
            w[b, :, c - n:c] = 0
            m = _rows(case, n)
            pos = torch.arange(c - m, c, device=DEV)
            hide = torch.arange(c, device=DEV) > pos[:, None]
            for h in range(Hkv if m else 0):
                k = st["k"][b, h, :c].to(f64)
                for e in range(h * g, h * g + g):
                    s = st["scale"] * (st["q"][t + n - m:t + n, e].to(f64) @ k.T)
                    s[hide] = -math.inf
                    w[b, h, :c] += torch.softmax(s, -1).sum(0)
            t += n
        return w
    if kind == "kv4_prompt":
        k, v, mask = st["k2"].to(f64), st["v2"].to(f64), st["mask"].clone()
        for b, (a, c) in enumerate(zip(st["lay"]["first"], st["lay"]["kv"])):
            k[b, :, a:c], v[b, :, a:c] = fours(st["k"][b, :, a:c]), fours(st["v"][b, :, a:c])
            mask[b, :, :c] = torch.arange(c - 1, -1, -1, device=DEV, dtype=torch.int32)
        return {"k": k, "v": v, "mask": mask}
    B, Hq, S = case["B"], case["Hq"], case["S"]
    g, mask = Hq // Hkv, st["mask"].clone()
    out = torch.zeros((B, Hq, d), dtype=f64, device=DEV)
    total = st["weights"].to(f64) if kind == "weights" else None
    chosen = torch.full((B, Hkv, case.get("k", 1)), -1, dtype=torch.int32, device=DEV)
    ks, vs = [], []
    ws = st["ws"].tolist()
    for b in range(B):
        if kind == "weights":
            k, v, nk, nv = st["k"][b].to(f64), st["v"][b].to(f64), st["nk"][b].to(f64), st["nv"][b].to(f64)
        else:
            k = _decode(st["k4"][b], st["ks"][b], K_PIECE)
            v = _decode(st["v4"][b], st["vs"][b], V_PIECE)
            nk, nv = fours(st["nk"][b]), fours(st["nv"][b])
        for h in range(Hkv):
            a = mask[b, h]
            if ws[b][h] >= 0:
                k[h, ws[b][h]], v[h, ws[b][h]] = nk[h], nv[h]
                if kind == "weights":
                    a += (a >= 0).int()
                    a[ws[b][h]] = 0
                    total[b, h, ws[b][h]] = 0
                else:
                    a[ws[b][h]].clamp_(min=0)
            live = torch.nonzero(a >= 0)[:, 0]
            if live.numel():
                s = st["scale"] * (st["q"][b, h * g:h * g + g].to(f64) @ k[h, live].T)
                p = torch.softmax(s, -1)
                out[b, h * g:h * g + g] = p @ v[h, live]
                if kind == "weights":
                    total[b, h, live] = total[b, h, live] * case["decay"] + p.sum(0)
            if kind == "weights":
                old = live[a[live] >= case["W"]]
                order = old[torch.sort(total[b, h, old], stable=True)[1]]
                if case["fill"]:
                    order = torch.cat([torch.nonzero(a < 0)[:, 0], order])
                order = order[:case["k"]]
                chosen[b, h, :order.numel()] = order.int()
        if case["write"]:
            ks.append(k)
            vs.append(v)
    if kind == "weights":
        got = {"out": out, "weights": total, "next": chosen}
        return dict(got, k=torch.stack(ks), v=torch.stack(vs), mask=mask) if case["write"] else got
    return {"out": out, "k": torch.stack(ks), "v": torch.stack(vs), "mask": mask} if case["write"] else out


def _decode(byte, scale, piece):
    """[Hkv, S, d] in 64 bits from the layout's definition, value by value of a row."""
    d = 2 * byte.shape[-1]
    c = torch.arange(d, device=DEV)
    g, r = c // GROUP, c % GROUP
    at = (r // piece * (d // GROUP) + g) * piece + r % piece
    code = (byte[..., at // 2].int() >> (at % 2 * 4).int()) & 15
    return (code - 8).double() * scale.double()[..., g]
