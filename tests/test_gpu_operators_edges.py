"""The prompt and shared-prefix operators where it is easy to go wrong: against their plain
fp64 definitions (tests/_plain.py, which also derives the bounds).

The attention divides by the sum of the rounded weights, so that rounding weight j by e_j <= 2^-8 of
it moves an output o by sum_j p_j e_j (v_j - o): at most 2^-8 * sum_j p_j |v_j - o|, with 2^-8 * |o|
for the output's own rounding. That is 0 where one key has the weight or all values are alike, and
exceeds _plain's 2^-8 * sum_j p_j |v_j| only where a few sharp weights add up values unlike the
output; the weights here are spread, or the test says what it allows.
"""
import math

import pytest
import torch

import decode_kv_cache_step_gb300 as lf

import _plain
from test_gpu_operators import BF, gen, ints, near, no_errors, normal

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.mark.parametrize("B,Hkv,S,P,live", [(2250, 8, 2112, 300, 0), (2250, 8, 2112, 300, 3), (64, 8, 2400, 300, 0),
                                            (1, 1, 700, 2000, 0), (7, 3, 2112, 64, 1)])
def test_prefix_counters_are_zero_before_the_step_counts(monkeypatch, B, Hkv, S, P, live):
    """Several chunks a unit, which count in words that the prefix's attention sets to 0; chunks
    without a live slot count at once. Every unit's merge runs, whatever the workspace held and
    however early the step starts."""
    g = gen(B)
    d = 64
    q, nk = normal(g, B, Hkv, d), normal(g, B, Hkv, d)
    k = torch.zeros(B, Hkv, S, d, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    k[:, :, :4], v[:, :, :4] = normal(g, B, Hkv, 4, d), normal(g, B, Hkv, 4, d)
    kp, vp = normal(g, 1, Hkv, P, d), normal(g, 1, Hkv, P, d)
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    start, plen = ints([0, B]), ints([P])
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    mask[:, :, :live] = 9
    ws = torch.empty(lf.decode_prefix_workspace(B, Hkv, Hkv, d, S, 1, P), dtype=torch.uint8, device="cuda")

    def step(fill):
        ws.fill_(fill)
        out = torch.full((B, Hkv, d), 7.0, dtype=BF, device="cuda")
        slots = torch.full((B, Hkv), 77, dtype=torch.int32, device="cuda")
        lf.decode_step_prefix(q, k, v, mask.clone(), nk, nk, write, kp, vp, start, plen, out, slots, 4, 0.125,
                              flags=lf.LF_STEP_FILL_EMPTY_FIRST, workspace=ws)
        return out, slots

    monkeypatch.setenv("LF_PDL", "0")
    want, slots = step(0)
    assert (slots == live).all()  # the first empty slot
    some = slice(0, B, max(1, B // 3))
    for b in range(B)[some]:
        one = _plain.prefix_step(q[b:b + 1], k[b:b + 1], v[b:b + 1], mask[b:b + 1], nk[b:b + 1], nk[b:b + 1],
                                 write[b:b + 1], kp, vp, [0, 1], [P], 0, 0.125, ageing=False)
        near(want[b:b + 1], one["out"], one["tol"])
    monkeypatch.delenv("LF_PDL")
    for fill in (0, 1, 255, 0x41, 255, 1):
        out, slots = step(fill)
        assert torch.equal(out, want) and (slots == live).all()
    no_errors()


def low_first(k, at, value):
    """Keys whose logit with a positive query is -infinity: 40 from `at`; the others' logits near
    value (a column of the query is 1)."""
    k[..., 0] = value
    k[..., at:at + 40, 0] = -math.inf


@pytest.mark.parametrize("value", [0.0, -300.0])
@pytest.mark.parametrize("kv,at,Hq,Hkv,d", [
    (128, 0, 1, 1, 64), (256, 128, 4, 1, 128), (256, 0, 2, 2, 64), (512, 0, 8, 1, 64), (512, 384, 4, 2, 128),
    (2048, 1920, 4, 1, 64), (2048, 896, 1, 1, 128)])
def test_minus_infinity_before_the_last_tiles_keys(kv, at, Hq, Hkv, d, value):
    """The first logits of a tile are -infinity and the rest are not, in tiles that no other of
    their stream follows, with the keys in parts and not; the finite logits large and small."""
    g = gen(kv + at)
    q, k, v = normal(g, 1, Hq, d), normal(g, 1, Hkv, kv, d), normal(g, 1, Hkv, kv, d)
    q[..., 0] = 1
    low_first(k, at, value)
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints([0, 1]), ints([kv]), out, 0, 0, 1.0 if value else 0.125)
    ref, tol = _plain.window_rows(q, k, v, [0, 1], [kv], 0, 0, 1.0 if value else 0.125)
    # A logit near -300 is held to 2^-16, and its weight to that: beyond _plain's bound for N(0, 1).
    near(out, ref, tol + 2.0 ** -10 * v.abs().max().double().cpu())
    no_errors()


@pytest.mark.parametrize("value", [0.0, -300.0])
@pytest.mark.parametrize("P,at,live", [(128, 0, 0), (256, 128, 30), (512, 0, 5), (2048, 1920, 0), (2048, 384, 64)])
def test_minus_infinity_in_a_shared_prefix(P, at, live, value):
    g = gen(P + at)
    B, Hq, Hkv, d, S = 3, 4, 2, 64, 64
    q, k, v = normal(g, B, Hq, d), normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    kp, vp, nk = normal(g, 1, Hkv, P, d), normal(g, 1, Hkv, P, d), normal(g, B, Hkv, d)
    q[..., 0] = 1
    k[..., 0] = value
    low_first(kp, at, value)
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    mask[:, :, :live] = 7
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    scale = 1.0 if value else 0.125
    lf.decode_attention_prefix(q, k, v, mask, nk, nk, write, kp, vp, ints([0, B]), ints([P]), out, scale)
    ref = _plain.prefix_step(q, k, v, mask, nk, nk, write, kp, vp, [0, B], [P], 0, scale, ageing=False)
    near(out, ref["out"], ref["tol"] + 2.0 ** -10 * vp.abs().max().double().cpu())
    no_errors()


def test_prefix_scores_wait_as_long_as_the_prefix_takes(monkeypatch):
    """Prefixes of 2^19 keys with an infinite value each: every row takes the second pass, more
    than a second. The scoring kernel behind the step waits for that, and scores as the step
    itself does. (Few enough units that the step's CTAs all run beside the prefixes'.)"""
    g = gen(31)
    N, Hq, Hkv, d, S, P = 80, 8, 1, 64, 128, 1 << 19
    B = 2 * N
    q, nk = normal(g, B, Hq, d), normal(g, B, Hkv, d)
    k, v = normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    kp, vp = (torch.zeros(N, Hkv, P, d, dtype=BF, device="cuda") for _ in range(2))
    vp[:, 0, 17, 3] = math.inf
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    mask = torch.randint(0, 90, (B, Hkv, S), generator=g, dtype=torch.int32).cuda()
    got = []
    for mode in ("0", "1"):
        monkeypatch.setenv("LF_SPLIT", mode)
        out, m = torch.empty_like(q), mask.clone()
        nxt = torch.full((B, Hkv), 7777, dtype=torch.int32, device="cuda")
        scores = torch.zeros(B, Hkv, S, device="cuda")
        lf.decode_step_prefix(q, k, v, m, nk, nk, write, kp, vp, ints(list(range(0, B + 1, 2))), ints([P] * N), out,
                              nxt, 5, 0.125, scores=scores)
        no_errors()
        got.append((out, nxt, scores, m))
    assert torch.isinf(got[0][0][..., 3]).all() and torch.isfinite(got[0][0][..., 4:]).all()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
def test_second_pass_of_every_row_outlasts_no_wait(d):
    """An infinite value in a prefix of 2^18 keys, for more query tiles than the GPU has SMs: every
    row of a CTA's items takes the second pass while its other warps wait."""
    g = gen(d)
    B, Hq, Hkv, S, P = 6000, 8, 1, 64, 1 << 18
    q, nk = normal(g, B, Hq, d), normal(g, B, Hkv, d)
    k = normal(g, B, Hkv, S, d)
    kp, vp = (normal(g, 1, Hkv, 2048, d).repeat(1, 1, P // 2048, 1) for _ in range(2))
    vp[0, 0, 17, 3] = math.inf
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    mask = torch.zeros(B, Hkv, S, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    lf.decode_attention_prefix(q, k, k, mask, nk, nk, write, kp, vp, ints([0, B]), ints([P]), out, 0.125)
    no_errors()
    assert torch.isinf(out[..., 3]).all()
    vp[0, 0, 17, 3] = 0.0  # the reference of the other columns
    for b in (0, 2999, 5999):
        one = slice(b, b + 1)
        ref = _plain.prefix_step(q[one], k[one], k[one], mask[one], nk[one], nk[one], write[one], kp, vp, [0, 1], [P],
                                 0, 0.125, ageing=False)
        # fp32 sums of P keys in sequence: P * 2^-24 of sum p |v| at most, 2^-6.
        near(out[one, :, 4:], ref["out"][..., 4:], (ref["tol"] * (1 + 2.0 ** 2))[..., 4:])


# Equal values in every key: an output is their weights' sum over the weights' sum. Where both
# sums are of the same (rounded) weights, only fp32 accumulation is left, below n * 2^-24 for n <=
# 5000 keys, 3e-4: less than half a step of bf16 (2^-9 of the value or more), so it is exact.
CONSTANT = [  # rows per sequence, lengths, window, sinks, Hq, Hkv, d
    ([1], [200], 0, 0, 8, 1, 64), ([1, 1, 1], [129, 1000, 4999], 0, 0, 4, 2, 128), ([1], [5000], 1024, 4, 2, 2, 64),
    ([1] * 40, [300 + 17 * i for i in range(40)], 256, 3, 8, 2, 128), ([700], [700], 0, 0, 4, 1, 64),
    ([300, 2, 150], [1300, 900, 150], 200, 70, 4, 2, 128), ([33, 5], [161, 512], 130, 0, 8, 1, 64)]


@pytest.mark.parametrize("sharp", [0.5, 3.0])
@pytest.mark.parametrize("nq,kv,window,sinks,Hq,Hkv,d", CONSTANT)
def test_equal_values_come_out_exactly(nq, kv, window, sinks, Hq, Hkv, d, sharp):
    g = gen(sum(kv))
    B, T, S = len(nq), sum(nq), max(kv)
    starts = [sum(nq[:i]) for i in range(B + 1)]
    q, k = normal(g, T, Hq, d), normal(g, B, Hkv, S, d)
    row = normal(g, Hkv, d)
    v = row[None, :, None].expand(B, Hkv, S, d).contiguous()
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints(starts), ints(kv), out, window, sinks, sharp * d ** -0.5)
    assert torch.equal(out, row.repeat_interleave(Hq // Hkv, 0).expand(T, Hq, d))
    no_errors()


@pytest.mark.parametrize("sharp", [0.5, 3.0])
@pytest.mark.parametrize("B,P,Hq,Hkv,d", [(1, 200, 8, 1, 64), (5, 1000, 4, 2, 128), (70, 4999, 8, 2, 64), (9, 129, 2, 2, 64)])
def test_equal_values_of_a_prefix_come_out_exactly(B, P, Hq, Hkv, d, sharp):
    """And the scores' normalisation stays that of the weights themselves: own slots with equal
    logits score alike to fp32, whatever the prefix's weights round to."""
    g = gen(B + P)
    S, W = 40, 2
    q, nk = normal(g, B, Hq, d), normal(g, B, Hkv, d)
    kp, row = normal(g, 1, Hkv, P, d), normal(g, Hkv, d)
    vp = row[None, :, None].expand(1, Hkv, P, d).contiguous()
    k, v = normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    out, nxt = torch.empty_like(q), torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    tail = (kp, vp, ints([0, B]), ints([P]))
    scale = sharp * d ** -0.5
    lf.decode_attention_prefix(q, k, v, mask, nk, nk, write, *tail, out, scale)
    assert torch.equal(out, row.repeat_interleave(Hq // Hkv, 0).expand(B, Hq, d))
    mask.fill_(9)
    scores = torch.empty(B, Hkv, S, device="cuda")
    lf.decode_step_prefix(q, k, v, mask, nk, nk, write, *tail, out, nxt, W, scale, scores=scores)
    one = slice(0, min(B, 9))
    ref = _plain.prefix_step(q[one], k[one], v[one], mask[one], nk[one], nk[one], write[one], kp, vp,
                             [0, min(B, 9)], [P], W, scale, ageing=False)
    # A logit is within d * 2^-24 * sum |q k| * scale of its value, with sum |q k| * scale <= 32 sharp
    # (2^-9 of a weight at most, less by the square root of d and of the terms); the approximate
    # exponential, the row's L1 norm and the sums are within 2^-18.
    s, r = scores[one].double().cpu(), ref["scores"]
    assert ((s - r).abs() <= (sharp * 2.0 ** -12 + 2.0 ** -18) * r + 1e-37).all(), float(((s - r).abs() / r).max())
    no_errors()


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter", [(500, 8, 2, 128, 128, False), (700, 4, 1, 64, 48, True),
                                                  (6500, 2, 1, 128, 112, True)])
@pytest.mark.parametrize("top", [1 << 24, 1 << 28, (1 << 31) - 1, -(1 << 31)])
def test_rotation_at_far_positions(T, Hq, Hkv, d, rot, inter, top):
    """Any int32 position, frequencies from 1e-6 to above 1 and below 0: the bound of _plain.rope_bound
    (its own angles, n * f in fp64, are within 2^-22)."""
    g = gen(T + rot)
    qkv = normal(g, T, Hq + 2 * Hkv, d)
    freq = (1e6 ** (-torch.arange(rot // 2).double() * 2 / rot)).float()
    freq[1], freq[2], freq[3], freq[4] = 1.9, -0.7, 0.0, 1e-30
    freq = freq.cuda()
    span = torch.randint(0, 4096, (T,), generator=g, dtype=torch.int32)
    pos = (torch.tensor(top, dtype=torch.int32) + (span if top < 0 else -span)).cuda()
    pos[0] = top
    q = torch.empty(T, Hq, d, dtype=BF, device="cuda")
    k, v = (torch.empty(T, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
    lf.qk_norm_rope(qkv, None, None, freq, pos, q, k, v, 1e-6, interleaved=inter)
    ref = _plain.rope(qkv[:, :Hq + Hkv], None, freq, pos, 1e-6, inter)
    near(torch.cat([q, k], 1), ref, _plain.rope_bound(ref))
    no_errors()


def test_rotation_by_large_frequencies():
    """Frequencies beyond a turn per position: what counts is their fraction of a turn."""
    g = gen(8)
    T, d = 300, 64
    qkv = normal(g, T, 3, d)
    freq = torch.exp2(torch.linspace(0, 24, 32).double()).float().cuda()
    pos = torch.randint(-1000, 1000, (T,), generator=g, dtype=torch.int32).cuda()
    q, k, v = (torch.empty(T, 1, d, dtype=BF, device="cuda") for _ in range(3))
    lf.qk_norm_rope(qkv, None, None, freq, pos, q, k, v, 1e-6)
    ref = _plain.rope(qkv[:, :2], None, freq, pos, 1e-6, False)  # |n f| < 2^34: exact in fp64
    near(torch.cat([q, k], 1), ref, _plain.rope_bound(ref))
    no_errors()


@pytest.mark.parametrize("T", [5, 6500])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("d", [64, 128])
def test_norm_of_the_largest_and_smallest_heads(T, eps, d):
    """Heads whose sum of squares leaves fp32's range either way: the norm is the formula's."""
    g = gen(d)
    qkv = normal(g, T, 4, d)
    scales = [3e38 / 8, 1e30, 1e20, 2e-19, 1e-25, 1e-36, 1.0]  # (below 8 standard deviations)
    for i, s in enumerate(scales):
        qkv[i::len(scales)] = (qkv[i::len(scales)].double() * s).to(BF)
    qkv[T - 1, 0, 0], qkv[T - 1, 0, 1:] = 3e38, 1e-38  # one value counts
    qkv[T - 2, 0] = 0.0
    qkv[T - 2, 1, 0] = 2e-39  # subnormal
    qkv[T - 2, 1, 1:] = 0.0
    w = normal(g, d)
    f = torch.full((d // 2,), 0.5, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    q = torch.empty(T, 2, d, dtype=BF, device="cuda")
    k, v = (torch.empty(T, 1, d, dtype=BF, device="cuda") for _ in range(2))
    lf.qk_norm_rope(qkv, w, w, f, pos, q, k, v, eps)
    ref = _plain.rope(qkv[:, :3], w, f, pos, eps, False)
    got = torch.cat([q, k], 1)
    if eps == 0.0:  # 0 / 0
        assert torch.isnan(got[T - 2, 0]).all() and torch.isnan(ref[T - 2, 0]).all()
        got[T - 2, 0], ref[T - 2, 0] = 0, 0
    # (Results below fp32's normal range are rounded to its steps.)
    near(got, ref, _plain.rope_bound(ref) + 2.0 ** -126)
    no_errors()


@pytest.mark.parametrize("scale,size", [(0.0, 1e17), (0.0, 1.0), (3e-33, 1e16), (-3e-33, 1e16), (1e-36, 1e17)])
@pytest.mark.parametrize("T,kv", [(1, 700), (200, 400)])
def test_scales_near_zero(scale, size, T, kv):
    """Queries and keys as large as bf16 holds them: a scale near zero is that scale."""
    g = gen(T + kv)
    q, k, v = normal(g, T, 4, 64), normal(g, 1, 2, kv, 64), normal(g, 1, 2, kv, 64)
    q, k = (q.double() * size).to(BF), (k.double() * size).to(BF)
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints([0, T]), ints([kv]), out, 150, 3, scale)
    ref, tol = _plain.window_rows(q, k, v, [0, T], [kv], 150, 3, scale)
    near(out, ref, tol)
    no_errors()


@pytest.mark.parametrize("Hq,Hkv,N", [(8, 1, 3), (1, 1, 3), (4, 2, 70)])
def test_row_starts_that_do_not_ascend_are_reported(Hq, Hkv, N):
    """A sequence that ends before it starts, behind whose start no later one lies: it has no rows
    to skip, and is reported all the same."""
    g = gen(N)
    T, S, d = 4000, 3904, 64
    q, k, v = normal(g, T, Hq, d), normal(g, N, Hkv, S, d), normal(g, N, Hkv, S, d)
    starts, lens = [0, 3900] + [3] * (N - 1), [3900] + [5] * (N - 1)
    out = torch.full_like(q, 7.0)
    lf.window_attention(q, k, v, ints(starts), ints(lens), out, 60, 0, 0.125)
    assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
    assert (out[3900:] == 7).all()
    lf.window_attention(q, k, v, ints([0] + [3900] * N), ints(lens), out, 60, 0, 0.125)
    no_errors()
    B = 40
    ws = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    mask = torch.zeros(B, Hkv, 70, dtype=torch.int32, device="cuda")
    own, nk = normal(g, B, Hkv, 70, d), normal(g, B, Hkv, d)
    lf.decode_attention_prefix(q[:B], own, own, mask, nk, nk, ws, k, v, ints([0, 39] + [3] * (N - 1)),
                               ints([100] * N), out[:B], 0.125)
    assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH


def marked(kv, d, part):
    """Values that count keys: 64 keys in turn mark each column, from key part * 64 * d on. [kv, d]"""
    j = torch.arange(kv)
    rel = j - part * 64 * d
    v = torch.zeros(kv, d, dtype=torch.float64)
    inside = (rel >= 0) & (rel < 64 * d)
    v[j[inside], rel[inside] % d] = 1
    return v


def seen_marks(v, T, kv, window, sinks):
    """How many keys that mark column c each of the last T rows sees, and how many keys at all."""
    c = torch.cat([torch.zeros(1, v.shape[1], dtype=F64), v.cumsum(0)])
    pos = torch.arange(kv - T, kv)
    lo = (pos + 1 - window).clamp(min=0) if window else torch.zeros(T, dtype=torch.long)
    first = lo.clamp(max=sinks)
    return c[pos + 1] - c[lo] + c[first], pos + 1 - lo + first


@pytest.mark.parametrize("T,kv,window,sinks,Hq,Hkv,d", [
    (1500, 1500, 0, 0, 4, 1, 128), (700, 3000, 1000, 16, 4, 2, 64), (1, 20000, 0, 0, 8, 2, 128),
    (1, 9000, 4096, 4, 4, 2, 64), (20, 5000, 0, 0, 8, 1, 64), (1, 16384, 4096, 100, 32, 8, 128),
    (3000, 3001, 1024, 4, 1, 1, 128), (130, 7777, 999, 333, 8, 8, 64), (9000, 9000, 0, 0, 8, 8, 64)])
def test_every_key_counts_once(T, kv, window, sinks, Hq, Hkv, d):
    """Queries of zero weigh all keys they see alike, so an output times the number of keys seen is
    a count of marked keys: at most 64 a column, which bf16's half step of 2^-8 (a quarter of a
    key) and fp32's sums tell apart exactly. Every row, every column, every key."""
    q = torch.zeros(T, Hq, d, dtype=BF, device="cuda")
    k = normal(gen(kv), 1, Hkv, kv, d)
    out = torch.empty_like(q)
    starts, lens = ints([0, T]), ints([kv])
    for part in range(-(-kv // (64 * d))):
        v = marked(kv, d, part)
        lf.window_attention(q, k, v.to(BF).cuda().expand(1, Hkv, kv, d).contiguous(), starts, lens, out, window,
                            sinks, 0.125)
        want, n = seen_marks(v, T, kv, window, sinks)
        got = (out.double().cpu() * n[:, None, None]).round()
        assert torch.equal(got, want[:, None].expand(T, Hq, d)), f"part {part}"
    no_errors()


@pytest.mark.parametrize("B,starts,plen,P,S,live", [
    (1, [0, 1], [20000], 20000, 300, 100), (40, [0, 40], [5003], 5003, 700, 650), (67, [0, 30, 60, 67], [5003, 0, 3001], 5003, 2400, 1999),
    (3, [0, 3], [129], 200, 9000, 8999)])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (4, 4, 64)])
def test_every_key_of_prefix_and_cache_counts_once(B, starts, plen, P, S, live, Hq, Hkv, d):
    q = torch.zeros(B, Hq, d, dtype=BF, device="cuda")
    N = len(plen)
    k, kp = torch.zeros(B, Hkv, S, d, dtype=BF, device="cuda"), torch.zeros(N, Hkv, P, d, dtype=BF, device="cuda")
    nk = torch.zeros(B, Hkv, d, dtype=BF, device="cuda")
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    mask[:, :, S - live:] = 3
    out = torch.empty_like(q)
    for part in range(-(-max(P, S) // (64 * d))):
        vp, v = marked(P, d, part), marked(S, d, part)
        # the cache marks the upper half of the columns, the prefix the lower
        vp[:, d // 2:], v[:, :d // 2] = 0, 0
        lf.decode_attention_prefix(q, k, v.to(BF).cuda().expand(B, Hkv, S, d).contiguous(), mask, nk, nk, write, kp,
                                   vp.to(BF).cuda().expand(N, Hkv, P, d).contiguous(), ints(starts), ints(plen), out,
                                   0.125)
        got = out.double().cpu()
        for b in range(B):
            n = plen[next(i for i in range(N) if starts[i] <= b < starts[i + 1])]
            want = vp[:n].sum(0) + v[S - live:].sum(0)
            assert torch.equal((got[b] * (n + live)).round(), want.expand(Hq, d)), f"sequence {b} part {part}"
    no_errors()


@pytest.mark.parametrize("S,P", [(8300, 3000), (2400, 700)])
def test_captured_step_with_a_prefix(S, P):
    """The step with its scoring kernel, and without, captured and replayed token by token: what
    the same calls give one by one."""
    g = gen(S)
    B, Hq, Hkv, d = 3, 8, 2, 64
    q, nk = normal(g, B, Hq, d), normal(g, B, Hkv, d)
    k, v = normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    kp, vp = normal(g, 2, Hkv, P, d), normal(g, 2, Hkv, P, d)
    mask = torch.randint(-30, 200, (B, Hkv, S), generator=g, dtype=torch.int32).clamp_(min=-1).cuda()
    starts, plen = ints([0, 2, 3]), ints([P, P // 3])

    def state():
        return dict(k=k.clone(), v=v.clone(), m=mask.clone(), ws=torch.zeros(B, Hkv, dtype=torch.int32, device="cuda"),
                    nx=torch.zeros(B, Hkv, dtype=torch.int32, device="cuda"), out=torch.zeros_like(q))

    def token(s):
        lf.decode_step_prefix(q, s["k"], s["v"], s["m"], nk, nk, s["ws"], kp, vp, starts, plen, s["out"], s["nx"], 5,
                              0.125)
        s["ws"].copy_(s["nx"])

    eager, graph = state(), state()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        token(graph)
        token(graph)
    for _ in range(4):
        token(eager)
        token(eager)
        gr.replay()
        for x in eager:
            assert torch.equal(eager[x], graph[x]), x
    no_errors()
