"""The prompt and shared-prefix operators against their plain fp64 definitions
(tests/_plain.py, which also derives the bounds)."""
import math

import pytest
import torch

import decode_kv_cache_step_gb300 as lf

import _plain

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN = float("nan")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(BF).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def near(got, ref, tol, what=""):
    got = got.double().cpu()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{torch.nonzero(bad)[0].tolist()}: {got[bad][0]} vs {ref[bad][0]} "
                           f"+- {tol[bad][0]}")


def no_errors():
    assert lf.device_errors(clear=True) == 0


# ------------------------------------------------------- norm and rotation --

ROPE = [  # T, Hq, Hkv, d, rot, interleaved, norm
    (1, 32, 8, 128, 128, False, True), (1, 1, 1, 64, 16, True, False), (7, 8, 1, 64, 64, False, True),
    (128, 32, 8, 128, 128, False, True), (33, 6, 3, 128, 48, False, True),
    (19, 4, 2, 64, 32, True, True), (65, 16, 2, 128, 112, True, False), (300, 2, 2, 64, 48, False, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,norm", ROPE)
def test_norm_rope(T, Hq, Hkv, d, rot, inter, norm):
    g = gen(T + rot)
    wide = normal(g, T, Hq + 2 * Hkv + 3, d)
    qkv = wide[:, :Hq + 2 * Hkv]                      # strided rows
    wq, wk = (normal(g, d), normal(g, d)) if norm else (None, None)
    freq = (1e4 ** (-torch.arange(rot // 2).double() * 2 / rot)).float().cuda()
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    pos[0], pos[-1] = 0, (1 << 20)
    pos = pos.cuda()
    q = torch.empty(T, Hq, d, dtype=BF, device="cuda")
    k, v = (torch.empty(T, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
    lf.qk_norm_rope(qkv, wq, wk, freq, pos, q, k, v, 1e-6, interleaved=inter)
    for got, x, w in ((q, qkv[:, :Hq], wq), (k, qkv[:, Hq:Hq + Hkv], wk)):
        ref = _plain.rope(x, w, freq, pos, 1e-6, inter)
        near(got, ref, _plain.rope_bound(ref))
    assert torch.equal(v, qkv[:, Hq + Hkv:])
    no_errors()


def test_norm_rope_extremes():
    """A zero head stays zero, large and tiny heads keep their norm, NaN stays in its head."""
    qkv = torch.ones(3, 4, 64, dtype=BF, device="cuda")
    qkv[0, 0] = 0
    qkv[1, 0] = 1e18
    qkv[2, 1] = 1e-12
    qkv[0, 1, 5] = NAN
    w = torch.ones(64, dtype=BF, device="cuda")
    f = torch.full((32,), 0.5, device="cuda")
    q, = (torch.empty(3, 2, 64, dtype=BF, device="cuda"),)
    k, v = (torch.empty(3, 1, 64, dtype=BF, device="cuda") for _ in range(2))
    lf.qk_norm_rope(qkv, w, w, f, ints([0, 0, 0]), q, k, v, 1e-6)
    assert (q[0, 0] == 0).all() and torch.isnan(q[0, 1]).all() and (q[1, 1] == 1).all()
    ref = _plain.rope(qkv[:, :2], w, f, torch.zeros(3), 1e-6, False)
    near(q[1:], ref[1:], _plain.rope_bound(ref[1:]))


APPEND = [  # rows per sequence, lengths after, S, rows beyond the last sequence
    ([5, 0, 17], [5, 0, 20], 24, 3), ([1], [1], 1, 0), ([64, 1, 2, 0], [64, 64, 30, 7], 64, 0),
    ([130, 257], [130, 300], 301, 11),
]


@pytest.mark.parametrize("nq,kv,S,extra", APPEND)
@pytest.mark.parametrize("Hq,Hkv,d,offset", [(4, 2, 64, None), (8, 1, 128, 4097)])
def test_append(nq, kv, S, extra, Hq, Hkv, d, offset):
    g = gen(S)
    B, T = len(nq), sum(nq) + extra
    starts = [sum(nq[:i]) for i in range(B + 1)]
    qkv = normal(g, T, Hq + 2 * Hkv, d)
    w = normal(g, d)
    freq = (1e4 ** (-torch.arange(d // 2).double() * 2 / d)).float().cuda()
    q = normal(g, T, Hq, d)
    k, v = normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    off = None if offset is None else ints([offset + b for b in range(B)])
    lf.prefill_append(qkv, w, w, freq, ints(starts), ints(kv), q, k, v, mask, pos_offset=off)
    assert torch.equal(q[sum(nq):], q0[sum(nq):])
    for b in range(B):
        rows, at = slice(starts[b], starts[b + 1]), slice(kv[b] - nq[b], kv[b])
        pos = torch.arange(kv[b] - nq[b], kv[b]) + (0 if offset is None else offset + b)
        ref = _plain.rope(qkv[rows, :Hq], w, freq, pos, 1e-6, False)
        near(q[rows], ref, _plain.rope_bound(ref))
        ref = _plain.rope(qkv[rows, Hq:Hq + Hkv], w, freq, pos, 1e-6, False)
        near(k[b, :, at].transpose(0, 1), ref, _plain.rope_bound(ref))
        assert torch.equal(v[b, :, at].transpose(0, 1), qkv[rows, Hq + Hkv:])
        k0[b, :, at], v0[b, :, at] = k[b, :, at], v[b, :, at]
        want = torch.full((S,), -1, dtype=torch.int32)
        want[:kv[b]] = torch.arange(kv[b] - 1, -1, -1)
        assert torch.equal(mask[b].cpu(), want.expand(Hkv, S))
    assert torch.equal(k, k0) and torch.equal(v, v0)  # every other slot as it was
    no_errors()


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,norm", [
    (7001, 2, 1, 64, 48, True, True), (6500, 4, 2, 128, 128, False, True), (8000, 1, 1, 64, 64, False, False),
    (6200, 6, 3, 128, 32, True, True)])
def test_norm_rope_many_tokens(T, Hq, Hkv, d, rot, inter, norm):
    """As many tokens as take a warp each."""
    test_norm_rope(T, Hq, Hkv, d, rot, inter, norm)


@pytest.mark.parametrize("nq,kv,S,extra", [
    ([3000, 0, 1, 3500], [3100, 0, 1, 3501], 3601, 5),  # rows of ages off 16 bytes
    ([5000, 1500], [5000, 4999], 5000, 0), ([1] * 100 + [6001], [7] * 100 + [6003], 6004, 1)])
@pytest.mark.parametrize("Hq,Hkv,d,offset", [(2, 1, 64, 3), (4, 2, 128, None)])
def test_append_many_tokens(nq, kv, S, extra, Hq, Hkv, d, offset):
    test_append(nq, kv, S, extra, Hq, Hkv, d, offset)


def test_bad_lengths_are_skipped_among_many_tokens():
    g = gen(3)
    qkv, f = normal(g, 7000, 3, 64), torch.ones(32, device="cuda")
    q = torch.zeros(7000, 1, 64, dtype=BF, device="cuda")
    k, v = (torch.zeros(3, 1, 4100, 64, dtype=BF, device="cuda") for _ in range(2))
    mask = torch.full((3, 1, 4100), -1, dtype=torch.int32, device="cuda")
    lf.prefill_append(qkv, None, None, f, ints([0, 3000, 3500, 7000]), ints([3000, 4101, 3500]),
                      q, k, v, mask)
    assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
    assert (q[3000:3500] == 0).all() and (k[1] == 0).all() and (v[1] == 0).all()
    assert (mask[1] == -1).all() and (mask[0, 0, :3000] >= 0).all()
    assert torch.equal(v[2, 0, :3500], qkv[3500:, 2]) and (v[2, 0, 3500:] == 0).all()


def test_bad_lengths_are_skipped():
    """A sequence whose lengths do not fit is skipped and reported; its neighbours are not."""
    g = gen(1)
    qkv, f = normal(g, 6, 4, 64), torch.ones(32, device="cuda")
    q = torch.zeros(6, 2, 64, dtype=BF, device="cuda")
    k, v = (torch.zeros(3, 1, 8, 64, dtype=BF, device="cuda") for _ in range(2))
    mask = torch.full((3, 1, 8), -1, dtype=torch.int32, device="cuda")
    for lens in ([2, 9, 2], [2, 1, 2], [2, -1, 2]):  # beyond S; fewer than its rows; negative
        q.zero_(), k.zero_(), v.zero_(), mask.fill_(-1)
        lf.prefill_append(qkv, None, None, f, ints([0, 2, 4, 6]), ints(lens), q, k, v, mask)
        assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
        assert (q[2:4] == 0).all() and (k[1] == 0).all() and (mask[1] == -1).all()
        assert (q[:2] != 0).any() and (q[4:] != 0).any() and (mask[2, 0, :2] >= 0).all()
        out = torch.full((6, 2, 64), 7.0, dtype=BF, device="cuda")
        lf.window_attention(normal(g, 6, 2, 64), k, v, ints([0, 2, 4, 6]), ints(lens), out, 0, 0, 0.1)
        assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
        assert (out[2:4] == 7).all() and (out[:2] != 7).all() and (out[4:] != 7).all()
    for bad in ([0, 9, 9, 9], [-1, 2, 4, 6], [0, 5, 3, 6]):  # beyond T; negative; not ascending
        lf.prefill_append(qkv, None, None, f, ints(bad), ints([8, 8, 8]), q, k, v, mask)
        lf.window_attention(q, k, v, ints(bad), ints([8, 8, 8]), out, 0, 0, 0.1)
        assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
    out = torch.zeros(6, 2, 64, dtype=BF, device="cuda")
    nk = normal(g, 6, 1, 64)
    kc = normal(g, 6, 1, 8, 64)
    m6 = torch.zeros(6, 1, 8, dtype=torch.int32, device="cuda")
    ws = torch.full((6, 1), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros_like(out)
    q = normal(g, 6, 2, 64)
    lf.decode_attention(q, kc, kc, m6, nk, nk, ws, ref, 0.1)
    lf.decode_attention_prefix(q, kc, kc, m6, nk, nk, ws, k, v, ints([0, 2, 4, 6]), ints([0, 9, 0]),
                               out, 0.1)
    assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
    assert torch.equal(out, ref)


# ------------------------------------------------------- window attention --

WINDOW = [  # rows per sequence, lengths, S, window, sinks
    ([1], [1], 1, 0, 0), ([1], [200], 200, 64, 4), ([1, 1, 1], [300, 1, 129], 301, 100, 3),
    ([40], [40], 40, 0, 0), ([40, 0, 3], [40, 0, 3], 64, 1, 0), ([33, 70], [161, 70], 200, 16, 2),
    ([129], [400], 400, 130, 5), ([257], [257], 260, 64, 200), ([1] * 37, list(range(1, 38)), 40, 7, 1),
    ([300, 1, 5], [300, 300, 300], 384, 0, 0), ([2, 150], [2, 511], 513, 127, 129),
    ([64, 64], [64, 128], 128, 1000, 7), ([5], [1024], 1024, 0, 0),
    ([64], [400], 400, 129, 5), ([2, 3], [500, 700], 704, 180, 64), ([1], [1000], 1000, 140, 65),
]
SHAPES = [(1, 1, 64), (8, 1, 64), (4, 2, 128), (8, 2, 128), (2, 1, 128)]


@pytest.mark.parametrize("nq,kv,S,window,sinks", WINDOW)
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_window(nq, kv, S, window, sinks, Hq, Hkv, d):
    g = gen(S + window)
    B, T = len(nq), sum(nq) + 2
    starts = [sum(nq[:i]) for i in range(B + 1)]
    q = normal(g, T, Hq, d)
    k, v = normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    for b in range(B):  # what no query may read
        k[b, :, kv[b]:], v[b, :, kv[b]:] = NAN, NAN
        if window and nq[b]:
            hidden = slice(min(sinks, kv[b]), max(sinks, kv[b] - nq[b] + 1 - window, 0))
            k[b, :, hidden], v[b, :, hidden] = NAN, math.inf
    out = torch.full((T, Hq, d), 7.0, dtype=BF, device="cuda")
    scale = d ** -0.5
    lf.window_attention(q, k, v, ints(starts), ints(kv), out, window, sinks, scale)
    ref, tol = _plain.window_rows(q, k, v, starts, kv, window, sinks, scale)
    near(out[:T - 2], ref[:T - 2], tol[:T - 2])
    assert (out[T - 2:] == 7).all()
    no_errors()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0, 40.0])
def test_window_scales(scale):
    """Negative, zero and large scales: the largest logits stand out by hundreds of nats, and an
    output is then a copy of a value row up to the weights' error, which grows with the logits:
    sum |q k| * scale * d * 2^-24 nats."""
    g = gen(5)
    q, k, v = normal(g, 90, 4, 64), normal(g, 1, 2, 200, 64), normal(g, 1, 2, 200, 64)
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints([0, 90]), ints([190]), out, 50, 3, scale)
    ref, tol = _plain.window_rows(q, k, v, [0, 90], [190], 50, 3, scale)
    slack = 64 * 2.0 ** -24 * abs(scale) * 64 * 4  # |q k| below 4 on average
    near(out, ref, tol + slack * v.abs().max().double().cpu())


def test_window_nonfinite_keys_stay_in_their_rows():
    """A NaN key or value reaches the rows that see it and no other, in the same tile too."""
    g = gen(6)
    q, k, v = normal(g, 100, 2, 64), normal(g, 1, 1, 100, 64), normal(g, 1, 1, 100, 64)
    k[0, 0, 40, 3], v[0, 0, 70, 9], v[0, 0, 71, 10] = NAN, math.inf, NAN
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints([0, 100]), ints([100]), out, 20, 2, 0.125)
    k2, v2 = k.clone(), v.clone()
    ref, tol = _plain.window_rows(q, k2, v2, [0, 100], [100], 20, 2, 0.125)
    got = out.double().cpu()
    assert torch.isnan(got[40:60]).all()
    clean = torch.ones(100, dtype=torch.bool)
    clean[40:60] = False
    assert (got[70:90, :, 9] == math.inf).all() and torch.isnan(got[71:91, :, 10]).all()
    cols = torch.ones(100, 2, 64, dtype=torch.bool)
    cols[40:60] = False
    cols[70:90, :, 9] = False
    cols[71:91, :, 10] = False
    ref2, tol2 = torch.nan_to_num(ref), torch.nan_to_num(tol)
    assert torch.isfinite(got[cols]).all()
    near(out.cpu()[cols], ref2[cols], tol2[cols])
    # minus infinity as a logit: weight zero, the row stays finite
    k[0, 0, 40, 3] = 1.0
    v[0, 0, 70, 9] = v[0, 0, 71, 10] = 0.0
    q.abs_()
    k[0, 0, 30, 0] = -math.inf
    lf.window_attention(q, k, v, ints([0, 100]), ints([100]), out, 20, 2, 0.125)
    ref, tol = _plain.window_rows(q, k, v, [0, 100], [100], 20, 2, 0.125)
    near(out, ref, tol)


@pytest.mark.parametrize("T,kv,window,sinks,Hq,Hkv,d", [
    (1500, 1500, 0, 0, 4, 1, 128), (700, 3000, 1000, 16, 4, 2, 64), (1, 20000, 0, 0, 8, 2, 128),
    (1, 9000, 4096, 4, 4, 2, 64), (20, 5000, 0, 0, 8, 1, 64)])
def test_window_long(T, kv, window, sinks, Hq, Hkv, d):
    """Long sequences: every 97th row against the definition."""
    g = gen(T + kv)
    q, k, v = normal(g, T, Hq, d), normal(g, 1, Hkv, kv, d), normal(g, 1, Hkv, kv, d)
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints([0, T]), ints([kv]), out, window, sinks, d ** -0.5)
    for i in list(range(0, T, 97)) + [T - 1]:
        ref, tol = _plain.window_rows(q[i:i + 1], k, v, [0, 1], [kv - T + i + 1], window, sinks,
                                      d ** -0.5)
        near(out[i:i + 1], ref, tol, f"row {i}")
    no_errors()


def test_window_many_sequences_and_repeats():
    """Hundreds of short sequences, the same bits at every call."""
    g = gen(9)
    nq = [int(x) for x in torch.randint(0, 4, (333,), generator=g)]
    kv = [n + int(x) for n, x in zip(nq, torch.randint(0, 90, (333,), generator=g))]
    starts = [sum(nq[:i]) for i in range(334)]
    q, k, v = normal(g, starts[-1], 4, 64), normal(g, 333, 2, 96, 64), normal(g, 333, 2, 96, 64)
    outs = []
    for _ in range(3):
        out = torch.full_like(q, 7.0)
        lf.window_attention(q, k, v, ints(starts), ints(kv), out, 33, 2, 0.125)
        outs.append(out)
    ref, tol = _plain.window_rows(q, k, v, starts, kv, 33, 2, 0.125)
    near(outs[0], ref, tol)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    no_errors()


# ----------------------------------------------------------- shared prefix --

PREFIX = [  # B, prefix starts, prefix lengths, P, S, live (None: random holes)
    (1, [0, 1], [1], 1, 1, 1), (4, [0, 4], [300], 301, 256, None), (3, [0, 1, 3], [0, 129], 200, 65, 0),
    (5, [1, 3, 3, 4], [64, 7, 500], 512, 100, None), (40, [0, 40], [1000], 1024, 70, None),
    (6, [0, 6], [0], 64, 64, 0),
]


def prefix_case(B, starts, plen, P, S, live, Hq, Hkv, d, seed=0):
    g = gen(B + P + S + seed)
    N = len(plen)
    c = dict(q=normal(g, B, Hq, d), k=normal(g, B, Hkv, S, d), v=normal(g, B, Hkv, S, d),
             nk=normal(g, B, Hkv, d), nv=normal(g, B, Hkv, d), kp=normal(g, N, Hkv, P, d),
             vp=normal(g, N, Hkv, P, d), starts=starts, plen=plen, scale=d ** -0.5)
    for n in range(N):
        c["kp"][n, :, plen[n]:], c["vp"][n, :, plen[n]:] = NAN, NAN
    m = torch.randint(-40, 100, (B, Hkv, S), generator=g, dtype=torch.int32).clamp_(min=-1)
    if live is not None:
        m = torch.where(torch.arange(S) < live, m.abs(), -1).to(torch.int32)
    c["mask"] = m.cuda()
    dead = (m < 0).cuda()
    c["k"][dead], c["v"][dead] = NAN, math.inf
    c["ws"] = torch.randint(-1, S, (B, Hkv), generator=g, dtype=torch.int32).cuda()
    return c


@pytest.mark.parametrize("B,starts,plen,P,S,live", PREFIX)
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (8, 1, 64), (4, 2, 128), (4, 1, 128)])
def test_prefix_attention_and_step(B, starts, plen, P, S, live, Hq, Hkv, d):
    c = prefix_case(B, starts, plen, P, S, live, Hq, Hkv, d)
    args = (c["nk"], c["nv"], c["ws"], c["kp"], c["vp"], ints(starts), ints(plen))
    out = torch.empty(B, Hq, d, dtype=BF, device="cuda")
    plain = (c["q"], c["k"], c["v"], c["mask"], c["nk"], c["nv"], c["ws"], c["kp"], c["vp"], starts,
             plen)
    ref = _plain.prefix_step(*plain, 0, c["scale"], ageing=False)
    k, v, mask = c["k"].clone(), c["v"].clone(), c["mask"].clone()
    lf.decode_attention_prefix(c["q"], k, v, mask, *args, out, c["scale"])
    near(out, ref["out"], ref["tol"])
    assert torch.equal(mask.cpu(), ref["mask"])
    # the step: the same attention, and scores normalised over prefix and slots
    W = 5
    ref = _plain.prefix_step(*plain, W, c["scale"])
    k, v, mask = c["k"].clone(), c["v"].clone(), c["mask"].clone()
    nxt = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    scores = torch.empty(B, Hkv, S, device="cuda")
    lf.decode_step_prefix(c["q"], k, v, mask, *args, out, nxt, W, c["scale"], scores=scores)
    near(out, ref["out"], ref["tol"])
    assert torch.equal(mask.cpu(), ref["mask"])
    for name, got in (("k", k), ("v", v)):
        assert torch.equal(torch.nan_to_num(got.double().cpu()), torch.nan_to_num(ref[name]))
    s = scores.double().cpu()
    liv = ref["mask"] >= 0
    assert torch.isinf(s[~liv]).all()
    assert ((s[liv] - ref["scores"][liv]).abs() <= 1e-3 * ref["scores"][liv] + 1e-30).all()
    nxt = nxt.cpu()
    for b in range(B):
        for u in range(Hkv):
            old = torch.nonzero(ref["mask"][b, u] >= W)[:, 0]
            if len(old) == 0:
                assert nxt[b, u] == -1
                continue
            vals = ref["scores"][b, u, old]
            assert ref["mask"][b, u, nxt[b, u]] >= W
            assert ref["scores"][b, u, nxt[b, u]] <= vals.min() * (1 + 1e-3)
            order = vals.sort().values
            if len(old) == 1 or order[1] > order[0] * (1 + 1e-3):
                assert nxt[b, u] == old[vals.argmin()]
    no_errors()


@pytest.mark.parametrize("k,flags", [(1, lf.LF_STEP_FILL_EMPTY_FIRST), (3, 0),
                                     (5, lf.LF_STEP_MASK_EVICTED)])
def test_prefix_step_choices(k, flags):
    """k slots at once and the flags, as lf_decode_step_ex has them."""
    c = prefix_case(3, [0, 3], [200], 200, 90, None, 4, 2, 64)
    out = torch.empty(3, 4, 64, dtype=BF, device="cuda")
    nxt = torch.empty(3, 2, k, dtype=torch.int32, device="cuda")
    kc, vc, mask = c["k"].clone(), c["v"].clone(), c["mask"].clone()
    lf.decode_step_prefix(c["q"], kc, vc, mask, c["nk"], c["nv"], c["ws"], c["kp"], c["vp"],
                          ints([0, 3]), ints([200]), out, nxt, 5, c["scale"], k=k, flags=flags)
    ref = _plain.prefix_step(c["q"], c["k"], c["v"], c["mask"], c["nk"], c["nv"], c["ws"], c["kp"],
                             c["vp"], [0, 3], [200], 5, c["scale"])
    for b in range(3):
        for u in range(2):
            m, s = ref["mask"][b, u], ref["scores"][b, u]
            if flags & lf.LF_STEP_FILL_EMPTY_FIRST:
                want = torch.nonzero(m < 0)[:k, 0]
            else:
                old = torch.nonzero(m >= 5)[:, 0]
                want = old[s[old].argsort()[:k]]
            assert nxt[b, u].tolist() == want.tolist()
            if flags & lf.LF_STEP_MASK_EVICTED:
                m = m.clone()
                m[want] = -1
            assert torch.equal(mask[b, u].cpu(), m)


def test_prefix_long_split_finish(monkeypatch):
    """Units long enough for the scoring kernel, with and without it: the same bits."""
    c = prefix_case(2, [0, 2], [3000], 3000, 8200, None, 4, 2, 64)
    got = []
    for mode in ("0", "1"):
        monkeypatch.setenv("LF_SPLIT", mode)
        kc, vc, mask = c["k"].clone(), c["v"].clone(), c["mask"].clone()
        out = torch.empty(2, 4, 64, dtype=BF, device="cuda")
        nxt = torch.empty(2, 2, dtype=torch.int32, device="cuda")
        lf.decode_step_prefix(c["q"], kc, vc, mask, c["nk"], c["nv"], c["ws"], c["kp"], c["vp"],
                              ints([0, 2]), ints([3000]), out, nxt, 5, c["scale"])
        got.append((out, nxt, mask))
    ref = _plain.prefix_step(c["q"], c["k"], c["v"], c["mask"], c["nk"], c["nv"], c["ws"], c["kp"],
                             c["vp"], [0, 2], [3000], 5, c["scale"])
    near(got[0][0], ref["out"], ref["tol"])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    no_errors()


# ------------------------------------------------- streams, graphs, a run --

def test_other_streams_and_graphs():
    """On another stream, without a workspace of the caller; captured, replayed on new inputs,
    two graphs in flight at once with workspaces of their own."""
    c = prefix_case(4, [0, 4], [700], 700, 128, None, 4, 2, 64)
    c["ws"].fill_(-1)
    k, v, m = c["k"], c["v"], c["mask"]
    starts, plen = ints([0, 4]), ints([700])
    q1, q2 = c["q"], c["q"].flip(0).contiguous()

    def run(q, out, stream=None, workspace=None):
        lf.decode_attention_prefix(q, k, v, m, c["nk"], c["nv"], c["ws"], c["kp"], c["vp"], starts,
                                   plen, out, c["scale"], workspace=workspace, stream=stream)

    def win(q, out, stream=None, workspace=None):
        lf.window_attention(q, c["kp"], c["vp"], ints([0, 4]) if stream is None else starts, plen,
                            out, 300, 4, c["scale"], workspace=workspace, stream=stream)

    for call in (run, win):
        want = [torch.empty_like(q1), torch.empty_like(q1)]
        call(q1, want[0]), call(q2, want[1])
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = [torch.empty_like(q1), torch.empty_like(q1)]
        torch.cuda.synchronize()
        call(q1, got[0], stream=s1)
        call(q2, got[1], stream=s2.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    n = lf.decode_prefix_workspace(4, 4, 2, 64, 128, 1, 700)
    graphs, ins, outs, keep = [], [], [], []
    for _ in range(2):
        qi, oi = torch.zeros_like(q1), torch.zeros_like(q1)
        work = torch.empty(n, dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run(qi, oi, workspace=work)
        graphs.append(gr), ins.append(qi), outs.append(oi), keep.append(work)
    want = [torch.empty_like(q1), torch.empty_like(q1)]
    run(q1, want[0]), run(q2, want[1])
    ins[0].copy_(q1), ins[1].copy_(q2)
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    no_errors()


def test_workspace_is_checked_and_bounded():
    """A workspace that is too small is refused; one that just fits is not overrun."""
    c = prefix_case(3, [0, 3], [500], 500, 100, None, 4, 2, 64)
    n = lf.decode_prefix_workspace(3, 4, 2, 64, 100, 1, 500)
    out = torch.empty(3, 4, 64, dtype=BF, device="cuda")
    args = (c["q"], c["k"], c["v"], c["mask"], c["nk"], c["nv"], c["ws"], c["kp"], c["vp"],
            ints([0, 3]), ints([500]), out, c["scale"])
    with pytest.raises(lf.LFError, match="workspace"):
        lf.decode_attention_prefix(*args, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    big = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    lf.decode_attention_prefix(*args, workspace=big[:n])
    assert (big[n:] == 0xAB).all()
    q = normal(gen(0), 2, 8, 64)
    kc = normal(gen(1), 2, 1, 4000, 64)
    n = lf.window_attention_workspace(2, 2, 8, 1, 64, 4000)
    big = torch.full((n + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    o1, o2 = torch.empty_like(q), torch.empty_like(q)
    lf.window_attention(q, kc, kc, ints([0, 1, 2]), ints([4000, 3999]), o1, 0, 0, 0.1, workspace=big[:n])
    lf.window_attention(q, kc, kc, ints([0, 1, 2]), ints([4000, 3999]), o2, 0, 0, 0.1)
    assert (big[n:] == 0xAB).all() and torch.equal(o1, o2)


def test_prompt_then_samples_together():
    """A prompt through norm, rotation and windowless attention into a prefix cache, in two chunks;
    then samples of it decoded with the evicting step, each token's q, k, v from the same pass."""
    g = gen(77)
    Hq, Hkv, d, P, B, S, steps = 4, 2, 64, 150, 3, 12, 20
    scale = d ** -0.5
    freq = (1e4 ** (-torch.arange(d // 2).double() * 2 / d)).float().cuda()
    w = normal(g, d)
    kp, vp = (torch.zeros(1, Hkv, P, d, dtype=BF, device="cuda") for _ in range(2))
    pm = torch.full((1, Hkv, P), -1, dtype=torch.int32, device="cuda")
    prompt = normal(g, P, Hq + 2 * Hkv, d)
    for lo, hi in ((0, 100), (100, 150)):
        n = hi - lo
        q, out = (torch.empty(n, Hq, d, dtype=BF, device="cuda") for _ in range(2))
        lf.prefill_append(prompt[lo:hi], w, w, freq, ints([0, n]), ints([hi]), q, kp, vp, pm)
        lf.window_attention(q, kp, vp, ints([0, n]), ints([hi]), out, 0, 0, scale)
        ref, tol = _plain.window_rows(q, kp, vp, [0, n], [hi], 0, 0, scale)
        near(out, ref, tol)
    want = _plain.rope(prompt[:, Hq:Hq + Hkv], w, freq, torch.arange(P), 1e-6, False)
    near(kp[0].transpose(0, 1), want, _plain.rope_bound(want))
    k, v = (torch.zeros(B, Hkv, S, d, dtype=BF, device="cuda") for _ in range(2))
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B, Hkv, dtype=torch.int32, device="cuda")
    nxt = torch.empty_like(ws)
    starts, plen = ints([0, B]), ints([P])
    q, out = (torch.empty(B, Hq, d, dtype=BF, device="cuda") for _ in range(2))
    nk, nv = (torch.empty(B, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
    for t in range(steps):
        tok = normal(g, B, Hq + 2 * Hkv, d)
        lf.qk_norm_rope(tok, w, w, freq, ints([P + t] * B), q, nk, nv)
        ref = _plain.prefix_step(q, k, v, mask, nk, nv, ws, kp, vp, [0, B], [P], 2, scale)
        lf.decode_step_prefix(q, k, v, mask, nk, nv, ws, kp, vp, starts, plen, out, nxt, 2, scale,
                              flags=lf.LF_STEP_FILL_EMPTY_FIRST)
        near(out, ref["out"], ref["tol"], f"step {t}")
        assert torch.equal(mask.cpu(), ref["mask"])
        for b in range(B):
            for u in range(Hkv):
                empty = torch.nonzero(ref["mask"][b, u] < 0)[:, 0]
                if len(empty):
                    assert nxt[b, u] == empty[0]
                else:
                    s = torch.where(ref["mask"][b, u] >= 2, ref["scores"][b, u], math.inf)
                    assert s[nxt[b, u]] <= s.min() * (1 + 1e-3)
        ws.copy_(nxt)
    assert (mask >= 0).all()
    no_errors()


def test_window_many_items_per_cta():
    """More query tiles than the GPU has SMs, long and short ones: each CTA takes several, in both
    ways the streams are paired; every 397th row against the definition."""
    for nq, kv, Hq, Hkv, window in (([9000], [9000], 8, 8, 0), ([5000, 40, 4001], [5000, 3000, 6000], 4, 4, 700),
                                    ([1] * 2500, [30 + i % 300 for i in range(2500)], 2, 1, 0)):
        g = gen(len(nq))
        B, T, S = len(nq), sum(nq), max(kv)
        starts = [sum(nq[:i]) for i in range(B + 1)]
        q, k, v = normal(g, T, Hq, 64), normal(g, B, Hkv, S, 64), normal(g, B, Hkv, S, 64)
        out = torch.empty_like(q)
        lf.window_attention(q, k, v, ints(starts), ints(kv), out, window, 3, 0.125)
        no_errors()
        for b in range(B):
            for i in range((97 * b) % 397 if nq[b] > 397 else 0, nq[b], 397):
                t = starts[b] + i
                ref, tol = _plain.window_rows(q[t:t + 1], k[b:b + 1], v[b:b + 1], [0, 1],
                                              [kv[b] - nq[b] + i + 1], window, 3, 0.125)
                near(out[t:t + 1], ref, tol, f"sequence {b} row {i}")


def test_held_workspaces_do_not_mix():
    """Calls without a workspace of the caller, from two threads on one stream and on two streams,
    of growing and shrinking sizes: each gives what it gives alone."""
    import threading

    cases = [prefix_case(B, [0, B], [p], p, 130, None, 4, 2, 64, seed=B) for B, p in
             ((3, 900), (9, 100), (2, 2500))]
    for c in cases:
        c["ws"].fill_(-1)
    extra = [(ints([0, c["q"].shape[0]]), ints(c["plen"])) for c in cases]

    def run(i, out):
        c = cases[i]
        lf.decode_attention_prefix(c["q"], c["k"], c["v"], c["mask"], c["nk"], c["nv"], c["ws"],
                                   c["kp"], c["vp"], *extra[i], out, c["scale"])

    want = [torch.empty_like(c["q"]) for c in cases]
    for i, w in enumerate(want):
        run(i, w)
    torch.cuda.synchronize()
    bad = []

    def work(order, stream):
        with torch.cuda.stream(stream):
            outs = [(i, torch.empty_like(want[i])) for i in order * 20]
            for i, out in outs:
                run(i, out)
            stream.synchronize()
            bad.extend(i for i, out in outs if not torch.equal(out, want[i]))

    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    for streams in ((main, main), (main, other)):
        threads = [threading.Thread(target=work, args=(o, s)) for o, s in
                   zip(([0, 1, 2], [2, 0, 1]), streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert not bad
    lf.release_workspace()
    out = torch.empty_like(want[0])
    run(0, out)
    assert torch.equal(out, want[0])


def test_waits_that_run_out_are_reported(monkeypatch):
    """With the wait limit cut to 1 ns the packed attention's waits give up before the copies
    land: the call retires and reports it, and the next one is right."""
    g = gen(3)
    q, k, v = normal(g, 300, 4, 64), normal(g, 1, 2, 400, 64), normal(g, 1, 2, 400, 64)
    out = torch.empty_like(q)
    for rows in (300, 3):
        monkeypatch.setenv("LF_WAIT_LIMIT_NS", "1")
        lf.window_attention(q[:rows], k, v, ints([0, rows]), ints([400]), out[:rows], 90, 2, 0.125)
        assert lf.device_errors(clear=True) & lf.LF_DEVERR_WAIT_TIMEOUT
        monkeypatch.delenv("LF_WAIT_LIMIT_NS")
        lf.window_attention(q[:rows], k, v, ints([0, rows]), ints([400]), out[:rows], 90, 2, 0.125)
        ref, tol = _plain.window_rows(q[:rows], k, v, [0, rows], [400], 90, 2, 0.125)
        near(out[:rows], ref, tol)
        no_errors()


def test_first_call_inside_a_capture():
    """Calls that allocate nothing but from the graph's pool: captured without a warm-up of their
    own shapes, replayed on new inputs."""
    g = gen(4)
    q, k, v = normal(g, 5, 8, 128), normal(g, 5, 2, 900, 128), normal(g, 5, 2, 900, 128)
    qs, kv = ints([0, 1, 2, 3, 4, 5]), ints([900, 1, 450, 129, 64])
    out = torch.empty_like(q)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lf.window_attention(q, k, v, qs, kv, out, 0, 0, 0.1)
    for _ in range(2):
        q.copy_(normal(g, 5, 8, 128))
        out.zero_()
        gr.replay()
        torch.cuda.synchronize()
        ref, tol = _plain.window_rows(q, k, v, [0, 1, 2, 3, 4, 5], [900, 1, 450, 129, 64], 0, 0, 0.1)
        near(out, ref, tol)
    no_errors()


def test_offsets_past_32_bits():
    """Caches, and packed rows, of more than 2^31 values: their last parts are right."""
    g = gen(12)
    B, Hkv, S, d = 33, 8, 65536, 128
    k, v = (torch.zeros(B, Hkv, S, d, dtype=BF, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 31
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    qkv, w = normal(g, 100, 8 + 16, d), normal(g, d)
    freq = (1e4 ** (-torch.arange(64).double() / 64)).float().cuda()
    q = torch.empty(100, 8, d, dtype=BF, device="cuda")
    starts, lens = [0] * B + [100], [0] * (B - 1) + [S]
    k[-1, :, S - 300:], v[-1, :, S - 300:] = normal(g, Hkv, 300, d), normal(g, Hkv, 300, d)
    lf.prefill_append(qkv, w, w, freq, ints(starts), ints(lens), q, k, v, mask)
    want = _plain.rope(qkv[:, 8:16], w, freq, torch.arange(S - 100, S), 1e-6, False)
    near(k[-1, :, S - 100:].transpose(0, 1), want, _plain.rope_bound(want))
    assert torch.equal(v[-1, :, S - 100:].transpose(0, 1), qkv[:, 16:])
    assert (mask[:-1] == -1).all() and mask[-1, -1, -1] == 0 and mask[-1, -1, 0] == S - 1
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints(starts), ints(lens), out, 150, 0, 0.09)
    at = slice(S - 300, S)
    ref, tol = _plain.window_rows(q, k[-1:, :, at], v[-1:, :, at], [0, 100], [300], 150, 0, 0.09)
    near(out, ref, tol)
    # the same caches as prefixes of one sequence each, the last one read
    own = prefix_case(B, [0, B], [1], 1, 40, None, 8, 8, d)
    o2 = torch.empty(B, 8, d, dtype=BF, device="cuda")
    lf.decode_attention_prefix(own["q"], own["k"], own["v"], own["mask"], own["nk"], own["nv"],
                               own["ws"], k, v, ints(list(range(B + 1))), ints(lens), o2, 0.09)
    i = B - 1
    ref = _plain.prefix_step(*(own[x][i:] for x in ("q", "k", "v", "mask", "nk", "nv", "ws")),
                             k[i:], v[i:], [0, 1], [S], 0, 0.09, ageing=False)
    near(o2[i:], ref["out"], ref["tol"])
    del k, v, mask
    T, Hq = 540000, 32
    k, v = normal(g, 1, 1, 1, d).expand(1, 4, T, d).contiguous(), torch.zeros(1, 4, T, d, dtype=BF, device="cuda")
    k[0, :, -400:], v[0, :, -400:] = normal(g, 4, 400, d), normal(g, 4, 400, d)
    q = torch.zeros(T, Hq, d, dtype=BF, device="cuda")
    assert q.numel() > 1 << 31
    q[-400:] = normal(g, 400, Hq, d)
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints([0, T]), ints([T]), out, 90, 0, 0.09)
    ref, tol = _plain.window_rows(q[-60:], k[:, :, -400:], v[:, :, -400:], [0, 60], [400], 90, 0, 0.09)
    near(out[-60:], ref, tol)
    assert (out[:1000] == 0).all()
    no_errors()


@pytest.mark.parametrize("seed", range(24))
def test_window_random_sweep(seed):
    """Random batches: lengths from none, windows, first keys, heads, garbage behind the lengths."""
    g = gen(1000 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    B, Hkv, gg, d = r(1, 9), r(1, 3), 1 << r(0, 3), 64 << r(0, 1)
    S = r(1, 700)
    kv = [r(0, S) for _ in range(B)]
    nq = [min(c, (0, 1, r(0, 40), r(0, S))[r(0, 3)]) for c in kv]
    if sum(nq) == 0:
        kv[0], nq[0] = S, 1
    window, sinks = (0, 1, r(1, 60), r(1, S), r(60, 260))[r(0, 4)], (0, r(0, 8), r(0, 200))[r(0, 2)]
    starts = [sum(nq[:i]) for i in range(B + 1)]
    lead, T = r(0, 3), starts[-1]
    starts = [s + lead for s in starts]
    T += lead + r(0, 5)
    q, k, v = normal(g, T, Hkv * gg, d), normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    k *= torch.exp(0.7 * torch.randn(B, Hkv, S, 1, generator=g)).cuda().to(BF)
    for b in range(B):
        k[b, :, kv[b]:], v[b, :, kv[b]:] = math.inf, NAN
    out = torch.full_like(q, 7.0)
    lf.window_attention(q, k, v, ints(starts), ints(kv), out, window, sinks, d ** -0.5)
    ref, tol = _plain.window_rows(q, k, v, starts, kv, window, sinks, d ** -0.5)
    inside = slice(starts[0], starts[-1])
    near(out[inside], ref[inside], tol[inside], f"window {window} sinks {sinks} nq {nq} kv {kv}")
    assert (out[:starts[0]] == 7).all() and (out[starts[-1]:] == 7).all()
    no_errors()


@pytest.mark.parametrize("seed", range(16))
def test_prefix_random_sweep(seed):
    g = gen(2000 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))
    B, Hkv, gg, d = r(1, 40), r(1, 3), 1 << r(0, 3), 64 << r(0, 1)
    N = r(1, 5)
    starts = sorted(r(0, B) for _ in range(N + 1))
    P = r(1, 900)
    plen = [r(0, P) for _ in range(N)]
    c = prefix_case(B, starts, plen, P, r(1, 300), None, Hkv * gg, Hkv, d, seed=seed)
    out = torch.empty_like(c["q"])
    ref = _plain.prefix_step(c["q"], c["k"], c["v"], c["mask"], c["nk"], c["nv"], c["ws"], c["kp"],
                             c["vp"], starts, plen, 0, c["scale"], ageing=False)
    lf.decode_attention_prefix(c["q"], c["k"], c["v"], c["mask"], c["nk"], c["nv"], c["ws"], c["kp"],
                               c["vp"], ints(starts), ints(plen), out, c["scale"])
    near(out, ref["out"], ref["tol"], f"starts {starts} lengths {plen}")
    assert torch.equal(c["mask"].cpu(), ref["mask"])
    no_errors()


def test_nonfinite_key_seen_by_a_long_prompt():
    """A NaN in the first key reaches every row of a causal prompt, and only it: the slower second
    pass of all rows stays within the waits' limit."""
    g = gen(21)
    q, k, v = normal(g, 6000, 8, 64), normal(g, 1, 2, 6000, 64), normal(g, 1, 2, 6000, 64)
    k[0, 1, 0, 0] = NAN
    out = torch.empty_like(q)
    lf.window_attention(q, k, v, ints([0, 6000]), ints([6000]), out, 0, 0, 0.125)
    no_errors()
    assert torch.isnan(out[:, 4:]).all()
    for i in (0, 777, 5999):
        ref, tol = _plain.window_rows(q[i:i + 1, :4], k[:, :1], v[:, :1], [0, 1], [i + 1], 0, 0, 0.125)
        near(out[i:i + 1, :4], ref, tol)


def test_without_programmatic_launch(monkeypatch):
    """LF_PDL=0: the same bits."""
    c = prefix_case(5, [0, 2, 5], [700, 33], 700, 200, None, 8, 2, 64)
    got = []
    for mode in ("1", "0"):
        monkeypatch.setenv("LF_PDL", mode)
        kc, vc, mask = c["k"].clone(), c["v"].clone(), c["mask"].clone()
        out, w = torch.empty_like(c["q"]), torch.empty_like(c["q"])
        nxt = torch.empty(5, 2, dtype=torch.int32, device="cuda")
        lf.decode_step_prefix(c["q"], kc, vc, mask, c["nk"], c["nv"], c["ws"], c["kp"], c["vp"],
                              ints([0, 2, 5]), ints([700, 33]), out, nxt, 5, c["scale"])
        lf.window_attention(c["q"], c["kp"], c["vp"], ints([0, 2, 5]), ints([700, 33]), w, 0, 0, 0.1)
        got.append((out, nxt, mask, w))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    no_errors()


@pytest.mark.parametrize("B,S,P,fill", [(1, 2400, 700, 255), (3, 700, 2000, 127), (40, 640, 300, 255), (2, 100, 90, 255)])
@pytest.mark.parametrize("score", [False, True])
def test_prefix_workspace_of_any_contents(B, S, P, fill, score):
    """The workspace needs no preparation: sequences with, beside and after the prefixes."""
    workspace_of_any_contents(B, S, P, fill, score)


def test_prefix_workspace_of_any_contents_split_finish():
    """Long caches, whose scores a second kernel takes."""
    workspace_of_any_contents(2, 20000, 300, 255, True)


def workspace_of_any_contents(B, S, P, fill, score):
    g = gen(B + S)
    Hq, Hkv, d, N = 8, 2, 64, 3
    q, k, v = normal(g, B, Hq, d), normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    nk, nv = normal(g, B, Hkv, d), normal(g, B, Hkv, d)
    kp, vp = normal(g, N, Hkv, P, d), normal(g, N, Hkv, P, d)
    start, plen = ints([0, B // 3, B // 3, max(B // 3, B - 1)]), ints([P, P // 2, P])
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(lf.decode_prefix_workspace(B, Hq, Hkv, d, S, N, P), dtype=torch.uint8, device="cuda")
    got = []
    for contents in (0, fill, 0x41):
        mask = torch.arange(S, dtype=torch.int32).flip(0).expand(B, Hkv, S).contiguous().cuda()
        out = torch.zeros(B, Hq, d, dtype=BF, device="cuda")
        slots = torch.zeros(B, Hkv, dtype=torch.int32, device="cuda")
        ws.fill_(contents)
        if score:
            lf.decode_step_prefix(q, k, v, mask, nk, nv, write, kp, vp, start, plen, out, slots, 4, 0.1,
                                  workspace=ws)
        else:
            lf.decode_attention_prefix(q, k, v, mask, nk, nv, write, kp, vp, start, plen, out, 0.1,
                                       workspace=ws)
        got.append((out, slots))
    no_errors()
    assert not torch.isnan(got[0][0]).any()
    for out, slots in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(slots, got[0][1])


@pytest.mark.parametrize("N", [129, 300, 1000])
def test_more_prefixes_than_threads(N):
    """Each of many sequences has its own prefix, or none: against the sequences one by one."""
    g = gen(N)
    Hq, Hkv, d, S, P, B = 4, 2, 64, 70, 9, N - 3
    q, k, v = normal(g, B, Hq, d), normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    nk, nv = normal(g, B, Hkv, d), normal(g, B, Hkv, d)
    kp, vp = normal(g, N, Hkv, P, d), normal(g, N, Hkv, P, d)
    starts = [min(max(n - 1, 0), B) for n in range(N + 1)]  # prefix 0 has none, n has n - 1
    lens = [n % (P + 1) for n in range(N)]
    mask = torch.zeros(B, Hkv, S, dtype=torch.int32, device="cuda")
    write = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    out, ref = (torch.zeros(B, Hq, d, dtype=BF, device="cuda") for _ in range(2))
    lf.decode_attention_prefix(q, k, v, mask, nk, nv, write, kp, vp, ints(starts), ints(lens), out, 0.2)
    for b in list(range(0, B, 41)) + [B - 1]:
        n = b + 1
        one = slice(b, b + 1)
        lf.decode_attention_prefix(q[one], k[one], v[one], mask[one], nk[one], nv[one], write[one],
                                   kp[n:n + 1], vp[n:n + 1], ints([0, 1]), ints([lens[n]]),
                                   ref[one], 0.2)
        # Two orders of the same sums, each rounded to bf16 once from fp32.
        a, c = out[b].double(), ref[b].double()
        assert ((a - c).abs() <= 2 ** -7 * c.abs() + 1e-3).all(), b
    no_errors()
