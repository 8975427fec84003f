"""Rotation with axes, eviction by accumulated weight and the 4-bit cache against
their plain fp64 definitions (tests/_plain_long.py, which also derives the bounds)."""
import math

import pytest
import torch

import decode_kv_cache_step_gb300 as lf

import _plain
import _plain_long as plain

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


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


# --------------------------------------------------------- rotation by axes --

AXES = [  # T, Hq, Hkv, d, rot, interleaved, norm, axes
    (1, 32, 8, 128, 128, False, True, 3), (7, 8, 1, 64, 64, True, True, 2),
    (33, 6, 3, 128, 48, False, False, 4), (130, 4, 4, 64, 16, True, False, 1),
    (700, 2, 1, 128, 112, False, True, 3), (7001, 1, 1, 64, 32, True, True, 3)]


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,norm,axes", AXES)
def test_axes(T, Hq, Hkv, d, rot, inter, norm, axes):
    g = gen(T + rot)
    wide = normal(g, T, Hq + 2 * Hkv + 1, d)
    qkv = wide[:, :Hq + 2 * Hkv]                      # strided rows
    wq, wk = (normal(g, d), normal(g, d)) if norm else (None, None)
    freq = (1e4 ** (-torch.arange(rot // 2).double() * 2 / rot)).float().cuda()
    pos = torch.randint(-1000, 1 << 20, (axes, T), generator=g, dtype=torch.int32)
    pos[0, 0], pos[-1, -1] = 0, (1 << 31) - 1
    pair = torch.randint(0, axes, (rot // 2,), generator=g).tolist()
    q = torch.empty(T, Hq, d, dtype=BF, device="cuda")
    k, v = (torch.empty(T, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
    lf.qk_norm_rope_axes(qkv, wq, wk, freq, pos.cuda(), pair, q, k, v, 1e-6, interleaved=inter)
    for got, x, w in ((q, qkv[:, :Hq], wq), (k, qkv[:, Hq:Hq + Hkv], wk)):
        ref = plain.axes_rope(x, w, freq, pos, pair, 1e-6, inter)
        near(got, ref, _plain.rope_bound(ref))
    assert torch.equal(v, qkv[:, Hq + Hkv:])
    no_errors()


@pytest.mark.parametrize("T,d,rot,inter", [(1, 128, 128, False), (90, 64, 32, True), (6500, 64, 64, False)])
def test_equal_axes_are_one_axis(T, d, rot, inter):
    """Text: the same position on every axis gives the bits of the rotation without axes."""
    g = gen(T)
    qkv, w = normal(g, T, 8, d), normal(g, d)
    freq = (1e6 ** (-torch.arange(rot // 2).double() * 2 / rot)).float().cuda()
    pos = torch.randint(0, 1 << 17, (T,), generator=g, dtype=torch.int32).cuda()
    a, b = ([torch.empty(T, h, d, dtype=BF, device="cuda") for h in (4, 2, 2)] for _ in range(2))
    lf.qk_norm_rope(qkv, w, w, freq, pos, *a, interleaved=inter)
    lf.qk_norm_rope_axes(qkv, w, w, freq, pos.expand(3, T).contiguous(), torch.arange(rot // 2) % 3, *b,
                         interleaved=inter)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("nq,kv,S,extra", [
    ([5, 0, 17], [5, 0, 20], 24, 3), ([130, 257], [130, 300], 301, 11),
    ([3000, 0, 1, 3500], [3100, 0, 1, 3501], 3601, 5)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_append_axes(nq, kv, S, extra, Hq, Hkv, d):
    g = gen(S)
    B, T = len(nq), sum(nq) + extra
    starts = [sum(nq[:i]) for i in range(B + 1)]
    qkv, w = normal(g, T, Hq + 2 * Hkv, d), normal(g, d)
    freq = (1e4 ** (-torch.arange(d // 2).double() * 2 / d)).float().cuda()
    pos = torch.randint(0, 5000, (3, T), generator=g, dtype=torch.int32)
    pair = [i % 3 for i in range(d // 2)]
    q, k, v = normal(g, T, Hq, d), normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    lf.prefill_append_axes(qkv, w, w, freq, ints(starts), ints(kv), pos.cuda(), pair, q, k, v, mask)
    assert torch.equal(q[sum(nq):], q0[sum(nq):])
    for b in range(B):
        rows, at = slice(starts[b], starts[b + 1]), slice(kv[b] - nq[b], kv[b])
        ref = plain.axes_rope(qkv[rows, :Hq], w, freq, pos[:, rows], pair, 1e-6, False)
        near(q[rows], ref, _plain.rope_bound(ref))
        ref = plain.axes_rope(qkv[rows, Hq:Hq + Hkv], w, freq, pos[:, rows], pair, 1e-6, False)
        near(k[b, :, at].transpose(0, 1), ref, _plain.rope_bound(ref))
        assert torch.equal(v[b, :, at].transpose(0, 1), qkv[rows, Hq + Hkv:])
        k0[b, :, at], v0[b, :, at] = k[b, :, at], v[b, :, at]
        want = torch.full((S,), -1, dtype=torch.int32)
        want[:kv[b]] = torch.arange(kv[b] - 1, -1, -1)
        assert torch.equal(mask[b].cpu(), want.expand(Hkv, S))
    assert torch.equal(k, k0) and torch.equal(v, v0)  # every other slot as it was
    no_errors()


# ------------------------------------------------- the step with its weights --

def step_case(g, B, Hq, Hkv, d, S, live=None, holes=0.1):
    mask = torch.randint(0, S, (B, Hkv, S), generator=g, dtype=torch.int32)
    mask[torch.rand((B, Hkv, S), generator=g) < holes] = -1
    for b in range(B if live is not None else 0):
        mask[b, :, live[b % len(live)]:] = -1
    dead = mask < 0
    k, v = normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    w = torch.exp(torch.randn((B, Hkv, S), generator=g))
    # What masked slots hold does not matter.
    k[dead.cuda()], v[dead.cuda()] = NAN, INF
    w[dead] = NAN
    return dict(q=normal(g, B, Hq, d), k=k, v=v, mask=mask.cuda(), weights=w.cuda(),
                nk=normal(g, B, Hkv, d), nv=normal(g, B, Hkv, d))


def run_step(c, ws, W, scale, decay=1.0, k=None, flags=0, **kw):
    B, Hq, d = c["q"].shape
    Hkv = c["k"].shape[1]
    out = torch.full((B, Hq, d), 7.0, dtype=BF, device="cuda")
    nxt = torch.full((B, Hkv) if k is None else (B, Hkv, k), -9, dtype=torch.int32, device="cuda")
    lf.decode_step_weights(c["q"], c["k"], c["v"], c["mask"], c["weights"], c["nk"], c["nv"], ws, out,
                           nxt, W, scale, decay=decay, k=k, flags=flags, **kw)
    return out, nxt


def check_step(c, ws, W, scale, decay=1.0, k=None, flags=0, **kw):
    before = {n: t.clone() for n, t in c.items()}
    fill = bool(flags & lf.LF_STEP_FILL_EMPTY_FIRST)
    want = plain.weights_step(before["q"], before["k"], before["v"], before["mask"], before["weights"],
                              before["nk"], before["nv"], ws, W, scale, decay, k or 1, fill)
    out, nxt = run_step(c, ws, W, scale, decay, k, flags, **kw)
    near(out, want["out"], want["tol"], "out")
    live = want["mask"] >= 0
    got = c["weights"].cpu()
    near(got[live], want["weights"][live], want["wtol"][live], "weights")
    assert torch.equal(got[~live].view(torch.int32), before["weights"].cpu()[~live].view(torch.int32))
    slots = plain.chosen(got, want["mask"], W, k or 1, fill)
    assert torch.equal(nxt.cpu().view(slots.shape), slots)
    if flags & lf.LF_STEP_MASK_EVICTED:
        for b, u, i in torch.nonzero(slots >= 0).tolist():
            want["mask"][b, u, slots[b, u, i]] = -1
    assert torch.equal(c["mask"].cpu(), want["mask"])
    for name in ("k", "v"):
        want_bits = want[name].to(BF)[live]
        assert torch.equal(c[name].cpu()[live], want_bits)
    return out, nxt


STEP = [  # B, Hq, Hkv, d, S, live lengths, W, decay, k, flags
    (1, 1, 1, 64, 1, None, 0, 1.0, None, 0), (1, 4, 1, 128, 5, [0], 0, 1.0, None, 0),
    (2, 4, 2, 64, 65, None, 3, 0.5, None, 0), (1, 32, 8, 128, 700, None, 32, 1.0, None, 0),
    (3, 8, 1, 128, 129, [129, 0, 70], 100, 0.9, None, lf.LF_STEP_FILL_EMPTY_FIRST),
    (2, 8, 4, 64, 1000, [1000, 333], 0, 0.0, None, lf.LF_STEP_MASK_EVICTED),
    (2, 16, 2, 128, 333, None, 50, 1.0, 7, 0),
    (2, 2, 2, 64, 40, [40, 3], 0, 1.0, 64, lf.LF_STEP_FILL_EMPTY_FIRST | lf.LF_STEP_MASK_EVICTED),
    (1, 8, 1, 64, 4500, [3000], 10, 1.0, None, 0), (1, 2, 1, 128, 9001, [9001], 64, 0.97, None, 0),
    (1, 4, 2, 64, 8200, [8200], 64, 0.97, 3, 0), (40, 8, 8, 64, 200, [200, 0, 17], 5, 1.0, None, 0),
]


@pytest.mark.parametrize("case", STEP)
@pytest.mark.parametrize("write", [True, False])
def test_weights_step(case, write):
    B, Hq, Hkv, d, S, live, W, decay, k, flags = case
    g = gen(S + B)
    c = step_case(g, B, Hq, Hkv, d, S, live)
    ws = torch.randint(0, S, (B, Hkv), generator=g, dtype=torch.int32) if write else torch.full((B, Hkv), -1, dtype=torch.int32)
    check_step(c, ws.cuda(), W, d ** -0.5, decay, k, flags)
    no_errors()


@pytest.mark.parametrize("env", [
    {"LF_CLUSTER": "0"}, {"LF_CLUSTER": "0", "LF_CHUNK_TILES": "1"}, {"LF_CLUSTER": "1", "LF_DEEP": "0"},
    {"LF_CLUSTER": "1", "LF_DEEP": "1"}, {"LF_CLUSTER": "0", "LF_SPLIT": "1"}, {"LF_STAGES": "3"},
    {"LF_CLUSTER": "0", "LF_SPLIT": "1", "LF_SPLIT_TAIL": "1", "LF_SCORE_PARTS": "2"},
    {"LF_PDL": "0"}, {"LF_CHUNK_TILES": "32"}])
@pytest.mark.parametrize("shape", [(1, 4, 1, 128, 1029, None), (3, 16, 2, 64, 700, [700, 30, 0])])
def test_weights_step_by_every_merge(monkeypatch, env, shape):
    """Each way to merge a unit's chunks; a second step continues from the first's state."""
    for name, value in env.items():
        monkeypatch.setenv(name, value)
    B, Hq, Hkv, d, S, live = shape
    g = gen(S)
    c = step_case(g, B, Hq, Hkv, d, S, live)
    ws = torch.randint(0, S, (B, Hkv), generator=g, dtype=torch.int32).cuda()
    _, nxt = check_step(c, ws, 16, d ** -0.5, 0.9)
    check_step(c, nxt, 16, d ** -0.5, 0.9, flags=lf.LF_STEP_FILL_EMPTY_FIRST)
    no_errors()


@pytest.mark.parametrize("env", [{"LF_CLUSTER": "0", "LF_SPLIT": "1"}, {"LF_SPLIT": "0"}, {"LF_CHUNK_TILES": "1"}])
def test_several_slots_by_every_finish(monkeypatch, env):
    for name, value in env.items():
        monkeypatch.setenv(name, value)
    g = gen(9)
    for S, k, flags in ((700, 20, 0), (9001, 1024, lf.LF_STEP_FILL_EMPTY_FIRST), (130, 200, lf.LF_STEP_MASK_EVICTED)):
        c = step_case(g, 2, 4, 1, 64, S, [S, S // 3])
        check_step(c, torch.randint(0, S, (2, 1), generator=g, dtype=torch.int32).cuda(), 5, 0.125, 0.9, k, flags)
    no_errors()


@pytest.mark.parametrize("S,k", [(300, 5), (2000, 1000), (50001, 7)])
def test_several_slots_with_equal_weights(S, k):
    """Ties go to the lowest slots; caches beyond what the selection stages."""
    g = gen(S)
    c = step_case(g, 1, 1, 1, 64, S, holes=0.05)
    live = c["mask"] >= 0
    c["k"][live] = 1.0  # every live slot weighs the same
    c["weights"][live] = 0.5
    c["weights"][0, 0, 3::7] = torch.where(live[0, 0, 3::7], 0.25, c["weights"][0, 0, 3::7])
    mask = c["mask"].cpu()
    _, nxt = run_step(c, ints([[-1]]), 11, 0.125, k=k)
    assert torch.equal(nxt.cpu(), plain.chosen(c["weights"].cpu(), mask, 11, k, False))
    assert torch.unique(c["weights"][live]).numel() == 2
    no_errors()


@pytest.mark.parametrize("env", [{}, {"LF_CLUSTER": "0", "LF_SPLIT": "0"}, {"LF_CLUSTER": "0", "LF_SPLIT": "1"},
                                 {"LF_CLUSTER": "0", "LF_SPLIT": "1", "LF_SPLIT_TAIL": "1"}])
@pytest.mark.parametrize("S,k", [(16384, 3), (16385, 8), (40000, 1), (40000, 7), (40000, 9), (70001, 6), (70001, 400),
                                 (100, 8)])
def test_several_slots_of_long_caches(monkeypatch, env, S, k):
    """Exactly the lowest (weight, slot), whatever the finish and the length, ties and empty units too."""
    for name, value in env.items():
        monkeypatch.setenv(name, value)
    g = gen(S + k)
    c = step_case(g, 3, 2, 1, 64, S, [S, min(S, k // 2), 0], holes=0.1)
    c["weights"].copy_(torch.randint(1000, 1050, (3, 1, S), generator=g).float() * 1e6)  # (an addition of under 1 is lost)
    mask = c["mask"].cpu()
    _, nxt = run_step(c, ints([[-1]] * 3), 11, 0.125, k=k)
    assert torch.equal(nxt.cpu().view(3, 1, k), plain.chosen(c["weights"].cpu(), mask, 11, k, False).view(3, 1, k))
    no_errors()


def test_a_switch_that_changes_after_the_first_call(monkeypatch):
    """A plan that needs a larger workspace than the one a call of these sizes last had."""
    g = gen(10)
    c = step_case(g, 2, 8, 2, 128, 3000)
    check_step(c, ints([[1, 2], [3, 4]]), 4, 0.1)
    lf.release_workspace()
    monkeypatch.setenv("LF_CHUNK_TILES", "1")
    monkeypatch.setenv("LF_CLUSTER", "0")
    check_step(c, ints([[5, 6], [7, 8]]), 4, 0.1)
    no_errors()


def test_weights_step_long_cache_off_16_bytes():
    """Arrays whose rows do not start on 16 bytes take the other way through the scan."""
    g = gen(3)
    c = step_case(g, 1, 4, 2, 64, 5000)
    for name in ("mask", "weights"):
        wide = torch.empty(c[name].numel() + 1, dtype=c[name].dtype, device="cuda")
        t = wide[1:].view(c[name].shape)
        t.copy_(c[name])
        c[name] = t
    check_step(c, ints([[0, 4999]]), 16, 0.125, 1.0, k=3)
    check_step(c, ints([[17, -1]]), 16, 0.125, 1.0)
    no_errors()


def test_weights_step_values_that_are_not_finite():
    """A live slot's NaN weight stays and is never returned; logits of -infinity weigh nothing."""
    g = gen(5)
    c = step_case(g, 1, 2, 2, 64, 100, holes=0.0)
    c["weights"][0, 0, 3] = NAN
    c["weights"][0, 0, 5] = INF
    c["q"][0, 1] = 1.0
    c["k"][0, 1] = -INF  # every logit of unit 1
    w1 = c["weights"][0, 1].clone()
    out, nxt = run_step(c, ints([[-1, -1]]), 0, 1.0, decay=0.5)
    w = c["weights"][0].cpu()
    assert torch.isnan(w[0, 3]) and w[0, 5] == INF and nxt[0, 0] not in (3, 5)
    assert (out[0, 1] == 0).all() and torch.equal(w[1], (0.5 * w1).cpu())
    assert int(nxt[0, 1]) == int(torch.argmin(w[1]))
    no_errors()


def test_weights_step_bad_write_slot():
    g = gen(6)
    c = step_case(g, 1, 2, 2, 64, 100)
    check_step(c, ints([[100, -2]]), 0, 0.125)
    assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_WRITE_SLOT


def test_weights_steps_in_place_of_the_slot():
    """next_slots may be write_slot's own buffer: a loop of steps on one buffer."""
    g = gen(7)
    c = step_case(g, 2, 8, 2, 128, 300, holes=0.0)
    d = {n: t.clone() for n, t in c.items()}
    slot = ints([[0, 1], [2, 3]])
    out = torch.empty_like(c["q"])
    for _ in range(5):
        lf.decode_step_weights(c["q"], c["k"], c["v"], c["mask"], c["weights"], c["nk"], c["nv"], slot, out,
                               slot, 8, 0.1)
    other = ints([[0, 1], [2, 3]])
    for _ in range(5):
        _, nxt = run_step(d, other, 8, 0.1)
        other = nxt
    assert torch.equal(slot, other) and torch.equal(c["weights"], d["weights"])


# ---------------------------------------------------------- a prompt's weights --

PROMPT = [  # rows per sequence, lengths, S, counted rows
    ([1], [1], 1, 0), ([1], [200], 200, 0), ([40], [40], 40, 0), ([40, 0, 3], [40, 0, 3], 64, 0),
    ([33, 70], [161, 70], 200, 32), ([129], [400], 401, 0), ([257], [257], 260, 5),
    ([300, 1, 5], [300, 300, 300], 384, 0), ([64, 64], [64, 128], 128, 200), ([1] * 37, list(range(1, 38)), 40, 0),
    ([2, 150], [2, 511], 513, 1), ([5], [1024], 1024, 0), ([0, 0], [0, 7], 8, 0),
    ([400, 300], [400, 500], 512, 150), ([17, 400, 0], [600, 400, 9], 700, 33), ([1, 2], [1000, 3], 1000, 7),
]


@pytest.mark.parametrize("nq,kv,S,rows", PROMPT)
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (2, 2, 64), (8, 1, 64), (2, 1, 128)])
def test_prompt_weights(nq, kv, S, rows, Hq, Hkv, d):
    g = gen(S + rows)
    B, T = len(nq), sum(nq) + 2
    starts = [sum(nq[:i]) for i in range(B + 1)]
    q, k = normal(g, T, Hq, d), normal(g, B, Hkv, S, d)
    for b in range(B):
        k[b, :, kv[b]:] = NAN
    q[sum(nq):] = NAN
    w = torch.randn((B, Hkv, S), generator=g).cuda()
    w0 = w.clone()
    lf.prompt_weights(q, k, ints(starts), ints(kv), w, d ** -0.5, rows=rows)
    ref, tol = plain.prompt_weights(q, k, starts, kv, w0, rows, d ** -0.5)
    near(w, ref, tol)
    for b in range(B):
        assert torch.equal(w[b, :, kv[b]:], w0[b, :, kv[b]:])
    no_errors()


@pytest.mark.parametrize("nq,kv,rows", [([150], [3000], 0), ([150, 0, 90], [3000, 5, 2000], 0), ([400, 300], [3000, 2500], 150),
                                        ([70], [1500], 65), ([130, 1], [2900, 2900], 129)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (2, 2, 64), (8, 1, 64)])
def test_prompt_weights_of_rows_in_pieces(nq, kv, rows, Hq, Hkv, d):
    """More rows than a tile, few enough that their keys are cut into pieces."""
    g = gen(sum(kv))
    B, T, S = len(nq), sum(nq) + 1, 3100
    starts = [sum(nq[:i]) for i in range(B + 1)]
    q, k = normal(g, T, Hq, d), normal(g, B, Hkv, S, d)
    q[sum(nq):] = NAN
    w = torch.zeros(B, Hkv, S, device="cuda")
    lf.prompt_weights(q, k, ints(starts), ints(kv), w, d ** -0.5, rows=rows)
    ref, tol = plain.prompt_weights(q, k, starts, kv, torch.zeros(B, Hkv, S), rows, d ** -0.5)
    near(w, ref, tol)
    no_errors()


@pytest.mark.parametrize("rows", [0, 20])
def test_prompt_weights_are_the_same_bits_again(rows):
    g = gen(3)
    q, k = normal(g, 900, 8, 128), normal(g, 2, 2, 900, 128)
    got = []
    for _ in range(3):
        w = torch.zeros(2, 2, 900, device="cuda")
        lf.prompt_weights(q, k, ints([0, 300, 900]), ints([900, 600]), w, 0.1, rows=rows)
        got.append(w)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("d,rows", [(128, 32), (64, 32), (128, 1), (128, 200)])
def test_prompt_weights_of_few_rows_over_long_prompts(d, rows):
    """Long streams past few rows, calls back to back: the same bits, and every row gives one."""
    g = gen(17)
    lens = [8192, 5000, 7001, 8000, 6144, 300, 8191, 4097]
    q, k = normal(g, 8 * rows, 32, d), normal(g, 8, 8, 8192, d)
    starts, kv = ints([rows * b for b in range(9)]), ints(lens)
    got = []
    for _ in range(12):
        w = torch.zeros(8, 8, 8192, device="cuda")
        lf.prompt_weights(q, k, starts, kv, w, d ** -0.5, rows=rows)
        got.append(w)
    assert all(torch.equal(got[0], w) for w in got[1:])
    # Rounding, of a weight's own size: its row's sum, some 70 additions one after another,
    # 2^-18; the logarithm, the argument (below 16) and the exponential 2^-20 each.
    assert (got[0].double().sum(2) - 4 * rows).abs().max() <= 4 * rows * 2.0 ** -17
    for b, n in enumerate(lens):
        assert (got[0][b, :, n:] == 0).all()
    no_errors()


@pytest.mark.parametrize("T,rows", [(900, 0), (900, 10)])
def test_prompt_weights_waits_that_run_out(monkeypatch, T, rows):
    """Waits with no time left end the call with an error, and the next call is right."""
    g = gen(6)
    q, k = normal(g, T, 4, 128), normal(g, 1, 1, T, 128)
    w = torch.zeros(1, 1, T, device="cuda")
    monkeypatch.setenv("LF_WAIT_LIMIT_NS", "1")
    lf.prompt_weights(q, k, ints([0, T]), ints([T]), w, 0.1, rows=rows)
    assert lf.device_errors(clear=True) == lf.LF_DEVERR_WAIT_TIMEOUT
    monkeypatch.delenv("LF_WAIT_LIMIT_NS")
    lf.prompt_weights(q, k, ints([0, T]), ints([T]), w, 0.1, rows=rows)
    assert abs(float(w.double().sum()) - 4 * (rows or T)) < 1e-2
    no_errors()


def test_prompt_weights_in_chunks_add_up():
    g = gen(1)
    q, k = normal(g, 300, 4, 64), normal(g, 1, 2, 300, 64)
    one, two = (torch.full((1, 2, 300), NAN, device="cuda") for _ in range(2))
    lf.prompt_weights(q, k, ints([0, 300]), ints([300]), one, 0.125)
    lf.prompt_weights(q[:111].clone(), k, ints([0, 111]), ints([111]), two, 0.125)
    lf.prompt_weights(q[111:].clone(), k, ints([0, 189]), ints([300]), two, 0.125)
    assert (one - two).abs().max() <= 2.0 ** -11 * one.max()
    # Every row of every head gives one in all.
    assert abs(float(one.double().sum()) - 1200) < 1e-3


@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
def test_prompt_weights_scales(scale):
    g = gen(2)
    q, k = normal(g, 150, 4, 64), normal(g, 1, 1, 170, 64)
    w = torch.zeros(1, 1, 170, device="cuda")
    lf.prompt_weights(q, k, ints([0, 150]), ints([170]), w, scale)
    ref, tol = plain.prompt_weights(q, k, [0, 150], [170], torch.zeros(1, 1, 170), 0, scale)
    near(w, ref, 8 * tol)  # logits of up to 24 times those of the bound's scale 0.125


def test_prompt_weights_infinite_logits():
    """Keys of -infinity weigh nothing; a row that sees no others gives none."""
    g = gen(4)
    q, k = torch.ones(200, 1, 64, dtype=BF, device="cuda"), normal(g, 1, 1, 200, 64)
    k[0, 0, :150] = -INF
    w = torch.zeros(1, 1, 200, device="cuda")
    lf.prompt_weights(q, k, ints([0, 200]), ints([200]), w, 0.125)
    assert (w[0, 0, :150] == 0).all() and abs(float(w.double().sum()) - 50) < 1e-3
    no_errors()


def test_prompt_weights_bad_lengths():
    g = gen(8)
    q, k = normal(g, 6, 2, 64), normal(g, 3, 1, 8, 64)
    for lens in ([2, 9, 2], [2, 1, 2], [2, -1, 2]):
        w = torch.full((3, 1, 8), 7.0, device="cuda")
        lf.prompt_weights(q, k, ints([0, 2, 4, 6]), ints(lens), w, 0.125)
        assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
        assert (w[1] == 7).all() and (w[0, 0, :2] != 7).all() and (w[2, 0, :2] != 7).all()
    for bad in ([0, 9, 9, 9], [-1, 2, 4, 6], [0, 5, 3, 6]):
        w = torch.full((3, 1, 8), 7.0, device="cuda")
        lf.prompt_weights(q, k, ints(bad), ints([8, 8, 8]), w, 0.125)
        assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH


# ----------------------------------------------------------------- 4-bit cache --

def empty4(B, Hkv, S, d, fill=0):
    return (torch.full((B, Hkv, S, d // 2), fill, dtype=torch.uint8, device="cuda"),
            torch.full((B, Hkv, S, d // 32), NAN if fill else 0.0, dtype=BF, device="cuda"))


def odd_rows(g, *shape):
    """Rows with groups of zeros, tiny, huge and outlying values, and exact ties."""
    x = torch.randn(shape, generator=g)
    f = torch.randint(0, 8, shape[:-1] + (shape[-1] // 32, 1), generator=g)
    y = x.unflatten(-1, (-1, 32))
    y = torch.where(f == 0, 0.0, torch.where(f == 1, y * 1e-38, torch.where(f == 2, y * 1e37, y)))
    y[..., 0] = torch.where(f[..., 0] == 3, 30.0, y[..., 0])
    ties = torch.randint(-7, 8, y.shape, generator=g).float() - 0.5
    ties[..., 0] = 7.0
    y = torch.where(f == 4, ties, y)
    y = torch.where(f == 5, torch.round(y * 3) * 2.0 ** -133, y)  # subnormal
    return y.flatten(-2).to(BF)


@pytest.mark.parametrize("B,Hkv,d,P,S", [(1, 1, 64, 1, 1), (2, 2, 128, 70, 90), (3, 1, 64, 333, 300),
                                         (1, 3, 128, 129, 129)])
def test_kv4_pack_and_unpack(B, Hkv, d, P, S):
    g = gen(P)
    k, v = odd_rows(g, B, Hkv, P, d).cuda(), odd_rows(g, B, Hkv, P, d).cuda()
    top = min(P, S)
    first = torch.randint(0, top + 1, (B,), generator=g)
    last = torch.maximum(first, torch.randint(0, top + 1, (B,), generator=g))
    first[0], last[0] = 0, top
    (k4, ks), (v4, vs) = empty4(B, Hkv, S, d, 0x5a), empty4(B, Hkv, S, d, 0x5a)
    mask = torch.full((B, Hkv, S), -5, dtype=torch.int32, device="cuda")
    lf.kv4_pack(k, v, first.int().cuda(), last.int().cuda(), k4, ks, v4, vs, mask)
    k2, v2 = (torch.full_like(k, 7.0) for _ in range(2))
    lf.kv4_unpack(k4, ks, v4, vs, first.int().cuda(), last.int().cuda(), k2, v2)
    for x, c, s, back, piece in ((k, k4, ks, k2, 8), (v, v4, vs, v2, 4)):
        code, scale, value = plain.quantise(x)
        laid = plain.lay(code, piece)
        for b in range(B):
            i, j = int(first[b]), int(last[b])
            assert torch.equal(c[b, :, i:j].cpu(), laid[b, :, i:j])
            assert torch.equal(s[b, :, i:j].double().cpu(), scale[b, :, i:j])
            assert torch.equal(back[b, :, i:j].cpu(), value[b, :, i:j].to(BF))
            assert (c[b, :, :i] == 0x5a).all() and (c[b, :, j:] == 0x5a).all()
            assert torch.isnan(s[b, :, :i]).all() and torch.isnan(s[b, :, j:]).all()
            assert (back[b, :, :i] == 7).all() and (back[b, :, j:] == 7).all()
            assert torch.equal(mask[b, :, :j].cpu(), torch.arange(j - 1, -1, -1, dtype=torch.int32).expand(Hkv, j))
            assert (mask[b, :, j:] == -5).all()
    no_errors()


def test_kv4_pack_every_pair_of_magnitudes():
    """Codes of every quotient that two bf16 magnitudes of a binade can have."""
    x = torch.zeros(128, 128, 32)
    m = 1 + torch.arange(128) / 128
    x[:, :, 0] = 7 * m[:, None]                    # scale m exactly
    steps = torch.arange(16) / 2                   # quotients by halves, and 1/8 below and above
    for i in range(15):
        x[:, :, 1 + 2 * i] = m[None, :] * steps[1 + i] / 2
        x[:, :, 2 + 2 * i] = -(m[:, None] * steps[1 + i]).to(BF).float()
    k = x.view(1, 1, -1, 128).to(BF).cuda()
    (k4, ks), (v4, vs) = empty4(1, 1, k.shape[2], 128), empty4(1, 1, k.shape[2], 128)
    mask = torch.zeros(1, 1, k.shape[2], dtype=torch.int32, device="cuda")
    lf.kv4_pack(k, k, None, ints([k.shape[2]]), k4, ks, v4, vs, mask)
    code, scale, _ = plain.quantise(k)
    assert torch.equal(ks.double().cpu(), scale) and torch.equal(vs.double().cpu(), scale)
    assert torch.equal(k4.cpu(), plain.lay(code, 8)) and torch.equal(v4.cpu(), plain.lay(code, 4))


def test_kv4_pack_groups_that_are_not_finite():
    k = torch.ones(1, 1, 3, 64, dtype=BF, device="cuda")
    k[0, 0, 0, 5], k[0, 0, 1, 40] = NAN, -INF
    (k4, ks), (v4, vs) = empty4(1, 1, 3, 64), empty4(1, 1, 3, 64)
    mask = torch.zeros(1, 1, 3, dtype=torch.int32, device="cuda")
    lf.kv4_pack(k, k, None, ints([3]), k4, ks, v4, vs, mask)
    k2, v2 = torch.zeros_like(k), torch.zeros_like(k)
    lf.kv4_unpack(k4, ks, v4, vs, None, ints([3]), k2, v2)
    want = torch.full((3, 64), float(torch.tensor(1 / 7).to(BF)) * 7, dtype=torch.float64).to(BF)
    want[0, :32], want[1, 32:] = NAN, NAN
    assert torch.equal(torch.nan_to_num(k2[0, 0].cpu(), nan=99.0), torch.nan_to_num(want, nan=99.0))
    assert torch.equal(torch.nan_to_num(v2[0, 0].cpu(), nan=99.0), torch.nan_to_num(want, nan=99.0))


def test_kv4_bad_lengths():
    g = gen(2)
    k = normal(g, 3, 1, 8, 64)
    for first, last in (([0, 3, 0], [8, 2, 8]), ([0, -1, 0], [8, 4, 8]), ([0, 0, 0], [8, 9, 8]), ([0, 0, 0], [8, -1, 8])):
        (k4, ks), (v4, vs) = empty4(3, 1, 8, 64, 0x5a), empty4(3, 1, 8, 64, 0x5a)
        mask = torch.full((3, 1, 8), -5, dtype=torch.int32, device="cuda")
        lf.kv4_pack(k, k, ints(first), ints(last), k4, ks, v4, vs, mask)
        assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
        assert (k4[1] == 0x5a).all() and (mask[1] == -5).all() and (mask[0] >= 0).all() and (mask[2] >= 0).all()
        k2, v2 = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
        lf.kv4_unpack(k4, ks, v4, vs, ints(first), ints(last), k2, v2)
        assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_LENGTH
        assert (k2[1] == 7).all() and (v2[0] != 7).any()


def kv4_case(g, B, Hq, Hkv, d, S, live=None, holes=0.1, spread=1.0):
    mask = torch.randint(0, S, (B, Hkv, S), generator=g, dtype=torch.int32)
    mask[torch.rand((B, Hkv, S), generator=g) < holes] = -1
    for b in range(B if live is not None else 0):
        mask[b, :, live[b % len(live)]:] = -1
    k, v = normal(g, B, Hkv, S, d), normal(g, B, Hkv, S, d)
    v = (v.float() * torch.exp(spread * torch.randn((B, Hkv, S, 1), generator=g)).cuda()).to(BF)
    (k4, ks), (v4, vs) = empty4(B, Hkv, S, d), empty4(B, Hkv, S, d)
    ages = torch.empty_like(mask).cuda()
    lf.kv4_pack(k, v, None, ints([S] * B), k4, ks, v4, vs, ages)
    dead = (mask < 0).cuda()
    for t in (ks, vs):
        t[dead] = torch.tensor([NAN, INF] * (t.shape[-1] // 2), dtype=BF, device="cuda")
    return dict(q=normal(g, B, Hq, d), k4=k4, ks=ks, v4=v4, vs=vs, mask=mask.cuda(),
                nk=normal(g, B, Hkv, d), nv=normal(g, B, Hkv, d))


def run_kv4(c, ws, scale, **kw):
    out = torch.full_like(c["q"], 7.0)
    lf.decode_attention_kv4(c["q"], c["k4"], c["ks"], c["v4"], c["vs"], c["mask"], c["nk"], c["nv"], ws,
                            out, scale, **kw)
    return out


def check_kv4(c, ws, scale, **kw):
    before = {n: t.clone() for n, t in c.items()}
    S = c["mask"].shape[2]
    for b, u in [(b, u) for b in range(ws.shape[0]) for u in range(ws.shape[1])]:
        w = int(ws[b, u])
        if not 0 <= w < S:
            continue
        for new, codes, scales, piece in (("nk", "k4", "ks", 8), ("nv", "v4", "vs", 4)):
            code, s, _ = plain.quantise(before[new][b, u])
            before[codes][b, u, w] = plain.lay(code, piece).cuda()
            before[scales][b, u, w] = s.to(BF).cuda()
        before["mask"][b, u, w].clamp_(min=0)
    out = run_kv4(c, ws, scale, **kw)
    for name in ("k4", "v4", "mask"):
        assert torch.equal(c[name], before[name]), name
    for name in ("ks", "vs"):
        assert torch.equal(c[name].view(torch.int16), before[name].view(torch.int16)), name
    k, v = plain.stand_for(c["k4"], c["ks"], 8), plain.stand_for(c["v4"], c["vs"], 4)
    ref, tol = plain.kv4_attention(c["q"], k, v, c["ks"], c["vs"], c["mask"], scale)
    near(out, ref, tol, "out")
    return out


KV4 = [  # B, Hq, Hkv, d, S, live lengths
    (1, 1, 1, 64, 1, None), (1, 8, 1, 128, 3, [0]), (2, 4, 2, 64, 17, None), (1, 32, 8, 128, 700, None),
    (3, 8, 1, 128, 129, [129, 0, 70]), (2, 8, 4, 64, 1000, [1000, 333]), (2, 16, 2, 128, 2050, None),
    (1, 2, 1, 64, 5001, [4999]), (40, 8, 8, 64, 200, [200, 0, 17]), (150, 4, 4, 128, 33, [33, 1, 16, 17]),
    (80, 8, 8, 64, 2500, [2500, 31]),
]


@pytest.mark.parametrize("case", KV4)
@pytest.mark.parametrize("write", [True, False])
def test_kv4_attention(case, write):
    B, Hq, Hkv, d, S, live = case
    g = gen(S + B)
    c = kv4_case(g, B, Hq, Hkv, d, S, live)
    ws = torch.randint(0, S, (B, Hkv), generator=g, dtype=torch.int32) if write else torch.full((B, Hkv), -1, dtype=torch.int32)
    check_kv4(c, ws.cuda(), d ** -0.5)
    no_errors()


def test_kv4_attention_fills_an_empty_cache():
    """A loop that starts from nothing, slot by slot."""
    g = gen(11)
    c = kv4_case(g, 2, 4, 2, 64, 70, live=[0])
    for t in range(6):
        c["nk"], c["nv"], c["q"] = normal(g, 2, 2, 64), normal(g, 2, 2, 64), normal(g, 2, 4, 64)
        check_kv4(c, ints([[t, 69 - t], [t * 11, 15 + t]]), 0.125)
    no_errors()


def test_kv4_attention_bad_write_slot():
    c = kv4_case(gen(12), 1, 2, 2, 64, 100)
    check_kv4(c, ints([[100, -2]]), 0.125)
    assert lf.device_errors(clear=True) == lf.LF_DEVERR_BAD_WRITE_SLOT


@pytest.mark.parametrize("d,factor", [(64, 1e-30), (128, 1e30), (64, 1e-4), (128, 3e4)])
def test_kv4_attention_of_any_size_of_values(d, factor):
    """Values far from 1, and queries whose keys make up for them."""
    g = gen(13)
    c = kv4_case(g, 1, 4, 2, d, 300)
    live = (c["mask"] >= 0)[..., None]
    c["vs"] = torch.where(live, (c["vs"].float() * factor).to(BF), c["vs"])
    c["ks"] = torch.where(live, (c["ks"].float() * factor).to(BF), c["ks"])
    c["q"] = (c["q"].float() / factor).to(BF)
    check_kv4(c, ints([[-1, -1]]), d ** -0.5)
    no_errors()


def test_kv4_attention_scales_that_grow():
    """Later slots with ever larger and smaller values, the small ones with the weight."""
    g = gen(14)
    c = kv4_case(g, 1, 4, 1, 128, 600, holes=0.0, spread=0.0)
    grow = 2.0 ** (torch.arange(600, device="cuda") / 40).floor()
    c["vs"] = (c["vs"].float() * grow[:, None]).to(BF)
    check_kv4(c, ints([[-1]]), 128 ** -0.5)
    c["ks"][0, 0, 64:] = 0  # logits of 0 but for the first slots
    check_kv4(c, ints([[-1]]), 1.0)
    no_errors()


def test_kv4_attention_offsets_past_32_bits():
    """The last sequence of a cache of more than 2^32 bytes of codes, and rows written there."""
    g = gen(17)
    S, n = 1 << 20, 300
    c = kv4_case(g, 1, 2, 1, 128, n, holes=0.05)
    B = 66
    big = {}
    for name, row in (("k4", 64), ("v4", 64), ("ks", 4), ("vs", 4)):
        big[name] = torch.empty((B, 1, S, row), dtype=c[name].dtype, device="cuda")
        big[name][-1, 0, S - n:] = c[name][0, 0]
    big["mask"] = torch.full((B, 1, S), -1, dtype=torch.int32, device="cuda")
    big["mask"][-1, 0, S - n:] = c["mask"][0, 0]
    big["q"] = c["q"].expand(B, 2, 128).contiguous()
    big["nk"], big["nv"] = (c[x].expand(B, 1, 128).contiguous() for x in ("nk", "nv"))
    ws = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    ws[-1] = S - n + 7
    out = run_kv4(big, ws, 0.1)
    check_kv4(c, ints([[7]]), 0.1)
    for name in ("k4", "v4", "mask"):
        assert torch.equal(big[name][-1, 0, S - n:], c[name][0, 0])
    k, v = plain.stand_for(c["k4"], c["ks"], 8), plain.stand_for(c["v4"], c["vs"], 4)
    ref, tol = plain.kv4_attention(c["q"], k, v, c["ks"], c["vs"], c["mask"], 0.1)
    near(out[-1:], ref, tol)
    assert (out[:-1] == 0).all()
    # Packed and unpacked there too.
    x = normal(g, 1, 1, n, 128)
    P = S
    src = torch.empty((B, 1, P, 128), dtype=BF, device="cuda")
    src[-1, 0, S - n:] = x[0, 0]
    first = torch.tensor([0] * (B - 1) + [S - n], dtype=torch.int32).cuda()
    last = torch.tensor([0] * (B - 1) + [S], dtype=torch.int32).cuda()
    lf.kv4_pack(src, src, first, last, big["k4"], big["ks"], big["v4"], big["vs"], big["mask"])
    code, scale, value = plain.quantise(x[0, 0])
    assert torch.equal(big["k4"][-1, 0, S - n:].cpu(), plain.lay(code, 8))
    assert torch.equal(big["v4"][-1, 0, S - n:].cpu(), plain.lay(code, 4))
    lf.kv4_unpack(big["k4"], big["ks"], big["v4"], big["vs"], first, last, src, src.clone())
    assert torch.equal(src[-1, 0, S - n:].cpu(), value.to(BF))
    no_errors()


def test_kv4_attention_values_that_are_not_finite():
    """A live group that stands for NaN reaches its own 32 outputs of its KV head alone."""
    g = gen(15)
    c = kv4_case(g, 1, 4, 2, 128, 200, holes=0.0)
    ref = run_kv4({n: t.clone() for n, t in c.items()}, ints([[-1, -1]]), 0.1)
    c["vs"][0, 1, 77, 2] = NAN
    out = run_kv4(c, ints([[-1, -1]]), 0.1)
    bad = torch.zeros(1, 4, 128, dtype=torch.bool)
    bad[:, 2:, 64:96] = True
    assert torch.equal(torch.isnan(out).cpu(), bad)
    assert torch.equal(out[~bad.cuda()], ref[~bad.cuda()])


@pytest.mark.parametrize("scale", [-0.125, 0.0, 2.0])
def test_kv4_attention_scales(scale):
    g = gen(16)
    c = kv4_case(g, 2, 8, 1, 64, 333)
    k, v = plain.stand_for(c["k4"], c["ks"], 8), plain.stand_for(c["v4"], c["vs"], 4)
    ref, tol = plain.kv4_attention(c["q"], k, v, c["ks"], c["vs"], c["mask"], scale)
    near(run_kv4(c, ints([[-1], [-1]]), scale), ref, 4 * tol)  # logits of 16 times the bound's scale


# -------------------------------------------------------- streams and graphs --

def test_other_streams_and_workspaces():
    """Calls on a stream of the caller's, with workspaces of their own, give the same bits."""
    g = gen(21)
    s = torch.cuda.Stream()
    c = kv4_case(g, 2, 8, 2, 128, 3000)
    ws = ints([[1, 2], [3, 4]])
    a = run_kv4({n: t.clone() for n, t in c.items()}, ws, 0.1)
    e = step_case(g, 2, 8, 2, 64, 900)
    f = {n: t.clone() for n, t in e.items()}
    out, nxt = run_step(e, ws, 4, 0.1)
    q, k = normal(g, 200, 8, 64), normal(g, 1, 2, 256, 64)
    w1, w2 = torch.zeros(1, 2, 256, device="cuda"), torch.zeros(1, 2, 256, device="cuda")
    lf.prompt_weights(q, k, ints([0, 200]), ints([256]), w1, 0.1)
    torch.cuda.synchronize()
    own = torch.full((lf.decode_kv4_workspace(2, 8, 2, 128, 3000),), 0xff, dtype=torch.uint8, device="cuda")
    own2 = torch.full((lf.decode_weights_workspace(2, 8, 2, 64, 900),), 0xff, dtype=torch.uint8, device="cuda")
    own3 = torch.full((lf.prompt_weights_workspace(200, 1, 8, 2, 64, 256),), 0xff, dtype=torch.uint8, device="cuda")
    starts, lens = ints([0, 200]), ints([256])
    torch.cuda.synchronize()
    b = run_kv4(c, ws, 0.1, workspace=own, stream=s)
    out2, nxt2 = run_step(f, ws, 4, 0.1, workspace=own2, stream=s)
    lf.prompt_weights(q, k, starts, lens, w2, 0.1, workspace=own3, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(out, out2) and torch.equal(nxt, nxt2) and torch.equal(w1, w2)
    live = e["mask"] >= 0
    assert torch.equal(e["weights"][live], f["weights"][live])
    no_errors()


def test_two_graphs_at_once():
    """Two captured graphs of each call, replayed on two streams at the same time."""
    g = gen(22)
    cases = [(kv4_case(g, 4, 8, 2, 64, 5000), step_case(g, 4, 8, 2, 64, 9000),
              normal(g, 500, 8, 64), normal(g, 1, 2, 600, 64)) for _ in range(2)]
    ws = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    starts, lens = ints([0, 500]), ints([600])
    want, graphs = [], []
    for c, e, q, k in cases:
        w = torch.zeros(1, 2, 600, device="cuda")
        lf.prompt_weights(q, k, starts, lens, w, 0.1, rows=100)
        a = run_kv4(c, ws, 0.1)
        f = {n: t.clone() for n, t in e.items()}
        out, nxt = run_step(f, ws, 4, 0.1, decay=0.0)
        want.append((a, out, nxt, w))
    torch.cuda.synchronize()
    for c, e, q, k in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w = torch.zeros(1, 2, 600, device="cuda")
            lf.prompt_weights(q, k, starts, lens, w, 0.1, rows=100)
            a = run_kv4(c, ws, 0.1)
            out, nxt = run_step(e, ws, 4, 0.1, decay=0.0)
        graphs.append((graph, (a, out, nxt, w)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, got), ref in zip(graphs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    no_errors()


@pytest.mark.parametrize("rows,T", [(0, 150), (120, 400), (20, 400), (0, 1500)])
def test_a_captured_call_sees_new_inputs_and_lengths(rows, T):
    """Every form of a prompt's weights, and steps that return several slots: a replay reads what
    lies in the tensors then."""
    g = gen(23 + T)
    S = 3000
    q, k = normal(g, T, 4, 128), normal(g, 2, 1, S, 128)
    starts, lens = ints([0, T - 40, T]), ints([S, 900])
    w = torch.zeros(2, 1, S, device="cuda")
    c = step_case(g, 2, 4, 1, 128, S)
    ws = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    few, many = (torch.full((2, 1, n), -9, dtype=torch.int32, device="cuda") for n in (3, 20))
    out = torch.empty_like(c["q"])

    def calls():
        lf.prompt_weights(q, k, starts, lens, w, 0.1, rows=rows)
        for nxt in (few, many):
            lf.decode_step_weights(c["q"], c["k"], c["v"], c["mask"], c["weights"], c["nk"], c["nv"], ws, out, nxt,
                                   4, 0.1, decay=0.5, k=nxt.shape[2])

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    state = (q, lens, w, c["weights"], c["q"])
    for n in (S, 1700):
        q.copy_(normal(g, T, 4, 128))
        c["q"].copy_(normal(g, 2, 4, 128))
        lens.copy_(ints([n, n // 2 if T < 1500 else 1500]))
        w.zero_()
        before = [t.clone() for t in state]
        graph.replay()
        got = [t.clone() for t in (w, few, many, out, c["weights"])]
        for t, old in zip(state, before):
            t.copy_(old)
        calls()
        # (Bits: what masked slots hold is NaN.)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
                   for x, y in zip(got, (w, few, many, out, c["weights"])))
    no_errors()


# ------------------------------------------------------------------- together --

def test_a_long_prompt_then_tokens():
    """An image prompt in two chunks into bf16 caches, its weights, then evicting tokens over a
    full budget; and the same prompt's cache in 4 bits with tokens appended to it."""
    g = gen(31)
    B, Hq, Hkv, d, S, n1, n2 = 2, 8, 2, 64, 96, 50, 46
    freq = (1e4 ** (-torch.arange(16).double() / 16)).float().cuda()
    pair, scale = [0] * 8 + [1] * 4 + [2] * 4, d ** -0.5
    k, v = (torch.full((B, Hkv, S, d), NAN, dtype=BF, device="cuda") for _ in range(2))
    mask = torch.full((B, Hkv, S), -1, dtype=torch.int32, device="cuda")
    weights = torch.full((B, Hkv, S), NAN, device="cuda")
    total = torch.zeros((B, Hkv, S), dtype=torch.float64)
    w = torch.ones(d, dtype=BF, device="cuda")
    done = 0
    for n in (n1, n2):
        qkv = normal(g, B * n, Hq + 2 * Hkv, d)
        pos = torch.randint(0, 200, (3, B * n), generator=g, dtype=torch.int32).cuda()
        q = torch.empty(B * n, Hq, d, dtype=BF, device="cuda")
        starts, lens = ints([0, n, 2 * n]), ints([done + n] * B)
        lf.prefill_append_axes(qkv, w, w, freq, starts, lens, pos, pair, q, k, v, mask)
        out = torch.empty_like(q)
        lf.window_attention(q, k, v, starts, lens, out, 0, 0, scale)
        lf.prompt_weights(q, k, starts, lens, weights, scale)
        total, _ = plain.prompt_weights(q, k, [0, n, 2 * n], [done + n] * B, total, 0, scale)
        done += n
    near(weights, total, 2.0 ** -11 * total)
    (k4, ks), (v4, vs) = empty4(B, Hkv, S + 8, d), empty4(B, Hkv, S + 8, d)
    mask4 = torch.full((B, Hkv, S + 8), -1, dtype=torch.int32, device="cuda")
    lf.kv4_pack(k, v, None, ints([S] * B), k4, ks, v4, vs, mask4)
    c = dict(k=k, v=v, mask=mask, weights=weights)
    c4 = dict(k4=k4, ks=ks, v4=v4, vs=vs, mask=mask4)
    ws = torch.full((B, Hkv), -1, dtype=torch.int32, device="cuda")
    for t in range(5):
        qkv = normal(g, B, Hq + 2 * Hkv, d)
        pos = torch.full((3, B), S + t, dtype=torch.int32, device="cuda")
        q = torch.empty(B, Hq, d, dtype=BF, device="cuda")
        nk, nv = (torch.empty(B, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
        lf.qk_norm_rope_axes(qkv, w, w, freq, pos, pair, q, nk, nv)
        c.update(q=q, nk=nk, nv=nv)
        _, ws = check_step(c, ws, 16, scale)
        c4.update(q=q, nk=nk, nv=nv)
        check_kv4(c4, torch.full_like(ws, S + t), scale)
    no_errors()


# ------------------------------------------- logits that are not finite numbers --

@pytest.mark.parametrize("nq,kv,S,rows", [
    ([20], [20], 24, 0), ([40, 7], [130, 7], 140, 32), ([300], [300], 300, 0), ([200, 150], [450, 150], 512, 0),
    ([1100], [1100], 1100, 0), ([700, 60], [700, 900], 1000, 600)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 128), (2, 2, 64), (8, 1, 64)])
@pytest.mark.parametrize("what", [NAN, INF])
def test_prompt_weights_of_rows_that_are_not_finite(nq, kv, S, rows, Hq, Hkv, d, what):
    """A counted row whose softmax is NaN gives NaN to the keys that it sees and nothing to the others."""
    g = gen(S + Hq)
    B, T = len(nq), sum(nq)
    starts = [sum(nq[:i]) for i in range(B + 1)]
    q, k = normal(g, T, Hq, d), normal(g, B, Hkv, S, d)
    for b in range(B):
        k[b, :, kv[b]:] = NAN
    at = starts[1] - 1 - min(nq[0], rows or nq[0]) // 3  # a counted row of the first sequence
    q[at, Hq - 1] = what
    w = torch.zeros(B, Hkv, S, device="cuda")
    lf.prompt_weights(q, k, ints(starts), ints(kv), w, d ** -0.5, rows=rows)
    ref, tol = plain.prompt_weights(q, k, starts, kv, torch.zeros(B, Hkv, S), rows, d ** -0.5)
    seen = kv[0] - nq[0] + at + 1
    assert torch.isnan(ref[0, -1, :seen]).all() and not torch.isnan(ref[0, -1, seen:]).any()
    assert torch.equal(torch.isnan(w).cpu(), torch.isnan(ref))
    fine = ~torch.isnan(ref)
    near(w.cpu()[fine], ref[fine], tol[fine])
    no_errors()


@pytest.mark.parametrize("env", [
    {}, {"LF_CLUSTER": "0"}, {"LF_CLUSTER": "0", "LF_CHUNK_TILES": "1"}, {"LF_CLUSTER": "1", "LF_DEEP": "0"},
    {"LF_CLUSTER": "1", "LF_DEEP": "1"}, {"LF_CLUSTER": "0", "LF_SPLIT": "1"},
    {"LF_CLUSTER": "0", "LF_SPLIT": "1", "LF_SPLIT_TAIL": "1"}])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (4, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("others", ["finite", "masked", "-inf"])
def test_weights_step_logits_that_are_nan(monkeypatch, env, Hq, Hkv, d, others):
    """A live key of NaN or a logit of +infinity: its unit's heads have no softmax, whatever
    the other slots hold."""
    for name, value in env.items():
        monkeypatch.setenv(name, value)
    g = gen(d + Hq)
    for S, at, what in ((70, 3, NAN), (70, 69, INF), (1029, 517, NAN), (4200, 4199, NAN), (4200, 100, INF)):
        for k in (None, 3):
            c = step_case(g, 1, Hq, Hkv, d, S, holes=0.05)
            c["mask"][0, 0, at] = 5
            if others == "masked":
                c["mask"][0, 0, :at] = c["mask"][0, 0, at + 1:] = -1
            if others == "-inf" or what == INF:
                c["q"][0, :Hq // Hkv] = 1.0
            if others == "-inf":
                c["k"][0, 0, :at] = c["k"][0, 0, at + 1:] = -INF
            c["k"][0, 0, at] = what
            c["weights"][0, 0, at] = 1.0
            mask, before = c["mask"].cpu(), c["weights"].cpu()
            want = plain.weights_step(c["q"][:, Hq // Hkv:], c["k"][:, 1:], c["v"][:, 1:], c["mask"][:, 1:],
                                      c["weights"][:, 1:], c["nk"][:, 1:], c["nv"][:, 1:], ints([[-1]]), 2,
                                      d ** -0.5, 0.9, 1)
            out, nxt = run_step(c, ints([[-1, -1]]), 2, d ** -0.5, decay=0.9, k=k)
            w = c["weights"].cpu()
            live = mask[0, 0] >= 0
            assert torch.isnan(out[0, :Hq // Hkv]).all() and torch.isnan(w[0, 0][live]).all()
            assert torch.equal(w[0, 0][~live].view(torch.int32), before[0, 0][~live].view(torch.int32))
            assert (nxt[0, 0] == -1).all()
            # The other unit knows nothing of it.
            near(out[:, Hq // Hkv:], want["out"], want["tol"])
            live = mask[:, 1:] >= 0
            near(w[:, 1:][live], want["weights"][live], want["wtol"][live])
            assert torch.equal(nxt.cpu()[:, 1:].view(1, 1, k or 1), plain.chosen(w[:, 1:], mask[:, 1:], 2, k or 1, False))
    no_errors()


# --------------------------------------------- how a prompt's weights split their work --

def pieces(T, B, Hq, Hkv, d, S, rows, kept):
    """Pieces of the keys, from the workspace: (m, l) of `kept` rows each."""
    n = lf.prompt_weights_workspace(T, B, Hq, Hkv, d, S, rows)
    assert n % (8 * kept * Hq) == 0
    return n // (8 * kept * Hq)


@pytest.mark.parametrize("B,S", [(8, 8192), (3, 16384), (64, 4096)])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_prompt_weights_cut_the_keys_of_few_rows_like_those_of_a_full_tile(B, S, G):
    """A sequence's rows take a tile whether or not they fill it, so the keys have as many pieces."""
    tile = 128 // G
    full = pieces(8 * tile * B, B, 8 * G, 8, 128, S, tile, tile * B)
    for rows in {1, 3, tile // 4, tile - 1}:
        assert pieces(8 * tile * B, B, 8 * G, 8, 128, S, rows, rows * B) == full
        # All rows of short chunks too.
        assert pieces(rows * B, B, 8 * G, 8, 128, S, rows, rows * B) == full


@pytest.mark.parametrize("B,n", [(32, 10), (64, 3), (16, 30)])
def test_prompt_weights_of_many_short_chunks_leave_the_keys_whole(B, n):
    """Sequences that fill the GPU by themselves gain nothing from pieces and their join."""
    assert B * 8 >= 100  # items, each on an SM of its own
    assert pieces(B * n, B, 32, 8, 128, 4096, 0, B * n) == 1


# ------------------------------------------------ small queries beside a large one --

@pytest.mark.parametrize("d,Hq", [(64, 2), (128, 8), (128, 1)])
@pytest.mark.parametrize("low,places", [(-20, "all"), (-26, "all"), (-30, "even"), (-30, "odd"), (-33, "all")])
def test_kv4_attention_of_queries_far_below_the_largest(d, Hq, low, places):
    """One large value that meets zero keys, and values of 2^low of it whose keys make up for that.

    A query is held to 2^-34 of its head's largest value, at even places to 2^-38, and
    exactly where its last bit is above that (2^-7 of 2^-26, or of 2^-30): an error of a logit of
    at most scale * sum |k| times that, which moves the output by at most twice as much of
    sum_j p_j (|v_j| + |o|).
    """
    g = gen(d - low)
    S, scale = 300, d ** -0.5
    q = torch.zeros(1, Hq, d)
    # Magnitudes of [1, 2) times 2^low, 8 bits: no last bit below 2^(low - 7).
    small = torch.randint(128, 256, (1, Hq, d), generator=g) / 128 * 2.0 ** low
    sign = torch.randint(0, 2, (1, Hq, d), generator=g) * 2 - 1
    at = torch.arange(d)
    there = (at >= 32) & ((at % 2 == 0) | (places != "even")) & ((at % 2 == 1) | (places != "odd"))
    q[:, :, there] = (small * sign)[:, :, there]
    q[:, :, 5] = 1.0
    q = q.to(BF).cuda()
    k, v = torch.randn((1, 1, S, d), generator=g) * 2.0 ** -low, normal(g, 1, 1, S, d)
    k[..., :32] = 0
    (k4, ks), (v4, vs) = empty4(1, 1, S, d), empty4(1, 1, S, d)
    mask = torch.full((1, 1, S), -1, dtype=torch.int32, device="cuda")
    lf.kv4_pack(k.to(BF).cuda(), v, None, ints([S]), k4, ks, v4, vs, mask)
    out = torch.full_like(q, 7.0)
    lf.decode_attention_kv4(q, k4, ks, v4, vs, mask, v[:, :, 0].contiguous(), v[:, :, 0].contiguous(),
                            ints([[-1]]), out, scale)
    kk, vv = plain.stand_for(k4, ks, 8), plain.stand_for(v4, vs, 4)
    ref, tol = plain.kv4_attention(q, kk, vv, ks, vs, mask, scale)
    held = torch.where(at % 2 == 0, 2.0 ** -38, 2.0 ** -34).double()
    held[~there] = 0
    held[(2.0 ** (low - 7) >= 2 * held)] = 0  # exact
    delta = float((kk[0, 0].abs() @ held).max() * scale)
    assert (delta == 0) == (low >= -26 or places == "even")
    for h in range(Hq):
        p = torch.softmax(kk[0, 0] @ q[0, h].cpu().double() * scale, 0)
        tol[0, h] += math.expm1(2 * delta) * (p @ vv[0, 0].abs() + ref[0, h].abs())
    near(out, ref, tol)
    # (The small values do count: without them every slot weighs the same.)
    assert (ref - vv[0, 0].mean(0)).abs().max() > 0.1
    no_errors()


# --------------------------------------------- a prompt's weights: bad lengths, long prompts --

def summed(q, k, starts, lens, rows, scale):
    """Weights [B, Hkv, S] of one call over zeros, in 64 bits on the GPU, some rows at a time."""
    q, k = q.double(), k.double()
    B, Hkv, S, _ = k.shape
    G = q.shape[1] // Hkv
    w = torch.zeros(B, Hkv, S, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, kv = starts[b + 1] - starts[b], lens[b]
        at = torch.arange(kv, device="cuda")
        for i in range(max(0, n - rows) if rows else 0, n, 512):
            tok = torch.arange(i, min(n, i + 512), device="cuda")
            for h in range(Hkv * G):
                s = q[starts[b] + tok, h] @ k[b, h // G, :kv].T * scale
                s.masked_fill_(at[None] > (kv - n + tok)[:, None], -math.inf)
                w[b, h // G, :kv] += torch.softmax(s, 1).sum(0)
    return w.cpu()


@pytest.mark.parametrize("nq,kv,rows,Hq,Hkv,d", [
    # One tile of rows held in both passes.
    ([100, 40], [70001, 12345], 32, 4, 1, 128), ([7, 3], [30000, 9001], 5, 8, 2, 64),
    ([20], [262144], 1, 8, 1, 64), ([4], [1 << 20], 0, 1, 1, 64),
    # Two tiles of rows, their keys in pieces that are joined.
    ([300], [20000], 0, 8, 2, 128), ([700, 200], [20000, 16001], 130, 2, 1, 64),
    # Keys held, alone and by clusters of two and four.
    ([2500, 3], [12000, 11000], 0, 4, 2, 64), ([9000], [12000], 0, 2, 1, 64), ([2000], [10000], 0, 4, 4, 128),
    # Clusters of eight.
    ([1100], [1100], 0, 8, 1, 128), ([2000], [2000], 0, 4, 1, 128), ([5000], [5000], 0, 1, 1, 128)])
def test_prompt_weights_of_long_prompts(nq, kv, rows, Hq, Hkv, d):
    """Against 64 bits past 8192 keys, and for clusters of eight.

    A weight is off by 2^-12 of itself as in _plain_long, and sums of many terms by their
    chains of fp32 additions: a row's sum over up to 2^20 keys has at most 300 one after another
    (16 pieces, four turns, halves of a tile), a key's over 9000 rows 150: below 2^-15.
    """
    g = gen(sum(kv) + d)
    B, T, S = len(nq), sum(nq) + 1, max(kv) + (0 if max(kv) == 1 << 20 else 5)
    starts = [sum(nq[:i]) for i in range(B + 1)]
    q, k = normal(g, T, Hq, d), normal(g, B, Hkv, S, d)
    q[sum(nq):] = NAN
    for b in range(B):
        k[b, :, kv[b]:] = NAN
    w = torch.zeros(B, Hkv, S, device="cuda")
    lf.prompt_weights(q, k, ints(starts), ints(kv), w, d ** -0.5, rows=rows)
    ref = summed(q, k, starts, kv, rows, d ** -0.5)
    near(w, ref, (2.0 ** -12 + 2.0 ** -15) * ref)
    no_errors()


BAD = [  # q_start as shares of T, kv_len
    ((0, 1 / 3, 2 / 3, 1), (1400, 9999, 1300)), ((0, 1 / 3, 2 / 3, 1), (1400, 100, 1300)),
    ((0, 1 / 3, 2 / 3, 1), (1400, -1, 1300)), ((0, 1 / 3, 2, 1), (1400, 1400, 1400)),
    ((-1, 1 / 3, 2 / 3, 1), (1400, 1400, 1400)), ((0, 2 / 3, 1 / 3, 1), (1400, 1400, 1400))]


@pytest.mark.parametrize("shares,kv", BAD)
@pytest.mark.parametrize("T,rows,Hq,d", [
    (600, 0, 4, 64),      # rows in pieces that are joined, keys held by clusters of four
    (1800, 0, 8, 128),    # clusters of eight
    (600, 100, 2, 128),   # counted rows, by sequence
    (600, 20, 4, 64),     # one tile of rows held
    (27, 0, 4, 64)])      # the same, packed
def test_prompt_weights_bad_lengths_in_every_form(shares, kv, T, rows, Hq, d):
    """A sequence that does not fit keeps its weights; those beside it are right, or (where
    q_start does not ascend) right or kept."""
    g = gen(T + Hq)
    S = 1500
    starts = [int(x * T) for x in shares]
    q, k = normal(g, T, Hq, d), normal(g, 3, 1, S, d)
    w = torch.full((3, 1, S), 7.0, device="cuda")
    lf.prompt_weights(q, k, ints(starts), ints(kv), w, d ** -0.5, rows=rows)
    rows_of = [(starts[b], starts[b + 1]) for b in range(3)]
    fits = [0 <= a <= e <= T and e - a <= kv[b] <= S for b, (a, e) in enumerate(rows_of)]
    # (A length of 100 fits 9 rows.)
    assert lf.device_errors(clear=True) == (0 if all(fits) else lf.LF_DEVERR_BAD_LENGTH)
    ascends = all(0 <= a <= e <= T for a, e in rows_of)
    for b, (a, e) in enumerate(rows_of):
        # Without counted rows of its own a sequence's rows are found by their order alone.
        if not fits[b] or (not ascends and (rows == 0 or (w[b] == 7).all())):
            assert (w[b] == 7).all(), b
            continue
        ref = summed(q, k[b:b + 1], [a, e], [kv[b]], rows, d ** -0.5)[0]
        ref[:, :kv[b] - (e - a)] += 7.0
        near(w[b, :, :kv[b]], ref[:, :kv[b]], (2.0 ** -12 + 2.0 ** -15) * ref[:, :kv[b]])
        assert (w[b, :, kv[b]:] == 7).all()


# ------------------------------------------------------------- the same bits again --

@pytest.mark.parametrize("B,Hq,Hkv,d,S,k", [(1, 32, 8, 128, 2400, None), (9, 16, 2, 64, 9001, 4), (2, 8, 1, 128, 40000, None),
                                            (40, 32, 8, 128, 1500, None), (3, 4, 1, 64, 20000, 20)])
def test_steps_by_weight_are_the_same_bits_again(B, Hq, Hkv, d, S, k):
    """By clusters, the last CTA and the scoring kernel, one slot and several."""
    g = gen(B + S)
    c = step_case(g, B, Hq, Hkv, d, S, [S, S // 2])
    ws = torch.randint(0, S, (B, Hkv), generator=g, dtype=torch.int32).cuda()
    ref = None
    for _ in range(6):
        e = {n: t.clone() for n, t in c.items()}
        out, nxt = run_step(e, ws, 16, d ** -0.5, decay=0.9, k=k)
        got = [t.view(torch.uint8) for t in (out, nxt, e["weights"], e["mask"], e["k"], e["v"])]
        assert ref is None or all(torch.equal(x, y) for x, y in zip(got, ref))
        ref = got
    no_errors()


@pytest.mark.parametrize("B,Hq,Hkv,d,S", [(1, 32, 8, 128, 16384), (64, 8, 2, 64, 300), (6, 8, 1, 128, 5001)])
def test_kv4_attention_is_the_same_bits_again(B, Hq, Hkv, d, S):
    g = gen(B + S)
    c = kv4_case(g, B, Hq, Hkv, d, S, [S, S // 2])
    ws = torch.randint(0, S, (B, Hkv), generator=g, dtype=torch.int32).cuda()
    ref = None
    for _ in range(6):
        e = {n: t.clone() for n, t in c.items()}
        out = run_kv4(e, ws, d ** -0.5)
        got = [t.view(torch.uint8) for t in (out, e["mask"], e["k4"], e["ks"], e["v4"], e["vs"])]
        assert ref is None or all(torch.equal(x, y) for x, y in zip(got, ref))
        ref = got
    no_errors()


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (4, 2, 128), (8, 1, 128)])
def test_weights_step_of_one_head_without_a_softmax(Hq, Hkv, d):
    """A query of NaN: its head's output and its unit's weights, and no other head's output."""
    g = gen(d)
    for S in (40, 900, 9000):
        c = step_case(g, 1, Hq, Hkv, d, S)
        c["q"][0, 0, 3] = NAN
        G, live = Hq // Hkv, c["mask"].cpu() >= 0
        want = plain.weights_step(*(c[x] for x in ("q", "k", "v", "mask", "weights", "nk", "nv")),
                                  ints([[-1] * Hkv]), 2, 0.1, 1.0, 1)
        out, nxt = run_step(c, ints([[-1] * Hkv]), 2, 0.1)
        w = c["weights"].cpu()
        assert torch.isnan(out[0, 0]).all() and torch.isnan(w[0, 0][live[0, 0]]).all() and nxt[0, 0] == -1
        near(out[:, 1:], want["out"][:, 1:], want["tol"][:, 1:])
        near(w[:, 1:][live[:, 1:]], want["weights"][:, 1:][live[:, 1:]], want["wtol"][:, 1:][live[:, 1:]])
        assert torch.equal(nxt.cpu()[:, 1:, None], plain.chosen(w[:, 1:], c["mask"].cpu()[:, 1:], 2, 1, False))
    no_errors()


@pytest.mark.parametrize("seed", range(40))
def test_prompt_weights_of_random_batches(seed):
    """Skewed lengths, empty sequences, counted rows of every size: whatever the plan makes of them."""
    g = gen(1000 + seed)

    def pick(lo, hi):  # over the logarithm
        return int(lo * (hi / lo) ** float(torch.rand((), generator=g)))

    B, Hkv, G, d = pick(1, 40), pick(1, 4), 2 ** int(torch.randint(0, 4, (), generator=g)), 64 + 64 * (seed % 2)
    nq = [0 if torch.rand((), generator=g) < 0.15 else pick(1, 2500 // B + 2) for _ in range(B)]
    nq[0] = max(nq[0], 1)
    kv = [n + (pick(1, 3000) if torch.rand((), generator=g) < 0.6 else 0) for n in nq]
    S = max(kv) + int(torch.randint(0, 9, (), generator=g))
    rows = 0 if torch.rand((), generator=g) < 0.4 else pick(1, 400)
    starts = [sum(nq[:i]) for i in range(B + 1)]
    T = starts[B] + int(torch.randint(0, 5, (), generator=g))
    q, k = normal(g, T, Hkv * G, d), normal(g, B, Hkv, S, d)
    q[starts[B]:] = NAN
    w = torch.full((B, Hkv, S), 2.0, device="cuda")
    for b in range(B):
        k[b, :, kv[b]:] = NAN
    lf.prompt_weights(q, k, ints(starts), ints(kv), w, d ** -0.5, rows=rows)
    ref = summed(q, k, starts, kv, rows, d ** -0.5)
    for b in range(B):
        past = kv[b] - nq[b]
        ref[b, :, :past] += 2.0
        ref[b, :, kv[b] if nq[b] else 0:] = 2.0
    near(w, ref, (2.0 ** -12 + 2.0 ** -15) * ref)
    no_errors()


@pytest.mark.parametrize("Hq,d,k", [(8, 64, None), (1, 128, 5), (2, 64, 300)])
def test_weights_step_of_the_longest_cache(Hq, d, k):
    """2^20 slots, in runs of live and masked ones."""
    g = gen(Hq)
    S = 1 << 20
    c = step_case(g, 1, Hq, 1, d, S, holes=0.0)
    c["mask"][0, 0, 70000:900000] = -1
    check_step(c, ints([[S - 1]]), 64, d ** -0.5, 0.97, k)
    no_errors()


def test_kv4_attention_of_the_longest_cache():
    g = gen(5)
    S = 1 << 20
    c = kv4_case(g, 1, 8, 1, 64, S, holes=0.01)
    check_kv4(c, ints([[S - 1]]), 0.125)
    no_errors()
