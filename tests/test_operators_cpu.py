"""Refusals of the prompt and shared-prefix operators, without a GPU: the C ABI
checks sizes, pointers and overlaps on the host, the binding its tensors."""
import ctypes

import pytest
import torch

import decode_kv_cache_step_gb300 as lf
from decode_kv_cache_step_gb300 import build as lfbuild

MB = 1 << 20
FAKE = [0x100000000 + i * 256 * MB for i in range(16)]  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    lfbuild.build()
    return lf.load_library()


def norm_rope(lib, **kw):
    a = dict(qkv=FAKE[0], stride=8 * 64, wq=FAKE[1], wk=FAKE[2], freq=FAKE[3], pos=FAKE[4],
             q=FAKE[5], k=FAKE[6], v=FAKE[7], T=3, Hq=4, Hkv=2, d=64, rot=64, inter=0, eps=1e-6)
    a.update(kw)
    return lib.lf_qk_norm_rope(a["qkv"], a["stride"], a["wq"], a["wk"], a["freq"], a["pos"], a["q"],
                               a["k"], a["v"], a["T"], a["Hq"], a["Hkv"], a["d"], a["rot"],
                               a["inter"], a["eps"], None)


BAD, NO = lf.LF_ERR_INVALID_ARG, lf.LF_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    ({"qkv": None}, BAD), ({"qkv": FAKE[0] + 8}, BAD), ({"wq": None}, BAD), ({"wk": None}, BAD),
    ({"wk": FAKE[2] + 2}, BAD), ({"freq": None}, BAD), ({"pos": None}, BAD), ({"q": None}, BAD),
    ({"k": FAKE[6] + 4}, BAD), ({"v": None}, BAD), ({"T": 0}, BAD), ({"T": (1 << 22) + 1}, NO),
    ({"stride": 8 * 64 - 8}, BAD), ({"stride": 8 * 64 + 4}, BAD), ({"Hkv": 3}, BAD),
    ({"Hq": 6}, NO), ({"d": 96}, NO), ({"rot": 0}, BAD), ({"rot": 24}, BAD), ({"rot": 80}, BAD),
    ({"eps": -1.0}, BAD), ({"eps": float("nan")}, BAD),
    ({"q": FAKE[0] + 256}, BAD), ({"k": FAKE[0]}, BAD), ({"v": FAKE[6]}, BAD),
    ({"v": FAKE[5] + 512}, BAD),
])
def test_norm_rope_refusals(lib, kw, status):
    assert norm_rope(lib, **kw) == status
    assert lib.lf_last_error() != b""


def append(lib, **kw):
    a = dict(qkv=FAKE[0], stride=8 * 64, wq=None, wk=None, freq=FAKE[3], qs=FAKE[4], kv=FAKE[5],
             off=None, q=FAKE[6], k=FAKE[7], v=FAKE[8], mask=FAKE[9], T=3, B=2, Hq=4, Hkv=2, d=64,
             S=16, rot=32, inter=1, eps=1e-6)
    a.update(kw)
    return lib.lf_prefill_append(a["qkv"], a["stride"], a["wq"], a["wk"], a["freq"], a["qs"],
                                 a["kv"], a["off"], a["q"], a["k"], a["v"], a["mask"], a["T"],
                                 a["B"], a["Hq"], a["Hkv"], a["d"], a["S"], a["rot"], a["inter"],
                                 a["eps"], None)


@pytest.mark.parametrize("kw,status", [
    ({"qs": None}, BAD), ({"kv": FAKE[5] + 1}, BAD), ({"off": FAKE[10] + 2}, BAD),
    ({"mask": None}, BAD), ({"B": 0}, BAD), ({"S": 0}, BAD), ({"S": MB + 1}, NO),
    ({"B": 40000}, NO), ({"T": 0}, BAD), ({"k": FAKE[8]}, BAD), ({"q": FAKE[0]}, BAD),
    ({"d": 80}, NO), ({"rot": 128}, BAD),
])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


def window(lib, **kw):
    a = dict(q=FAKE[0], k=FAKE[1], v=FAKE[2], qs=FAKE[3], kv=FAKE[4], out=FAKE[5], T=3, B=2, Hq=4,
             Hkv=2, d=64, S=16, w=4, sinks=1, scale=0.1, ws=FAKE[6], n=1 << 30)
    a.update(kw)
    return lib.lf_window_attention(a["q"], a["k"], a["v"], a["qs"], a["kv"], a["out"], a["T"],
                                   a["B"], a["Hq"], a["Hkv"], a["d"], a["S"], a["w"], a["sinks"],
                                   a["scale"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, BAD), ({"k": FAKE[1] + 8}, BAD), ({"v": None}, BAD), ({"qs": None}, BAD),
    ({"kv": None}, BAD), ({"out": None}, BAD), ({"out": FAKE[0]}, BAD), ({"T": 0}, BAD),
    ({"T": (1 << 22) + 1}, NO), ({"w": -1}, BAD), ({"sinks": -1}, BAD), ({"w": (1 << 30) + 1}, BAD),
    ({"scale": float("inf")}, BAD), ({"d": 32}, NO), ({"Hq": 32}, NO), ({"S": MB + 1}, NO),
    ({"B": 0}, BAD), ({"out": FAKE[0] + 1024}, BAD), ({"out": FAKE[1]}, BAD),
    ({"out": FAKE[2] + 256}, BAD), ({"T": 1 << 22, "Hq": 1024, "Hkv": 1024}, NO),
])
def test_window_refusals(lib, kw, status):
    assert window(lib, **kw) == status


def prefix(lib, step, **kw):
    a = dict(q=FAKE[0], k=FAKE[1], v=FAKE[2], mask=FAKE[3], nk=FAKE[4], nv=FAKE[5], ws=FAKE[6],
             kp=FAKE[7], vp=FAKE[8], ps=FAKE[9], pl=FAKE[10], out=FAKE[11], nxt=FAKE[12], topk=1,
             flags=0, scores=None, B=2, Hq=4, Hkv=2, d=64, S=16, N=1, P=100, W=2, scale=0.1,
             work=FAKE[13], n=1 << 30)
    a.update(kw)
    head = [a[x] for x in ("q", "k", "v", "mask", "nk", "nv", "ws", "kp", "vp", "ps", "pl", "out")]
    size = [a[x] for x in ("B", "Hq", "Hkv", "d", "S", "N", "P")]
    if step:
        return lib.lf_decode_step_prefix(*head, a["nxt"], a["topk"], a["flags"], a["scores"], *size,
                                         a["W"], a["scale"], a["work"], a["n"], None)
    return lib.lf_decode_attention_prefix(*head, *size, a["scale"], a["work"], a["n"], None)


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("kw,status", [
    ({"q": None}, BAD), ({"k": None}, BAD), ({"kp": None}, BAD), ({"kp": FAKE[7] + 8}, BAD),
    ({"vp": None}, BAD), ({"ps": None}, BAD), ({"pl": FAKE[10] + 2}, BAD), ({"work": None}, BAD),
    ({"work": FAKE[13] + 16}, BAD), ({"N": 0}, BAD), ({"P": 0}, BAD), ({"P": MB + 1}, NO),
    ({"N": 40000}, NO), ({"kp": FAKE[1]}, BAD), ({"vp": FAKE[2]}, BAD), ({"out": FAKE[0]}, BAD),
    ({"kp": FAKE[2]}, BAD), ({"vp": FAKE[1]}, BAD), ({"out": FAKE[7]}, BAD), ({"out": FAKE[8]}, BAD),
    ({"d": 256}, NO), ({"B": 0}, BAD), ({"scale": float("nan")}, BAD),
])
def test_prefix_refusals(lib, step, kw, status):
    assert prefix(lib, step, **kw) == status


@pytest.mark.parametrize("kw", [{"nxt": None}, {"topk": 0}, {"topk": 1025}, {"flags": 64},
                                {"W": -1}, {"scores": FAKE[14] + 2}])
def test_prefix_step_refusals(lib, kw):
    assert prefix(lib, True, **kw) == BAD


def test_workspace_queries_refuse(lib):
    n = ctypes.c_size_t(0)
    assert lib.lf_window_attention_workspace(1, 1, 4, 2, 64, 16, 0, 0, None) == BAD
    assert lib.lf_window_attention_workspace(0, 1, 4, 2, 64, 16, 0, 0, ctypes.byref(n)) == BAD
    assert lib.lf_window_attention_workspace(1, 1, 4, 2, 96, 16, 0, 0, ctypes.byref(n)) == NO
    assert lib.lf_decode_prefix_workspace(1, 4, 2, 64, 16, 1, 16, None) == BAD
    assert lib.lf_decode_prefix_workspace(1, 4, 2, 64, 16, 0, 16, ctypes.byref(n)) == BAD
    assert lib.lf_decode_prefix_workspace(1, 4, 2, 64, 16, 1, MB + 1, ctypes.byref(n)) == NO


def test_binding_checks_tensors():
    bf = torch.bfloat16
    qkv = torch.zeros(3, 8, 64, dtype=bf)
    q, kv = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf)
    f, pos = torch.ones(32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lf.qk_norm_rope(qkv, None, None, f, pos, q, kv, kv.clone())
    with pytest.raises(ValueError, match="k_out"):
        lf.qk_norm_rope(qkv, None, None, f, pos, q, kv[0], kv)
    cache, ln = torch.zeros(1, 2, 16, 64, dtype=bf), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lf.window_attention(q, cache, cache, torch.zeros(2, dtype=torch.int32), ln, q, 0, 0, 0.1)
    with pytest.raises(ValueError, match="k_cache"):
        lf.prefill_append(qkv, None, None, f, ln, ln, q, kv, kv, ln)
    with pytest.raises(ValueError, match="CUDA"):
        lf.decode_attention_prefix(q[:1], cache, cache, ln, kv[:1], kv[:1], ln, cache, cache, ln, ln,
                                   q[:1], 0.1)
