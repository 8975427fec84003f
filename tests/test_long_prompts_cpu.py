"""Refusals of the rotation with axes, of eviction by accumulated weight and of the
4-bit cache, without a GPU; the plain definitions' own pins; the binding's checks."""
import ctypes
import os
import subprocess
import sys

import numpy
import pytest
import torch

import decode_kv_cache_step_gb300 as lf
from decode_kv_cache_step_gb300 import _binding as binding
from decode_kv_cache_step_gb300 import build as lfbuild

import _plain_long as plain

MB = 1 << 20
FAKE = [0x100000000 + i * 256 * MB for i in range(16)]  # never dereferenced
BAD, NO = lf.LF_ERR_INVALID_ARG, lf.LF_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    lfbuild.build()
    return lf.load_library()


# -------------------------------------------------------------------- the C ABI --

def axes(lib, **kw):
    a = dict(qkv=FAKE[0], stride=8 * 64, wq=FAKE[1], wk=FAKE[2], freq=FAKE[3], pos=FAKE[4],
             pair=bytes([0, 1, 2, 0] * 8), axes=3, q=FAKE[5], k=FAKE[6], v=FAKE[7], T=3, Hq=4, Hkv=2,
             d=64, rot=64, inter=0, eps=1e-6)
    a.update(kw)
    return lib.lf_qk_norm_rope_axes(
        a["qkv"], a["stride"], a["wq"], a["wk"], a["freq"], a["pos"], a["pair"], a["axes"], a["q"],
        a["k"], a["v"], a["T"], a["Hq"], a["Hkv"], a["d"], a["rot"], a["inter"], a["eps"], None)


@pytest.mark.parametrize("kw,status", [
    ({"qkv": None}, BAD), ({"pos": None}, BAD), ({"pos": FAKE[4] + 2}, BAD), ({"pair": None}, BAD),
    ({"axes": 0}, BAD), ({"axes": lf.LF_MAX_AXES + 1}, BAD), ({"axes": 2}, BAD), ({"axes": -1}, BAD),
    ({"pair": bytes([255] * 32)}, BAD), ({"T": 0}, BAD), ({"rot": 24}, BAD),
    ({"rot": 128, "pair": bytes(64)}, BAD),
    ({"d": 96}, NO), ({"Hq": 6}, NO), ({"v": FAKE[6]}, BAD), ({"eps": float("nan")}, BAD),
    ({"stride": 8 * 64 + 4}, BAD), ({"wk": None}, BAD),
])
def test_axes_refusals(lib, kw, status):
    assert axes(lib, **kw) == status
    assert lib.lf_last_error() != b""


def append_axes(lib, **kw):
    a = dict(qkv=FAKE[0], stride=8 * 64, wq=None, wk=None, freq=FAKE[3], qs=FAKE[4], kv=FAKE[5],
             pos=FAKE[10], pair=bytes([0, 1] * 8), axes=2, q=FAKE[6], k=FAKE[7], v=FAKE[8], mask=FAKE[9],
             T=3, B=2, Hq=4, Hkv=2, d=64, S=16, rot=32, inter=1, eps=1e-6)
    a.update(kw)
    return lib.lf_prefill_append_axes(
        a["qkv"], a["stride"], a["wq"], a["wk"], a["freq"], a["qs"], a["kv"], a["pos"], a["pair"],
        a["axes"], a["q"], a["k"], a["v"], a["mask"], a["T"], a["B"], a["Hq"], a["Hkv"], a["d"],
        a["S"], a["rot"], a["inter"], a["eps"], None)


@pytest.mark.parametrize("kw,status", [
    ({"qs": None}, BAD), ({"kv": FAKE[5] + 1}, BAD), ({"pos": None}, BAD), ({"mask": None}, BAD),
    ({"axes": 1}, BAD), ({"axes": 5}, BAD), ({"pair": None}, BAD), ({"B": 0}, BAD), ({"S": MB + 1}, NO),
    ({"k": FAKE[8]}, BAD), ({"q": FAKE[0]}, BAD), ({"rot": 144}, BAD),
    ({"rot": 128, "pair": bytes([0, 1] * 32)}, BAD),
])
def test_append_axes_refusals(lib, kw, status):
    assert append_axes(lib, **kw) == status


def weights(lib, **kw):
    a = dict(q=FAKE[0], k=FAKE[1], v=FAKE[2], mask=FAKE[3], w=FAKE[4], nk=FAKE[5], nv=FAKE[6],
             ws=FAKE[7], out=FAKE[8], next=FAKE[9], topk=1, flags=0, B=2, Hq=4, Hkv=2, d=64, S=16, W=2,
             scale=0.1, decay=1.0, work=FAKE[10], n=1 << 30)
    a.update(kw)
    return lib.lf_decode_step_weights(
        a["q"], a["k"], a["v"], a["mask"], a["w"], a["nk"], a["nv"], a["ws"], a["out"], a["next"],
        a["topk"], a["flags"], a["B"], a["Hq"], a["Hkv"], a["d"], a["S"], a["W"], a["scale"],
        a["decay"], a["work"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, BAD), ({"k": FAKE[1] + 8}, BAD), ({"v": None}, BAD), ({"mask": None}, BAD),
    ({"w": None}, BAD), ({"w": FAKE[4] + 2}, BAD), ({"nk": None}, BAD), ({"nv": FAKE[6] + 2}, BAD),
    ({"ws": None}, BAD), ({"out": None}, BAD), ({"next": None}, BAD), ({"topk": 0}, BAD),
    ({"topk": lf.LF_MAX_TOPK + 1}, BAD), ({"flags": 8}, BAD), ({"flags": lf.LF_STEP_LOG2_SCORES}, BAD),
    ({"W": -1}, BAD), ({"scale": float("inf")}, BAD), ({"decay": -0.1}, BAD), ({"decay": 1.5}, BAD),
    ({"decay": float("nan")}, BAD), ({"S": 0}, BAD), ({"S": MB + 1}, NO), ({"Hq": 6}, NO), ({"Hkv": 3}, BAD),
    ({"d": 32}, NO), ({"B": 40000}, NO), ({"w": FAKE[3]}, BAD), ({"w": FAKE[1] + 64}, BAD),
    ({"w": FAKE[2]}, BAD), ({"w": FAKE[8]}, BAD), ({"out": FAKE[0]}, BAD), ({"work": None}, BAD),
    ({"work": FAKE[10] + 128}, BAD),
])
def test_weights_step_refusals(lib, kw, status):
    assert weights(lib, **kw) == status


def prompt(lib, **kw):
    a = dict(q=FAKE[0], k=FAKE[1], qs=FAKE[2], kv=FAKE[3], w=FAKE[4], T=3, B=2, Hq=4, Hkv=2, d=64, S=16,
             rows=0, scale=0.1, work=FAKE[5], n=1 << 30)
    a.update(kw)
    return lib.lf_prompt_weights(a["q"], a["k"], a["qs"], a["kv"], a["w"], a["T"], a["B"], a["Hq"],
                                 a["Hkv"], a["d"], a["S"], a["rows"], a["scale"], a["work"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, BAD), ({"k": FAKE[1] + 8}, BAD), ({"qs": None}, BAD), ({"kv": None}, BAD),
    ({"w": None}, BAD), ({"w": FAKE[4] + 1}, BAD), ({"T": 0}, BAD), ({"T": (1 << 22) + 1}, NO),
    ({"rows": -1}, BAD), ({"scale": float("nan")}, BAD), ({"d": 32}, NO), ({"Hq": 32}, NO),
    ({"S": MB + 1}, NO), ({"B": 0}, BAD), ({"w": FAKE[0]}, BAD), ({"w": FAKE[1] + 256}, BAD),
    ({"work": None}, BAD), ({"work": FAKE[5] + 64}, BAD), ({"T": 1 << 22, "Hq": 1024, "Hkv": 1024}, NO),
])
def test_prompt_weights_refusals(lib, kw, status):
    assert prompt(lib, **kw) == status


def pack(lib, unpack, **kw):
    a = dict(k=FAKE[0], v=FAKE[1], first=FAKE[2], kv=FAKE[3], k4=FAKE[4], ks=FAKE[5], v4=FAKE[6],
             vs=FAKE[7], mask=FAKE[8], B=2, Hkv=2, d=64, P=16, S=32)
    a.update(kw)
    if unpack:
        return lib.lf_kv4_unpack(a["k4"], a["ks"], a["v4"], a["vs"], a["first"], a["kv"], a["k"], a["v"],
                                 a["B"], a["Hkv"], a["d"], a["P"], a["S"], None)
    return lib.lf_kv4_pack(a["k"], a["v"], a["first"], a["kv"], a["k4"], a["ks"], a["v4"], a["vs"],
                           a["mask"], a["B"], a["Hkv"], a["d"], a["P"], a["S"], None)


@pytest.mark.parametrize("kw,status", [
    ({"k": None}, BAD), ({"v": FAKE[1] + 8}, BAD), ({"first": FAKE[2] + 2}, BAD), ({"kv": None}, BAD),
    ({"k4": None}, BAD), ({"k4": FAKE[4] + 8}, BAD), ({"ks": None}, BAD), ({"v4": None}, BAD),
    ({"vs": FAKE[7] + 4}, BAD), ({"B": 0}, BAD), ({"B": 40000}, NO), ({"d": 32}, NO), ({"P": 0}, BAD),
    ({"S": 0}, BAD), ({"P": MB + 1}, NO), ({"S": MB + 1}, NO), ({"v4": FAKE[4]}, BAD),
    ({"vs": FAKE[5] + 16}, BAD), ({"k4": FAKE[0]}, BAD), ({"ks": FAKE[1]}, BAD),
])
@pytest.mark.parametrize("unpack", [False, True])
def test_kv4_pack_refusals(lib, unpack, kw, status):
    assert pack(lib, unpack, **kw) == status


def test_kv4_pack_needs_a_mask_and_unpack_two_outputs(lib):
    assert pack(lib, False, mask=None) == BAD
    assert pack(lib, True, v=FAKE[0]) == BAD


def kv4(lib, **kw):
    a = dict(q=FAKE[0], k4=FAKE[1], ks=FAKE[2], v4=FAKE[3], vs=FAKE[4], mask=FAKE[5], nk=FAKE[6],
             nv=FAKE[7], ws=FAKE[8], out=FAKE[9], B=2, Hq=4, Hkv=2, d=64, S=16, scale=0.1, work=FAKE[10],
             n=1 << 30)
    a.update(kw)
    return lib.lf_decode_attention_kv4(
        a["q"], a["k4"], a["ks"], a["v4"], a["vs"], a["mask"], a["nk"], a["nv"], a["ws"], a["out"],
        a["B"], a["Hq"], a["Hkv"], a["d"], a["S"], a["scale"], a["work"], a["n"], None)


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, BAD), ({"k4": FAKE[1] + 8}, BAD), ({"ks": None}, BAD), ({"v4": None}, BAD),
    ({"vs": None}, BAD), ({"mask": FAKE[5] + 2}, BAD), ({"nk": None}, BAD), ({"nv": FAKE[7] + 8}, BAD),
    ({"ws": None}, BAD), ({"out": None}, BAD), ({"scale": float("inf")}, BAD), ({"S": 0}, BAD),
    ({"S": MB + 1}, NO), ({"Hq": 6}, NO), ({"d": 256}, NO), ({"B": 40000}, NO), ({"out": FAKE[0]}, BAD),
    ({"out": FAKE[1]}, BAD), ({"v4": FAKE[1] + 16}, BAD), ({"q": FAKE[4]}, BAD),
])
def test_kv4_attention_refusals(lib, kw, status):
    assert kv4(lib, **kw) == status


def test_workspace_sizes_refuse(lib):
    n = ctypes.c_size_t(0)
    p = ctypes.byref(n)
    assert lib.lf_decode_weights_workspace(1, 4, 2, 64, 16, 1, None) == BAD
    assert lib.lf_decode_weights_workspace(1, 4, 2, 64, 16, 0, p) == BAD
    assert lib.lf_decode_weights_workspace(1, 4, 2, 48, 16, 1, p) == NO
    assert lib.lf_prompt_weights_workspace(3, 1, 4, 2, 64, 16, 0, None) == BAD
    assert lib.lf_prompt_weights_workspace(3, 1, 4, 2, 64, 16, -1, p) == BAD
    assert lib.lf_prompt_weights_workspace(0, 1, 4, 2, 64, 16, 0, p) == BAD
    assert lib.lf_decode_kv4_workspace(1, 4, 2, 64, 16, None) == BAD
    assert lib.lf_decode_kv4_workspace(1, 4, 3, 64, 16, p) == BAD


# ------------------------------------------------------------------ the binding --

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    with pytest.raises(ValueError, match="q_out"):
        lf.qk_norm_rope_axes(t(3, 8, 64), None, None, t(16, dtype=f32), t(2, 3, dtype=i32), [0] * 16,
                             t(3, 4, 64), t(3, 2, 64), t(3, 2, 64))
    with pytest.raises(ValueError, match="pair_axis"):
        lf.qk_norm_rope_axes(t(3, 8, 64), None, None, t(16, dtype=f32), t(2, 3, dtype=i32), [0] * 15,
                             t(3, 4, 64), t(3, 2, 64), t(3, 2, 64))
    with pytest.raises(ValueError, match="pair_axis"):
        lf.qk_norm_rope_axes(t(3, 8, 64), None, None, t(16, dtype=f32), t(2, 3, dtype=i32), [300] * 16,
                             t(3, 4, 64), t(3, 2, 64), t(3, 2, 64))
    with pytest.raises(ValueError, match="positions"):
        lf.prefill_append_axes(t(3, 8, 64), None, None, t(16, dtype=f32), t(2, dtype=i32), t(1, dtype=i32),
                               t(3, dtype=i32), [0] * 16, t(3, 4, 64), t(1, 2, 8, 64), t(1, 2, 8, 64),
                               t(1, 2, 8, dtype=i32))
    c = t(1, 2, 8, 64)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lf.decode_step_weights(t(1, 4, 64), c, c, t(1, 2, 8, dtype=i32), t(1, 2, 8, dtype=f32), t(1, 2, 64),
                               t(1, 2, 64), t(1, 2, dtype=i32), t(1, 4, 64), t(1, 2, dtype=i32), 0, 0.1)
    with pytest.raises(ValueError, match="q must be"):
        lf.prompt_weights(t(3, 64), c, t(2, dtype=i32), t(1, dtype=i32), t(1, 2, 8, dtype=f32), 0.1)
    with pytest.raises(TypeError, match="expected torch.Tensors"):
        lf.prompt_weights(None, c, t(2, dtype=i32), t(1, dtype=i32), t(1, 2, 8, dtype=f32), 0.1)
    with pytest.raises(ValueError, match="k4"):
        lf.kv4_pack(c, c, None, t(1, dtype=i32), t(2, 8, 32, dtype=u8), t(1, 2, 8, 2), t(1, 2, 8, 32, dtype=u8),
                    t(1, 2, 8, 2), t(1, 2, 8, dtype=i32))
    with pytest.raises(TypeError, match="mask"):
        lf.kv4_pack(c, c, None, t(1, dtype=i32), t(1, 2, 8, 32, dtype=u8), t(1, 2, 8, 2),
                    t(1, 2, 8, 32, dtype=u8), t(1, 2, 8, 2), None)
    with pytest.raises(TypeError, match="kv_len"):
        lf.kv4_unpack(t(1, 2, 8, 32, dtype=u8), t(1, 2, 8, 2), t(1, 2, 8, 32, dtype=u8), t(1, 2, 8, 2), None,
                      None, c, c)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        lf.decode_attention_kv4(t(1, 4, 64), t(1, 2, 8, 32, dtype=u8), t(1, 2, 8, 2),
                                t(1, 2, 8, 32, dtype=u8), t(1, 2, 8, 2), t(1, 2, 8, dtype=i32), t(1, 2, 64),
                                t(1, 2, 64), t(1, 2, dtype=i32), t(1, 4, 64), 0.1)


# ---------------------------------------------------- the plain definitions' pins --

def test_quantise_by_hand():
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 7.0, 2.5, -3.5, 0.5   # scale 1: ties to even
    code, s, value = plain.quantise(x)
    assert s.tolist() == [[1.0, 0.0]] and code[0, :4].tolist() == [7, 2, -4, 0]
    assert value[0, :4].tolist() == [7.0, 2.0, -4.0, 0.0] and (code[0, 32:] == 0).all()
    keys, values = plain.lay(code, 8), plain.lay(code, 4)
    # Group 0's first piece lies first; group 1's (codes 0 + 8) follows it.
    assert keys[0, :8].tolist() == [0xaf, 0x84, 0x88, 0x88, 0x88, 0x88, 0x88, 0x88]
    assert values[0, :4].tolist() == [0xaf, 0x84, 0x88, 0x88]
    g = torch.Generator().manual_seed(1)
    x = torch.randn((3, 128), generator=g).to(torch.bfloat16)
    code, s, value = plain.quantise(x)
    for piece in (4, 8):
        assert torch.equal(plain.stand_for(plain.lay(code, piece), s, piece), value)


def test_chosen_by_hand():
    w = torch.tensor([[[3.0, 1.0, 1.0, float("nan"), 0.5, 9.0]]])
    mask = torch.tensor([[[5, 5, 5, 5, 0, -1]]], dtype=torch.int32)
    assert plain.chosen(w, mask, 1, 4, False).tolist() == [[[1, 2, 0, -1]]]
    assert plain.chosen(w, mask, 1, 2, True).tolist() == [[[5, 1]]]


def test_prompt_weights_by_hand():
    # Two tokens, one head, equal logits: the first gets 1 + 1/2, the second 1/2.
    q, k = torch.zeros(2, 1, 64), torch.zeros(1, 1, 3, 64)
    w, _ = plain.prompt_weights(q, k, [0, 2], [2], torch.full((1, 1, 3), 7.0), 0, 1.0)
    assert w.tolist() == [[[1.5, 0.5, 7.0]]]
    w, _ = plain.prompt_weights(q, k, [0, 2], [3], torch.full((1, 1, 3), 7.0), 1, 1.0)
    assert torch.allclose(w, torch.tensor([[[7 + 1 / 3, 1 / 3, 1 / 3]]], dtype=torch.float64))


# ------------------------------------------------------------ the compiled checks --

def test_importing_the_package_maps_no_library(lib):
    """Both libraries are loaded by the first call, not by the import."""
    code = ("import decode_kv_cache_step_gb300 as lf\n"
            "ours = lambda: {n for n in ('liblf_decode', '_lf_check') if n in open('/proc/self/maps').read()}\n"
            "assert not ours(), ours()\n"
            "lf.load_library()\n"
            "print(sorted(ours()))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
    assert "liblf_decode" in r.stdout
    assert ("_lf_check" in r.stdout) == os.path.exists(lfbuild.CHECK_PATH)


@pytest.fixture
def own_lib(tmp_path, monkeypatch):
    """The build's output in a folder of its own, compilers replaced by a record of their calls."""
    for name in ("LIB_PATH", "CHECK_PATH", "STAMP_PATH"):
        monkeypatch.setattr(lfbuild, name, str(tmp_path / os.path.basename(getattr(lfbuild, name))))
    monkeypatch.setattr(lfbuild, "LIB_DIR", str(tmp_path))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(lfbuild.subprocess, "run", run)
    open(lfbuild.LIB_PATH, "w").close()  # newer than every source
    return ran


def compiled(ran):
    n = sum(lfbuild.CHECK_SRC in cmd for cmd in ran)
    assert n == len(ran)  # nothing else
    ran.clear()
    return n


def test_build_renews_stale_checks_alone(own_lib, monkeypatch):
    lfbuild.build()
    assert compiled(own_lib) == 1  # missing
    lfbuild.build()
    assert compiled(own_lib) == 0
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "9.9.9")
        lfbuild.build()
        assert compiled(own_lib) == 1  # for another torch
        lfbuild.build()
        assert compiled(own_lib) == 0
    lfbuild.build()
    assert compiled(own_lib) == 1
    os.utime(lfbuild.CHECK_PATH, (1, 1))  # older than its source
    lfbuild.build()
    assert compiled(own_lib) == 1
    os.unlink(lfbuild.STAMP_PATH)
    lfbuild.build()
    assert compiled(own_lib) == 1


def test_build_warns_where_the_checks_do_not_compile(own_lib, monkeypatch):
    """Whatever fails there, the library is built and the binding checks in Python."""
    def fails(cmd, **kw):
        return subprocess.CompletedProcess(cmd, 1, "", "no such header")

    lfbuild.build()
    os.unlink(lfbuild.STAMP_PATH)
    with monkeypatch.context() as m:
        m.setattr(lfbuild.subprocess, "run", fails)
        with pytest.warns(UserWarning, match="no such header"):
            assert lfbuild.build() == lfbuild.LIB_PATH
    assert not os.path.exists(lfbuild.CHECK_PATH)  # nor a stale one, or pieces of one
    assert sorted(os.listdir(lfbuild.LIB_DIR)) == [os.path.basename(lfbuild.LIB_PATH)]
    with monkeypatch.context() as m:
        m.delattr(torch._C, "_GLIBCXX_USE_CXX11_ABI")
        with pytest.warns(UserWarning, match="_GLIBCXX_USE_CXX11_ABI"):
            assert lfbuild.build() == lfbuild.LIB_PATH
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)  # import torch raises ImportError
        with pytest.warns(UserWarning, match="was not built"):
            assert lfbuild.build() == lfbuild.LIB_PATH


# -------------------------------------------------------------- the pairs' axes --

@pytest.mark.parametrize("make", [list, tuple, bytes, bytearray, numpy.array, torch.tensor,
                                  lambda x: numpy.array(x, dtype=numpy.uint8),
                                  lambda x: torch.tensor(x, dtype=torch.uint8), iter])
def test_pair_axis_is_read_entry_by_entry(make):
    pairs = [0, 1, 2, 0, 1, 2, 0, 1]
    got = binding._check_axes(torch.zeros(3, 5, dtype=torch.int32), make(pairs), 16)
    assert got == (3, bytes(pairs))


@pytest.mark.parametrize("wrong", [
    numpy.array([1]), numpy.int64(1), numpy.array([1, 2], dtype=numpy.int32),  # 8 bytes of memory each
    8, 2.0, None, "01201201", [0, 1, 2], [0.0] * 8, [0, 1, 2, 0, 1, 2, 0, 256], [0, 1, 2, 0, 1, 2, 0, -1],
    numpy.zeros(8), torch.zeros(8), torch.zeros(2, 4, dtype=torch.int32)])
def test_pair_axis_of_another_length_or_kind_is_refused(wrong):
    with pytest.raises(ValueError, match="pair_axis"):
        binding._check_axes(torch.zeros(3, 5, dtype=torch.int32), wrong, 16)
