"""The vocabulary-head operators' boundary without a GPU: exported names, workspace
sizes, and the refusal of bad arguments before anything is enqueued, in C and in
the torch front end."""
import ctypes
import os
import re

import pytest

import draft_verification_spec_amd as sv

torch = pytest.importorskip("torch")

FAKE = 0x1000                                         # never dereferenced: every call below is refused first
WS = 0x100000
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


def test_exports_every_declared_function(lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "sv_head.h")).read()
    names = set(re.findall(r"^(?:int|size_t) (sv_\w+)\(", text, flags=re.M))
    assert names == {"sv_act8_pack", "sv_act8_unpack", "sv_head_logits", "sv_head_logits_workspace_bytes", "sv_head_ce",
                     "sv_head_ce_workspace_bytes", "sv_head_kd", "sv_head_kd_workspace_bytes"}
    for n in names:
        assert hasattr(lib, n), n


def test_act8_refusals(lib):
    def pack(N=4, H=8, dt=0, x=FAKE, xs=0, c=FAKE, cs=0, s=FAKE):
        return lib.sv_act8_pack(N, H, dt, x, xs, c, cs, s, None)

    def unpack(N=4, H=8, c=FAKE, cs=0, s=FAKE, dt=0, y=FAKE):
        return lib.sv_act8_unpack(N, H, c, cs, s, dt, y, None)
    for f in (pack, unpack):
        assert f(dt=2) == f(dt=-1) == sv.SV_ERR_DTYPE
        assert f(N=-1) == f(H=0) == f(H=131073) == f(cs=7) == f(cs=-1) == sv.SV_ERR_SHAPE
        assert f(c=None) == f(s=None) == sv.SV_ERR_NULL
        assert f(N=0, c=None, s=None) == sv.SV_OK
    assert pack(xs=7) == sv.SV_ERR_SHAPE and pack(x=None) == sv.SV_ERR_NULL and unpack(y=None) == sv.SV_ERR_NULL


def test_logits_refusals(lib):
    def shape(N=4, H=64, V=100, hd=0, od=1, hs=0, ws=0, os=0):
        return sv.sv_logits_shape_t(N, H, V, hd, od, hs, ws, os)

    def call(s, h=FAKE, hsc=FAKE, c=FAKE, sc=FAKE, o=FAKE, w=WS, wb=1 << 40):
        return lib.sv_head_logits(None if s is None else ctypes.byref(s), h, hsc, c, sc, o, w, wb, None)

    def need(s):
        return lib.sv_head_logits_workspace_bytes(ctypes.byref(s))
    assert call(None) == sv.SV_ERR_NULL
    assert call(shape(hd=3)) == call(shape(od=2)) == call(shape(od=-1)) == sv.SV_ERR_DTYPE
    for bad in (shape(N=-1), shape(H=0), shape(H=131073), shape(V=0), shape(V=(1 << 24) + 1), shape(hs=63), shape(ws=63),
                shape(os=99), shape(hs=-64), shape(N=2147483647, V=1 << 24)):
        assert call(bad) == sv.SV_ERR_SHAPE and need(bad) == 0
    good = shape()
    for k in ("h", "c", "sc", "o"):
        assert call(good, **{k: None}) == sv.SV_ERR_NULL, k
    assert call(shape(hd=2), hsc=None) == sv.SV_ERR_NULL
    assert call(good, w=None) == call(good, wb=need(good) - 1) == call(good, w=WS + 8) == sv.SV_ERR_WORKSPACE
    assert call(shape(N=0)) == sv.SV_OK
    assert 0 < need(good) < need(shape(N=1024, H=4096, V=128256))


def head(N=4, H=64, V=100, dt=1, hd=None, g=3, hs=0, ws=0, T=1.0, S=4, G=2, wm=INF):
    return sv.sv_head_shape_t(N, H, V, dt, dt if hd is None else hd, g, hs, ws, T, -1, S, G, wm)


@pytest.mark.parametrize("kd", [False, True])
def test_loss_refusals(lib, kd):
    need = lambda s: (lib.sv_head_kd_workspace_bytes if kd else lib.sv_head_ce_workspace_bytes)(ctypes.byref(s))  # noqa: E731

    def call(s, **over):
        a = dict(h=FAKE, hsc=FAKE, w=FAKE, t=FAKE, t2=FAKE, t3=FAKE, t4=FAKE, rows=FAKE, more=None, st=None, loss=FAKE,
                 gh=FAKE, gw=FAKE, ws=WS, wb=1 << 50)
        a.update(over)
        ins = [a["t"], a["t2"], a["t3"], a["t4"]] if kd else [a["t"], None]
        f = lib.sv_head_kd if kd else lib.sv_head_ce
        return f(None if s is None else ctypes.byref(s), a["h"], a["hsc"], a["w"], *ins, a["rows"], a["more"], a["st"],
                 a["loss"], a["gh"], a["gw"], a["ws"], a["wb"], None)
    assert call(None) == sv.SV_ERR_NULL
    assert call(head(dt=2)) == call(head(dt=5)) == call(head(dt=1, hd=0)) == call(head(hd=9)) == sv.SV_ERR_DTYPE
    for T in (0.0, -1.0, float("nan"), INF):
        assert call(head(T=T)) == sv.SV_ERR_TEMPERATURE
    bad = [head(N=-1), head(N=(1 << 20) + 1), head(H=0), head(H=131073), head(V=0), head(V=(1 << 24) + 1), head(g=4),
           head(g=-1), head(hs=63), head(ws=63), head(hs=-64)]
    if kd:
        bad += [head(T=0.5), head(S=0), head(S=3), head(G=0), head(wm=0.0), head(wm=float("nan"))]
    for s in bad:
        assert call(s) == sv.SV_ERR_SHAPE and need(s) == 0
    good = head()
    for k in ["h", "w", "t", "rows", "loss", "gh", "gw"] + (["t2", "t3", "t4"] if kd else []):
        assert call(good, **{k: None}) == sv.SV_ERR_NULL, k
    assert call(head(hd=2), hsc=None) == sv.SV_ERR_NULL
    assert call(good, ws=None) == call(good, wb=need(good) - 1) == call(good, ws=WS + 8) == sv.SV_ERR_WORKSPACE
    assert call(head(N=0)) == sv.SV_OK
    assert need(head(g=0)) < need(head(g=2)) <= need(head(g=3))


@pytest.mark.parametrize("kd", [False, True])
@pytest.mark.parametrize("dt", [0, 1])
def test_workspace_of_an_empty_batch(lib, kd, dt):
    """A batch without rows has a size like any other, whatever gradients are asked for."""
    f = lib.sv_head_kd_workspace_bytes if kd else lib.sv_head_ce_workspace_bytes
    for g in range(4):
        for h, v in ((1, 1), (64, 100), (4096, 151936), (131072, 1 << 24)):
            assert f(ctypes.byref(head(N=0, H=h, V=v, dt=dt, g=g, S=0))) > 0


def test_workspace_does_not_grow_with_the_logits(lib):
    """A rollout batch: the workspace is a fraction of its float32 logits, and a
    larger vocabulary adds two numbers per row and 128 entries at most, 1/64 of
    its logits (and what a piece's rounding to whole tiles adds)."""
    f = lambda **k: lib.sv_head_ce_workspace_bytes(ctypes.byref(head(**k)))  # noqa: E731
    big = f(N=4096, H=4096, V=151936)
    assert big < 4096 * 151936 * 4 // 3
    assert f(N=4096, H=4096, V=607744) - big < 4096 * (607744 - 151936) * 4 / 64 + (64 << 20)


def test_front_end_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(10, 8)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        sv.head_ce(x, w, t)                           # not on the GPU
    with pytest.raises(ValueError):
        sv.act8_pack(x)
    with pytest.raises(TypeError):
        sv.act8_pack(x.half())
    with pytest.raises(TypeError):
        sv.head_ce(x.bfloat16(), w, t)
    with pytest.raises(ValueError):
        sv.head_ce(x, w, t, grad="both")
    with pytest.raises(ValueError):
        sv.head_ce(x, w[0], t)
    with pytest.raises(ValueError):
        sv.head_ce(x, w, t, ignore_index=1 << 31)
    with pytest.raises(TypeError):
        sv.head_logits(x, w)
    with pytest.raises(TypeError):
        sv.head_logits(x, sv.Act8(w, torch.zeros(10)))
    with pytest.raises(TypeError):
        sv.act8_unpack(sv.Act8(x, torch.zeros(4)))
