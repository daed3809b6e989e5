"""The boundary of the 4-bit rows and head logits without a GPU: exported names, workspace
sizes, the refusal of bad arguments before anything is enqueued, in C and in the torch front
end, and the host code (csrc/sv_mx4_host.h) under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import ctypes
import os
import re
import subprocess

import pytest

import draft_verification_spec_amd as sv

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, WS = 0x1000, 0x100000                           # never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


def test_exports_every_declared_function(lib):
    text = open(os.path.join(ROOT, "include", "sv_mx4.h")).read()
    names = set(re.findall(r"^(?:int|size_t) (sv_\w+)\(", text, flags=re.M))
    assert names == {"sv_mx4_pack", "sv_mx4_unpack", "sv_head_logits4", "sv_head_logits4_workspace_bytes"}
    for n in names:
        assert hasattr(lib, n), n


def test_row_refusals(lib):
    def pack(N=4, H=65, dt=0, x=FAKE, xs=0, c=FAKE, cs=0, s=FAKE, ss=0):
        return lib.sv_mx4_pack(N, H, dt, x, xs, c, cs, s, ss, None)

    def unpack(N=4, H=65, c=FAKE, cs=0, s=FAKE, ss=0, dt=0, y=FAKE):
        return lib.sv_mx4_unpack(N, H, c, cs, s, ss, dt, y, None)
    for f in (pack, unpack):
        assert f(dt=2) == f(dt=3) == f(dt=-1) == sv.SV_ERR_DTYPE
        assert f(N=-1) == f(H=0) == f(H=131073) == f(cs=32) == f(cs=-33) == f(ss=2) == f(ss=-3) == sv.SV_ERR_SHAPE
        assert f(c=None) == f(s=None) == sv.SV_ERR_NULL
        assert f(N=0, c=None, s=None) == sv.SV_OK
    assert pack(xs=64) == sv.SV_ERR_SHAPE and pack(x=None) == sv.SV_ERR_NULL and unpack(y=None) == sv.SV_ERR_NULL


def shape(N=100, H=65, V=100, hd=0, od=1, hs=0, hss=0, ws=0, wss=0, os=0):
    return sv.sv_logits4_shape_t(N, H, V, hd, od, hs, hss, ws, wss, os)


def test_logits_refusals(lib):
    def call(s, h=FAKE, hsc=FAKE, c=FAKE, sc=FAKE, o=FAKE, w=WS, wb=1 << 40):
        return lib.sv_head_logits4(None if s is None else ctypes.byref(s), h, hsc, c, sc, o, w, wb, None)

    def need(s):
        return lib.sv_head_logits4_workspace_bytes(ctypes.byref(s))
    assert call(None) == sv.SV_ERR_NULL
    assert call(shape(hd=2)) == call(shape(hd=4)) == call(shape(od=2)) == call(shape(od=-1)) == sv.SV_ERR_DTYPE
    for bad in (shape(N=-1), shape(H=0), shape(H=131073), shape(V=0), shape(V=(1 << 24) + 1), shape(hs=64), shape(hs=-65),
                shape(hd=3, hs=32), shape(hd=3, hss=2), shape(ws=32), shape(wss=2), shape(os=99),
                shape(N=2147483647, V=1 << 24), shape(N=1 << 20, V=1 << 24)):
        assert call(bad) == sv.SV_ERR_SHAPE and need(bad) == 0
    good = shape()
    for k in ("h", "c", "sc", "o"):
        assert call(good, **{k: None}) == sv.SV_ERR_NULL, k
    assert call(shape(hd=3), hsc=None) == sv.SV_ERR_NULL
    assert need(good) > 0
    assert call(good, w=None) == call(good, wb=need(good) - 1) == call(good, w=WS + 8) == sv.SV_ERR_WORKSPACE
    assert call(shape(N=0)) == sv.SV_OK
    assert need(shape(N=1)) == 0 < need(shape(N=1, hd=3)) < need(shape(N=1024, H=4096, V=128256))


def test_front_end_refusals():
    x = torch.zeros(4, 64)
    a = sv.Mx4(torch.zeros(10, 32, dtype=torch.uint8), torch.zeros(10, 2, dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        sv.mx4_pack(x)                                # not on the GPU
    with pytest.raises(ValueError):
        sv.mx4_unpack(a)
    with pytest.raises(ValueError):
        sv.head_logits(x, a)
    with pytest.raises(TypeError):
        sv.mx4_pack(x.half())
    with pytest.raises(ValueError):
        sv.mx4_pack(torch.zeros(4, 0))
    with pytest.raises(TypeError):
        sv.mx4_unpack(sv.Act8(a.codes, a.scale))
    with pytest.raises(TypeError):
        sv.mx4_unpack(a, torch.float16)
    with pytest.raises(TypeError):
        sv.mx4_unpack(a._replace(codes=a.codes.char()))
    with pytest.raises(TypeError):
        sv.mx4_unpack(a._replace(scale=a.scale.float()))
    for bad in (a._replace(width=62), a._replace(width=0), a._replace(width=131073), a._replace(scale=a.scale[:9]),
                a._replace(scale=a.scale[:, :1])):
        with pytest.raises(ValueError):
            sv.mx4_unpack(bad)
        with pytest.raises(ValueError):
            sv.head_logits(x, bad)
    with pytest.raises(TypeError):
        sv.head_logits(x, sv.Mx4(a.codes[0], a.scale[0], 64))
    with pytest.raises(TypeError):
        sv.head_logits(x.half(), a)
    with pytest.raises(TypeError):
        sv.head_logits(x, a, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        sv.head_logits(sv.Mx4(a.codes[:, :31], a.scale, 62), a)
    a8 = sv.Act8(torch.zeros(10, 64, dtype=torch.int8), torch.zeros(10))
    with pytest.raises(TypeError):
        sv.head_logits(a8, a)
    with pytest.raises(TypeError):
        sv.head_logits(a, a8)
    with pytest.raises(TypeError):
        sv.head_ce(a, x, torch.zeros(10, dtype=torch.int64))


DRIVER = r"""
#include <stdio.h>
#include "sv_mx4_host.h"
using namespace sv_mx4_host;

#define NEED(x) do { if (!(x)) { printf("%s: N %d H %d V %d hd %d od %d\n", #x, s.N, s.H, s.V, s.hidden_dtype, s.out_dtype); \
                                 return 1; } } while (0)

int main() {
  const int Ns[] = {-1, 0, 1, 4, 16, 17, 32, 33, 64, 65, 128, 129, 300, 4096, 1 << 20, 0x7fffffff};
  const int Hs[] = {0, 1, 7, 32, 64, 100, 128, 129, 1000, 1024, 4096, 12000, 131071, 131072, 131073};
  const int Vs[] = {0, 1, 15, 255, 256, 257, 1000, 65536, 151936, 1 << 24, (1 << 24) + 1};
  const int dts[] = {-1, 0, 1, 2, 3, 4};
  const long long strides[] = {0, -1, 8, 200000, 5000000000LL};
  char *const mem = (char *)4096;        // never dereferenced
  long long valid = 0, refused = 0;
  for (int N : Ns) for (int H : Hs) for (int V : Vs) for (int hd : dts) for (int od : dts) for (long long st : strides) {
    sv_logits4_shape_t s = {N, H, V, hd, od, st, st, st, st, st > V ? st : 0};
    bool nothing = false;
    const int rc = check_logits(&s, mem, mem, mem, mem, mem, mem, (size_t)-1, &nothing);
    if (rc != SV_OK) { ++refused; continue; }
    ++valid;
    const Plan p = plan_for(&s);
    if (p.held) {
      // a workgroup's hidden rows fit its LDS, in whole 16-byte pieces
      NEED(N <= 16 * p.frags && p.frags >= 1 && p.frags <= 8 && p.frags != 7);
      NEED(held_bytes(N, H) <= LDS_ROWS && p.image + p.x_scales == held_bytes(N, H) && p.image % 16 == 0 && p.x_scales % 16 == 0);
      NEED(p.nks * 128 >= H && (p.nks - 1) * 128 < H);
      NEED(!p.fused || (hd != SV_MX4 && p.total == 0 && p.frags == 1));
      if (!p.fused && N) NEED(p.scales - p.codes >= (size_t)p.image && p.total - p.scales >= (size_t)p.x_scales);
    } else {
      NEED(p.Kp % SPAN == 0 && 2 * p.Kp >= H && p.groups * SPAN == p.Kp && p.groups * 16 * BLOCK >= H);
      NEED(p.piece % 256 == 0 && p.piece >= 256 && p.scaled % 256 == 0 && p.scaled >= 256);
      NEED(p.x_ld >= p.Kp && p.x_ld % 16 == 0 && p.x_ld <= MAX_LD && p.scales - p.codes >= (size_t)N * p.x_ld && p.weight - p.scales >= (size_t)(up(N, 256) * p.groups * 16));
      NEED(p.wscale - p.weight >= (size_t)(p.piece * p.x_ld));
      NEED(p.total - p.wscale >= (size_t)((p.piece > p.scaled ? p.piece : p.scaled) * p.groups * 16));
      // a launch of the scales' words, and a tile's offsets
      NEED((p.piece > p.scaled ? p.piece : p.scaled) * p.groups * 4 < 0xffffffffLL && 255 * p.x_ld < 0x7fffffffLL);
    }
    if (p.total && !nothing)
      NEED(check_logits(&s, mem, mem, mem, mem, mem, mem, p.total - 1, &nothing) == SV_ERR_WORKSPACE);
  }
  for (int N : Ns) for (int H : Hs) for (int dt : dts) for (long long st : strides)
    check_rows(N, H, dt, mem, st, mem, st, mem, st) == SV_OK ? ++valid : ++refused;
  printf("valid %lld refused %lld\n", valid, refused);
  return valid > 1000 && refused > 1000 ? 0 : 1;
}
"""


def test_host_code(tmp_path):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    subprocess.check_call(["g++", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                           "-fno-omit-frame-pointer", "-g", "-O1", "-I", os.path.join(ROOT, "include"), "-I",
                           os.path.join(ROOT, "draft_verification_spec_amd", "csrc"), "-o", str(exe), str(src)])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
