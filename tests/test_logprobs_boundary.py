"""The log-probability operators' boundary without a GPU: exported names, workspace sizes,
the refusal of bad arguments before anything is enqueued, in C and in the torch front end,
and the host code (csrc/sv_logprobs_host.h) under AddressSanitizer and
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
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    return sv.load_library()


def test_exports_every_declared_function(lib):
    text = open(os.path.join(ROOT, "include", "sv_logprobs.h")).read()
    names = set(re.findall(r"^(?:int|size_t) (sv_\w+)\(", text, flags=re.M))
    assert names == {"sv_logprobs", "sv_logprobs_workspace_bytes", "sv_logprobs_grad"}
    for n in names:
        assert hasattr(lib, n), n


def shape(N=4, V=400000, dt=1, top=3, rs=0, T=1.0):
    return sv.sv_logprobs_shape_t(N, V, dt, top, rs, T, -1)


BAD_T = (0.0, -1.0, float("nan"), INF, 1e-39)


def test_forward_refusals(lib):
    def call(s, z=FAKE, t=FAKE, p=FAKE, tv=FAKE, ti=FAKE, w=WS, wb=1 << 40):
        return lib.sv_logprobs(None if s is None else ctypes.byref(s), z, t, p, None, None, None, None, tv, ti, w, wb, None)

    def need(s):
        return lib.sv_logprobs_workspace_bytes(ctypes.byref(s))
    assert call(None) == sv.SV_ERR_NULL
    assert call(shape(dt=2)) == call(shape(dt=-1)) == sv.SV_ERR_DTYPE
    for T in BAD_T:
        assert call(shape(T=T)) == sv.SV_ERR_TEMPERATURE and need(shape(T=T)) == 0
    for bad in (shape(N=-1), shape(N=(1 << 20) + 1), shape(V=0), shape(V=(1 << 24) + 1), shape(top=-1), shape(top=33),
                shape(rs=399999), shape(rs=-400000)):
        assert call(bad) == sv.SV_ERR_SHAPE and need(bad) == 0
    good = shape()
    for k in ("z", "t", "p", "tv", "ti"):
        assert call(good, **{k: None}) == sv.SV_ERR_NULL, k
    assert need(good) > 0
    assert call(good, w=None) == call(good, wb=need(good) - 1) == call(good, w=WS + 8) == sv.SV_ERR_WORKSPACE
    assert call(shape(N=0), z=None, t=None, p=None, w=None) == sv.SV_OK
    assert need(shape(N=4096)) == need(shape(V=100)) == 0     # a workgroup a row: none needed


def test_gradient_refusals(lib):
    def gs(N=4, V=1000, dt=1, gd=1, rs=0, gst=0, T=1.0):
        return sv.sv_logprobs_grad_shape_t(N, V, dt, gd, rs, gst, T, -1)

    def call(s, z=FAKE, t=FAKE, m=FAKE, e=FAKE, g=FAKE, h=FAKE, o=2 * FAKE):
        return lib.sv_logprobs_grad(None if s is None else ctypes.byref(s), z, t, m, e, g, h, o, None)
    assert call(None) == sv.SV_ERR_NULL
    assert call(gs(dt=2)) == call(gs(gd=2)) == call(gs(gd=-1)) == sv.SV_ERR_DTYPE
    for T in BAD_T:
        assert call(gs(T=T)) == sv.SV_ERR_TEMPERATURE
    for bad in (gs(N=-1), gs(N=(1 << 20) + 1), gs(V=0), gs(V=(1 << 24) + 1), gs(rs=999), gs(gst=999), gs(gst=-1000)):
        assert call(bad) == sv.SV_ERR_SHAPE
    for k in ("z", "t", "m", "e", "g", "o"):
        assert call(gs(), **{k: None}) == sv.SV_ERR_NULL, k
    # in place: another type or distance of rows would overwrite what is still to be read
    assert call(gs(gd=0), o=FAKE) == call(gs(rs=1008), o=FAKE) == call(gs(gst=1008), o=FAKE) == sv.SV_ERR_SHAPE
    assert call(gs(N=0), z=None, t=None, m=None, g=None, o=None) == sv.SV_OK


def test_front_end_refusals():
    z, t = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    r = sv.LogprobsResult(*[torch.zeros(4)] * 3, torch.zeros(2, 4), None, None, None)
    with pytest.raises(ValueError):
        sv.logprobs(z, t)                             # not on the GPU
    with pytest.raises(ValueError):
        sv.logprobs_grad(z, t, r, torch.zeros(4))
    with pytest.raises(TypeError):
        sv.logprobs(z.half(), t)
    with pytest.raises(ValueError):
        sv.logprobs(torch.zeros(4, 0), t)
    with pytest.raises(ValueError):
        sv.logprobs(z, t, ignore_index=1 << 31)
    with pytest.raises(ValueError):
        sv.logprobs(z, t, top=33)
    with pytest.raises(ValueError):
        sv.logprobs(z, t, top=-1)
    with pytest.raises(ValueError):
        sv.logprobs_grad(z, t, r._replace(norm=torch.zeros(4, 2)), torch.zeros(4))
    with pytest.raises(TypeError):
        sv.logprobs_grad(z, t, r, torch.zeros(4), out_dtype=torch.float16)
    with pytest.raises(ValueError):
        sv.logprobs_grad(z, t, r, torch.zeros(4), out=torch.zeros(4, 9))


DRIVER = r"""
#include <stdio.h>
#include "sv_logprobs_host.h"
using namespace sv_logprobs_host;

#define NEED(x) do { if (!(x)) { printf("%s: N %d V %d dt %d top %d\n", #x, s.N, s.V, s.dtype, s.top); return 1; } } while (0)

int main() {
  const int Ns[] = {-1, 0, 1, 2, 31, 64, 127, 128, 1023, 1024, 5000, 1 << 20, (1 << 20) + 1};
  const int Vs[] = {0, 1, 31, 16384, 32768, 32769, 65537, 151936, 262145, 1 << 24, (1 << 24) + 1};
  const int tops[] = {-1, 0, 1, 32, 33};
  const float Ts[] = {1.f, 0.7f, 0.f, -1.f, 1e-39f, 3e38f, INFINITY, NAN};
  const long long strides[] = {0, -1, 31, 200000000000LL};
  char *const mem = (char *)4096;        // never dereferenced
  long long valid = 0, refused = 0;
  for (int N : Ns) for (int V : Vs) for (int dt = -1; dt < 3; ++dt) for (int top : tops) for (float T : Ts) for (long long st : strides) {
    sv_logprobs_shape_t s = {N, V, dt, top, st, T, -1};
    bool nothing = false;
    const int rc = check(&s, mem, mem, mem, mem, mem, mem, (size_t)-1, &nothing);
    sv_logprobs_grad_shape_t g = {N, V, dt, dt, st, 0, T, -1};
    bool none;
    if (top == 0 && (check_grad(&g, mem, mem, mem, mem, mem, mem, mem + 1, &none) == SV_OK) != (rc == SV_OK)) {
      printf("gradient\n");
      return 1;
    }
    if (rc != SV_OK) { ++refused; continue; }
    ++valid;
    const Plan p = plan_for(&s);
    // the parts are runs of whole steps, none empty, and cover the row; a wave joins them
    NEED(p.waves == 4 || p.waves == 16);
    NEED(p.batch == (int64_t)p.waves * 64 * VECS * (dt == SV_F32 ? 4 : 8));
    NEED(p.batches * p.batch >= V && (p.batches - 1) * p.batch < V);
    NEED(p.parts >= 1 && p.parts <= 64 && p.parts <= p.batches && (p.parts == 1 || N < 128));
    NEED((int64_t)(N ? N : 1) * p.parts * 64 * p.waves <= 0xffffffffLL);
    if (p.parts > 1) {
      NEED(p.keys % 256 == 0 && p.keys >= (size_t)N * p.parts * 24);
      NEED(p.total >= p.keys + (top ? (size_t)N * p.parts * LIST * 8 : 0));
      if (!nothing) NEED(check(&s, mem, mem, mem, mem, mem, mem, p.total - 1, &nothing) == SV_ERR_WORKSPACE);
    } else {
      NEED(p.total == 0 && check(&s, mem, mem, mem, mem, mem, nullptr, 0, &nothing) == SV_OK);
    }
  }
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
