"""The vocabulary-head operators' host code (csrc/sv_head_host.h: argument checks,
piece sizes, workspace layouts) built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer and driven over valid and invalid shapes.  Every plan it
accepts has to hold what the kernels assume of it.  No GPU is involved."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")

DRIVER = r"""
#include <stdio.h>
#include "sv_head_host.h"
using namespace sv_head_host;

#define NEED(x) do { if (!(x)) { printf("%s: N %d H %d V %d dt %d hd %d g %d kd %d direct %d\n", #x, s.N, s.H, s.V, \
                                        s.dtype, s.hidden_dtype, s.grads, kd, direct); return 1; } } while (0)

static int plan_holds(const sv_head_shape_t &s, bool kd, bool direct) {
  const Plan p = plan_for(&s, kd, direct);
  const int64_t e = p.e, q = STEP / e;
  NEED(p.Kp % q == 0 && p.Kp >= s.H && p.Kp < s.H + q && p.Np % q == 0 && p.Np >= s.N);
  NEED(p.piece % 256 == 0 && p.piece >= 256 && p.pieces * p.piece >= s.V && (p.pieces - 1) * p.piece < s.V);
  NEED(p.x_ld >= p.Kp * e && p.x_ld % 256 == 128 && p.dz_ld >= p.piece * e && p.dz_ld % 16 == 0);
  NEED(p.xw_ld >= p.Kp * 16 && p.dzw_ld >= p.piece * 16);
  // a step of columns or blocks, or a tile of rows, stays in 31-bit offsets
  NEED(255 * p.x_ld < 0x7fffffffLL && 255 * p.dz_ld < 0x7fffffffLL && 8 * p.dzw_ld < 0x7fffffffLL && 8 * p.xw_ld < 0x7fffffffLL);
  const int64_t tiles = cdiv(s.N, p.bm) * cdiv(s.H, p.bn), full = p.piece * e / STEP;
  NEED(p.groups >= 1 && p.slots >= 1 && full >= 1);
  // whatever part of the rows has a gradient: the runs cover its tiles, and no run touches more than its slots
  for (int64_t m = 1; m <= s.N; m = m * 3 + 1) {
    const int64_t total = cdiv(m, p.bm) * cdiv(s.H, p.bn) * full;
    int64_t per = cdiv(total, p.groups);
    if (per < RUN) per = RUN;
    NEED(per <= 0x7fffffffLL && per * p.groups >= total);
    for (int64_t b = 0; b < p.groups && b < 40; ++b)
      if (b * per < total) {
        const int64_t last = (b + 1) * per < total ? (b + 1) * per - 1 : total - 1;
        NEED(last / full - b * per / full < p.slots);
      }
  }
  (void)tiles;
  const size_t sec[] = {p.counts, p.perm, p.alpha, p.ga, p.lse2, p.w, p.flags, p.zt, p.pt, p.term, p.part, p.xs, p.xw,
                        p.dz, p.dzw, p.wt, p.acc, p.total};
  for (int i = 0; i < 18; ++i) {
    NEED(sec[i] % 256 == 0 || i == 17);
    if (i) NEED(sec[i] >= sec[i - 1]);
  }
  NEED(p.total <= head_bytes(&s, kd));
  NEED(p.xw - p.xs >= (size_t)s.N * p.x_ld && p.wt - p.dzw >= (size_t)((s.grads & SV_GRAD_WEIGHT) ? p.Np * e / 16 * p.dzw_ld : 0));
  return 0;
}

int main() {
  const int Ns[] = {-1, 0, 1, 31, 32, 33, 64, 65, 191, 192, 1000, 4096, 1 << 20, (1 << 20) + 1};
  const int Hs[] = {0, 1, 7, 64, 100, 1024, 4096, 131072, 131073};
  const int Vs[] = {0, 1, 255, 256, 257, 1000, 65535, 65536, 151936, 1 << 24, (1 << 24) + 1};
  const int dts[] = {0, 1, 2, 7};
  const long long strides[] = {0, -1, 8, 200000};
  long long valid = 0, refused = 0;
  char *const mem = (char *)4096;        // never dereferenced
  for (int N : Ns) for (int H : Hs) for (int V : Vs) for (int dt : dts) for (int hd : dts) for (int g = -1; g < 5; ++g)
    for (long long st : strides) for (int kd = 0; kd < 2; ++kd) {
      sv_head_shape_t s = {N, H, V, dt, hd, g, st, st, 1.f, -1, 4, 2, 1.f};
      bool nothing = false;
      const int rc = check_head(&s, kd, mem, mem, mem, mem, mem, mem, mem, mem, mem, mem, mem, mem, (size_t)-1, &nothing);
      if (rc != SV_OK) { ++refused; continue; }
      ++valid;
      if (nothing) continue;
      for (int direct = 0; direct <= (weight_direct(&s, 0) ? 1 : 0); ++direct)   // the plans that a call may use
        if (plan_holds(s, kd, direct)) return 1;
      if (check_head(&s, kd, mem, mem, mem, mem, mem, mem, mem, mem, mem, mem, mem, mem, head_bytes(&s, kd) - 1, &nothing) !=
          SV_ERR_WORKSPACE) { printf("short workspace\n"); return 1; }
    }
  for (int N : Ns) for (int H : Hs) for (int V : Vs) for (int hd : dts) for (int od : dts) for (long long st : strides) {
    sv_logits_shape_t s = {N, H, V, hd, od, st, st, st};
    bool nothing = false;
    const int rc = check_logits(&s, mem, mem, mem, mem, mem, mem, (size_t)-1, &nothing);
    if (rc != SV_OK) { ++refused; continue; }
    ++valid;
    const LogitsLayout L = logits_layout(&s);
    if (L.Kp % STEP || L.Kp < H || L.piece % 256 || L.codes % 256 || L.scale % 256 || L.weight % 256 ||
        L.total < L.weight + (size_t)L.piece * L.Kp) { printf("logits layout\n"); return 1; }
  }
  for (int N : Ns) for (int H : Hs) for (int dt : dts) for (long long st : strides)
    check_act8(N, H, dt, mem, st, mem, st, mem) == SV_OK ? ++valid : ++refused;
  printf("valid %lld refused %lld\n", valid, refused);
  return valid > 1000 && refused > 1000 ? 0 : 1;
}
"""


def test_host_code(tmp_path):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    subprocess.check_call(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I",
                           os.path.join(ROOT, "draft_verification_spec_amd", "csrc"), "-o", str(exe), str(src)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=ENV, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
