"""What the losses' host plan (csrc/sv_head_host.h) promises the kernels, built with g++
under AddressSanitizer and UndefinedBehaviorSanitizer.  No GPU is involved."""
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")


def run(tmp_path, source, *args):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(source)
    subprocess.check_call(["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I",
                           os.path.join(ROOT, "draft_verification_spec_amd", "csrc"), "-o", str(exe), str(src)])
    r = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True, env=ENV, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    return r.stdout


PIECES = r"""
#include <stdio.h>
#include <stdlib.h>
#include "sv_head_host.h"
using namespace sv_head_host;
int main(int n, char **a) {
  for (int i = 1; i + 4 < n; i += 5) {
    sv_head_shape_t s = {atoi(a[i]), atoi(a[i + 1]), atoi(a[i + 2]), atoi(a[i + 3]), atoi(a[i + 4]), 3, 0, 0, 1.f, -1, 4, 2, 1.f};
    const Plan p = plan_for(&s, true, weight_direct(&s, 0));
    printf("%lld %lld\n", (long long)p.pieces, (long long)p.piece);
  }
}
"""


def test_pieces_of_the_distillation_tests(tmp_path):
    """The shapes that the GPU tests take for several pieces are cut where they say."""
    from test_gpu_head_edges import KD_PIECES
    args = []
    for n, h, v, dtype, kind, _, _ in KD_PIECES:
        dt = 1 if dtype is torch.bfloat16 else 0
        args += [n, h, v, dt, 2 if kind == "i8" else dt]
    got = [tuple(map(int, line.split())) for line in run(tmp_path, PIECES, *args).splitlines()]
    assert got == [(c[5], c[6]) for c in KD_PIECES]
    assert all(p > 1 for p, _ in got)


SHARES = r"""
#include <stdio.h>
#include "sv_head_host.h"
using namespace sv_head_host;

#define NEED(x) do { if (!(x)) { printf("%s: N %d H %d V %d dt %d hd %d g %d kd %d direct %d M %lld\n", #x, s.N, s.H, s.V, \
                                        s.dtype, s.hidden_dtype, s.grads, kd, direct, (long long)M); return 1; } } while (0)

struct Tile { int bm, bn, threads, frags; };             // frags: fragment rows that are joined
const Tile BIG = {256, 256, 512, 64}, MID = {128, 128, 256, 16}, SQUARE = {64, 64, 256, 8}, FEW = {32, 128, 256, 8},
           PAIR = {64, 128, 256, 8}, NARROW = {32, 64, 256, 4};

// the shares of the hidden gradient as the kernels form them, for every number of rows with a
// gradient, and the sections that they write
static int holds(const sv_head_shape_t &s, bool kd, bool direct) {
  const Plan p = plan_for(&s, kd, direct);
  const bool bf = s.dtype == SV_BF16, gh = s.grads & SV_GRAD_HIDDEN, gw = s.grads & SV_GRAD_WEIGHT;
  const Tile T = bf ? (p.bm == 256 ? BIG : p.bm == 128 ? MID : PAIR) : p.bm == 64 ? SQUARE : FEW;   // dx
  const Tile S = p.bm > 32 ? T : p.narrow ? NARROW : FEW;                                           // against the weight's rows
  const bool both = bf && p.bm == 32;    // two terms of 32 rows in a tile of 64, whose sums are of 32
  const int64_t e = p.e, steps = p.piece * e / STEP, runs = p.groups / p.chunks, nt = cdiv(s.H, T.bn);
  int64_t M = 0;
  NEED(p.bm == (both ? 32 : T.bm) && p.bn == T.bn);
  NEED(p.chunks >= 1 && p.chunks <= 8 && p.groups >= p.chunks && p.groups % p.chunks == 0);
  NEED((int64_t)p.chunks * p.full >= steps && (int64_t)(p.chunks - 1) * p.full <= steps && p.full >= 1);
  const int64_t rows[] = {1, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 1000, s.N / 3, s.N / 2, s.N - 1, s.N};
  for (int64_t m : rows) {
    if (m < 1 || m > s.N) continue;
    M = m;
    const int64_t mt = both ? 1 : cdiv(M, T.bm), total = mt * nt * p.full;
    const int64_t q = cdiv(total, runs), per = q > RUN ? q : RUN;
    NEED(per <= 0x7fffffffLL && per * runs >= total);
    for (int64_t b = 0; b < runs; ++b) {                 // a run's tiles have a slot each
      if (b * per >= total) break;
      const int64_t end = (b + 1) * per < total ? (b + 1) * per : total;
      NEED((end - 1) / p.full - b * per / p.full < p.slots);
    }
    const int64_t tiles = mt * nt;
    for (int64_t t = 0; t < tiles; t += tiles > 4096 && t > 64 && t < tiles - 64 ? 61 : 1) {
      const int64_t b0 = t * p.full / per, b1 = ((t + 1) * p.full - 1) / per, k0 = t - b0 * per / p.full;
      NEED(b1 < runs && k0 >= 0 && k0 < p.slots);        // its first sum lies in b0's slot k0,
      for (int64_t b = b0 + 1; b <= b1 && b < b0 + 40; ++b) NEED(b * per / p.full == t);   // the others are their runs' first
      NEED(b1 == b0 || b1 * per / p.full == t);
    }
    NEED(cdiv(M, T.bm) * nt * T.frags < 0x7fffffffLL);
  }
  // sections
  const int terms = (s.grads & SV_GRAD_TWO_TERMS) && bf && p.bm > 32 ? 2 : 1;
  NEED(p.terms == terms);
  int64_t columns = 0;
  const int64_t part = direct ? s.V : p.piece, most = launch_columns(cdiv(s.N, S.bm), S.bn, S.threads);
  NEED(most >= 256 && most % 256 == 0);
  NEED(!p.keep || most >= s.V);                           // kept logits: one launch
  for (int64_t v = 0; v < s.V; v += part)
    for (int64_t c = 0, n = s.V - v < part ? s.V - v : part; c < n; c += most) {
      const int64_t tiles = cdiv(n - c < most ? n - c : most, S.bn);
      NEED(cdiv(s.N, S.bm) * tiles * S.threads <= 0xffffffffLL && cdiv(s.N, S.bm) * tiles <= 0x7fffffffLL);
      columns += tiles;
    }
  NEED((int64_t)(p.xs - p.part) >= columns * s.N * 8);
  NEED((int64_t)(p.xw - p.xs) >= p.Np * p.x_ld);
  if (gw) NEED((int64_t)(p.dz - p.xw) >= terms * p.Np * e / 16 * p.xw_ld && (int64_t)(p.wt - p.dzw) >= terms * p.Np * e / 16 * p.dzw_ld);
  if (gh || p.keep) NEED((int64_t)(p.dzw - p.dz) >= terms * p.Np * p.dz_ld);
  if (!direct) NEED((int64_t)(p.acc - p.wt) >= p.piece * p.x_ld);
  if (gh) NEED((int64_t)(p.total - p.acc) >= (int64_t)p.groups * p.slots * T.bm * T.bn / (both ? 2 : 1) * 4);
  // launches over a piece
  if (s.grads) {
    NEED((cdiv(both ? 32 : p.Np, S.bm) * cdiv(p.piece, S.bn) + p.Np * e / 16 + 1) * S.threads <= 0xffffffffLL);
    NEED(cdiv(p.piece, 64) * cdiv(s.H, 64) * 256 <= 0xffffffffLL);
  }
  return 0;
}

int main() {
  const int Ns[] = {1, 5, 24, 32, 33, 64, 65, 100, 128, 129, 191, 250, 256, 257, 520, 750, 1000, 1025, 2772, 4096, 20000, 1 << 20};
  const int Hs[] = {1, 7, 64, 72, 100, 192, 512, 1001, 1024, 2048, 4096, 8192, 131072};
  const int Vs[] = {1, 40, 255, 257, 1000, 4343, 20000, 32768, 33000, 65535, 65536, 100000, 151936, 262144, 600000, 1 << 24};
  const int Gs[] = {0, 1, 2, 3, 5, 7};
  long long plans = 0;
  for (int N : Ns) for (int H : Hs) for (int V : Vs) for (int dt = 0; dt < 2; ++dt) for (int g : Gs)
    for (int kd = 0; kd < 2; ++kd) {
      if ((double)N * H * V > 4e15 && (g == 1 || kd)) continue;
      sv_head_shape_t s = {N, H, V, dt, dt, g, 0, 0, 1.f, -1, 4, 2, 1.f};
      if (!head_shape_ok(&s, kd)) { printf("refused\n"); return 1; }
      for (int direct = 0; direct <= (weight_direct(&s, 0) ? 1 : 0); ++direct, ++plans)
        if (holds(s, kd, direct)) return 1;
    }
  printf("plans %lld\n", plans);
  return plans > 10000 ? 0 : 1;
}
"""


def test_shares_and_sections(tmp_path):
    """Every step of the hidden gradient in one run, every run's tiles in its slots, every
    tile's sums where they are joined; sections as large as what is written to them."""
    print(run(tmp_path, SHARES))
