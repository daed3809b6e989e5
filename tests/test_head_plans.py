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
