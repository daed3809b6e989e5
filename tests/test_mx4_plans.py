"""The 4-bit head logits' plan where the hidden rows of a call are staged by several launches,
on the CPU under AddressSanitizer and UndefinedBehaviorSanitizer: each launch's codes and
scales lie where one launch over all rows would put them."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <stdio.h>
#include "sv_mx4_host.h"
using namespace sv_mx4_host;

#define NEED(x) do { if (!(x)) { printf("%s: H %d rows %lld\n", #x, H, (long long)p.rows); return 1; } } while (0)

int main() {
  int seen = 0;
  for (int H = 1; H <= SV_HEAD_MAX_H; H += H < 600 ? 1 : 511) {
    sv_logits4_shape_t s = {0x7fffffff, H, 1, SV_MX4, SV_BF16, 0, 0, 0, 0, 0};
    const Plan p = plan_for(&s);
    NEED(!p.held && p.rows > 0);
    // no more than a launch's worth, in threads of four items and of one
    const int64_t lanes = p.Kp / 4;
    NEED(cdiv(p.rows * lanes, 1024) <= sv_head_host::max_groups(256));
    // the scale of block b of a row, as the kernel puts it: in the whole, and in its own launch's memory
    const int64_t blocks_of[] = {0, 5, blocks(H) - 1};
    for (int64_t k = 0; k < 3; ++k)
      for (int64_t d = -70; d < 70; ++d) {
        const int64_t row = k * p.rows + d;
        if (row < 0) continue;
        const int64_t first = row / p.rows * p.rows, mine = row - first;
        for (int64_t b : blocks_of) {
          if (b >= blocks(H)) continue;
          const int64_t lane = b % 4 * 16, at = tiled_scale(row, b / 16, lane + row % 16, p.groups) * 4 + b / 4 % 4;
          const int64_t there = first * p.groups * 16 + tiled_scale(mine, b / 16, lane + mine % 16, p.groups) * 4 + b / 4 % 4;
          NEED(at == there);
          ++seen;
        }
      }
    // rows of a group share no byte with another's
    NEED(tiled_scale(SCALE_ROWS, 0, 0, p.groups) * 4 == SCALE_ROWS * p.groups * 16);
  }
  printf("seen %d\n", seen);
  return seen > 100000 ? 0 : 1;
}
"""


def test_staging_in_launches(tmp_path):
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    subprocess.check_call(["g++", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                           "-fno-omit-frame-pointer", "-g", "-O1", "-I", os.path.join(ROOT, "include"), "-I",
                           os.path.join(ROOT, "draft_verification_spec_amd", "csrc"), "-o", str(exe), str(src)])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
