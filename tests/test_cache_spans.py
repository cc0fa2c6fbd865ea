"""The arithmetic that keeps an attention call's queries and tokens inside its
arrays, compiled for the host and run under UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "vector_codebook_codec_amd", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "cache_spans.h"

int main() {
  const int64_t low = -(int64_t(1) << 31), high = (int64_t(1) << 31) - 1;
  const int64_t entries[] = {low, low + 1, low + 5, -(int64_t(1) << 30), -4, -1, 0, 1, 5, 6, 7, 100, (int64_t(1) << 30) - 1,
                             int64_t(1) << 30, high - 1, high};
  const int64_t totals[] = {1, 5, 6, 100, int64_t(1) << 30};
  int wrong = 0;
  for (int64_t T : totals)
    for (int64_t s0 : entries)
      for (int64_t s1 : entries)
        for (int64_t len : entries) {
          const int64_t most = int64_t(1) << 30;
          const qamw::Sequence s = qamw::clamped_sequence(s0, s1, T, len, most);
          // the queries of [s0, s1) that there are
          const int64_t a = s0 < 0 ? 0 : s0, b = s1 < T ? s1 : T, n = b > a ? b - a : 0;
          const int64_t length = len < 0 ? 0 : len < most ? len : most;
          const bool held = s.first >= 0 && s.first <= T && s.n >= 0 && s.first + s.n <= T;
          if (!held || s.n != n || (n && s.first != a) || s.length != length) {
            if (!wrong++)
              std::printf("T=%lld starts %lld, %lld length %lld: first %lld n %d length %d\n", (long long)T, (long long)s0,
                          (long long)s1, (long long)len, (long long)s.first, s.n, s.length);
          }
        }
  if (wrong) std::printf("%d wrong\n", wrong);
  return wrong != 0;
}
"""


def test_queries_and_tokens_stay_inside(tmp_path):
    """Of starts and lengths of any value, those of 32 bits' ends among them, what lies inside the arrays is taken."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    source, program = tmp_path / "spans.cpp", tmp_path / "spans"
    source.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", CSRC, str(source),
                    "-o", str(program)], check=True, capture_output=True, text=True, timeout=120)
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    res = subprocess.run([str(program)], capture_output=True, text=True, timeout=60, env=env)
    assert res.returncode == 0, res.stdout + res.stderr
