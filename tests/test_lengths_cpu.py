"""Lengths near 2^31, checked without a GPU: on the GPU a length that passes for a small one may read
out of range, so the kernels' test of lengths is compiled for the host, and their sources use it."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "self_speculative_sparse_paged_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "lengths.h"
using namespace vegas;
int main() {
  long bad = 0, n = 0;
  const int caps[] = {16, 32, 48, 4096, 131072, 1 << 24};
  for (int cap : caps)
    for (int rows = 1; rows <= 16; ++rows) {
      auto check = [&](long long x) {
        if (x < -2147483648ll || x > 2147483647ll) return;
        const int L = (int)x;
        const bool fits = x >= 0 && x + rows <= cap;
        const long long near = fits ? x : x < 0 ? 0 : cap - rows;
        bad += length_fits(L, rows, cap) != fits;
        bad += nearest_length(L, rows, cap) != near;
        ++n;
      };
      for (long long d = -40; d <= 40; ++d) {
        check(d);
        check(cap + d);
        check(2147483647ll + d);
        check(-2147483648ll + d);
        check(1073741824ll + d);
      }
    }
  std::printf("%ld %ld\n", n, bad);
  return bad != 0;
}
"""


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _uses_the_test_of_lengths(name):
    text = _source(name)
    assert "length_fits(" in text and "nearest_length(" in text
    assert not re.search(r"\+ T > cap", text)           # (wraps for lengths near 2^31)


def test_lengths_near_2_to_31_do_not_fit(tmp_path):
    src, exe = tmp_path / "lengths.cpp", tmp_path / "lengths"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    assert int(run.stdout.split()[0]) > 10000


def test_the_8_bit_verify_uses_it():
    _uses_the_test_of_lengths("verify_kv8.cu")


def test_the_bf16_verifies_use_it():
    _uses_the_test_of_lengths("verify_tc.cu")
    _uses_the_test_of_lengths("verify_attn.cu")
