"""Host arithmetic of the query/key norm, checked without a GPU."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "scaled_dot_product_gb300", "csrc")

SPLIT = r"""
#include <cstdio>
#include "norm_split.h"
int main() {
  const int heads[] = {1, 2, 3, 7, 8, 31, 100, 303, 304, 606, 607, 608, 1000, 4096, 1 << 20};
  const int want[] = {1, 2, 3, 150, 151, 152, 153, 302, 303, 304, 305, 606, 607, 608, 100000, 1 << 29};
  int bad = 0;
  auto check = [&](int nq, int nk, int wq, int wk) {
    const sdpa::NormBwdBlocks b = sdpa::norm_bwd_blocks(nq, nk, wq, wk);
    const bool ok = b.q >= 1 && b.k >= 1 && b.q <= (wq > 1 ? wq : 1) && b.k <= (wk > 1 ? wk : 1) &&
                    b.q + b.k <= sdpa::kNormBwdMaxBlocks;
    if (!ok && bad++ < 8) std::printf("Nq %d Nkv %d want %d %d: %d + %d\n", nq, nk, wq, wk, b.q, b.k);
  };
  for (int nq : heads) for (int nk : heads) for (int wq : want) for (int wk : want) check(nq, nk, wq, wk);
  check(4, 2, 0, 0);                                   // no rows: the sums over none are still written
  const sdpa::NormBwdBlocks even = sdpa::norm_bwd_blocks(32, 8, 1 << 20, 1 << 20);
  if (even.q != 243 || even.k != 61) { ++bad; std::printf("32 : 8 heads as %d : %d\n", even.q, even.k); }
  return bad != 0;
}
"""


def test_the_gradients_blocks_fit_its_workspace(tmp_path):
    """The workspace holds a row of partial sums for kNormBwdMaxBlocks blocks: no pair of head counts
    may launch more."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("needs g++")
    src = tmp_path / "split.cpp"
    src.write_text(SPLIT)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(tmp_path / "split")], check=True)
    r = subprocess.run([str(tmp_path / "split")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
