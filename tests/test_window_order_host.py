"""The order of a windowed unit's key tiles has one source: decode_unit reads
it from the parameters, the roles of the kernel from win_gap_first(D), and the
launch writes the first from the second whatever the caller left there.  With
them apart, the second query tile would skip another tile than the loader
placed there."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_tiled_attention_14_gb300", "csrc")
INCLUDE = os.path.join(ROOT, "include")

PROGRAM = r'''
#include <cstdio>
#include "fa_launch.cuh"
template <int D>
int check() {
  int units = 0;
  for (int left : {0, 1})
    for (int win : {100, 300, 1000}) {
      fa::FwdParams p{};
      p.gap_first = left;
      p.BH = p.H = p.Hk = p.hgroup = 1;
      p.N = p.Nk = 2048;
      p.n_qblk = p.num_units = 8;
      p.win = win;
      p.sinks = 4;
      p.align_br = 1;
      const fa::FwdParams q = fa::win_launch_params<D>(p);
      for (int s = 0; s < 8; ++s) {
        const fa::Unit x = fa::decode_unit<true, true, true>(s, q);
        fa::Piece u{};
        u.n0 = x.n0; u.n1 = x.n1; u.ns = x.ns; u.wa = x.wa; u.nl = x.nl; u.gap = x.gap;
        if (u.gap < 0) continue;
        ++units;   // the skipped tile is the first window's, in the kernel's own order
        if (fa::win_tile(u, u.gap, fa::win_gap_first(D)) != u.wa) return -1;
      }
    }
  return units;
}
int main() {
  std::printf("%d %d\n", check<64>(), check<128>());
  return 0;
}
'''


def test_launch_and_kernel_agree_on_the_order(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc) and not shutil.which("nvcc"):
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "order.cu", tmp_path / "order"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                    "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE, str(src), "-o", str(exe)],
                   check=True, capture_output=True, timeout=600)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout
    d64, d128 = (int(x) for x in out.split())
    assert d64 > 0 and d128 > 0
