"""Drafted tokens under a window near the number of marks a row can have
(dec_row of fa_decode_win_kernel.cuh, compiled for the host): positions of
drafted tokens lie 0 to 64 apart (a row of 0 at c - 1, one of 64 marks at
c + 63), so a window of 64 still hides some.  Rows are arbitrary words, among
them all ones and 0, checked token by token against the definition."""
import os
import random
import shutil
import subprocess

import pytest

import window_common as wc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_tiled_attention_14_gb300", "csrc")
INCLUDE = os.path.join(ROOT, "include")

PROGRAM = r'''
#include <cstdio>
#include "fa_decode_win_kernel.cuh"
int main() {
  int Nq, len, win, sinks;
  while (std::scanf("%d %d %d %d", &Nq, &len, &win, &sinks) == 4) {
    unsigned long long rows[64];
    for (int i = 0; i < Nq; ++i)
      if (std::scanf("%llx", rows + i) != 1) return 1;
    for (int i = 0; i < Nq; ++i)
      std::printf("%llx ", fa::dec_row(rows, i, Nq, len, win, sinks).bits);
    std::printf("\n");
  }
  return 0;
}
'''


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc) and not shutil.which("nvcc"):
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("tree")
    src, exe = d / "tree.cu", d / "tree"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", CSRC, "-I", INCLUDE, str(src), "-o", str(exe)], check=True,
                   capture_output=True, timeout=600)
    return str(exe)


def test_windows_about_the_number_of_marks(program):
    rng = random.Random(21)
    cases = []
    for win in (1, 2, 33, 62, 63, 64, 65, 66):
        for Nq in (1, 5, 63, 64):
            for sinks in (0, 3, 1000, 1010):
                rows = [rng.getrandbits(64) for _ in range(Nq)]
                rows[0] = 0
                rows[-1] = 2 ** 64 - 1
                if Nq > 2:
                    rows[1] = 1
                cases.append((Nq, 1000, win, sinks, rows))
    text = "".join(f"{n} {c} {w} {s} " + " ".join(f"{r:x}" for r in rows) + "\n"
                   for n, c, w, s, rows in cases)
    out = subprocess.run([program], input=text, capture_output=True, text=True, check=True,
                         timeout=60).stdout.splitlines()
    assert len(out) == len(cases)
    for line, (Nq, c, win, sinks, rows) in zip(out, cases):
        vis = wc.tree_mask(rows, c + Nq, c, win, sinks)[:, c:]
        for i, word in enumerate(line.split()):
            got = [int(word, 16) >> j & 1 == 1 for j in range(Nq)]
            assert got == vis[i].tolist(), (Nq, win, sinks, i)
