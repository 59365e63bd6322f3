"""Index arithmetic of the sliding-window and drafted-tree kernels, compiled
for the host and checked against the mask's definition key by key:

* forward units (decode_unit with kWin): every (row, visible key) pair lies in
  exactly one listed tile that the row's query tile computes, listed tiles
  stay inside the batch's keys, and the rows that are cleared in a V tile
  hold no key that some row of the unit sees;
* backward items (bwd_win_q_end, bwd_win_keys): the same for the dQ items, and
  every visible pair is in the query range of its key tile;
* decoding (dec_span, dec_tile, dec_row, dec_visible, dec_run_start): every
  visible key is in one row of one tile's list, loads stay inside a tile and
  start at no negative row, the visible columns of every row are exactly the
  mask's, and the runs partition the tiles.
"""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_tiled_attention_14_gb300", "csrc")
INCLUDE = os.path.join(ROOT, "include")

PROGRAM = r'''
#include <cstdio>
#include <vector>
#include "fa_fwd_kernel.cuh"
#include "fa_bwd_kernel.cuh"
#include "fa_decode_win_kernel.cuh"
#define BAD(...) do { std::printf(__VA_ARGS__); std::printf("\n"); return 1; } while (0)

static bool sees(long long pos, long long key, int len, int win, int sinks) {
  return key < len && key <= pos && (key > pos - win || key < sinks);
}

// one head: Nq queries, Nk keys of which len count, window, sinks, alignment
static int check_prompt(int Nq, int Nk, int len, int win, int sinks, int br, int gap_first = 0) {
  fa::FwdParams p{};
  p.gap_first = gap_first;
  p.BH = p.H = p.Hk = 1;
  p.N = Nq;
  p.Nk = Nk;
  p.n_qblk = (Nq + 255) / 256;
  p.num_units = p.n_qblk;
  p.hgroup = 1;
  p.win = win;
  p.sinks = sinks;
  p.align_br = br;
  int counts[1] = {len};
  p.seqlens_k = counts;
  const int off = br ? len - Nq : 0;
  for (int s = 0; s < p.num_units; ++s) {
    const fa::Unit x = fa::decode_unit<true, true, true>(s, p);
    fa::Piece u{};
    u.mblk = x.mblk; u.n0 = x.n0; u.n1 = x.n1; u.ns = x.ns; u.wa = x.wa; u.nl = x.nl;
    u.gap = x.gap; u.lo = x.lo; u.hi = x.hi;
    std::vector<int> pos_in_list((Nk + 127) / 128 + 1, -1);
    int active[2] = {0, 0};
    for (int j = 0; j < u.nl; ++j) {
      const int kt = fa::win_tile(u, j, gap_first);
      if (kt < 0 || kt * 128 >= len) BAD("fwd tile %d of unit %d", kt, s);
      if (pos_in_list[kt] >= 0) BAD("fwd tile twice %d", kt);
      pos_in_list[kt] = j;
      if (!fa::win_active(u, 0, j) && !fa::win_active(u, 1, j)) BAD("idle tile %d", kt);
      for (int w = 0; w < 2; ++w)
        if (fa::win_active(u, w, j) && fa::win_pos(u, w, active[w]++) != j) BAD("position %d", j);
      // the tiles with rows to clear come in order, and no other needs it
      bool unseen = false;
      for (int key = kt * 128; key < kt * 128 + 128; ++key)
        unseen |= !(key < sinks && key < x.hi) && !(key >= x.lo && key < x.hi);
      if (unseen != (fa::win_next_cut(u, j, sinks, gap_first) == j)) BAD("cut %d of %d", j, u.nl);
    }
    if (u.nl && fa::win_next_cut(u, u.nl, sinks, gap_first) != u.nl) BAD("cut after the list");
    if (active[0] != u.n0 || active[1] != u.n1) BAD("fwd active %d %d", active[0], active[1]);
    for (int w = 0; w < 2; ++w)
      for (int r = 0; r < 128; ++r) {
        const int row = (2 * u.mblk + w) * 128 + r;
        if (row >= Nq) continue;
        for (int key = 0; key < len; ++key)
          if (sees(row + off, key, len, win, sinks)) {
            const int kt = key / 128;
            if (pos_in_list[kt] < 0 || !fa::win_active(u, w, pos_in_list[kt])) BAD("fwd pair %d %d", row, key);
            if (!(key < sinks && key < x.hi) && !(key >= x.lo && key < x.hi))
              BAD("fwd cleared key %d", key);
          }
      }
  }
  if (!gap_first) {
    const int rc = check_prompt(Nq, Nk, len, win, sinks, br, 1);
    if (rc) return rc;
  } else {
    return 0;
  }
  const int n_tiles = (Nq + 127) / 128, n_ktiles = (Nk + 127) / 128;
  const int nkv = (len + 127) / 128;
  for (int qt = 0; qt < n_tiles; ++qt) {
    const int r0 = qt * 128, r1 = r0 + 128 < Nq ? r0 + 128 : Nq;
    const int last = r1 - 1 + off;
    const int n_end = last < 0 ? 0 : (last / 128 + 1 < nkv ? last / 128 + 1 : nkv);
    const fa::BwdWinKeys k = fa::bwd_win_keys(r0, r1, len, off, n_end, win, sinks);
    std::vector<int> listed(n_ktiles + 1, 0);
    for (int j = 0; j < k.count; ++j) {
      const int kt = j < k.ns ? j : k.wa + (j - k.ns);
      if (kt < 0 || kt * 128 >= len || listed[kt]++) BAD("dq tile %d", kt);
    }
    for (int row = r0; row < r1; ++row)
      for (int key = 0; key < len; ++key)
        if (sees(row + off, key, len, win, sinks)) {
          if (!listed[key / 128]) BAD("dq pair %d %d", row, key);
          if (!(key < sinks && key < k.hi) && !(key >= k.lo && key < k.hi))
            BAD("dq cleared key %d", key);
          const int kt = key / 128, first = kt * 128 - off;
          const int i0 = first <= 0 ? 0 : first / 128;
          if (qt < i0 || qt >= fa::bwd_win_q_end(kt, len, off, n_tiles, win, sinks))
            BAD("dkdv pair %d %d", row, key);
        }
  }
  for (int kt = 0; kt < n_ktiles; ++kt)
    if (fa::bwd_win_q_end(kt, len, off, n_tiles, win, sinks) > n_tiles) BAD("q end");
  return 0;
}

// tree: 0 a window call, else a seed for the drafted rows
static int check_decode(int Nq, int Nk, int count, int win, int sinks, int tree) {
  const fa::DecSpan s = fa::dec_span(count, Nk, Nq, win, sinks, tree != 0);
  const int nt = fa::dec_tiles(s);
  std::vector<unsigned long long> rows(Nq);
  unsigned long long x = tree * 0x9E3779B97F4A7C15ull;
  for (int i = 0; tree && i < Nq; ++i) {
    x = x * 6364136223846793005ull + 1442695040888963407ull;
    const int up = static_cast<int>((x >> 33) % (i + 1)) - 1;     // parent, -1: the history
    rows[i] = (up >= 0 ? rows[up] : 0ull) | (1ull << i);
    if ((x >> 20) % 7 == 0) rows[i] = 0;                          // padding
    if (Nq < 64 && (x >> 24) % 3 == 0) rows[i] |= 1ull << 63;     // a bit that means nothing
  }
  const unsigned long long* tr = tree ? rows.data() : nullptr;
  std::vector<fa::DecRow> me(Nq);
  std::vector<int> pos(Nq);
  for (int i = 0; i < Nq; ++i) {
    me[i] = fa::dec_row(tr, i, Nq, s.len, win, sinks);
    int marks = 0;
    for (int j = 0; j < Nq; ++j) marks += tree && (rows[i] >> j & 1);
    pos[i] = tree ? s.len - 1 + marks : s.len - Nq + i;
    if (me[i].pos != pos[i]) BAD("position %d", i);
  }
  std::vector<std::vector<int>> where(Nq, std::vector<int>(Nk + 1, 0));
  for (int t = 0; t < nt; ++t) {
    const fa::DecTile d = fa::dec_tile(s, t);
    if (d.ns % 16 || d.ns < 0 || d.ns > 128 || d.nw < 0 || d.ns + d.nw > 128) BAD("tile %d", t);
    if (d.nw > 112 && d.ns) BAD("full box beside sinks");
    const int bs = d.ns / 16, bw = (d.nw + 15) / 16;
    if (bs + bw > 8) BAD("boxes");
    if (d.nw > 0 && d.key0 < 0) BAD("negative load");
    if (bs == 0 && bw == 0 && d.key0 < 0) BAD("negative empty load");
    if (d.ns && d.sink0 + d.ns > s.sink_rows) BAD("sink rows");
    for (int i = 0; i < Nq; ++i) {
      uint32_t vis[4];
      for (int q = 0; q < 4; ++q)
        vis[q] = fa::dec_visible(s, d, me[i], tree != 0, win, sinks, q);
      const fa::DecRange w = fa::dec_whole(s, me[i], tree != 0, win);
      const bool all = vis[0] == ~0u && vis[1] == ~0u && vis[2] == ~0u && vis[3] == ~0u;
      if (t >= w.from && t < w.to && (d.ns || d.nw != 128 || d.key0 != w.base + 128 * t))
        BAD("tile %d is not plain", t);
      if (t >= w.from && t < w.to && !all) BAD("tile %d is not whole", t);
      if (all && d.ns == 0 && !(t >= w.from && t < w.to) && sinks == 0 && !tree)
        BAD("whole tile %d missed", t);
      for (int c = 0; c < 128; ++c) {
        if (!(vis[c >> 5] >> (c & 31) & 1)) continue;
        const int key = c < d.ns ? d.sink0 + c : d.key0 + c - d.ns;
        // a visible column is a loaded key, not one of the cleared rows
        if (c < d.ns ? key >= s.sink : c - d.ns >= d.nw) BAD("cleared column %d of tile %d", c, t);
        if (key < 0 || key >= Nk) BAD("key %d past the cache", key);
        ++where[i][key];
      }
    }
  }
  for (int i = 0; i < Nq; ++i)
    for (int key = 0; key < Nk; ++key) {
      bool want;
      if (!tree) {
        want = sees(pos[i], key, s.len, win, sinks);
      } else if (key < s.len) {
        want = key > pos[i] - win || key < sinks;
      } else {
        const int j = key - s.len;
        want = j < Nq && (rows[i] >> j & 1) && (pos[j] > pos[i] - win || pos[j] < sinks);
      }
      if (where[i][key] != (want ? 1 : 0)) BAD("row %d key %d: %d", i, key, where[i][key]);
    }
  return 0;
}

int main() {
  int op, a, b, c, d, e, f;
  while (std::scanf("%d %d %d %d %d %d %d", &op, &a, &b, &c, &d, &e, &f) == 7) {
    const int bad = op == 0 ? check_prompt(a, b, c, d, e, f) : check_decode(a, b, c, d, e, f);
    if (bad) {
      std::printf("case %d: %d %d %d %d %d %d\n", op, a, b, c, d, e, f);
      return 1;
    }
  }
  for (int total : {1, 7, 151, 152, 153, 100000, 2000000000})
    for (int grid : {1, 7, 152}) {
      const fa::DecDeal d = fa::dec_deal(total, grid);
      if (d.runs < 1 || d.runs > grid || d.runs > total) BAD("runs %d %d", total, grid);
      int prev = 0;
      for (int i = 0; i <= d.runs; ++i) {
        const int st = fa::dec_run_start(d, i);
        if ((i == 0 && st) || (i == d.runs && st != total)) BAD("run %d %d", total, i);
        if (i && (st <= prev || st - prev > d.per + 1)) BAD("uneven run");
        if (i && (fa::dec_run_of(d, prev) != i - 1 || fa::dec_run_of(d, st - 1) != i - 1))
          BAD("run of tile %d", prev);
        prev = st;
      }
    }
  std::printf("ok\n");
  return 0;
}
'''


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc) and not shutil.which("nvcc"):
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("window")
    src, exe = d / "window.cu", d / "window"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", CSRC, "-I", INCLUDE, str(src), "-o", str(exe)], check=True,
                   capture_output=True, timeout=600)
    return str(exe)


def run(program, cases):
    text = "".join(" ".join(str(int(x)) for x in c) + "\n" for c in cases)
    out = subprocess.run([program], input=text, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout


def test_prompt_units_and_backward_items(program):
    rng = random.Random(11)
    cases = [(0, 1, 1, 1, 1, 0, 1), (0, 1, 1, 0, 1, 0, 0), (0, 300, 200, 200, 64, 4, 1),
             (0, 512, 512, 512, 128, 128, 0), (0, 512, 512, 512, 129, 129, 1),
             (0, 900, 900, 100, 64, 0, 0), (0, 256, 2000, 1999, 600, 300, 1)]
    for _ in range(400):
        Nq, Nk = rng.randint(1, 900), rng.randint(1, 1500)
        length = rng.choice((Nk, rng.randint(0, Nk)))
        win = min(rng.choice((1, 2, 64, 127, 128, 129, 500, 5000)), max(Nq, Nk) + 1)
        cases.append((0, Nq, Nk, length, win, min(rng.choice((0, 0, 1, 4, 127, 128, 129, 400)), Nk),
                      rng.randint(0, 1)))
    run(program, cases)


def test_decode_tiles_and_runs(program):
    rng = random.Random(12)
    cases = [(1, 1, 1, 1, 1, 0, 0), (1, 16, 4, 4, 3, 2, 0), (1, 64, 64, 0, 70, 0, 1),
             (1, 64, 300, 236, 5, 3, 2), (1, 33, 500, 490, 600, 0, 3)]
    for n in range(1500):
        tree = rng.randint(0, 1) * (n + 1)
        Nq = rng.randint(1, 64 if tree else 16)
        Nk = rng.randint(Nq if tree else 1, 900)
        count = rng.choice((Nk, Nk - Nq, rng.randint(0, Nk), -3, Nk + 9))
        win = min(rng.choice((1, 3, 17, 64, 128, 300, 9000)), Nk + Nq + 1)
        cases.append((1, Nq, Nk, count, win, min(rng.choice((0, 1, 4, 15, 16, 17, 130, 400)), Nk),
                      tree))
    run(program, cases)
