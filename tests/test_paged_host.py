"""Index arithmetic of the paged-cache and rotary kernels, compiled for the host
and checked against the definitions slot by slot:

* decoding (paged_span, paged_key0, paged_sees): every key that some token sees
  is in exactly one tile of the list, tiles start inside the sequence, every
  sequence has a tile, and the runs' tiles stay below the host's bound;
* shared memory (dp_row, dp_chunk): slots are a permutation of a tile's rows,
  chunks of a row cover it, and the reads of a quarter (half) warp touch every
  bank once;
  (dt_piece, dt_place) codes turned to half precision cover a tile, go where the
  128-byte swizzle puts them, and do the same;
* append (append_span, append_pages): new slots are those of the definition,
  and the launch has a block for each page that they touch;
* scales (page_scale): the smallest power of two (e4m3) and the 127th part
  (int8), at and around every boundary;
* rotary units cover a row's columns once, partners together."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_tiled_attention_14_gb300", "csrc")
INCLUDE = os.path.join(ROOT, "include")

PROGRAM = r'''
#include <cmath>
#include <cstdio>
#include <cstring>
#include <set>
#include <vector>
#include "fa_decode_paged_tc_kernel.cuh"
#include "fa_rotary.cuh"
#define BAD(...) do { std::printf(__VA_ARGS__); std::printf("\n"); return 1; } while (0)

static int check_span(int Nq, int capacity, int count, int win, int sinks, int keys) {
  const fa::PagedSpan s = fa::paged_span(count, capacity, Nq, win, sinks, keys);
  const int len = count < 0 ? 0 : count > capacity ? capacity : count;
  if (s.len != len || s.tiles < 1) BAD("len %d tiles %d", s.len, s.tiles);
  if (s.tiles > (capacity + keys - 1) / keys + 1 || s.tiles * keys > capacity + 2 * keys) BAD("tiles %d", s.tiles);
  std::vector<int> listed(capacity + 2 * keys, 0);
  for (int t = 0; t < s.tiles; ++t) {
    const int k0 = fa::paged_key0(s, t, keys);
    if (k0 < 0 || k0 % keys || (len > 0 && k0 >= len)) BAD("tile %d at %d", t, k0);
    for (int i = 0; i < keys; ++i)
      if (listed[k0 + i]++) BAD("key %d twice", k0 + i);
    // a block of keys is seen by a row iff one of its keys is
    for (int i = 0; i < keys; i += 16)
      for (int r = 0; r < Nq; ++r) {
        const int pos = len - Nq + r;
        bool any = false;
        for (int key = k0 + i; key < k0 + i + 16; ++key)
          any |= key <= pos && (key > pos - win || key < sinks);
        if (any != fa::paged_sees(k0 + i, 16, pos, win, sinks)) BAD("sees %d row %d", k0 + i, r);
      }
    // and seen at all iff by some row
    for (int i = 0; i < keys; i += 16) {
      bool some = false;
      for (int r = 0; r < Nq; ++r) some |= fa::paged_sees(k0 + i, 16, len - Nq + r, win, sinks);
      if (some != fa::paged_seen(s, Nq, k0 + i, 16, win, sinks)) BAD("seen %d", k0 + i);
    }
  }
  for (int r = 0; r < Nq; ++r) {
    const int pos = len - Nq + r;
    for (int key = 0; key < len; ++key)
      if (key <= pos && (key > pos - win || key < sinks) && !listed[key]) BAD("key %d unlisted", key);
  }
  return 0;
}

template <int D>
static int check_layout() {
  std::set<int> rows;
  for (int s = 0; s < 8; ++s) {
    const int r = fa::dp_row<D>(s);
    if (r < 0 || r > 7) BAD("row %d", r);
    rows.insert(r);
  }
  if (rows.size() != 8) BAD("rows of %d", D);
  // where the swizzled copy puts a chunk: the bits above the row's 16-byte
  // chunks are added to the chunk's number, row * D + chunk * 16 in the tile
  const int keys = fa::dp_keys(D);
  std::set<unsigned> all;
  for (int r = 0; r < keys; ++r)
    for (int c = 0; c < D / 16; ++c) {
      const unsigned plain = r * D + c * 16;
      const unsigned want = D == 128 ? plain ^ ((plain >> 7 & 7) << 4) : plain ^ ((plain >> 7 & 3) << 4);
      if (fa::dp_chunk<D>(r, c) != want) BAD("chunk %d of row %d", c, r);
      all.insert(want);
    }
  if (static_cast<int>(all.size()) * 16 != fa::kDpTileBytes) BAD("tile bytes");
  // K: 16 bytes a lane, eight lanes at a time
  for (int i = 0; i < D / 64; ++i)
    for (int q = 0; q < 4; ++q) {
      std::set<unsigned> banks;
      for (int lane = 8 * q; lane < 8 * q + 8; ++lane)
        banks.insert(fa::dp_chunk<D>(fa::dp_row<D>(lane >> 2), (lane & 3) * (D / 64) + i) % 128 / 16);
      if (banks.size() != 8) BAD("K banks of %d", D);
    }
  // V: 16 bytes and eight lanes, or 8 bytes and sixteen lanes at a time
  for (int e = 0; e < 2; ++e)
    for (int q = 0; q < (D == 128 ? 4 : 2); ++q) {
      std::set<unsigned> banks;
      const int n = D == 128 ? 8 : 16;
      for (int lane = n * q; lane < n * q + n; ++lane) {
        const int g = lane >> 2, t = lane & 3, r = fa::dp_row<D>(2 * t + e);
        const unsigned at = D == 128 ? fa::dp_chunk<D>(r, g) : fa::dp_chunk<D>(r, g >> 1) + (g & 1) * 8;
        banks.insert(at % 128 / (D == 128 ? 16 : 8));
      }
      if (static_cast<int>(banks.size()) != n) BAD("V banks of %d", D);
    }
  return 0;
}

// Turning codes to half precision: every piece of a step's rows once, no bank
// twice in a quarter warp, neither reading nor writing.
template <int D>
static int check_pieces() {
  const int step = D == 128 ? 4 : 8;
  std::set<int> all;
  for (int k = 0; k < 128 / step; ++k)
    for (int q = 0; q < 4; ++q) {
      std::set<unsigned> read, write[2];
      for (int lane = 8 * q; lane < 8 * q + 8; ++lane) {
        const fa::DtPiece m = fa::dt_piece<D>(lane, k);
        if (m.row < 0 || m.row > 7 || m.piece < 0 || m.piece >= D / 16) BAD("piece of lane %d", lane);
        const int r = (k * step & ~7) + m.row;
        all.insert(r * 8 + m.piece);
        read.insert(fa::dp_chunk<D>(r, m.piece) % 128 / 16);
        for (int h = 0; h < 2; ++h) {
          const unsigned at = fa::dt_place(r, m.piece, h);
          write[h].insert(at % 128 / 16);
          if (at != (fa::dt_place(r, m.piece, 0) ^ (16u * h))) BAD("halves of row %d", r);
          const int col = m.piece * 16 + h * 8;             // the 128-byte swizzle of a 64-column chunk
          const unsigned plain = (col / 64) * 16384u + r * 128u + col % 64 * 2;
          if (at != (plain ^ ((plain >> 7 & 7) << 4))) BAD("place of row %d column %d", r, col);
        }
      }
      if (read.size() != 8 || write[0].size() != 8 || write[1].size() != 8) BAD("banks of %d", D);
    }
  if (static_cast<int>(all.size()) != 128 * D / 16) BAD("pieces of %d", D);
  return 0;
}

static int check_append(int len, int count, int T, int page, int per_seq) {
  const int capacity = page * per_seq;
  const fa::AppendSpan a = fa::append_span(len, count, T, capacity);
  const int c = count < 0 ? 0 : count > T ? T : count, n = len < 0 ? 0 : len;
  std::set<int> want, got;
  for (int i = 0; i < c; ++i) {
    const int slot = n - c + i;
    if (slot >= 0 && slot < capacity) want.insert(slot);
  }
  const int lo = a.first + a.skip, blocks = fa::append_pages(T, page);
  for (int j = 0; j < blocks; ++j) {
    const int nth = lo / page + j, slot0 = nth * page;
    if (slot0 >= a.end || lo >= a.end) continue;
    if (nth < 0 || nth >= per_seq) BAD("page %d", nth);
    for (int r = 0; r < page; ++r) {
      const int slot = slot0 + r;
      if (slot < lo || slot >= a.end) continue;
      const int token = slot - a.first;
      if (token < 0 || token >= c || slot != n - c + token) BAD("token %d at %d", token, slot);
      got.insert(slot);
    }
  }
  if (want != got) BAD("slots: %d, %d wanted", (int)got.size(), (int)want.size());
  return 0;
}

static int check_scales() {
  auto bits = [](float x) { unsigned u; std::memcpy(&u, &x, 4); return u; };
  for (int e = -126; e < 128; ++e)
    for (int step = -2; step <= 2; ++step)
      for (float m : {1.0f, 1.75f}) {
        float x = std::ldexp(m, e);
        for (int i = 0; i < std::abs(step); ++i) x = std::nextafter(x, step < 0 ? 0.0f : INFINITY);
        if (!std::isfinite(x)) continue;
        const float s = fa::page_scale<false>(bits(x)), t = fa::page_scale<true>(bits(x));
        int k;
        if (std::frexp(s, &k) != 0.5f || s < fa::kMinPageScale) BAD("scale of %g: %g", x, s);
        if (448.0 * s < x || (s > fa::kMinPageScale && 224.0 * s >= x)) BAD("scale of %g: %g", x, s);
        const float want = x / 127.0f > fa::kMinPageScale ? x / 127.0f : fa::kMinPageScale;
        if (t != want) BAD("int8 scale of %g: %g", x, t);
      }
  for (float x : {0.0f, 1e-42f})
    if (fa::page_scale<false>(bits(x)) != fa::kMinPageScale ||
        fa::page_scale<true>(bits(x)) != fa::kMinPageScale) BAD("scale of %g", x);
  for (float x : {INFINITY, NAN})
    if (fa::page_scale<false>(bits(x)) == fa::page_scale<false>(bits(x)) ||
        fa::page_scale<true>(bits(x)) == fa::page_scale<true>(bits(x))) BAD("scale of %g", x);
  if (fa::kMinPageScale != std::ldexp(1.0f, -100)) BAD("smallest scale");
  return 0;
}

static int check_rotary() {
  for (int d : {64, 128})
    for (int rot = 0; rot <= d; rot += 16)
      for (bool inter : {false, true}) {
        std::vector<int> seen(d, 0);
        for (int u = 0; u < d / 16; ++u) {
          const fa::RotaryUnit r = fa::rotary_unit(u, rot, inter);
          if (r.first % 8 || r.second % 8) BAD("alignment");
          for (int i = 0; i < 8; ++i) {
            ++seen[r.first + i];
            ++seen[r.second + i];
            if (r.turned != (r.first + i < rot) || r.turned != (r.second + i < rot)) BAD("turned");
            if (r.turned && !inter && (r.second != r.first + rot / 2 || r.first + i >= rot / 2)) BAD("halves");
          }
          if ((inter || !r.turned) && r.second != r.first + 8) BAD("neighbours");
        }
        for (int x : seen) if (x != 1) BAD("columns of %d %d", d, rot);
      }
  return 0;
}

int main() {
  if (check_layout<64>() || check_layout<128>() || check_pieces<64>() || check_pieces<128>() || check_scales() || check_rotary()) return 1;
  int op, a, b, c, d, e, f;
  while (std::scanf("%d %d %d %d %d %d %d", &op, &a, &b, &c, &d, &e, &f) == 7) {
    const int bad = op == 0 ? check_span(a, b, c, d, e, f) : check_append(a, b, c, d, e);
    if (bad) {
      std::printf("case %d: %d %d %d %d %d %d\n", op, a, b, c, d, e, f);
      return 1;
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
    d = tmp_path_factory.mktemp("paged")
    src, exe = d / "paged.cu", d / "paged"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", CSRC, "-I", INCLUDE, str(src), "-o", str(exe)], check=True,
                   capture_output=True, timeout=600)
    return str(exe)


def run(program, cases):
    text = "".join(" ".join(str(int(x)) for x in c) + "\n" for c in cases)
    out = subprocess.run([program], input=text, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout


def test_tiles_of_a_sequence(program):
    rng = random.Random(21)
    cases = []
    for _ in range(1500):
        keys, cap = rng.choice((32, 64, 128)), 16 * rng.randint(1, 60)
        Nq = rng.randint(1, 16)
        win = min(rng.choice((1, 2, 15, 31, 32, 33, 64, 100, 300, 9999)), cap + Nq + 1)
        count = rng.choice((cap, 0, 1, Nq - 1, rng.randint(0, cap), -5, cap + 7))
        sinks = min(rng.choice((0, 1, 4, 31, 32, 33, 64, 130, 400)), cap)
        cases.append((0, Nq, cap, count, win, sinks, keys))
    run(program, cases)


def test_slots_of_an_append(program):
    rng = random.Random(22)
    cases = [(1, 0, 0, 1, 16, 1, 0), (1, 5, 9, 9, 16, 1, 0), (1, 2 ** 31 - 1, 7, 7, 16, 3, 0),
             (1, -2 ** 31, 7, 7, 16, 3, 0), (1, 17, -1, 3, 16, 2, 0)]
    for _ in range(3000):
        page, per_seq, T = 16 * rng.randint(1, 8), rng.randint(1, 9), rng.randint(1, 200)
        cases.append((1, rng.randint(-3, page * per_seq + 40), rng.choice((T, rng.randint(-2, T + 5))), T,
                      page, per_seq, 0))
    run(program, cases)
