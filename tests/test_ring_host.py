"""Soundness of the waits on the forward kernel's K/V ring, on the CPU.

A wait by parity for use u of a ring slot returns at once while the slot's
use u - 1 on the same barrier is still in flight (its parity is that of use
u - 2).  It is sound only if use u - 1 is known to be over when the wait
begins, whatever time each load, product and softmax step takes.  The test
reads each variant's ring from the header (stages, query buffers, whether K
and V tiles take rings of their own or share slots), writes the kernel's roles down
as a graph of what must come before what, and asks of every ring wait
whether the landing of the barrier's previous use comes before it.
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
#include "fa_fwd_kernel.cuh"
template <int D, bool kDrop, bool kWin>
void show() {
  using L = fa::Smem<D, kDrop, kWin>;
  std::printf("%d %d %d %d %d %d %d %d\n", D, kDrop, kWin, L::kStages, L::kQBufs, L::kTwoRings,
              L::bVFull - L::bKFull, L::bKvEmpty - L::bVFull);
}
int main() {
  show<64, false, false>(); show<64, true, false>(); show<64, false, true>();
  show<128, false, false>(); show<128, true, false>(); show<128, false, true>();
  return 0;
}
'''

VARIANTS = [(d, drop, win) for d in (64, 128) for drop, win in ((0, 0), (1, 0), (0, 1))]


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc) and not shutil.which("nvcc"):
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("ring")
    src, exe = d / "ring.cu", d / "ring"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", CSRC, "-I", INCLUDE, str(src), "-o", str(exe)], check=True,
                   capture_output=True, timeout=600)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout
    rows = [tuple(int(x) for x in line.split()) for line in out.splitlines()]
    return {r[:3]: r[3:] for r in rows}


def unsound_waits(pieces, stages, q_bufs, form):
    """Ring waits of one CTA that may pass early, as (kind, piece, key tile).
    pieces: the two query tiles' numbers of key tiles, piece by piece; form:
    "shared" (one ring, one full barrier a slot), "apart" (one ring, a full
    barrier a slot for K and one for V) or "two" (half of the slots a ring for
    K, half for V)."""
    before, last = {}, {}

    def after(node, *earlier):
        before.setdefault(node, []).extend(e for e in earlier if e is not None)

    def step(role, node, *earlier):      # the next thing that a role does
        after(node, last.get(role), *earlier)
        last[role] = node

    # the producer: K0 Q K1 V0 K2 V1 ... V_{n-1} of each piece
    tiles = []
    for k, nn in enumerate(pieces):
        tiles.append(("K", k, 0))
        for j in range(max(nn)):
            if j + 1 < max(nn):
                tiles.append(("K", k, j + 1))
            tiles.append(("V", k, j))
    rings = ([[t for t in tiles if t[0] == kind] for kind in "KV"] if form == "two" else [tiles])
    depth = stages // len(rings)
    ring_of = {t: ring for ring in rings for t in ring}
    slot_use = {t: i for ring in rings for i, t in enumerate(ring)}

    def previous(t, same_kind=False):    # the tile that had t's slot (and barrier) before it
        i = slot_use[t] - depth
        while same_kind and i >= 0 and ring_of[t][i][0] != t[0]:
            i -= depth
        return ring_of[t][i] if i >= 0 else None

    for t in tiles:
        step("load", ("issue", t), ("free", previous(t)) if previous(t) else None)
        after(("landed", t), ("issue", t))
        if t[0] == "K" and t[2] == 0:
            step("load", ("issue q", t[1]), ("free q", t[1] - q_bufs) if t[1] >= q_bufs else None)
            after(("landed q", t[1]), ("issue q", t[1]))
    waits = []

    def ring_wait(role, t):
        step(role, ("wait", t))
        waits.append(t)
        step(role, ("passed", t), ("landed", t))

    # the S issuer, one softmax group per query tile, the P V issuer
    read_before = [None, None]
    for k, nn in enumerate(pieces):
        step("S", ("q", k), ("landed q", k))
        for j in range(max(nn)):
            ring_wait("S", ("K", k, j))
            took = [w for w in (0, 1) if j < nn[w]]
            for w in took:
                step("S", ("S", w, k, j), read_before[w])
                read_before[w] = ("read", w, k, j)
            after(("free", ("K", k, j)), ("S", took[-1], k, j))
            if j + 1 == max(nn):
                after(("free q", k), ("S", took[-1], k, j))
    for w in (0, 1):
        for k, nn in enumerate(pieces):
            for j in range(nn[w]):
                step(("softmax", w), ("read", w, k, j), ("S", w, k, j))
                step(("softmax", w), ("P", w, k, j), ("PV", w, k, j - 1) if j else None)
            if nn[w]:
                step(("softmax", w), ("O read", w, k), ("PV", w, k, nn[w] - 1))
    out_before = [None, None]
    for k, nn in enumerate(pieces):
        for j in range(max(nn)):
            ring_wait("PV", ("V", k, j))
            took = [w for w in (0, 1) if j < nn[w]]
            for w in took:
                step("PV", ("PV", w, k, j), ("P", w, k, j), None if j else out_before[w])
            after(("free", ("V", k, j)), ("PV", took[-1], k, j))
        for w in (0, 1):
            if nn[w]:
                out_before[w] = ("O read", w, k)

    def comes_before(target, node):
        seen, todo = set(), [node]
        while todo:
            x = todo.pop()
            if x == target:
                return True
            if x not in seen:
                seen.add(x)
                todo.extend(before.get(x, ()))
        return False

    bad = []
    for t in waits:
        use = previous(t, same_kind=form == "apart")
        if use and not comes_before(("landed", use), ("wait", t)):
            bad.append(t)
    return bad


def test_the_model_finds_shared_barriers_unsound():
    # V_0 is the second use of slot 0 in a ring of two; with three stages V_1
    # follows K_1, with eight K_3 may follow a V that only the other query
    # tile's products wait for
    assert ("V", 0, 0) in unsound_waits([(2, 2)], 2, 1, "shared")
    assert ("V", 0, 1) in unsound_waits([(4, 4)], 3, 1, "shared")
    assert unsound_waits([(2, 0), (1, 0), (0, 4)], 8, 2, "shared") == [("K", 2, 3)]


@pytest.mark.parametrize("variant", VARIANTS)
def test_no_ring_wait_passes_early(rings, variant):
    stages, q_bufs, two, k_bars, v_bars = rings[variant]
    form = "two" if two else ("apart" if k_bars else "shared")
    # a barrier a slot of each ring, or two a slot
    assert (k_bars, v_bars) == ((stages // 2, stages // 2) if two else (stages, stages))
    rng = random.Random(5)
    lengths = (1, 1, 2, 3, 4, 5, 6, 9)
    for _ in range(400):
        pieces = []
        for _ in range(rng.randint(1, 5)):
            n, m = rng.choice(lengths), rng.choice(lengths)
            pieces.append(rng.choice(((n, n), (n, n + 1), (n, 0), (0, n), (n + 1, n), (n, m))))
        assert unsound_waits(pieces, stages, q_bufs, form) == [], pieces
