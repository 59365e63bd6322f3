"""Decoding under a sliding window with sinks (fa_decode_window) and of drafted
trees (fa_decode_tree) against the float64 definition, and the run of the
window's operators together: a prompt, single tokens, a drafted tree."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa
import window_common as wc
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def status_ok():
    torch.cuda.synchronize()
    code, word = fa.fa_status()
    assert code == fa.FA_OK, f"device status {word:#x}"


def inputs(B, H, Hk, Nq, Nk, d, dtype, seed=0):
    return (wc.normal((B, H, Nq, d), dtype, seed), wc.normal((B, Hk, Nk, d), dtype, seed + 1),
            wc.normal((B, Hk, Nk, d), dtype, seed + 2))


def counts(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


WINDOW_CASES = [
    # B, H, Hk, Nq, Nk, d, dtype, window, sinks, lens
    (1, 1, 1, 1, 1, 64, "bf16", 1, 0, None),
    (1, 8, 2, 1, 1000, 128, "bf16", 256, 4, None),
    (1, 8, 8, 1, 129, 64, "fp16", 128, 0, None),
    (2, 4, 1, 4, 700, 64, "fp16", 100, 3, [700, 350]),
    (3, 6, 2, 16, 900, 128, "fp16", 300, 5, [900, 7, 0]),          # rows before the first key
    (2, 16, 1, 16, 1500, 64, "bf16", 700, 16, [1500, 801]),        # 256 rows
    (1, 24, 1, 16, 600, 128, "bf16", 1000000, 0, None),            # 384 rows, no limit
    (5, 2, 2, 3, 400, 64, "bf16", 17, 130, [400, 399, 131, 146, 2]),   # more than a tile of sinks
    (2, 3, 3, 2, 333, 128, "fp16", 1, 0, None),
    (40, 2, 1, 1, 500, 64, "fp16", 200, 4, [11 * b % 501 for b in range(40)]),
    (1, 2, 1, 8, 5000, 128, "bf16", 4000, 1, [4999]),
    (300, 2, 2, 1, 130, 64, "bf16", 64, 2, [(7 * b) % 131 for b in range(300)]),   # runs of units
]


def window_masks(B, Nq, Nk, lens, win, sinks):
    return [wc.window_mask(Nq, Nk, Nk if lens is None else lens[b], "bottom_right", win, sinks)
            for b in range(B)]


@pytest.mark.parametrize("case", WINDOW_CASES, ids=["-".join(map(str, c[:9])) for c in WINDOW_CASES])
def test_decode_window_against_definition(case):
    B, H, Hk, Nq, Nk, d, dtype, win, sinks, lens = case
    q, k, v = inputs(B, H, Hk, Nq, Nk, d, dtype)
    o, lse = fa.attention_decode_window(q.cuda(), k.cuda(), v.cuda(), win, sinks,
                                        seqlens_k=counts(lens))
    status_ok()
    val, tol = wc.reference(q, k, v, window_masks(B, Nq, Nk, lens, win, sinks), wc.scale_of(d),
                            dtype)
    wc.check(dict(o=o, lse=lse), val, tol, str(case))


def random_parents(B, T, seed):
    rng = np.random.default_rng(seed)
    p = np.full((B, T), -1, dtype=np.int64)
    for i in range(1, T):
        p[:, i] = rng.integers(-1, i, size=B)
    return torch.from_numpy(p)


TREE_CASES = [
    # B, H, Hk, Nq, Nk, d, dtype, window, sinks, lens (history)
    (1, 1, 1, 1, 1, 64, "bf16", None, 0, None),                 # no history
    (1, 8, 2, 7, 600, 64, "fp16", None, 0, None),
    (2, 4, 1, 33, 700, 128, "bf16", None, 0, [600, 1]),
    (2, 4, 1, 64, 800, 64, "fp16", None, 0, [736, 100]),        # 256 rows
    (1, 12, 2, 50, 500, 128, "fp16", None, 0, [0]),             # 300 rows, only the tree
    (3, 6, 3, 20, 900, 64, "bf16", 200, 4, [880, 300, 64]),
    (2, 2, 1, 40, 300, 64, "fp16", 5, 3, [250, 3]),             # drafted tokens leave the window
    (2, 2, 2, 64, 400, 128, "bf16", 63, 0, [300, 400]),         # slots past the cache
    (1, 4, 2, 64, 2000, 64, "fp16", 1, 2, None),
    (2, 8, 1, 16, 260, 128, "fp16", 128, 20, [128, 244]),
]


@pytest.mark.parametrize("case", TREE_CASES, ids=["-".join(map(str, c[:9])) for c in TREE_CASES])
def test_decode_tree_against_definition(case):
    B, H, Hk, T, Nk, d, dtype, win, sinks, lens = case
    q, k, v = inputs(B, H, Hk, T, Nk, d, dtype, seed=50)
    rows = fa.tree_rows(random_parents(B, T, 4))
    if T > 4:
        rows[0, 3] = 0                                # a padding row: the history alone
    if T < 64:
        rows[:, 0] |= torch.tensor(-2 ** 63)          # a bit past Nq means nothing
    o, lse = fa.attention_decode_tree(q.cuda(), k.cuda(), v.cuda(), rows.cuda(),
                                      seqlens_k=counts(lens), window=win, sinks=sinks)
    status_ok()
    hist = [Nk - T] * B if lens is None else lens
    masks = [wc.tree_mask(rows[b].tolist(), Nk, hist[b], win, sinks) for b in range(B)]
    val, tol = wc.reference(q, k, v, masks, wc.scale_of(d), dtype)
    wc.check(dict(o=o, lse=lse), val, tol, str(case))


@pytest.mark.parametrize("junk", [float("nan"), float("-inf")])
@pytest.mark.parametrize("G,Nq", [(2, 3), (8, 16)])
def test_stale_cache_may_hold_anything(G, Nq, junk):
    """Cache slots that no token sees (evicted between sinks and window, past
    the count) reach no result, in one row tile and in two, nor do they in
    the drafted form."""
    B, Hk, Nk, d, win, sinks = 3, 2, 700, 128, 90, 5
    lens = [700, 411, 203]
    q, k, v = inputs(B, G * Hk, Hk, Nq, Nk, d, "fp16", seed=60)
    ms = window_masks(B, Nq, Nk, lens, win, sinks)
    for b in range(B):
        unseen = torch.from_numpy(~ms[b].any(0))
        k[b, :, unseen] = junk
        v[b, :, unseen] = junk
    o, lse = fa.attention_decode_window(q.cuda(), k.cuda(), v.cuda(), win, sinks,
                                        seqlens_k=counts(lens))
    status_ok()
    val, tol = wc.reference(q, k, v, ms, wc.scale_of(d), "fp16")
    wc.check(dict(o=o, lse=lse), val, tol, f"junk {junk}")
    # the same queries as a drafted chain: all of them see what they saw
    rows = fa.tree_rows(torch.arange(-1, Nq - 1).expand(B, Nq))
    o2, lse2 = fa.attention_decode_tree(q.cuda(), k.cuda(), v.cuda(), rows.cuda(),
                                        seqlens_k=counts([n - Nq for n in lens]), window=win,
                                        sinks=sinks)
    status_ok()
    wc.check(dict(o=o2, lse=lse2), val, tol, f"chain, junk {junk}")


@pytest.mark.parametrize("d", [64, 128])
def test_drafted_slots_that_no_row_marks_may_hold_anything(d):
    """Padded trees: a batch's last rows are 0 and its last slots stale; the
    keys before the window too, one key earlier where a padding row sits."""
    B, H, Hk, T, Nk, win, sinks = 2, 4, 1, 20, 500, 70, 2
    lens = [480, 130]
    q, k, v = inputs(B, H, Hk, T, Nk, d, "bf16", seed=65)
    rows = fa.tree_rows(random_parents(B, T, 5))
    rows[1, 13:] = 0
    masks = [wc.tree_mask(rows[b].tolist(), Nk, lens[b], win, sinks) for b in range(B)]
    for b in range(B):
        unseen = torch.from_numpy(~masks[b].any(0))
        assert unseen[lens[b] + 13] == (b == 1)
        k[b, :, unseen] = float("nan")
        v[b, :, unseen] = float("nan")
    o, lse = fa.attention_decode_tree(q.cuda(), k.cuda(), v.cuda(), rows.cuda(),
                                      seqlens_k=counts(lens), window=win, sinks=sinks)
    status_ok()
    val, tol = wc.reference(q, k, v, masks, wc.scale_of(d), "bf16")
    wc.check(dict(o=o, lse=lse), val, tol, "padded tree")


def test_captured_graphs_with_their_own_workspaces():
    """Two captured calls replay with new inputs and counts, on two streams."""
    B, H, Hk, Nk, d = 4, 8, 2, 900, 64
    made = []
    for g in range(2):
        q, k, v = (t.cuda() for t in inputs(B, H, Hk, 1, Nk, d, "bf16", seed=70 + g))
        sl = counts([900, 10, 500, 333])
        ws = fa.make_decode_workspace(q, k)
        out = torch.empty_like(q)
        lse = torch.empty(B, H, 1, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        fa.attention_decode_window(q, k, v, 300, 2, seqlens_k=sl, out=out, lse=lse, workspace=ws,
                                   stream=s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fa.attention_decode_window(q, k, v, 300, 2, seqlens_k=sl, out=out, lse=lse,
                                       workspace=ws)
        made.append((graph, s, q, k, v, sl, out, lse, ws))
    for step in range(3):
        refs = []
        for g, (graph, s, q, k, v, sl, out, lse, ws) in enumerate(made):
            new = inputs(B, H, Hk, 1, Nk, d, "bf16", seed=90 + 2 * step + g)
            for t, x in zip((q, k, v), new):
                t.copy_(x)
            lens = [(123 * (step + g) + 77 * b) % 901 for b in range(B)]
            sl.copy_(torch.tensor(lens, dtype=torch.int32))
            refs.append((new, lens))
        torch.cuda.synchronize()
        for m in made:
            with torch.cuda.stream(m[1]):
                m[0].replay()
        status_ok()
        for m, (new, lens) in zip(made, refs):
            val, tol = wc.reference(*new, window_masks(B, 1, Nk, lens, 300, 2), wc.scale_of(d),
                                    "bf16")
            wc.check(dict(o=m[6], lse=m[7]), val, tol, f"replay {step}")


def test_results_do_not_depend_on_the_run():
    q, k, v = (t.cuda() for t in inputs(3, 8, 2, 4, 3001, 128, "bf16", seed=80))
    first = fa.attention_decode_window(q, k, v, 2500, 4)
    for _ in range(5):
        again = fa.attention_decode_window(q, k, v, 2500, 4)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    status_ok()


def test_cache_past_two_to_the_31_elements():
    """Heads whose keys start past element 2^31 of the cache."""
    B, Hk, Nk, d = 5, 8, 1 << 19, 128                       # 2.7e9 elements, 5.4 GB each
    k = torch.zeros(B, Hk, Nk, d, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    lens = [900, 1, 400, 700, Nk]
    win, sinks = 500, 3
    q = wc.normal((B, Hk, 2, d), "fp16", 1)
    tail = wc.normal((2, Hk, 1000, d), "fp16", 2)
    kc, vc = tail[0][None].repeat(B, 1, 1, 1), tail[1][None].repeat(B, 1, 1, 1)
    for b, n in enumerate(lens):                            # the last 1000 keys, and the sinks
        m = min(n, 1000)
        k[b, :, n - m:n] = kc[b, :, :m].cuda()
        v[b, :, n - m:n] = vc[b, :, :m].cuda()
    o, lse = fa.attention_decode_window(q.cuda(), k, v, win, sinks, seqlens_k=counts(lens))
    status_ok()
    for b, n in enumerate(lens):
        m = min(n, 1000)
        keys = torch.cat((k[b, :, :sinks], k[b, :, n - m:n]), 1).cpu() if n > m else kc[b, :, :m]
        vals = torch.cat((v[b, :, :sinks], v[b, :, n - m:n]), 1).cpu() if n > m else vc[b, :, :m]
        L = keys.shape[1]
        # sinks first, then the span: the window's mask over this shortened list
        mask = [wc.window_mask(2, L, L, "bottom_right", win, sinks)]
        val, tol = wc.reference(q[b:b + 1], keys[None], vals[None], mask, wc.scale_of(d), "fp16")
        wc.check(dict(o=o[b:b + 1], lse=lse[b:b + 1]), val, tol, f"batch {b}")


def test_prompt_tokens_and_a_drafted_tree_agree():
    """A prompt through fa_fwd_window, two tokens through fa_decode_window and
    a tree through fa_decode_tree on one cache: every row equals the same
    position's row of one long prompt over its own path."""
    H, Hk, d, win, sinks, N, steps, T = 4, 2, 64, 60, 3, 200, 2, 12
    total = N + steps
    cap = total + T + 5
    q, k, v = inputs(1, H, Hk, cap, cap, d, "fp16", seed=100)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    o, lse = fa.attention_forward_window(qd[:, :, :N].contiguous(), kd, vd, win, sinks,
                                         causal="upper_left", seqlens_k=counts([N]))
    rows = [(o, lse)]
    for s in range(steps):
        n = N + s + 1
        rows.append(fa.attention_decode_window(qd[:, :, n - 1:n].contiguous(), kd, vd, win, sinks,
                                               seqlens_k=counts([n])))
    got = dict(o=torch.cat([r[0] for r in rows], 2), lse=torch.cat([r[1] for r in rows], 2))
    status_ok()
    mask = [wc.window_mask(total, total, total, "upper_left", win, sinks)]
    val, tol = wc.reference(q[:, :, :total], k[:, :, :total], v[:, :, :total], mask,
                            wc.scale_of(d), "fp16")
    wc.check(got, val, tol, "prompt and tokens")
    parents = random_parents(1, T, 8)
    qt = qd[:, :, total:total + T].contiguous()
    o, lse = fa.attention_decode_tree(qt, kd, vd, fa.tree_rows(parents).cuda(),
                                      seqlens_k=counts([total]), window=win, sinks=sinks)
    status_ok()
    for i in range(T):
        path, at = [i], int(parents[0, i])
        while at >= 0:
            path.insert(0, at)
            at = int(parents[0, at])
        slots = list(range(total)) + [total + j for j in path]
        L = len(slots)
        mask = [wc.window_mask(1, L, L, "bottom_right", win, sinks)]
        val, tol = wc.reference(qt[:, :, i:i + 1].cpu(), k[:, :, slots], v[:, :, slots], mask,
                                wc.scale_of(d), "fp16")
        wc.check(dict(o=o[:, :, i:i + 1], lse=lse[:, :, i:i + 1]), val, tol, f"drafted {i}")


def test_no_keys():
    q = torch.ones(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_decode_window(q, k, k, 8)
    status_ok()
    assert not o.any() and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Nq", [(1, 1), (3, 15), (2, 50), (4, 64), (5, 60)])
def test_long_runs_of_tiles(G, Nq, d):
    """Many tiles and several units a CTA, from HBM, for every number of rows'
    variant (1, 45, 100, 256, 300 rows): first, last and a cut unit against the
    definition, and the same call again bit for bit."""
    B, Hk, Nk = 2, 50, 6000
    g = torch.Generator(device="cuda").manual_seed(7)
    dt = torch.float16
    k = torch.randn(B, Hk, Nk, d, generator=g, device="cuda", dtype=dt)
    v = torch.randn(B, Hk, Nk, d, generator=g, device="cuda", dtype=dt)
    q = torch.randn(B, G * Hk, Nq, d, generator=g, device="cuda", dtype=dt)
    rows = fa.tree_rows(random_parents(B, Nq, 3))
    lens = [Nk - Nq, 4321]
    args = (q, k, v, rows.cuda())
    o, lse = fa.attention_decode_tree(*args, seqlens_k=counts(lens))
    for _ in range(20):      # back to back: the last one is compared
        o2, lse2 = fa.attention_decode_tree(*args, seqlens_k=counts(lens))
    status_ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b, hk in ((0, 0), (0, 31), (1, 20), (1, Hk - 1)):
        hq = slice(hk * G, hk * G + G)
        masks = [wc.tree_mask(rows[b].tolist(), Nk, lens[b], None, 0)]
        val, tol = wc.reference(q[b:b + 1, hq].cpu(), k[b:b + 1, hk:hk + 1].cpu(),
                                v[b:b + 1, hk:hk + 1].cpu(), masks, wc.scale_of(d), "fp16")
        wc.check(dict(o=o[b:b + 1, hq], lse=lse[b:b + 1, hq]), val, tol, f"batch {b} head {hk}")


def test_counts_out_of_range_are_clamped():
    B, H, Hk, Nk, d = 4, 4, 2, 300, 64
    lens = [-7, 301, 2**31 - 1, -2**31]
    q, k, v = inputs(B, H, Hk, 2, Nk, d, "fp16", seed=17)
    o, lse = fa.attention_decode_window(q.cuda(), k.cuda(), v.cuda(), 60, 3, seqlens_k=counts(lens))
    rows = fa.tree_rows(torch.tensor([[-1, 0]]).expand(B, 2))
    o2, lse2 = fa.attention_decode_tree(q.cuda(), k.cuda(), v.cuda(), rows.cuda(),
                                        seqlens_k=counts(lens), window=60, sinks=3)
    status_ok()
    val, tol = wc.reference(q, k, v, window_masks(B, 2, Nk, lens, 60, 3), wc.scale_of(d), "fp16")
    wc.check(dict(o=o, lse=lse), val, tol, "clamped")
    ms = [wc.tree_mask(rows[b].tolist(), Nk, lens[b], 60, 3) for b in range(B)]
    val, tol = wc.reference(q, k, v, ms, wc.scale_of(d), "fp16")
    wc.check(dict(o=o2, lse=lse2), val, tol, "clamped tree")


def test_streams_and_workspaces():
    """Two calls at once on two streams, each with its workspace and on a
    stream given as an object and as a handle; a short workspace is refused."""
    B, H, Hk, Nk, d = 2, 16, 4, 20000, 128
    k, v = (torch.randn(B, Hk, Nk, d, device="cuda", dtype=torch.float16) for _ in range(2))
    qs = [torch.randn(B, H, 4, d, device="cuda", dtype=torch.float16) for _ in range(2)]
    want = [fa.attention_decode_window(q, k, v, 15000, 4) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [fa.attention_decode_window(q, k, v, 15000, 4,
                                          stream=s if i else s.cuda_stream)
               for i, (q, s) in enumerate(zip(qs, streams))]
        status_ok()
        for (a, b), (c, d2) in zip(want, got):
            assert torch.equal(a, c) and torch.equal(b, d2)
    o, lse = fa.attention_decode_window(qs[0], k, v, 15000, 4, stream=0)
    status_ok()
    assert torch.equal(o, want[0][0])
    with pytest.raises(fa.FaError):
        fa.attention_decode_window(qs[0], k, v, 15000, 4,
                                   workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
