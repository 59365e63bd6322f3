"""Sliding-window attention with sinks and shared key/value heads
(fa_fwd_window, fa_bwd_window) against the float64 definition."""
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
            wc.normal((B, Hk, Nk, d), dtype, seed + 2), wc.normal((B, H, Nq, d), dtype, seed + 3))


def lens_tensor(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


def run(q, k, v, do, win, sinks, causal, lens):
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    sl = lens_tensor(lens)
    o, lse = fa.attention_forward_window(q, k, v, win, sinks, causal=causal, seqlens_k=sl)
    dq, dk, dv = fa.attention_backward_window(q, k, v, o, lse, do, win, sinks, causal=causal,
                                              seqlens_k=sl)
    status_ok()
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


def masks(B, Nq, Nk, lens, causal, win, sinks):
    return [wc.window_mask(Nq, Nk, Nk if lens is None else lens[b], causal, win, sinks)
            for b in range(B)]


CASES = [
    # B, H, Hk, Nq, Nk, d, dtype, causal, window, sinks, lens
    (1, 1, 1, 1, 1, 64, "bf16", "upper_left", 1, 0, None),
    (1, 2, 1, 128, 128, 128, "fp16", "upper_left", 128, 0, None),
    (1, 2, 2, 300, 300, 64, "fp16", "upper_left", 1, 0, None),          # only itself
    (2, 4, 2, 333, 333, 64, "bf16", "upper_left", 100, 4, None),
    (1, 6, 2, 700, 700, 128, "fp16", "bottom_right", 129, 5, None),
    (1, 8, 1, 520, 520, 64, "fp16", "upper_left", 64, 130, None),       # two sink tiles
    (1, 3, 3, 600, 600, 128, "bf16", "upper_left", 256, 1, None),
    (2, 4, 1, 200, 1000, 64, "fp16", "bottom_right", 300, 4, None),     # a chunk after a cache
    (2, 2, 1, 129, 900, 128, "fp16", "bottom_right", 200, 3, [900, 371]),
    (3, 2, 2, 257, 512, 64, "bf16", "bottom_right", 77, 0, [512, 130, 0]),   # an empty batch
    (3, 6, 3, 333, 333, 64, "fp16", "upper_left", 50, 0, [333, 100, 1]),     # rows past their keys
    (2, 2, 1, 300, 128, 128, "fp16", "bottom_right", 64, 2, None),      # Nq > Nk: empty rows
    (1, 2, 1, 100, 900, 64, "bf16", "upper_left", 40, 2, None),         # Nq < Nk
    (1, 4, 4, 640, 640, 64, "fp16", "upper_left", 100000, 0, None),     # no limit: causal
    (1, 2, 1, 400, 400, 128, "bf16", "upper_left", 50, 1000, None),     # every key a sink
    (5, 4, 2, 140, 300, 64, "bf16", "bottom_right", 90, 16, [300, 17, 140, 139, 5]),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:10])) + ("p" if c[10] else "")
                                              for c in CASES])
def test_window_against_definition(case):
    B, H, Hk, Nq, Nk, d, dtype, causal, win, sinks, lens = case
    q, k, v, do = inputs(B, H, Hk, Nq, Nk, d, dtype)
    got = run(q, k, v, do, win, sinks, causal, lens)
    val, tol = wc.reference(q, k, v, masks(B, Nq, Nk, lens, causal, win, sinks), wc.scale_of(d),
                            dtype, do)
    wc.check(got, val, tol, str(case))


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_unseen_places_may_hold_anything(d, junk):
    """Keys and values past the counts and between sinks and window, and
    queries and dO of rows that see nothing, do not reach any result."""
    B, H, Hk, Nq, Nk, win, sinks = 3, 4, 2, 200, 700, 60, 3
    lens = [700, 333, 150]            # the last: 50 rows at negative positions
    q, k, v, do = inputs(B, H, Hk, Nq, Nk, d, "fp16", seed=7)
    ms = masks(B, Nq, Nk, lens, "bottom_right", win, sinks)
    for b in range(B):
        keys, rows = torch.from_numpy(ms[b].any(0)), torch.from_numpy(ms[b].any(1))
        k[b, :, ~keys] = junk
        v[b, :, ~keys] = junk
        q[b, :, ~rows] = junk
        do[b, :, ~rows] = junk
    got = run(q, k, v, do, win, sinks, "bottom_right", lens)
    val, tol = wc.reference(q, k, v, ms, wc.scale_of(d), "fp16", do)
    wc.check(got, val, tol, f"junk {junk}")


def test_rows_whose_window_starts_past_the_keys_may_hold_anything():
    B, H, Hk, N, d, win = 2, 2, 1, 300, 64, 40
    lens = [300, 100]
    q, k, v, do = inputs(B, H, Hk, N, N, d, "bf16", seed=9)
    ms = masks(B, N, N, lens, "upper_left", win, 0)
    rows = torch.from_numpy(ms[1].any(1))
    assert (~rows).sum() == 300 - 139
    q[1, :, ~rows] = float("nan")
    do[1, :, ~rows] = float("nan")
    k[1, :, 100:] = float("nan")
    v[1, :, 100:] = float("nan")
    got = run(q, k, v, do, win, 0, "upper_left", lens)
    val, tol = wc.reference(q, k, v, ms, wc.scale_of(d), "bf16", do)
    wc.check(got, val, tol, "past the keys")


def test_wide_window_equals_the_causal_entry_point():
    """A window past every length is the causal mask; shared heads equal
    repeated ones, and their gradients the sum over the group."""
    B, H, Hk, N, d = 1, 4, 2, 777, 128
    q, k, v, do = (t.cuda() for t in inputs(B, H, Hk, N, N, d, "bf16", seed=3))
    kr, vr = k.repeat_interleave(2, 1).contiguous(), v.repeat_interleave(2, 1).contiguous()
    o, lse = fa.attention_forward_window(q, k, v, 2**40, causal="upper_left")
    o2, lse2 = fa.attention_forward_kv(q, kr, vr, causal="upper_left")
    status_ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = fa.attention_backward_window(q, k, v, o, lse, do, 2**40, causal="upper_left")
    g2 = fa.attention_backward_kv(q, kr, vr, o2, lse2, do, causal="upper_left")
    status_ok()
    assert torch.equal(g[0], g2[0])
    for a, b in zip(g[1:], g2[1:]):
        b = b.float().view(B, Hk, 2, N, d)
        # one rounding of the sum against one of each part, and fp32 order
        tol = 2 ** -8 * (b.abs().sum(2) + a.float().abs()) + 1e-4
        assert bool(((a.float() - b.sum(2)).abs() <= tol).all())


def test_results_are_reproducible_and_stream_safe():
    B, H, Hk, N, d = 2, 8, 2, 1000, 64
    q, k, v, do = (t.cuda() for t in inputs(B, H, Hk, N, N, d, "fp16", seed=5))
    ref = run(q.cpu(), k.cpu(), v.cpu(), do.cpu(), 200, 4, "upper_left", None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o, lse = fa.attention_forward_window(q, k, v, 200, 4, causal="upper_left", stream=side)
        g = fa.attention_backward_window(q, k, v, o, lse, do, 200, 4, causal="upper_left",
                                         stream=side)
        torch.cuda.current_stream().wait_stream(side)
        status_ok()
        for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *g)):
            assert torch.equal(x, ref[name]), name


def test_captured_and_replayed_with_new_counts():
    """Forward and backward captured once; replays read new inputs and counts."""
    B, H, Hk, N, d = 2, 4, 2, 400, 64
    q, k, v, do = (t.cuda() for t in inputs(B, H, Hk, N, N, d, "bf16", seed=21))
    sl = lens_tensor([400, 400])

    def step():
        o, lse = fa.attention_forward_window(q, k, v, 90, 3, seqlens_k=sl)
        return (o, lse, *fa.attention_backward_window(q, k, v, o, lse, do, 90, 3, seqlens_k=sl))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for lens, seed in (([400, 123], 31), ([77, 400], 32)):
        new = inputs(B, H, Hk, N, N, d, "bf16", seed=seed)
        for t, x in zip((q, k, v, do), new):
            t.copy_(x)
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        status_ok()
        val, tol = wc.reference(*new[:3], masks(B, N, N, lens, "bottom_right", 90, 3),
                                wc.scale_of(d), "bf16", new[3])
        wc.check(dict(zip(("o", "lse", "dq", "dk", "dv"), out)), val, tol, f"replay {lens}")


def test_autograd_wrapper_and_differences():
    """flash_attention_window's gradients equal the entry point's, and follow
    central differences of a float64 loss."""
    B, H, Hk, N, d = 1, 4, 2, 150, 64
    q, k, v, do = inputs(B, H, Hk, N, N, d, "fp16", seed=41)
    leaves = [t.cuda().requires_grad_() for t in (q, k, v)]
    o, lse = fa.flash_attention_window(*leaves, 40, 2, causal="upper_left")
    assert not lse.requires_grad
    o.backward(do.cuda())
    got = run(q, k, v, do, 40, 2, "upper_left", None)
    for t, name in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(t.grad, got[name]), name
    ms = masks(B, N, N, None, "upper_left", 40, 2)
    rng = np.random.default_rng(0)
    _, tol = wc.reference(q, k, v, ms, wc.scale_of(d), "fp16", do)
    for which, name in enumerate(("dq", "dk", "dv")):
        dirn = rng.standard_normal(tuple(leaves[which].shape))
        h = 1e-4
        loss = []
        for sign in (1, -1):
            ts = [t.double() for t in (q, k, v)]
            ts[which] = ts[which] + sign * h * torch.from_numpy(dirn)
            val, _ = wc.reference(*ts, ms, wc.scale_of(d), "fp16")
            loss.append((val["o"] * do.double().numpy()).sum())
        slope = (loss[0] - loss[1]) / (2 * h)
        mine = (got[name].cpu().double().numpy() * dirn).sum()
        assert abs(mine - slope) <= (np.abs(dirn) * tol[name]).sum() + 1e-4 * (1 + abs(slope))


def test_no_queries_or_no_keys():
    q = torch.zeros(2, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(2, 2, 50, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_forward_window(q, k, k, 8)
    dq, dk, dv = fa.attention_backward_window(q, k, k, o, lse, q, 8)
    status_ok()
    assert o.numel() == 0 and dq.numel() == 0
    assert not dk.any() and not dv.any()
    q = torch.ones(2, 4, 70, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 0, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.attention_forward_window(q, k, k, 8)
    dq, dk, dv = fa.attention_backward_window(q, k, k, o, lse, q, 8)
    status_ok()
    assert not o.any() and bool(torch.isneginf(lse).all()) and not dq.any() and dk.numel() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_many_tiles_a_unit_and_many_units_a_cta(d):
    """Windows of many whole tiles, more units than SMs: rows of a few heads
    against the definition, key by key from the whole cache."""
    B, H, Hk, N, win, sinks = 1, 48, 12, 2500, 1100, 4
    q, k, v, do = inputs(B, H, Hk, N, N, d, "bf16", seed=13)
    got = run(q, k, v, do, win, sinks, "upper_left", None)
    ms = masks(B, N, N, None, "upper_left", win, sinks)
    for hk in (0, 11):
        hq = slice(hk * 4, hk * 4 + 4)
        val, tol = wc.reference(q[:, hq], k[:, hk:hk + 1], v[:, hk:hk + 1], ms, wc.scale_of(d),
                                "bf16", do[:, hq])
        part = {n: got[n][:, hq] if n in ("o", "lse", "dq") else got[n][:, hk:hk + 1] for n in got}
        wc.check(part, val, tol, f"head {hk}")


def test_counts_out_of_range_are_clamped():
    B, H, Hk, Nq, Nk, d = 4, 2, 1, 130, 300, 64
    q, k, v, do = inputs(B, H, Hk, Nq, Nk, d, "fp16", seed=17)
    lens = [-7, 301, 2**31 - 1, -2**31]
    got = run(q, k, v, do, 60, 3, "bottom_right", lens)
    val, tol = wc.reference(q, k, v, masks(B, Nq, Nk, lens, "bottom_right", 60, 3), wc.scale_of(d),
                            "fp16", do)
    wc.check(got, val, tol, "clamped")
    assert not got["dk"][0].any() and not got["dv"][3].any() and not got["dq"][0].any()


def test_given_buffers_are_filled_and_nothing_else():
    """Outputs given as slices of a larger buffer: the rest stays as it was."""
    B, H, Hk, N, d = 1, 4, 2, 200, 64
    q, k, v, _ = (t.cuda() for t in inputs(B, H, Hk, N, N, d, "fp16", seed=19))
    big = torch.full((3, B, H, N, d), 7.0, dtype=torch.float16, device="cuda")
    biglse = torch.full((3, B, H, N), 7.0, device="cuda")
    o, lse = fa.attention_forward_window(q, k, v, 50, 1, out=big[1], lse=biglse[1])
    o2, lse2 = fa.attention_forward_window(q, k, v, 50, 1)
    status_ok()
    assert o.data_ptr() == big[1].data_ptr()
    assert torch.equal(big[1], o2) and torch.equal(biglse[1], lse2)
    assert bool((big[0] == 7).all() & (big[2] == 7).all())
    assert bool((biglse[0] == 7).all() & (biglse[2] == 7).all())
    with pytest.raises(ValueError):
        fa.attention_forward_window(q, k, v, 50, 1, out=big[1].transpose(1, 2))
    with pytest.raises(ValueError):
        fa.attention_forward_window(q, k, v, 50, 1, lse=biglse[1].half())
    with pytest.raises(ValueError):
        fa.attention_forward_window(q.transpose(1, 2), k, v, 50, 1)


@pytest.mark.parametrize("causal,lens", [("bottom_right", [1000, 100, 0]), ("upper_left", [1000, 128, 3])])
def test_parts_of_sink_tiles_without_steps(causal, lens):
    """Sink tiles cut into parts, of which a short batch fills few or none."""
    B, H, Hk, N, d, win, sinks = 3, 4, 2, 1000, 64, 100, 200
    assert fa.fa_bwd_window_workspace_size(B, H, Hk, N, N, d, win, sinks) > 0
    q, k, v, do = inputs(B, H, Hk, N, N, d, "bf16", seed=23)
    got = run(q, k, v, do, win, sinks, causal, lens)
    val, tol = wc.reference(q, k, v, masks(B, N, N, lens, causal, win, sinks), wc.scale_of(d),
                            "bf16", do)
    wc.check(got, val, tol, f"{causal} {lens}")


def test_rows_past_two_to_the_31_elements():
    """Q, O, dO and dQ of more than 2^31 elements: the last rows of the last
    head, and the last keys, against the definition of the last 300 tokens."""
    B, H, Hk, N, d, win, m = 1, 2, 1, 2**24 + 300, 64, 40, 300
    gen = torch.Generator(device="cuda").manual_seed(29)
    q, do = (torch.randn(B, H, N, d, dtype=torch.bfloat16, device="cuda", generator=gen)
             for _ in range(2))
    k, v = (torch.randn(B, Hk, N, d, dtype=torch.bfloat16, device="cuda", generator=gen)
            for _ in range(2))
    o, lse = fa.attention_forward_window(q, k, v, win, causal="upper_left")
    dq, dk, dv = fa.attention_backward_window(q, k, v, o, lse, do, win, causal="upper_left")
    status_ok()
    last = [t[:, :, -m:].contiguous() for t in (q, k, v, do, o, lse, dq, dk, dv)]
    del q, k, v, do, o, lse, dq, dk, dv
    torch.cuda.empty_cache()
    val, tol = wc.reference(*(t.cpu() for t in last[:3]), masks(B, m, m, None, "upper_left", win, 0),
                            wc.scale_of(d), "bf16", last[3].cpu())
    # the first `win` rows and keys of the cut lack what lies before it
    cut = lambda t: t[:, :, win:]
    got = dict(zip(("o", "lse", "dq", "dk", "dv"), map(cut, last[4:])))
    wc.check(got, {n: cut(x) for n, x in val.items()}, {n: cut(x) for n, x in tol.items()}, "last rows")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [1, 16, 31, 32, 33, 128, 129, 300])
def test_sinks_far_behind_the_window(d, sinks):
    """Units whose windows lie past the sinks, whole and ragged lengths: a sink
    tile of its own, narrow up to 32 sinks, before or behind the first tile of
    the windows."""
    B, H, Hk, Nq, Nk, win = 2, 4, 2, 700, 1300, 200
    lens = [1300, 911]
    q, k, v, do = inputs(B, H, Hk, Nq, Nk, d, "bf16", seed=100 + sinks)
    ms = masks(B, Nq, Nk, lens, "bottom_right", win, sinks)
    for b in range(B):      # what nobody sees must not matter here either
        unseen = ~torch.from_numpy(ms[b].any(0))
        k[b, :, unseen] = float("nan")
        v[b, :, unseen] = float("nan")
    got = run(q, k, v, do, win, sinks, "bottom_right", lens)
    val, tol = wc.reference(q, k, v, ms, wc.scale_of(d), "bf16", do)
    wc.check(got, val, tol, f"{sinks} sinks")


def test_large_scores_move_the_reference_at_every_tile():
    """Scores that grow along the keys, and largest at the sinks: the running
    maximum moves at each tile, also at a narrow sink tile behind the first."""
    B, H, Hk, N, win = 1, 2, 1, 900, 300
    for d in (64, 128):
        for sign in (1, -1):
            q, k, v, do = inputs(B, H, Hk, N, N, d, "bf16", seed=55)
            ramp = torch.linspace(0.2, 3, N) if sign > 0 else torch.linspace(3, 0.2, N)
            k = (k.float() * ramp[None, None, :, None]).to(k.dtype)
            k[:, :, :4] *= 6
            got = run(q, k, v, do, win, 4, "upper_left", None)
            val, tol = wc.reference(q, k, v, masks(B, N, N, None, "upper_left", win, 4),
                                    wc.scale_of(d), "bf16", do)
            wc.check(got, val, tol, f"d {d} sign {sign}")


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("Nq,Nk,sinks", [(1, 506, 1), (5, 9, 4), (254, 395, 0), (130, 200, 180)])
def test_keys_after_the_last_query_may_hold_anything(Nq, Nk, sinks, junk):
    """Keys of a query tile's key tile that come after its last query."""
    B, H, Hk, win = 2, 4, 2, 35
    for d in (64, 128):
        q, k, v, do = inputs(B, H, Hk, Nq, Nk, d, "bf16", seed=61)
        k[:, :, Nq:] = junk
        v[:, :, Nq:] = junk
        got = run(q, k, v, do, win, sinks, "upper_left", None)
        val, tol = wc.reference(q, k, v, masks(B, Nq, Nk, None, "upper_left", win, sinks),
                                wc.scale_of(d), "bf16", do)
        wc.check(got, val, tol, f"{Nq} of {Nk}, {junk}")
