"""A key that is not finite, in places that queries see: the rows that see it
are NaN in O and LSE, as the softmax's definition gives (a NaN score, or
+inf - +inf), and every other row is what a call with a finite key gives, bit
for bit.  Never O = 0 with LSE = -inf, which says that a row sees no key, and
never the softmax over the remaining keys."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa
import window_common as wc
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu

JUNK = [float("nan"), float("inf")]
ONE_KIND = pytest.mark.parametrize("junk", JUNK, ids=["nan", "inf"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def inputs(B, H, Hk, Nq, Nk, d, dtype="fp16", seed=90):
    """Queries whose first column is positive: a key with +inf there has score +inf."""
    q = wc.normal((B, H, Nq, d), dtype, seed)
    q[..., 0] = q[..., 0].abs() + 0.125
    return (q.cuda(), wc.normal((B, Hk, Nk, d), dtype, seed + 1).cuda(),
            wc.normal((B, Hk, Nk, d), dtype, seed + 2).cuda())


def check(call, k, places, masks, junk):
    """call(k) -> O, LSE; places: (batch, key/value head, key) to spoil."""
    o0, lse0 = call(k)
    bad = k.clone()
    for b, h, j in places:
        bad[b, h, j, 0] = junk
    o, lse = call(bad)
    torch.cuda.synchronize()
    assert fa.fa_status()[0] == fa.FA_OK
    B, H = lse.shape[:2]
    G = H // k.shape[1]
    hit = np.zeros(lse.shape, dtype=bool)
    for b, h, j in places:
        hit[b, h * G:(h + 1) * G] |= masks[b][:, j][None, :]
    hit = torch.from_numpy(hit).cuda()
    assert bool(hit.any()) and not bool(hit.all())
    assert bool(torch.isnan(lse[hit]).all()) and bool(torch.isnan(o[hit]).all())
    assert torch.equal(o[~hit], o0[~hit]) and torch.equal(lse[~hit], lse0[~hit])
    assert not bool(torch.isnan(lse0).any())


def masks_of(Nq, Nk, lens, win, sinks, causal="bottom_right"):
    return [wc.window_mask(Nq, Nk, n, causal, win, sinks) for n in lens]


# rows of a key/value head: 6 (four copies), 48 (two), 128 (one), 256 (two row tiles)
@ONE_KIND
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Nq", [(2, 3), (3, 16), (8, 16), (16, 16)])
def test_decode_window(G, Nq, d, junk):
    """Units of a few tiles and, with one sequence, one unit cut over many CTAs."""
    lens = [700, 411, 203]
    q, k, v = inputs(3, 2 * G, 2, Nq, 700, d)
    ms = masks_of(Nq, 700, lens, 500, 5)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    run = lambda kk: fa.attention_decode_window(q, kk, v, 500, 5, seqlens_k=n)
    check(run, k, [(0, 0, 2), (1, 1, 400 - Nq)], ms, junk)     # a sink, a key inside
    check(run, k, [(0, 1, 699), (2, 0, 202)], ms, junk)        # the last token's own key
    q, k, v = inputs(1, G, 1, Nq, 9000, d, seed=95)
    ms = masks_of(Nq, 9000, [9000], 8000, 3)
    run = lambda kk: fa.attention_decode_window(q, kk, v, 8000, 3)
    check(run, k, [(0, 0, 8999)], ms, junk)
    q2, k2 = q.expand(2, G, Nq, d).contiguous(), k.expand(2, 1, 9000, d).contiguous()
    v2 = v.expand(2, 1, 9000, d).contiguous()
    ms = masks_of(Nq, 9000, [9000, 9000], 8000, 3)
    run = lambda kk: fa.attention_decode_window(q2, kk, v2, 8000, 3)
    for key in (1, 1100, 5000, 8990 - Nq):
        check(run, k2, [(1, 0, key)], ms, junk)


@ONE_KIND
@pytest.mark.parametrize("T,G,Nk", [(20, 1, 600), (20, 3, 4000), (64, 4, 4000)])
def test_decode_tree(T, G, Nk, junk):
    hist = [Nk - T, 150]
    q, k, v = inputs(2, G, 1, T, Nk, 128)
    rng = np.random.default_rng(3)
    up = torch.tensor([[-1] + [int(rng.integers(-1, i)) for i in range(1, T)]] * 2)
    rows = fa.tree_rows(up).cuda()
    ms = [wc.tree_mask(rows[b].tolist(), Nk, hist[b], None, 0) for b in range(2)]
    n = torch.tensor(hist, dtype=torch.int32, device="cuda")
    run = lambda kk: fa.attention_decode_tree(q, kk, v, rows, seqlens_k=n)
    check(run, k, [(0, 0, hist[0] // 2)], ms, junk)
    check(run, k, [(0, 0, hist[0] + 1), (1, 0, 150 + T - 1)], ms, junk)


@ONE_KIND
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_window(d, junk):
    lens = [700, 650]
    q, k, v = inputs(2, 4, 2, 600, 700, d)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for win, sinks in ((300, 5), (100, 40)):
        ms = masks_of(600, 700, lens, win, sinks)
        run = lambda kk: fa.attention_forward_window(q, kk, v, win, sinks, seqlens_k=n)
        check(run, k, [(0, 0, 400)], ms, junk)
        check(run, k, [(1, 1, 649), (0, 1, 699)], ms, junk)


@ONE_KIND
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["plain", "causal", "split", "split causal", "dropout"])
def test_square_forward(form, d, junk):
    """Heads with one bad key; with dropout a row that dropped it has a sum of NaN too."""
    B, H, N = 2, 40, 600
    q, k, v = inputs(B, H, H, N, N, d, "bf16")
    causal = "causal" in form
    ms = [np.tril(np.ones((N, N), dtype=bool)) if causal else np.ones((N, N), dtype=bool)] * B
    if form == "dropout":
        run = lambda kk: fa.flash_attention(q, kk, v, dropout_p=0.5, seed=3)
    else:
        ws = "auto" if "split" in form else None
        run = lambda kk: fa.attention_forward(q, kk, v, causal=causal, workspace=ws)
    places = [(b, h, (37 * h) % N) for b in range(B) for h in range(0, H, 3)]
    check(run, k, places, ms, junk)


@ONE_KIND
@pytest.mark.parametrize("Nk", [700, 20000])
def test_decode(Nk, junk):
    B, H, Nq, d = 1, 2, 3, 128
    q, k, v = inputs(B, H, H, Nq, Nk, d, "bf16")
    ms = masks_of(Nq, Nk, [Nk], 1 << 30, 0)
    run = lambda kk: fa.attention_decode(q, kk, v, causal=True)
    for key in (0, Nk // 2, Nk - 1):
        check(run, k, [(0, 1, key)], ms, junk)
