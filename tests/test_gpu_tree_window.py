"""Drafted trees whose window is as long as a row has marks: rows of arbitrary
64-bit words, one of all ones that marks a row of 0, against the definition."""
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa
import window_common as wc
from gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("win", [63, 64, 65])
@pytest.mark.parametrize("G,d", [(1, 64), (4, 128)])
def test_rows_of_all_marks(G, d, win):
    require_gpu()
    B, T, Nk, hist = 2, 64, 400, [300, 20]
    q = wc.normal((B, G, T, d), "bf16", 31)
    k, v = wc.normal((B, 1, Nk, d), "bf16", 32), wc.normal((B, 1, Nk, d), "bf16", 33)
    g = torch.Generator().manual_seed(34)
    rows = torch.randint(-2 ** 63, 2 ** 63 - 1, (B, T), generator=g, dtype=torch.int64)
    rows[:, 0], rows[:, 1], rows[:, 63] = 0, 1, -1
    masks = [wc.tree_mask(rows[b].tolist(), Nk, hist[b], win, 2) for b in range(B)]
    # the row of all marks sits 64 positions past the row of 0
    assert masks[0][63, 300] == (win > 64)
    o, lse = fa.attention_decode_tree(q.cuda(), k.cuda(), v.cuda(), rows.cuda(),
                                      seqlens_k=torch.tensor(hist, dtype=torch.int32).cuda(),
                                      window=win, sinks=2)
    torch.cuda.synchronize()
    assert fa.fa_status()[0] == fa.FA_OK
    val, tol = wc.reference(q, k, v, masks, wc.scale_of(d), "bf16")
    wc.check(dict(o=o, lse=lse), val, tol, f"window {win}")
