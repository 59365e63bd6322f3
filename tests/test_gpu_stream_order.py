"""Work queued behind a backward call starts only when the call's D pass is
done too, also where no query sees a key and no item waits for D: the D
scratch is overwritten on the same stream right behind the call, and must
keep what was written (the D pass of these sizes takes some hundred
microseconds, the items without steps far less)."""
import pytest
import torch

import exact_tiled_attention_14_gb300 as fa

pytestmark = pytest.mark.gpu
B, H, N, D = 4, 16, 16384, 128


@pytest.fixture(scope="module")
def tensors():
    q = torch.ones(B, H, N, D, dtype=torch.bfloat16, device="cuda")
    return q, torch.ones_like(q), torch.empty_like(q), torch.empty(B, H, N, device="cuda")


def refill(tensors, call):
    """The call, a fill of delta behind it, twice; delta holds the second fill."""
    q, dout, dq, delta = tensors
    lse = torch.full((B, H, N), float("-inf"), device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    for value in (3.0, 7.0):
        assert call(q, dout, dq, lse, delta, st) == fa.FA_OK
        delta.fill_(value)
    torch.cuda.synchronize()
    assert fa.fa_status()[0] == fa.FA_OK
    assert bool((delta == 7.0).all()) and not dq.any()


@pytest.mark.parametrize("Nk,count,causal", [(0, 0, 2), (300, 0, 1), (300, -5, 2)])
def test_window_backward_that_sees_nothing(tensors, Nk, count, causal):
    k = torch.ones(B, 4, Nk, D, dtype=torch.bfloat16, device="cuda")
    dk, dv = torch.empty_like(k), torch.empty_like(k)
    lens = torch.full((B,), count, dtype=torch.int32, device="cuda")
    refill(tensors, lambda q, do, dq, lse, delta, st: fa.fa_bwd_window(
        q, k, k, q, lse, do, dq, dk, dv, delta, B, H, 4, N, Nk, D, causal, 100, 0, lens,
        D ** -0.5, fa.FA_BF16, None, 0, st))
    assert not dk.any() and not dv.any()


@pytest.mark.parametrize("Nk,count", [(0, 0), (300, 0)])
def test_kv_backward_that_sees_nothing(tensors, Nk, count):
    k = torch.ones(B, H, Nk, D, dtype=torch.bfloat16, device="cuda")
    dk, dv = torch.empty_like(k), torch.empty_like(k)
    lens = torch.full((B,), count, dtype=torch.int32, device="cuda")
    refill(tensors, lambda q, do, dq, lse, delta, st: fa.fa_bwd_kv(
        q, k, k, q, lse, do, dq, dk, dv, delta, B, H, N, Nk, D, D, 2, lens, D ** -0.5,
        fa.FA_BF16, st))
    assert not dk.any() and not dv.any()
