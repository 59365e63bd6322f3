"""Refusals of the sliding-window and drafted-tree entry points (CPU): return
codes of the C ABI in their documented order, before any device work, and the
binding's TypeError and ValueError."""
import ctypes
import os

import pytest
import torch

import exact_tiled_attention_14_gb300 as fa

FAKE = 0x10000   # 256-byte aligned, never dereferenced (errors are returned first)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(fa.LIB_PATH):
        fa.build()
    return fa.load_library()


FWD = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=2, H=6, Hk=3, Nq=300, Nk=500, d=64, causal=2,
           window=100, sinks=4, seqlens_k=FAKE, scale=0.1, dtype=fa.FA_FP16)
COMMON = [
    (dict(B=-1), fa.FA_ERR_SHAPE), (dict(H=-2), fa.FA_ERR_SHAPE), (dict(Hk=0), fa.FA_ERR_SHAPE),
    (dict(Hk=4), fa.FA_ERR_SHAPE), (dict(H=3, Hk=6), fa.FA_ERR_SHAPE), (dict(Nk=-1), fa.FA_ERR_SHAPE),
    (dict(d=0), fa.FA_ERR_SHAPE), (dict(d=96), fa.FA_ERR_UNSUPPORTED_D),
    (dict(window=0), fa.FA_ERR_SHAPE), (dict(window=-5), fa.FA_ERR_SHAPE),
    (dict(sinks=-1), fa.FA_ERR_SHAPE), (dict(dtype=2), fa.FA_ERR_DTYPE),
    (dict(scale=0.0), fa.FA_ERR_SCALE), (dict(scale=NAN), fa.FA_ERR_SCALE),
    (dict(scale=INF), fa.FA_ERR_SCALE), (dict(B=0, q=None), fa.FA_OK),
    (dict(H=0, Hk=0, q=None), fa.FA_OK), (dict(q=None), fa.FA_ERR_NULLPTR),
    (dict(k=None), fa.FA_ERR_NULLPTR), (dict(lse=None), fa.FA_ERR_NULLPTR),
    (dict(v=FAKE + 8), fa.FA_ERR_ALIGN), (dict(o=FAKE + 2), fa.FA_ERR_ALIGN),
    (dict(lse=FAKE + 1), fa.FA_ERR_ALIGN), (dict(seqlens_k=FAKE + 2), fa.FA_ERR_ALIGN),
]


@pytest.mark.parametrize("args,code", COMMON + [
    (dict(causal=0), fa.FA_ERR_SHAPE), (dict(causal=3), fa.FA_ERR_SHAPE),
    (dict(Nq=-1), fa.FA_ERR_SHAPE), (dict(Nq=0, q=None, o=None), fa.FA_OK),
    (dict(Nq=1 << 30), fa.FA_ERR_SHAPE), (dict(B=1 << 15, H=1 << 15, Hk=1 << 15), fa.FA_ERR_SHAPE),
])
def test_forward(args, code):
    assert fa.fa_fwd_window(**{**FWD, **args}) == code


BWD = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, delta=FAKE,
           B=2, H=6, Hk=3, Nq=3000, Nk=3000, d=64, causal=1, window=100, sinks=4, seqlens_k=None,
           scale=0.1, dtype=fa.FA_BF16, workspace=FAKE, workspace_bytes=1 << 40)


@pytest.mark.parametrize("args,code", COMMON + [
    (dict(causal=0), fa.FA_ERR_SHAPE), (dict(dout=None), fa.FA_ERR_NULLPTR),
    (dict(delta=None), fa.FA_ERR_NULLPTR), (dict(dv=FAKE + 4), fa.FA_ERR_ALIGN),
    (dict(Nq=0, Nk=0, q=None), fa.FA_OK), (dict(workspace=None), fa.FA_ERR_WORKSPACE),
    (dict(workspace_bytes=100), fa.FA_ERR_WORKSPACE), (dict(workspace=FAKE + 16), fa.FA_ERR_ALIGN),
])
def test_backward(args, code):
    assert fa.fa_bwd_window(**{**BWD, **args}) == code


def test_backward_workspace_size(lib):
    size = fa.fa_bwd_window_workspace_size
    assert size(2, 6, 3, 3000, 3000, 64, 100, 0) == 0            # no sinks
    assert size(2, 6, 3, 200, 200, 64, 100, 4) == 0              # as many steps as a window's tile
    # 24 query tiles in parts of 100 // 128 + 2: 12 parts of 128 x 2 d floats a head and sink tile
    assert size(2, 6, 3, 3000, 3000, 64, 100, 4) == 2 * 3 * 12 * 128 * 2 * 64 * 4
    assert size(2, 6, 3, 3000, 3000, 64, 100, 129) == 2 * 2 * 3 * 12 * 128 * 2 * 64 * 4
    with pytest.raises(fa.FaError):
        size(2, 6, 4, 3000, 3000, 64, 100, 4)
    assert lib.fa_bwd_window_workspace_size(2, 6, 3, 3000, 3000, 64, 100, 4, None) == fa.FA_ERR_NULLPTR


@pytest.mark.parametrize("B,Hk,N,window,sinks", [(1, 8, 16384, 2048, 64), (8, 8, 131072, 1, 131072),
                                                 (1, 1, 1 << 20, 1, 70000), (64, 32, 65536, 100, 4)])
def test_backward_workspace_is_bounded(lib, B, Hk, N, window, sinks):
    """However many sink tiles there are, at most 608 parts of 128 x 2 d floats."""
    n = ctypes.c_size_t(1)
    assert lib.fa_bwd_window_workspace_size(B, Hk, Hk, N, N, 128, window, sinks, ctypes.byref(n)) == fa.FA_OK
    assert n.value <= 608 * 128 * 256 * 4
    assert (n.value > 0) == (B * Hk * -(-sinks // 128) <= 304)


DEC = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=2, H=6, Hk=3, Nq=4, Nk=500, d=128, window=100,
           sinks=4, seqlens_k=FAKE, scale=0.1, dtype=fa.FA_FP16, workspace=FAKE,
           workspace_bytes=1 << 40)


@pytest.mark.parametrize("args,code", COMMON + [
    (dict(Nq=0), fa.FA_ERR_SHAPE), (dict(Nq=17), fa.FA_ERR_SHAPE),
    (dict(B=1 << 20, H=1 << 10, Hk=1 << 10), fa.FA_ERR_SHAPE),
    (dict(B=1 << 10, H=1 << 10, Hk=1 << 10, Nk=1 << 20), fa.FA_ERR_SHAPE),
])
def test_decode_window(args, code):
    assert fa.fa_decode_window(**{**DEC, **args}) == code


TREE = dict(DEC, Nq=64, tree=FAKE)


@pytest.mark.parametrize("args,code", [c for c in COMMON if c[0] != dict(window=0)] + [
    (dict(Nq=0), fa.FA_ERR_SHAPE), (dict(Nq=65), fa.FA_ERR_SHAPE), (dict(Nk=63), fa.FA_ERR_SHAPE),
    (dict(tree=None), fa.FA_ERR_NULLPTR), (dict(tree=FAKE + 4), fa.FA_ERR_ALIGN),
])
def test_decode_tree(args, code):
    assert fa.fa_decode_tree(**{**TREE, **args}) == code


def test_decode_workspace_size_refusals(lib):
    out = ctypes.c_size_t(7)
    size = lib.fa_decode_window_workspace_size
    assert size(1, 2, 1, 4, 500, 64, None) == fa.FA_ERR_NULLPTR
    for args, code in (((1, 2, 0, 4, 500, 64), fa.FA_ERR_SHAPE), ((1, 2, 1, 65, 500, 64), fa.FA_ERR_SHAPE),
                       ((1, 2, 1, 4, 500, 32), fa.FA_ERR_UNSUPPORTED_D), ((0, 2, 1, 4, 500, 64), fa.FA_OK)):
        assert size(*args, ctypes.byref(out)) == code
    assert out.value == 0


def test_a_valid_call_needs_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert fa.fa_fwd_window(**FWD) == fa.FA_ERR_DEVICE
    assert fa.fa_bwd_window(**BWD) == fa.FA_ERR_DEVICE
    assert fa.fa_decode_window(**DEC) == fa.FA_ERR_DEVICE
    assert fa.fa_decode_tree(**TREE) == fa.FA_ERR_DEVICE


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding():
    q, k = t(1, 4, 8, 64), t(1, 2, 16, 64)
    calls = [lambda q, k, v, **a: fa.attention_forward_window(q, k, v, a.pop("window", 4), **a),
             lambda q, k, v, **a: fa.attention_decode_window(q, k, v, a.pop("window", 4), **a),
             lambda q, k, v, **a: fa.attention_decode_tree(q, k, v, t(1, 8, dtype=torch.int64),
                                                           window=a.pop("window", 4), **a),
             lambda q, k, v, **a: fa.attention_backward_window(
                 q, k, v, q, torch.zeros(1, 4, 8), q, a.pop("window", 4), **a)]
    for call in calls:
        with pytest.raises(TypeError):
            call(q, k, t(1, 2, 16, 64, dtype=torch.float16))
        with pytest.raises(TypeError):
            call(q.float(), k.float(), k.float())
        with pytest.raises(ValueError):
            call(q[0], k[0], k[0])                                 # rank
        with pytest.raises(ValueError):
            call(q, k, t(1, 2, 15, 64))                            # k, v lengths
        with pytest.raises(ValueError):
            call(q, t(2, 2, 16, 64), t(2, 2, 16, 64))              # batch
        with pytest.raises(ValueError):
            call(q, t(1, 2, 16, 128), t(1, 2, 16, 128))            # width
        with pytest.raises(ValueError):
            call(q, t(1, 3, 16, 64), t(1, 3, 16, 64))              # 4 heads on 3
        with pytest.raises(ValueError):
            call(q, k, k, window=0)
        with pytest.raises(ValueError):
            call(q, k, k, sinks=-1)
        with pytest.raises(ValueError):
            call(q, k, k)                                          # host tensors


def test_tree_rows():
    rows = fa.tree_rows(torch.tensor([[-1, 0, 0, 2, -1], [-1, 0, 1, 2, 3]]))
    assert rows.dtype == torch.int64
    assert rows.tolist() == [[1, 3, 5, 13, 16], [1, 3, 7, 15, 31]]
    chain = fa.tree_rows(torch.arange(-1, 63)[None])
    assert chain[0, 63].item() == -1 and chain[0, 62].item() == 2 ** 63 - 1
    with pytest.raises(ValueError):
        fa.tree_rows(torch.tensor([[0]]))                          # its own parent
    with pytest.raises(ValueError):
        fa.tree_rows(torch.tensor([[-1, -2]]))
    with pytest.raises(ValueError):
        fa.tree_rows(torch.zeros(1, 65, dtype=torch.int64))
