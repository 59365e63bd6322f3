"""Cases, plain forms and exact results of the windowed and drafted-tree
attention operators.

Four calls of the package are covered, all of them exact attention under a
mask that the plain entry points do not have, with K/V heads that may be
shared by a group of G = H / Hk query heads (query head h reads K/V head
h // G):

``prompt``  ``attention_forward_window``: queries at positions p see key j
            when j <= p and (j > p - window or j < sinks).
``train``   the same forward and ``attention_backward_window``: O, LSE, dQ,
            dK, dV of one step.
``token``   ``attention_decode_window``: the last few tokens of each cache.
``tree``    ``attention_decode_tree``: up to 64 drafted tokens whose keys sit
            behind the history in the cache; a token sees the history and
            the drafted tokens its 64-bit row marks.

``run`` takes one pass through an operator: in its plain form (elementary
torch operations in float32) or, where ``own`` is true, through the package.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    """The listed cases.  ``lens`` is "full" (every batch uses all ``Nk`` keys)
    or "ragged" (key counts spread from Nk / 4 to Nk, dealt to the batches by
    the seed).  For ``token`` the counts include the new tokens, for ``tree``
    they are the history before the drafted ones."""
    return [
        # a short prompt of a small model: a few tiles, the launch counts
        dict(name="prompt_short", op="prompt", B=1, H=8, Hk=2, Nq=200, Nk=200, d=64, window=64,
             sinks=4, align="bottom_right", lens="full", dtype="fp16"),
        # chunked prefill: 2048 new tokens of four users against their caches
        dict(name="prompt_chunk", op="prompt", B=4, H=32, Hk=8, Nq=2048, Nk=16384, d=128,
             window=4096, sinks=4, align="bottom_right", lens="ragged", dtype="bf16"),
        # one long document in one call
        dict(name="prompt_long", op="prompt", B=1, H=32, Hk=8, Nq=32768, Nk=32768, d=128,
             window=4096, sinks=16, align="bottom_right", lens="full", dtype="bf16"),
        # a padded batch of short sequences, no shared heads, no sinks: rows
        # far behind a short sequence's end see no key
        dict(name="train_padded", op="train", B=3, H=6, Hk=6, Nq=333, Nk=333, d=64, window=100,
             sinks=0, align="upper_left", lens="ragged", dtype="fp16"),
        # an ordinary training step of narrow heads
        dict(name="train_d64", op="train", B=4, H=16, Hk=4, Nq=4096, Nk=4096, d=64, window=1024,
             sinks=4, align="upper_left", lens="full", dtype="bf16"),
        # long-context training, wide heads in groups of four
        dict(name="train_long", op="train", B=1, H=32, Hk=8, Nq=16384, Nk=16384, d=128,
             window=2048, sinks=64, align="upper_left", lens="full", dtype="bf16"),
        # one user's next token: latency
        dict(name="token_single", op="token", B=1, H=32, Hk=8, Nq=1, Nk=8192, d=128, window=1024,
             sinks=4, lens="full", dtype="bf16"),
        # several tokens a user (odd capacity and window), no shared heads
        dict(name="token_few", op="token", B=16, H=16, Hk=16, Nq=4, Nk=10007, d=64, window=2000,
             sinks=5, lens="ragged", dtype="fp16"),
        # a serving batch of 64 users at mixed lengths
        dict(name="token_batch", op="token", B=64, H=32, Hk=8, Nq=1, Nk=16384, d=128,
             window=4096, sinks=4, lens="ragged", dtype="bf16"),
        # one user's small draft: latency
        dict(name="tree_single", op="tree", B=1, H=16, Hk=4, Nq=7, Nk=1500, d=64, window=0,
             sinks=0, lens="full", dtype="fp16"),
        # drafts of 32 tokens for 16 users at mixed lengths, whole history visible
        dict(name="tree_batch", op="tree", B=16, H=32, Hk=8, Nq=32, Nk=8192, d=128, window=0,
             sinks=0, lens="ragged", dtype="bf16"),
        # the widest drafts over long caches
        dict(name="tree_long", op="tree", B=8, H=32, Hk=8, Nq=64, Nk=131072, d=128, window=0,
             sinks=0, lens="full", dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """Rough seconds of a pass at one card's rates (compares cases only)."""
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.0e15)


def draw(rng):
    """One more case of the listed ranges."""
    limit = {op: max(_cost(c) for c in listed() if c["op"] == op)
             for op in ("prompt", "train", "token", "tree")}
    while True:
        op = rng.choice(("prompt", "train", "token", "tree"))
        Hk = rng.choice((1, 2, 3, 4, 8, 16))
        G = rng.choice((1, 1, 2, 3, 4, 6, 8))
        c = dict(op=op, H=Hk * G, Hk=Hk, d=rng.choice((64, 128)),
                 dtype=rng.choice(("bf16", "fp16")), lens=rng.choice(("full", "ragged")),
                 sinks=rng.choice((0, 1, 4, 5, 16, 64, 130)))
        if c["H"] > 64:
            continue
        if op == "prompt":
            c.update(B=rng.choice((1, 1, 2, 3, 4)), Nq=_log_int(rng, 64, 32768),
                     window=_log_int(rng, 32, 8192))
            c["Nk"] = c["Nq"] + rng.choice((0, _log_int(rng, 64, 16384)))
            c["align"] = "bottom_right"
        elif op == "train":
            c.update(B=rng.choice((1, 2, 3, 4)), Nq=_log_int(rng, 128, 16384),
                     window=_log_int(rng, 32, 4096))
            c["Nk"] = c["Nq"]
            c["align"] = "upper_left"
        elif op == "token":
            c.update(B=_log_int(rng, 1, 64), Nq=rng.choice((1, 1, 1, 2, 3, 4, 5, 8, 16)),
                     Nk=_log_int(rng, 256, 65536), window=_log_int(rng, 128, 16384))
        else:
            c.update(B=_log_int(rng, 1, 32), Nq=_log_int(rng, 4, 64),
                     Nk=_log_int(rng, 512, 131072),
                     window=rng.choice((0, 0, _log_int(rng, 256, 16384))))
        cache = c["B"] * c["Hk"] * c["Nk"] * c["d"] * 4
        if cache <= (9 << 30) and _cost(c) <= limit[op]:
            return c


# ---------------------------------------------------------------- inputs

def _spread(case):
    """Key counts of the batches, in an order that the seed deals."""
    B, top = case["B"], case["Nk"] - (case["Nq"] if case["op"] == "tree" else 0)
    if case["lens"] == "full":
        return [top] * B
    low = max(case["Nk"] // 4, min(case["Nq"], top))
    if B == 1:
        return [(low + top) // 2]
    return [low + (top - low) * b // (B - 1) for b in range(B)]


def _lens(case, seed):
    lens = _spread(case)
    random.Random(seed).shuffle(lens)
    return lens


def _tree_rows(B, T, seed):
    """[B, T] int64 ancestor rows of random drafted trees: token i's parent is
    one of the last few tokens before it (or the last committed token), and
    its row marks itself and its ancestors."""
    rng = random.Random(seed ^ 0x7EE)
    rows = np.zeros((B, T), dtype=np.uint64)
    for b in range(B):
        for i in range(T):
            parent = rng.randint(max(-1, i - 6), i - 1) if i else -1
            up = int(rows[b, parent]) if parent >= 0 else 0
            rows[b, i] = up | (1 << i)
    return torch.from_numpy(rows.view(np.int64))


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    B, H, Hk, Nq, Nk, d = (case[x] for x in ("B", "H", "Hk", "Nq", "Nk", "d"))
    lens = _lens(case, seed)
    s = dict(case)
    s["q"] = normal(B, H, Nq, d)
    s["k"] = normal(B, Hk, Nk, d)
    s["v"] = normal(B, Hk, Nk, d)
    s["lens"] = lens
    # a program whose batches are all full passes no counts
    s["seqlens"] = (None if case["lens"] == "full" else
                    torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["op"] == "train":
        s["dout"] = normal(B, H, Nq, d)
    if case["op"] in ("token", "tree"):   # a decoding loop keeps its buffers
        s["out"] = torch.empty(B, H, Nq, d, dtype=dt, device="cuda")
        s["lse"] = torch.empty(B, H, Nq, dtype=torch.float32, device="cuda")
        s["workspace"] = None
    if case["op"] == "tree":
        s["tree"] = _tree_rows(B, Nq, seed).cuda()
        if s["seqlens"] is None:
            s["seqlens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    if state["op"] in ("prompt", "train"):
        return _plain_window(state)
    return _plain_decode(state)


def _run_own(s):
    import exact_tiled_attention_14_gb300 as fa
    if s["op"] in ("prompt", "train"):
        o, lse = fa.attention_forward_window(s["q"], s["k"], s["v"], s["window"], s["sinks"],
                                             causal=s["align"], seqlens_k=s["seqlens"])
        if s["op"] == "prompt":
            return o, lse
        dq, dk, dv = fa.attention_backward_window(s["q"], s["k"], s["v"], o, lse, s["dout"],
                                                  s["window"], s["sinks"], causal=s["align"],
                                                  seqlens_k=s["seqlens"])
        return o, lse, dq, dk, dv
    if s["workspace"] is None:
        s["workspace"] = fa.make_decode_workspace(s["q"], s["k"])
    if s["op"] == "token":
        return fa.attention_decode_window(s["q"], s["k"], s["v"], s["window"], s["sinks"],
                                          seqlens_k=s["seqlens"], out=s["out"], lse=s["lse"],
                                          workspace=s["workspace"])
    return fa.attention_decode_tree(s["q"], s["k"], s["v"], s["tree"], seqlens_k=s["seqlens"],
                                    window=s["window"] or None, sinks=s["sinks"], out=s["out"],
                                    lse=s["lse"], workspace=s["workspace"])


# ---------------------------------------------------------------- plain forms

def _softmax_rows(sc, vis):
    """exp(sc - LSE) on the visible entries, and LSE; rows that see nothing get
    zeros and -inf."""
    sc = torch.where(vis, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(sc - m)
    l = e.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    return e / torch.where(l > 0, l, 1.0), lse.squeeze(-1)


def _plain_window(s):
    """Blocks of query rows against the sinks and the block's span of keys,
    all query heads of a K/V head together."""
    B, H, Hk, Nq, Nk, d, W, S = (s[x] for x in ("B", "H", "Hk", "Nq", "Nk", "d", "window",
                                                "sinks"))
    G, dev, dt = H // Hk, s["q"].device, s["q"].dtype
    scale = 1.0 / math.sqrt(d)
    train = s["op"] == "train"
    o = torch.zeros(B, H, Nq, d, dtype=dt, device=dev)
    lse = torch.full((B, H, Nq), -math.inf, device=dev)
    if train:
        dq = torch.zeros(B, H, Nq, d, dtype=dt, device=dev)
        dk, dv = (torch.zeros(B, Hk, Nk, d, device=dev) for _ in range(2))
    step = 512
    for b in range(B):
        n = s["lens"][b]
        off = n - Nq if s["align"] == "bottom_right" else 0
        for r0 in range(0, Nq, step):
            r1 = min(r0 + step, Nq)
            lo, hi = max(r0 + off - W + 1, 0), min(r1 + off, n)
            ns = max(min(S, lo, hi), 0)
            if hi <= lo and ns == 0:
                continue
            lo = min(lo, max(hi, 0))
            kk = torch.cat((s["k"][b, :, :ns], s["k"][b, :, lo:hi]), 1).float()
            vv = torch.cat((s["v"][b, :, :ns], s["v"][b, :, lo:hi]), 1).float()
            key = torch.cat((torch.arange(ns, device=dev), torch.arange(lo, hi, device=dev)))
            pos = torch.arange(r0 + off, r1 + off, device=dev)[:, None]
            vis = (key <= pos) & ((key > pos - W) | (key < S))
            vis = vis.repeat(G, 1)
            qq = s["q"][b, :, r0:r1].float().reshape(Hk, G * (r1 - r0), d)
            p, l = _softmax_rows(qq @ kk.transpose(1, 2) * scale, vis)
            ob = p @ vv
            o[b, :, r0:r1] = ob.reshape(H, r1 - r0, d).to(dt)
            lse[b, :, r0:r1] = l.reshape(H, r1 - r0)
            if train:
                do = s["dout"][b, :, r0:r1].float().reshape(Hk, G * (r1 - r0), d)
                ds = p * (do @ vv.transpose(1, 2) - (do * ob).sum(-1, keepdim=True))
                dq[b, :, r0:r1] = (ds @ kk * scale).reshape(H, r1 - r0, d).to(dt)
                gk, gv = ds.transpose(1, 2) @ qq * scale, p.transpose(1, 2) @ do
                for acc, grad in ((dk, gk), (dv, gv)):
                    acc[b, :, :ns] += grad[:, :ns]
                    acc[b, :, lo:hi] += grad[:, ns:]
    if train:
        return o, lse, dq, dk.to(dt), dv.to(dt)
    return o, lse


def _plain_decode(s):
    """Batch by batch: the new tokens' rows of all query heads of a K/V head
    against the sinks and the span of the cache that they see."""
    B, H, Hk, Nq, d, W, S = (s[x] for x in ("B", "H", "Hk", "Nq", "d", "window", "sinks"))
    G, dev, dt = H // Hk, s["q"].device, s["q"].dtype
    scale = 1.0 / math.sqrt(d)
    o = torch.zeros(B, H, Nq, d, dtype=dt, device=dev)
    lse = torch.full((B, H, Nq), -math.inf, device=dev)
    slot = torch.arange(Nq, device=dev)
    for b in range(B):
        n = s["lens"][b]
        if s["op"] == "tree":
            bits = ((s["tree"][b][:, None] >> slot) & 1).bool()      # [row, drafted token]
            first, hi = n, n + Nq
            pos = n + bits.sum(1) - 1
        else:
            first, hi = n, n
            pos = n - Nq + slot
        lo = max(0, n - (0 if s["op"] == "tree" else Nq) - W) if W else 0
        ns = min(S, lo)
        key = torch.cat((torch.arange(ns, device=dev), torch.arange(lo, hi, device=dev)))
        kpos = key
        vis = key <= pos[:, None]
        if s["op"] == "tree":
            draft = key >= first
            slot_of = (key - first).clamp(min=0)
            kpos = torch.where(draft, pos[slot_of], key)
            vis = torch.where(draft, bits[:, slot_of], key < first)
        if W:
            vis = vis & ((kpos > pos[:, None] - W) | (kpos < S))
        kk = torch.cat((s["k"][b, :, :ns], s["k"][b, :, lo:hi]), 1).float()
        vv = torch.cat((s["v"][b, :, :ns], s["v"][b, :, lo:hi]), 1).float()
        qq = s["q"][b].float().reshape(Hk, G * Nq, d)
        p, l = _softmax_rows(qq @ kk.transpose(1, 2) * scale, vis.repeat(G, 1))
        o[b] = (p @ vv).reshape(H, Nq, d).to(dt)
        lse[b] = l.reshape(H, Nq)
    return o, lse


# ---------------------------------------------------------------- exact results

def exact(case, seed):
    """The definition in float64: for every batch and block of rows the full
    truth table of visible keys, the softmax over it, and for training the
    gradients that torch derives from that expression."""
    s = prepare(case, seed)
    B, H, Hk, Nq, Nk, d = (case[x] for x in ("B", "H", "Hk", "Nq", "Nk", "d"))
    W, S, op = case["window"], case["sinks"], case["op"]
    G, dev = H // Hk, s["q"].device
    train = op == "train"
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device=dev)
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device=dev)
    grads = [torch.zeros(t.shape, dtype=torch.float64, device=dev)
             for t in ((s["q"], s["k"], s["v"]) if train else ())]
    j = torch.arange(Nk, device=dev)
    for b in range(B):
        n = s["lens"][b]
        rows = torch.arange(Nq, device=dev)
        if op == "tree":
            m = s["tree"][b]
            pos = torch.full_like(rows, n - 1)
            for t in range(Nq):
                pos += (m >> t) & 1
        else:
            pos = rows + (0 if case.get("align") == "upper_left" else n - Nq)
        block = 256
        for r0 in range(0, Nq, block):
            r = rows[r0:r0 + block]
            pr = pos[r0:r0 + block].view(-1, 1)
            if op == "tree":
                see = (j < n).expand(len(r), Nk).clone()
                jpos = j.clone()
                for t in range(Nq):
                    see[:, n + t] = ((m[r0:r0 + block] >> t) & 1) == 1
                    jpos[n + t] = pos[t]
                if W:
                    see &= (pr - jpos < W) | (jpos < S)
            else:
                see = (j <= pr) & (j < n) & ((pr - j < W) | (j < S))
            used = see.any(0).nonzero().view(-1)
            live = see.any(1)
            if used.numel() == 0:
                continue
            see = see[:, used]
            for h0 in range(0, Hk, 4):       # a few K/V heads at a time
                hk = slice(h0, min(h0 + 4, Hk))
                hq = slice(h0 * G, min(h0 + 4, Hk) * G)
                leaf = [t.double().requires_grad_(train)
                        for t in (s["q"][b, hq, r0:r0 + block], s["k"][b, hk][:, used],
                                  s["v"][b, hk][:, used])]
                q, k, v = leaf[0], *(t.repeat_interleave(G, 0) for t in leaf[1:])
                with torch.set_grad_enabled(train):
                    z = torch.einsum("hrd,hjd->hrj", q, k) / math.sqrt(d)
                    z = z.masked_fill(~see, -math.inf)[:, live]
                    lz = torch.logsumexp(z, -1)
                    out = torch.einsum("hrj,hjd->hrd", torch.exp(z - lz[..., None]), v)
                hidx = torch.arange(H, device=dev)[hq].view(-1, 1)
                o[b][hidx, r[live]] = out.detach()
                lse[b][hidx, r[live]] = lz.detach()
                if train:
                    do = s["dout"][b, hq, r0:r0 + block].double()[:, live]
                    gq, gk, gv = torch.autograd.grad(out, leaf, do)
                    grads[0][b, hq, r0:r0 + block] = gq
                    grads[1][b, hk] = grads[1][b, hk].index_add(1, used, gk)
                    grads[2][b, hk] = grads[2][b, hk].index_add(1, used, gv)
    return (o, lse, *grads)


# ---------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass: every visible key and value once per
    K/V head, every (row, visible key) pair's products (a training step forms
    S twice, and O, dP, dV, dQ, dK once each)."""
    B, H, Hk, Nq, d = (case[x] for x in ("B", "H", "Hk", "Nq", "d"))
    op, S = case["op"], case["sinks"]
    pairs = keys = 0
    for n in _spread(case):
        if op == "tree":
            W = case["window"] or n + Nq
            span = min(n, W + min(S, max(n - W, 0)))
            keys += span + Nq
            pairs += Nq * (span + 1)           # the history and the token itself
            continue
        W = case["window"]
        pos = np.arange(Nq, dtype=np.int64) + (0 if case.get("align") == "upper_left" else n - Nq)
        hi = np.clip(pos + 1, 0, n)
        first = np.minimum(hi, S)
        lo = np.maximum(np.maximum(pos - W + 1, 0), first)
        pairs += int((first + np.maximum(hi - lo, 0)).sum())
        keys += int(max(first.max(), 0) + max(hi.max() - max(lo.min(), first.max()), 0))
    rows = B * H * Nq
    nbytes = 2 * rows * d * 2 + rows * 4 + 2 * keys * Hk * d * 2
    flops = 4 * d * pairs * H
    if op == "train":
        nbytes += 2 * rows * d * 2 + 2 * B * Hk * case["Nk"] * d * 2
        flops += 10 * d * pairs * H
    return {"bytes": nbytes, "flops": flops}
