"""Cases, plain forms and exact results of the rotary-position and paged-cache
operators: what stands between a model's projections and its attention, and
the attention of new tokens over a cache held in 8 bits.

A cache is a pool of pages, ``[pages, Hk, page_size, d]`` in 8 bits (float8
e4m3, or int8) with one float32 scale for each page and K/V head; a page table
names the pages of each sequence in order.

``rotary``   ``rotary_forward`` (and, for training, ``rotary_backward``): the
             rotation of q and k by their positions, on strided views of a
             fused projection's output.
``append``   ``cache_append``: the last tokens of each sequence, keys rotated
             on the way, quantised into their pages.  A page's scale is that
             of its largest element; when a new token raises it, the tokens
             that the page holds are quantised again.
``read``     ``cache_read``: the cache's tokens as 16-bit keys and values, for
             a prompt chunk's attention; with ``T`` new tokens appended first.
``attend``   ``attention_decode_paged``: up to 16 new tokens of each sequence
             over its pages, under a window with sinks or over everything.

``run`` takes one pass through an operator: in its plain form (elementary
torch operations in float32) or, where ``own`` is true, through the package.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}
LOWEST = 2.0 ** -100            # smallest scale of a page


# ---------------------------------------------------------------- cases

def listed():
    """The listed cases.  ``lens`` is "full" (every sequence has the cache's
    capacity) or "ragged" (from a quarter of it up, dealt by the seed).
    ``scaling`` is that of the rotation's frequencies for long contexts."""
    return [
        # one decoding step of 32 users, positions behind each user's history
        dict(name="rotary_token", op="rotary", train=False, B=32, H=32, Hk=8, N=1, d=128, rot=128,
             interleaved=False, scaling="none", at="seqlens", far=16384, dtype="bf16"),
        # a padded batch of a small model: part of the head, interleaved pairs
        dict(name="rotary_part", op="rotary", train=True, B=3, H=6, Hk=6, N=333, d=64, rot=32,
             interleaved=True, scaling="linear", at="positions", far=100000, dtype="fp16"),
        # long-context training, one layer: q and k there, their gradients back
        dict(name="rotary_train", op="rotary", train=True, B=1, H=32, Hk=8, N=16384, d=128, rot=128,
             interleaved=False, scaling="parts", at="start", far=16384, dtype="bf16"),
        # one new token of 64 users
        dict(name="append_token", op="append", B=64, Hk=8, T=1, hist=8192, page=64, d=128, rot=128,
             interleaved=False, scaling="none", lens="ragged", code="e4m3", dtype="bf16"),
        # prompts of different lengths, padded to the longest
        dict(name="append_prompt", op="append", B=4, Hk=8, T=8192, hist=0, page=64, d=128, rot=128,
             interleaved=False, scaling="none", lens="ragged", code="e4m3", dtype="bf16"),
        # a short chunk into half-full pages of another size, then all of it back
        dict(name="read_chunk", op="read", B=2, Hk=3, T=77, hist=1000, page=48, d=64, rot=48,
             interleaved=True, scaling="none", lens="ragged", code="int8", dtype="fp16"),
        # four users' caches before a chunk's attention
        dict(name="read_long", op="read", B=4, Hk=8, T=0, hist=16384, page=64, d=128, rot=0,
             interleaved=False, scaling="none", lens="ragged", code="e4m3", dtype="bf16"),
        # one user's next token: latency
        dict(name="attend_single", op="attend", B=1, H=32, Hk=8, Nq=1, Nk=8192, page=64, d=128,
             window=0, sinks=0, lens="full", code="e4m3", dtype="bf16"),
        # several tokens a user under a window, small pages, no shared heads
        dict(name="attend_few", op="attend", B=16, H=16, Hk=16, Nq=4, Nk=10007, page=16, d=64,
             window=2000, sinks=5, lens="ragged", code="int8", dtype="fp16"),
        # a serving batch of 64 users at mixed lengths
        dict(name="attend_batch", op="attend", B=64, H=32, Hk=8, Nq=1, Nk=16384, page=64, d=128,
             window=0, sinks=0, lens="ragged", code="e4m3", dtype="bf16"),
        # two-token steps over long caches in int8
        dict(name="attend_long", op="attend", B=8, H=32, Hk=8, Nq=2, Nk=131072, page=128, d=128,
             window=0, sinks=0, lens="full", code="int8", dtype="bf16"),
        # many rows a K/V head: eight tokens of eight query heads each
        dict(name="attend_rows", op="attend", B=8, H=32, Hk=4, Nq=8, Nk=32768, page=32, d=128,
             window=0, sinks=0, lens="ragged", code="e4m3", dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """Rough seconds of a pass at one card's rates (compares cases only)."""
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.0e15)


def draw(rng):
    """One more case of the listed ranges."""
    ops = ("rotary", "append", "read", "attend")
    limit = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ops}
    while True:
        op = rng.choice(ops)
        Hk, d = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((64, 128))
        G = rng.choice((1, 1, 2, 3, 4, 6, 8))
        c = dict(op=op, Hk=Hk, d=d, dtype=rng.choice(("bf16", "fp16")))
        if op in ("rotary", "attend"):
            c["H"] = Hk * G
            if c["H"] > 64:
                continue
        if op != "attend":
            c.update(rot=rng.choice((16, 32, 48, d // 2, d, d)), interleaved=rng.random() < 0.5,
                     scaling=rng.choice(("none", "none", "linear", "base", "parts")))
        if op != "rotary":
            c.update(page=rng.choice((16, 32, 48, 64, 80, 128)), lens=rng.choice(("full", "ragged")),
                     code=rng.choice(("e4m3", "int8")))
        if op == "rotary":
            c.update(train=rng.random() < 0.5, B=_log_int(rng, 1, 64), N=_log_int(rng, 1, 16384),
                     at=rng.choice(("start", "seqlens", "positions")), far=_log_int(rng, 64, 1 << 20))
            c["far"] = max(c["far"], c["N"])
        elif op == "append":
            c.update(B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 8192), code="e4m3",
                     hist=rng.choice((0, _log_int(rng, 16, 16384))))
        elif op == "read":
            c.update(B=_log_int(rng, 1, 16), T=rng.choice((0, _log_int(rng, 1, 2048))),
                     hist=_log_int(rng, 16, 16384))
        else:
            c.update(B=_log_int(rng, 1, 64), Nq=rng.choice((1, 1, 1, 2, 3, 4, 5, 8, 16)),
                     Nk=_log_int(rng, 64, 131072), sinks=0, window=0)
            if rng.random() < 0.5:
                c.update(window=_log_int(rng, 16, 16384), sinks=rng.choice((0, 1, 4, 5, 64, 130)))
        if op != "rotary":
            tokens = c["Nk"] if op == "attend" else c["hist"] + c["T"]
            if c["B"] * Hk * tokens * d * 2 > (3 << 30):
                continue
        if _cost(c) <= limit[op]:
            return c


# ---------------------------------------------------------------- inputs

def _spread(case, top, low=None):
    """Lengths of the sequences up to ``top``, in an order that the seed deals."""
    B = case["B"]
    if case.get("lens", "full") == "full":
        return [top] * B
    low = max(top // 4, 0) if low is None else min(low, top)
    if B == 1:
        return [(low + top) // 2]
    return [low + (top - low) * b // (B - 1) for b in range(B)]


def _lengths(case, seed=None):
    """(history, new tokens) of the sequences of a cache's case."""
    if case["op"] == "attend":
        low = min(max(case["Nk"] // 4, case["Nq"]), case["Nk"])
        hist, new = _spread(case, case["Nk"], low), [0] * case["B"]
    else:
        hist = _spread(case, case["hist"])
        new = _spread(case, case["T"], (case["T"] + 3) // 4)[::-1]
    if seed is not None:
        order = list(range(case["B"]))
        random.Random(seed).shuffle(order)
        hist, new = [hist[i] for i in order], [new[i] for i in order]
    return hist, new


SCALING = {   # arguments of the frequencies: factor and the length the model was trained at
    "none": dict(), "linear": dict(factor=4.0), "base": dict(factor=8.0),
    "parts": dict(factor=16.0, original_length=4096)}


def _frequencies(case):
    """Angle per position of each pair in float64: base^(-2 j / rot), for long
    contexts divided by the factor, of a raised base, or (in parts) divided
    where a pair turns less than once over the original length, left alone
    where it turns more than 32 times, and between the two in between."""
    rot, how = case["rot"], case["scaling"]
    j = torch.arange(rot // 2, dtype=torch.float64)
    base, f = 10000.0, SCALING[how].get("factor", 1.0)
    if how == "base":
        base *= f ** (rot / max(rot - 2, 1))
    inv = base ** (-2.0 * j / max(rot, 1))
    if how == "linear":
        inv = inv / f
    if how == "parts":
        turns = SCALING[how]["original_length"] * inv / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        inv = inv * keep + inv / f * (1.0 - keep)
    return inv


def _mscale(case):
    return 0.1 * math.log(SCALING[case["scaling"]]["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def prepare(case, seed):
    dt, dev = DTYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt)

    s = dict(case)
    B, Hk, d, op = case["B"], case["Hk"], case["d"], case["op"]
    if op != "attend":
        s["inv"] = _frequencies(case).to(dev)
        s["mscale"] = _mscale(case)
    if op == "rotary":
        H, N = case["H"], case["N"]
        # the projections' output as a program has it: one row of all heads a token
        qkv = normal(B, N, H + 2 * Hk, d)
        s["q"], s["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
        s["seqlens"] = s["positions"] = None
        if case["at"] == "seqlens":
            s["seqlens"] = torch.randint(N, case["far"] + 1, (B,), generator=g, device=dev,
                                         dtype=torch.int32)
        if case["at"] == "positions":
            s["positions"] = torch.randint(0, case["far"], (B, N), generator=g, device=dev,
                                           dtype=torch.int32)
        if case["train"]:
            s["dq"], s["dk"] = normal(B, H, N, d), normal(B, Hk, N, d)
        return s
    # a pool with a few pages to spare, dealt to the sequences in random order
    page, code = case["page"], case["code"]
    hist, new = _lengths(case, seed)
    lens = [a + b for a, b in zip(hist, new)]
    per = max(-(-max(lens) // page), 1)
    pages = B * per + 3
    s["page_table"] = torch.randperm(pages, generator=g, device=dev)[:B * per].view(B, per).int()
    s["seqlens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["counts"] = torch.tensor(new, dtype=torch.int32, device=dev)
    for x in ("k", "v"):
        held = normal(pages, Hk, page, d)
        held.mul_(100.0 if code == "e4m3" else 32.0).clamp_(-TOP[code], TOP[code])
        if code == "int8":
            held.round_()
        s[x + "_cache"] = held.to(CODES[code])
        del held
        r = torch.rand(pages, Hk, generator=g, device=dev)
        # values of about one standard deviation a page
        s[x + "_scale"] = (torch.exp2(torch.floor(r * 3.0) - 8.0) if code == "e4m3"
                           else 0.02 + 0.02 * r)
    if op == "attend":
        H, Nq = case["H"], case["Nq"]
        s["q"] = normal(B, H, Nq, d)
        s["out"] = torch.empty(B, H, Nq, d, dtype=dt, device=dev)     # a decoding loop keeps its
        s["lse"] = torch.empty(B, H, Nq, dtype=torch.float32, device=dev)   # buffers
        s["workspace"] = None
    elif case["T"]:
        kv = normal(B, case["T"], 2 * Hk, d)
        s["k"], s["v"] = kv[:, :, :Hk].transpose(1, 2), kv[:, :, Hk:].transpose(1, 2)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "rotary":
        return _plain_rotary(state)
    if state["op"] == "attend":
        return _plain_attend(state)
    if state["op"] == "append":
        return _plain_append(state)
    if state["T"]:
        return (*_plain_read({**state, **dict(zip(HELD, _plain_append(state)))}),
                state["k_scale"], state["v_scale"])
    return _plain_read(state)


HELD = ("k_cache", "v_cache", "k_scale", "v_scale")


def _run_own(s):
    import exact_tiled_attention_14_gb300 as fa
    op = s["op"]
    if op != "attend" and s["rot"] and "freqs" not in s:      # laid out once, as weights are
        s["freqs"] = fa.rotary_frequencies(s["rot"], scaling=None if s["scaling"] == "none" else
                                           s["scaling"], device="cuda", **SCALING[s["scaling"]])
    if op == "rotary":
        turn = dict(positions=s["positions"], seqlens=s["seqlens"], mscale=s["mscale"],
                    interleaved=s["interleaved"])
        out = fa.rotary_forward(s["q"], s["k"], s["freqs"], **turn)
        if s["train"]:
            out += fa.rotary_backward(s["dq"], s["dk"], s["freqs"], **turn)
        return out
    cache = fa.PagedCache(*(s[x] for x in HELD))
    if op == "attend":
        if s["workspace"] is None:
            s["workspace"] = fa.make_paged_workspace(s["q"], cache, s["page_table"])
        return fa.attention_decode_paged(s["q"], cache, s["page_table"], s["seqlens"],
                                         window=s["window"] or None, sinks=s["sinks"],
                                         out=s["out"], lse=s["lse"], workspace=s["workspace"])
    if s["T"]:
        fa.cache_append(s["k"], s["v"], cache, s["page_table"], s["seqlens"], counts=s["counts"],
                        freqs=s["freqs"], mscale=s["mscale"], interleaved=s["interleaved"])
    if op == "append":
        return tuple(cache)
    k, v = fa.cache_read(cache, s["page_table"], s["seqlens"], dtype=DTYPES[s["dtype"]])
    return (k, v, cache.k_scale, cache.v_scale) if s["T"] else (k, v)


# ---------------------------------------------------------------- plain forms

def _cos_sin(s, pos):
    """cos and sin [..., 1, n, rot / 2] in float32 of angles in float64 (a far
    position's angle needs more than 32 bits)."""
    angle = pos.double()[:, None, :, None] * s["inv"]
    return (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()


def _turn(x, cos, sin, rot, interleaved):
    """The rotation of x [..., d] in float32; elements from rot on stay."""
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rotary(s):
    B, N, dt, dev = s["B"], s["N"], DTYPES[s["dtype"]], s["q"].device
    at = torch.arange(N, device=dev).expand(B, N)
    if s["seqlens"] is not None:
        at = at + (s["seqlens"].long()[:, None] - N)
    if s["positions"] is not None:
        at = s["positions"]
    cos, sin = _cos_sin(s, at)
    turn = (s["rot"], s["interleaved"])
    out = tuple(_turn(x, cos, sin, *turn).to(dt) for x in (s["q"], s["k"]))
    if s["train"]:     # the transposed rotation
        out += tuple(_turn(x, cos, -sin, *turn).to(dt) for x in (s["dq"], s["dk"]))
    return out


def _scale_of(top, code):
    """A page's scale by its largest magnitude: for e4m3 the smallest power of
    two under which it fits, for int8 the 127th part of it; not finite: NaN."""
    if code == "e4m3":
        m, e = torch.frexp(top)
        scale = torch.ldexp(torch.ones_like(top), e - torch.where(m <= 0.875, 9, 8))
    else:
        scale = top / 127.0
    scale = scale.clamp(min=LOWEST)
    return torch.where(torch.isfinite(top), scale, math.nan)


def _codes_of(x, code):
    if code == "e4m3":
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _plain_append(s):
    """All pages that the new tokens touch at once: [B, Hk, J, page, d]."""
    B, Hk, T, page, d, code = (s[x] for x in ("B", "Hk", "T", "page", "d", "code"))
    dev, table = s["k"].device, s["page_table"].long()
    start = (s["seqlens"] - s["counts"]).long()                      # slot of the first new token
    pos = start[:, None] + torch.arange(T, device=dev)
    cos, sin = _cos_sin(s, pos)
    J = (T - 1) // page + 2
    nth = start[:, None] // page + torch.arange(J, device=dev)       # [B, J] pages by number
    slot = nth[..., None] * page + torch.arange(page, device=dev)    # [B, J, page]
    i = slot - start[:, None, None]
    fresh = ((i >= 0) & (i < s["counts"].long()[:, None, None]))[:, None, ..., None]
    old = (i < 0)[:, None, ..., None]
    touched = (nth * page < s["seqlens"].long()[:, None]) & (s["counts"][:, None] > 0)
    # untouched pages stand in as the first one again, with the same contents
    use = torch.where(touched, torch.arange(J, device=dev), 0)
    ids = table.gather(1, nth.gather(1, use).clamp(max=table.shape[1] - 1))   # [B, J]
    pick = i.clamp(0, T - 1).view(B, 1, J * page, 1).expand(B, Hk, J * page, d)
    for x in ("k", "v"):
        val = s[x].float()
        if x == "k" and s["rot"]:
            val = _turn(s["k"], cos, sin, s["rot"], s["interleaved"])
        val = val.gather(2, pick).view(B, Hk, J, page, d)
        top = torch.where(fresh, val, 0.0).abs().amax((3, 4))        # [B, Hk, J]
        raw = s[x + "_cache"].view(torch.uint8)
        held = raw[ids].transpose(1, 2)                              # [B, Hk, J, page, d]
        before = s[x + "_scale"][ids].transpose(1, 2)
        need = _scale_of(top, code)
        partly = old.any(3).squeeze(-1)
        scale = torch.where(partly, torch.maximum(before, need), need)
        inverse = 1.0 / scale
        again = held.view(CODES[code]).float() * (before * inverse)[..., None, None]
        again = torch.where((scale == before)[..., None, None], held, _codes_of(again, code))
        codes = _codes_of(val * inverse[..., None, None], code)
        codes = torch.where(fresh, codes, torch.where(old, again, held))
        scale = torch.where(touched[:, None], scale, before)
        codes = torch.where(touched[:, None, :, None, None], codes, held)
        first = use[:, None].expand(B, Hk, J)
        scale = scale.gather(2, first)
        codes = codes.gather(2, first[..., None, None].expand(codes.shape))
        raw[ids] = codes.transpose(1, 2)
        s[x + "_scale"][ids] = scale.transpose(1, 2)
    return tuple(s[x] for x in HELD)


def _gathered(s, x):
    """The pages of every sequence in order, as float32 [B, Hk, capacity, d]."""
    ids = s["page_table"].long()
    val = s[x + "_cache"].view(torch.uint8)[ids].view(CODES[s["code"]]).float()
    val = val * s[x + "_scale"][ids][..., None, None]                # [B, per, Hk, page, d]
    return val.transpose(1, 2).reshape(s["B"], s["Hk"], -1, s["d"])


def _plain_read(s):
    out = []
    for x in ("k", "v"):
        val = _gathered(s, x)
        seen = torch.arange(val.shape[2], device=val.device) < s["seqlens"][:, None]
        out.append(torch.where(seen[:, None, :, None], val, 0.0).to(DTYPES[s["dtype"]]))
    return tuple(out)


def _plain_attend(s):
    """All sequences at once over their whole capacity, masked."""
    B, H, Hk, Nq, d, W, S = (s[x] for x in ("B", "H", "Hk", "Nq", "d", "window", "sinks"))
    G, dev = H // Hk, s["q"].device
    k, v = _gathered(s, "k"), _gathered(s, "v")
    n = s["seqlens"].long()[:, None, None]
    key = torch.arange(k.shape[2], device=dev)
    pos = n - Nq + torch.arange(Nq, device=dev)[:, None]             # [B, Nq, 1]
    vis = (key <= pos) & (key < n)
    if W:
        vis = vis & ((key > pos - W) | (key < S))
    vis = vis[:, None].expand(B, G, Nq, -1).reshape(B, 1, G * Nq, -1)
    q = s["q"].float().reshape(B, Hk, G * Nq, d)
    sc = torch.where(vis, q @ k.transpose(2, 3) / math.sqrt(d), -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    e = torch.exp(sc - m)
    l = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(l > 0, l, 1.0)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    return o.reshape(B, H, Nq, d).to(DTYPES[s["dtype"]]), lse.reshape(B, H, Nq)


# ---------------------------------------------------------------- exact results

def exact(case, seed):
    """The definitions in float64, sequence by sequence and page by page."""
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    hist, new = _lengths(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s, hist)
    held = [s[x].double() for x in HELD]
    if case["T"]:
        _exact_append(s, held, hist, new)
    if case["op"] == "append":
        return tuple(held)
    out = []
    for x in (0, 1):
        cap = s["page_table"].shape[1] * case["page"]
        full = torch.zeros(case["B"], case["Hk"], cap, case["d"], dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            n = hist[b] + new[b]
            full[b, :, :n] = _sequence(s, held[x], held[2 + x], b, n)
        out.append(full)
    return (*out, held[2], held[3]) if case["T"] else tuple(out)


def _sequence(s, codes, scales, b, n):
    """The first n tokens of sequence b as values [Hk, n, d]."""
    ids = s["page_table"][b, :-(-n // s["page"])].long()
    if not len(ids):
        return codes.new_zeros(s["Hk"], 0, s["d"])
    pages = [codes[p].double() * scales[p].double()[:, None, None] for p in ids.tolist()]
    return torch.cat(pages, 1)[:, :n]


def _spun(s, x, pos, sign=1.0):
    """x [..., n, d] with its pairs, as complex numbers, times mscale e^(i angle)."""
    rot, y = s["rot"], x.double().clone()
    if not rot:
        return y
    if s["interleaved"]:
        z = torch.complex(y[..., 0:rot:2].contiguous(), y[..., 1:rot:2].contiguous())
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous())
    angle = sign * torch.outer(pos.double(), s["inv"])
    z = z * torch.polar(torch.full_like(angle, s["mscale"]), angle)
    if s["interleaved"]:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_rotary(s):
    names = ("q", "k", "dq", "dk") if s["train"] else ("q", "k")
    out = []
    for name in names:
        rows = []
        for b in range(s["B"]):
            pos = torch.arange(s["N"], device="cuda")
            if s["at"] == "seqlens":
                pos = pos + int(s["seqlens"][b]) - s["N"]
            if s["at"] == "positions":
                pos = s["positions"][b]
            rows.append(_spun(s, s[name][b], pos, -1.0 if name[0] == "d" else 1.0))
        out.append(torch.stack(rows))
    return tuple(out)


def _rounded(x, code):
    """The nearest code's value, ties to even."""
    if code == "int8":
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x)                              # x = m 2^e with m in [1/2, 1)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_append(s, held, hist, new):
    page, code = s["page"], s["code"]
    for b in range(s["B"]):
        c, h = new[b], hist[b]
        if c == 0:
            continue
        pos = torch.arange(h, h + c, device="cuda")
        for x, val in enumerate((_spun(s, s["k"][b, :, :c], pos), s["v"][b, :, :c].double())):
            codes, scales = held[x], held[2 + x]
            for n in range(h // page, (h + c - 1) // page + 1):
                p = int(s["page_table"][b, n])
                lo, hi = max(h, n * page), min(h + c, (n + 1) * page)     # new slots of the page
                part = val[:, lo - h:hi - h]
                top = part.abs().amax((1, 2))
                if code == "e4m3":
                    fit = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
                    fit = torch.where(top <= 448.0 * fit / 2, fit / 2, fit)
                else:
                    fit = (top / 127.0).float().double()                  # kept in 32 bits
                fit = fit.clamp(min=LOWEST)
                k = lo - n * page                                         # tokens already there
                if k:
                    fit = torch.maximum(fit, scales[p])
                    again = _rounded(codes[p, :, :k] * (scales[p] / fit)[:, None, None], code)
                    codes[p, :, :k] = torch.where((fit == scales[p])[:, None, None],
                                                  codes[p, :, :k], again)
                scales[p] = fit
                codes[p, :, k:hi - n * page] = _rounded(part / fit[:, None, None], code)


def _exact_attend(s, lens):
    B, H, Hk, Nq, d, W, S = (s[x] for x in ("B", "H", "Hk", "Nq", "d", "window", "sinks"))
    G = H // Hk
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        k = _sequence(s, s["k_cache"], s["k_scale"], b, n)
        v = _sequence(s, s["v_cache"], s["v_scale"], b, n)
        j = torch.arange(n, device="cuda")
        for t in range(Nq):
            p = n - Nq + t
            if p < 0:
                continue
            see = (j <= p) & ((p - j < W) | (j < S) if W else (j >= 0))
            q = s["q"][b, :, t].double().view(Hk, G, d)
            z = torch.einsum("hgd,hjd->hgj", q, k[:, see]) / math.sqrt(d)
            lz = torch.logsumexp(z, -1)
            lse[b, :, t] = lz.reshape(H)
            o[b, :, t] = torch.einsum("hgj,hjd->hgd", torch.exp(z - lz[..., None]),
                                      v[:, see]).reshape(H, d)
    return o, lse


# ---------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass: every tensor element that the
    operator has to read or write once (8-bit keys and values of the tokens
    that some new token sees; the frequencies and lengths are left out)."""
    B, Hk, d, op = (case[x] for x in ("B", "Hk", "d", "op"))
    if op == "rotary":
        n = B * (case["H"] + Hk) * case["N"] * d * (2 if case["train"] else 1)
        return {"bytes": 4 * n, "flops": 3 * n}
    hist, new = _lengths(case)
    page = case["page"]
    if op in ("append", "read"):
        n, pages = sum(new), sum(-(-(h + c) // page) - h // page for h, c in zip(hist, new) if c)
        nbytes = 2 * (n * Hk * d * 3 + pages * Hk * 4)
        flops = 5 * n * Hk * d
        if op == "read":
            held = sum(hist) + n
            per = max(-(-max(h + c for h, c in zip(hist, new)) // page), 1)
            nbytes += 2 * Hk * (held * d + B * per * page * d * 2)
            flops += 2 * held * Hk * d
        return {"bytes": nbytes, "flops": flops}
    H, Nq, W, S = case["H"], case["Nq"], case["window"], case["sinks"]
    keys = pairs = scales = 0
    for n in hist:
        lo = max(n - Nq - W + 1, 0) if W else 0
        first = min(S, lo)
        keys += n - lo + first
        scales += -(-n // page) - lo // page + -(-first // page)
        for t in range(Nq):
            p = n - Nq + t
            low = max(p - W + 1, 0) if W else 0
            pairs += max(p + 1 - low, 0) + min(S, low)
    rows = B * H * Nq
    return {"bytes": 2 * keys * Hk * d + 8 * scales * Hk + rows * (4 * d + 4),
            "flops": 4 * d * pairs * H}
