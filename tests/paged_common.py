"""Plain float64 forms of rotary positions and of a paged 8-bit cache, written
from their definitions, and error bounds of the kernels' results.

u(t) = eps / 2 is half a step of a 16-bit type, E = 2^-24 half a step of float32.

Rotation.  cos and sin come from an angle cut to at most an eighth of a turn;
its float32 rounding is off by at most pi / 4 * E, sincospif by 2 steps of
values up to 1 (4 E), the product with mscale by E: under 2^-21 in all, relative
to mscale.  A result adds a product's and a sum's rounding, 2 E (|a| + |b|):
    |dy| <= r,  r = mscale (|a| + |b|) 2^-20,   then |dy| <= r + u |y| + 2^-25
in 16 bits (2^-25 is half of fp16's smallest step).

Codes.  x off by r as above (0 for values) is multiplied by 1 / s, off by E, and
rounded to E: |x / s| 2^-22 covers both, then half a code's step.

Attention over code * scale: the products are exact and accumulate in float32,
so a score is off by at most e = 128 * 2 E * scale * ks * sum |q||a| (which
covers its three scalings too); weights are rounded to half precision whatever
the queries' type (2^-12 relative to a power of two's range: 2^-11 at most, and
2^-25 absolute where a row's sum is at least 1); sums over up to 2^14 keys take
fewer than 2^7 additions in a row in any accumulator: 2^-17 covers them, the
exponential, the factors of merging and the division.  With n visible keys
    |dO| <= (2^-11 + 2 e + 2^-17) A + u |O| + n 2^-25 max |v| + 2^-25,
    A = sum_j p_j |v_j|;  |dLSE| <= e + 2^-17 + 2^-21 |LSE|.
"""
import math

import numpy as np
import torch

import window_common as wc

DT = wc.DT
CODE_DT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
normal, window_mask = wc.normal, wc.window_mask


def frequencies(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def rotate(x, pos, w, mscale=1.0, interleaved=False, sign=1.0):
    """x float64 [..., n, d] at integer positions pos [n] (or [..., n]) by
    frequencies w [rot / 2]; returns the result and the bound r."""
    rot = 2 * len(w)
    y, r = x.copy(), np.zeros_like(x)
    # the angle from the position's whole and remaining turns, in extended precision
    a = np.longdouble(1) * pos[..., None] * w.astype(np.longdouble)
    c, s = (np.asarray(f(a), dtype=np.float64) for f in (np.cos, np.sin))
    s = sign * s
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., ia] = mscale * (x[..., ia] * c - x[..., ib] * s)
    y[..., ib] = mscale * (x[..., ib] * c + x[..., ia] * s)
    r[..., ia] = r[..., ib] = mscale * (np.abs(x[..., ia]) + np.abs(x[..., ib])) * 2.0 ** -20
    return y, r


def numpy_codes(t):
    """The numbers that a tensor of codes stands for, float64 (NaN for 0x7f)."""
    if t.dtype == torch.int8:
        return t.cpu().numpy().astype(np.float64)
    b = t.view(torch.uint8).cpu().numpy().astype(np.int64)
    e, m = b >> 3 & 15, b & 7
    val = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    val = np.where((b & 127) == 127, np.nan, val)
    return np.where(b >> 7, -val, val)


def half_code(x, code):
    """Half a code's step next to x."""
    if code == "int8":
        return np.full_like(x, 0.5)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x) * (1 + 2.0 ** -20), 2.0 ** -60)))
    return 2.0 ** (np.maximum(e, -6) - 4)


def values(cache, table, lens):
    """k, v float64 [B, Hk, capacity, d]: code * scale of every slot of the
    sequences, zeros in pages outside the pool, NaN left in."""
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes, s = numpy_codes(x), s.double().cpu().numpy()
        pages, Hk, page, d = codes.shape
        B, per = table.shape
        full = np.zeros((B, Hk, per * page, d))
        for b in range(B):
            for j in range(per):
                p = int(table[b, j])
                if 0 <= p < pages:
                    full[b, :, j * page:(j + 1) * page] = codes[p] * s[p][:, None, None]
        out.append(full)
    return out


def random_cache(pages, Hk, page, d, code, seed, spread=1.0):
    """A cache of codes of about unit variance, scales between 1 / 2 and 2 times
    the usual ones (times up to 2^+-spread)."""
    import exact_tiled_attention_14_gb300 as fa
    g = torch.Generator().manual_seed(seed)
    parts = []
    for _ in range(2):
        x = torch.randn(pages, Hk, page, d, generator=g)
        x = (x * 100).clamp(-448, 448) if code == "e4m3" else (x * 30).round().clamp(-127, 127)
        parts.append(x.to(CODE_DT[code]).cuda())
    for _ in range(2):
        r = torch.rand(pages, Hk, generator=g) * 2 - 1
        parts.append((torch.exp2(r * spread) / (100 if code == "e4m3" else 30)).cuda())
    return fa.PagedCache(*parts)


def reference(q, k, v, masks, scale, dtype):
    """float64 O, LSE of q [B, H, Nq, d] on float64 k, v [B, Hk, N, d] under
    masks[b] [Nq, N], and their bounds."""
    B, H, Nq, d = q.shape
    Hk = k.shape[1]
    G, u = H // Hk, wc.half_step(dtype)
    val = {"o": np.zeros((B, H, Nq, d)), "lse": np.full((B, H, Nq), -np.inf)}
    tol = {"o": np.zeros((B, H, Nq, d)), "lse": np.zeros((B, H, Nq))}
    qd = q.double().cpu().numpy()
    for b in range(B):
        m = masks[b]
        rows, keys = m.any(1), m.any(0)
        if not rows.any():
            continue
        m = m[np.ix_(rows, keys)]
        n = m.sum(1).max()
        for h in range(H):
            kk, vv, qq = k[b, h // G][keys], v[b, h // G][keys], qd[b, h][rows]
            s = np.where(m, scale * (qq @ kk.T), -np.inf)
            e = 128 * 2.0 ** -23 * scale * (np.abs(qq) @ np.abs(kk).T)[m].max()
            mx = s.max(1, keepdims=True)
            w = np.exp(s - mx)
            l = w.sum(1, keepdims=True)
            p = w / l
            o, lse = p @ vv, (mx + np.log(l))[:, 0]
            val["o"][b, h, rows], val["lse"][b, h, rows] = o, lse
            tol["o"][b, h, rows] = ((2.0 ** -11 + 2 * e + 2.0 ** -17) * (p @ np.abs(vv)) + u * np.abs(o)
                                    + n * 2.0 ** -25 * np.abs(vv).max() + 2.0 ** -25)
            tol["lse"][b, h, rows] = e + 2.0 ** -17 + 2.0 ** -21 * np.abs(lse)
    return val, tol


def check(got, val, tol, what):
    wc.check(got, val, tol, what)


def scale_of(d):
    return 1.0 / math.sqrt(d)
