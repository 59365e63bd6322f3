"""Plain float64 forms of windowed and drafted-tree attention, written from the
mask's definition, and error bounds for results that the kernels compute with
16-bit weights.

Bounds.  u = eps / 2 is half a step of the 16-bit type.  The kernels round
each weight p_ij (and each dS_ij) once to 16 bits for the tensor core and each
result once; everything else is fp32.  A score is a sum of d <= 128 products,
each addition off by at most 2^-23 of the running sum of |q||k|, so with
m = max over the pairs of scale * sum |q||k| the exponent is off by at most
e = 128 * 2^-23 * m, and so is each weight, relatively (LSE, the sum's own
additions and the exponential itself add a few 2^-21):  s = 2 e + 2^-18.
fp16 weights below its normal range are off by up to 2^-25 each, at a scale
where the row's sum is at least 1 (n keys).
  |dO|   <= (u + s) A + u |O| + n 2^-25 max|v|,  A = sum_j p_ij |v_j|
  |dLSE| <= e + (n + 8) 2^-23 + 2^-21 |LSE| + 2^-20
  D = rowsum(dO * O) from the rounded O: |dD| <= sum |dO| tol_O
  |ddV| <= (u + s) P^T |dO| + u |dV| + n 2^-25 max|dO|
  |ddS| <= (u + s) P (|dP| + |D|) + P |dD|
  |ddQ| <= scale (|ddS| |K| + n 2^-25 max|K|) + u |dQ|, and dK alike.
"""
import math

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def normal(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def window_mask(Nq, Nk, length, causal, win, sinks):
    """[Nq, Nk] visible pairs of one batch."""
    n = max(0, min(Nk, length))
    pos = np.arange(Nq)[:, None] + (n - Nq if causal == "bottom_right" else 0)
    j = np.arange(Nk)[None, :]
    return (j < n) & (j <= pos) & ((j > pos - win) | (j < sinks))


def tree_mask(rows, Nk, count, win, sinks):
    """[Nq, Nk] visible keys of drafted tokens with 64-bit rows."""
    Nq = len(rows)
    rows = [int(r) & ((1 << Nq) - 1) for r in rows]
    c = max(0, min(Nk, count))
    pos = [c - 1 + bin(r).count("1") for r in rows]
    vis = np.zeros((Nq, Nk), dtype=bool)
    j = np.arange(Nk)
    for i in range(Nq):
        vis[i] = j < c
        if win is not None:
            vis[i] &= (j > pos[i] - win) | (j < sinks)
        for t in range(Nq):
            if rows[i] >> t & 1 and c + t < Nk:
                vis[i, c + t] = win is None or pos[t] > pos[i] - win or pos[t] < sinks
    return vis


def reference(q, k, v, masks, scale, dtype, dout=None):
    """float64 O, LSE (and dQ, dK, dV) of q [B, H, Nq, d], k, v [B, Hk, Nk, d]
    under masks[b] [Nq, Nk], with their bounds: two dicts name -> array.  Keys
    and values that no row sees, and queries that see none, may hold anything."""
    B, H, Nq, d = q.shape
    Hk = k.shape[1]
    G = H // Hk
    u = half_step(dtype)
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    val = {"o": np.zeros((B, H, Nq, d)), "lse": np.full((B, H, Nq), -np.inf)}
    tol = {"o": np.zeros((B, H, Nq, d)), "lse": np.zeros((B, H, Nq))}
    if dout is not None:
        for name, t in (("dq", q), ("dk", k), ("dv", k)):
            val[name], tol[name] = np.zeros(t.shape), np.zeros(t.shape)
    for b in range(B):
        vis = masks[b]
        rows, keys = vis.any(1), vis.any(0)
        if not rows.any():
            continue
        m = vis[np.ix_(rows, keys)]
        n = m.sum(1).max()
        for h in range(H):
            hk = h // G
            qq = q[b, h].double().numpy()[rows]
            kk = k[b, hk].double().numpy()[keys]
            vv = v[b, hk].double().numpy()[keys]
            s = np.where(m, scale * (qq @ kk.T), -np.inf)
            e = 128 * 2.0 ** -23 * scale * (np.abs(qq) @ np.abs(kk).T)[m].max()
            us = u + 2 * e + 2.0 ** -18
            mx = s.max(1, keepdims=True)
            w = np.exp(s - mx)
            l = w.sum(1, keepdims=True)
            p = w / l
            o = p @ vv
            lse = (mx + np.log(l))[:, 0]
            t_o = us * (p @ np.abs(vv)) + u * np.abs(o) + n * tiny * np.abs(vv).max()
            val["o"][b, h, rows], val["lse"][b, h, rows] = o, lse
            tol["o"][b, h, rows] = t_o
            tol["lse"][b, h, rows] = (e + (n + 8) * 2.0 ** -23 + 2.0 ** -21 * np.abs(lse)
                                      + 2.0 ** -20)
            if dout is None:
                continue
            do = dout[b, h].double().numpy()[rows]
            dp = do @ vv.T
            D = (do * o).sum(1, keepdims=True)
            ds = p * (dp - D)
            dD = (np.abs(do) * t_o).sum(1, keepdims=True)
            e_ds = us * p * (np.abs(dp) + np.abs(D)) + p * dD
            nq = m.sum(0).max()
            kidx = np.flatnonzero(keys)
            val["dq"][b, h, rows] = scale * (ds @ kk)
            tol["dq"][b, h, rows] = scale * (e_ds @ np.abs(kk) + n * tiny * np.abs(kk).max())
            val["dk"][b, hk, kidx] += scale * (ds.T @ qq)
            tol["dk"][b, hk, kidx] += scale * (e_ds.T @ np.abs(qq) + nq * tiny * np.abs(qq).max())
            val["dv"][b, hk, kidx] += p.T @ do
            tol["dv"][b, hk, kidx] += us * (p.T @ np.abs(do)) + nq * tiny * np.abs(do).max()
    if dout is not None:
        for name in ("dq", "dk", "dv"):
            tol[name] += u * np.abs(val[name])
    return val, tol


def check(got, val, tol, what):
    """Every result within its bound; rows that see nothing exactly O = 0,
    LSE = -inf, and gradients that are 0 by definition exactly 0."""
    for name, x in got.items():
        x = x.detach().cpu().double().numpy()
        ref, t = val[name], tol[name]
        if name == "lse":
            empty = np.isneginf(ref)
            assert np.all(np.isneginf(x[empty])), f"{what}: LSE of empty rows"
            x, ref, t = x[~empty], ref[~empty], t[~empty]
        if not x.size:
            continue
        assert np.all(np.isfinite(x)), f"{what}: {name} not finite"
        err = np.abs(x - ref)
        worst = np.unravel_index(np.argmax(err - t), err.shape)
        assert np.all(err <= t), (f"{what}: {name}{list(map(int, worst))} {x[worst]:.6e} against "
                                  f"{ref[worst]:.6e}, off {err[worst]:.3e}, bound {t[worst]:.3e}; "
                                  f"{int((err > t).sum())} of {err.size} out")


def scale_of(d):
    return 1.0 / math.sqrt(d)
