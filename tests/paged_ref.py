"""Plain 64-bit forms of the paged 8-bit cache's operators, for the GPU tests, and a small
pool builder.  Everything here is numpy on the host, one row at a time where that is clearer.

Tolerances (u = 2^-24, the f32 half step; a bf16 rounding is within 2^-8 of its value):

* a rotated row: the angle is reduced to within 2^-24 turns of its exact value and sincospi is
  good to 2 u, so cos and sin are within 2 pi 2^-24 + 2 u < 2^-21; the norm factor adds the sum
  of 16 squares a lane and up to 4 tree levels (20 u, halved by the root) and 2 u of rsqrt.
  Together a component is within 2^-20 of the length of its pair (Y_TOL).
* a scale: the largest component over 127, within sqrt(2) 2^-20 + u < 2^-19 of exact (S_TOL).
* a code c of y under scale s: |c - y / s| <= 1/2 + 127 (Y_TOL sqrt(2) + S_TOL + 2 u)
  <= 1/2 + 127 * 2^-18 (C_TOL); the same for a re-rounded code.
"""
import numpy as np
import torch

Y_TOL = 2.0 ** -20
S_TOL = 2.0 ** -19
C_TOL = 0.5 + 127 * 2.0 ** -18
BF16 = 2.0 ** -8


def ragged(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def make_table(rng, counts, max_pages, spare=2, fill=None):
    """(table [batch, max_pages], pages of the pool): shuffled pages, `fill` in unused entries."""
    num = int(sum(counts)) + spare
    order = rng.permutation(num)
    t = np.full((len(counts), max_pages), num + 7 if fill is None else fill, dtype=np.int32)
    at = 0
    for b, c in enumerate(counts):
        t[b, :c] = order[at:at + c]
        at += c
    return t, num


def make_pool(rng, num, nkv, ps, hd):
    codes = [np.clip(np.rint(rng.standard_normal((num, nkv, ps, hd)) * 36), -127, 127).astype(np.int8)
             for _ in range(2)]
    scales = [(np.exp(rng.standard_normal((num, nkv)) * 0.3) * 0.028).astype(np.float32) for _ in range(2)]
    return codes[0], scales[0], codes[1], scales[1]


def norm_rows(x, w, eps):
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * w


def rotate_rows(x, pos, theta, factors):
    half = x.shape[-1] // 2
    f = theta ** (-2.0 * np.arange(half) / (2 * half))
    if factors is not None:
        f = f / factors.astype(np.float64)
    a = np.asarray(pos, dtype=np.float64)[:, None, None] * f
    c, s = np.cos(a), np.sin(a)
    lo, hi = x[..., :half], x[..., half:]
    return np.concatenate([lo * c - hi * s, lo * s + hi * c], -1)


def pair_len(x):
    """Length of each component's rotation pair."""
    half = x.shape[-1] // 2
    r = np.sqrt(x[..., :half] ** 2 + x[..., half:] ** 2)
    return np.concatenate([r, r], -1)


def append_pages(rows, cu, start, table, ps, codes, scales):
    """The exact (unrounded) codes and the scales after an append of rows [T, nkv, hd]: returns
    (real codes f64 with NaN where the call leaves the byte alone, scales f64)."""
    real = np.full(codes.shape, np.nan)
    sc = scales.astype(np.float64).copy()
    tiny = float(np.finfo(np.float32).tiny)
    for b in range(len(start)):
        n, s0 = int(cu[b + 1] - cu[b]), int(start[b])
        for j in range(s0 // ps, (s0 + n - 1) // ps + 1 if n else s0 // ps):
            pg = table[b, j]
            lo, hi = max(s0, j * ps), min(s0 + n, (j + 1) * ps)
            x = rows[cu[b] + lo - s0:cu[b] + hi - s0].transpose(1, 0, 2)  # [nkv, m, hd]
            fin = np.where(np.isfinite(x), np.abs(x), 0).max((1, 2))
            old = sc[pg].copy() if lo > j * ps else np.zeros_like(sc[pg])
            new = np.maximum(old, fin / 127)
            new[new < tiny] = 0
            with np.errstate(divide="ignore", invalid="ignore"):
                if lo > j * ps:
                    r = np.where(new > 0, old / new, 0)
                    grown = new != old
                    kept = codes[pg, :, :lo - j * ps].astype(np.float64) * r[:, None, None]
                    real[pg, :, :lo - j * ps] = np.where(grown[:, None, None], kept, np.nan)
                v = np.where(new[:, None, None] > 0, x / new[:, None, None], 0)
            v = np.clip(np.where(np.isnan(v), 0, v), -127, 127)
            real[pg, :, lo - j * ps:hi - j * ps] = v
            sc[pg] = new
    return real, sc


def rows_of(codes, scales, table, ps, b, n):
    """Decoded rows 0 .. n - 1 of sequence b: f64 [nkv, n, hd]."""
    p = np.arange(n)
    pg = table[b][p // ps]
    return (codes[pg, :, p % ps].astype(np.float64) * scales[pg].astype(np.float64)[..., None]).transpose(1, 0, 2)


def attend(q, cu, lens, codes, table, ps, scale, softcap=0.0, window=0, bidir=False):
    """(o, bound) f64 [T, nh, hd]: the attention, and the f32-level error a kernel that keeps
    22 bits of q, P and the codes may make: a logit is off by at most 2^-19 of its absolute
    sum L (products and f32 sums of up to 256 terms in 16-wide tensor-core steps), so each
    weight by a factor exp(+-2 2^-19 L) with its own f32 roundings (2^-19 covers exp, the
    running sums' corrections and the final division): bound = (2 2^-19 max L + 2^-19) sum
    p |v|.  With a softcap the slope of the cap is at most 1."""
    kc, ks, vc, vs = codes
    T, nh, hd = q.shape
    nkv = kc.shape[1]
    G = nh // nkv
    o, bound = np.zeros((T, nh, hd)), np.zeros((T, nh, hd))
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        K = rows_of(kc, ks, np.clip(table, 0, kc.shape[0] - 1), ps, b, L)
        V = rows_of(vc, vs, np.clip(table, 0, kc.shape[0] - 1), ps, b, L)
        for i in range(n):
            P = L - n + i
            hi = L if bidir else P + 1
            lo = max(0, P - window + 1) if window else 0
            if hi <= lo:
                continue
            for h in range(nh):
                k, v = K[h // G, lo:hi], V[h // G, lo:hi]
                x = q[cu[b] + i, h].astype(np.float64)
                s = scale * (k @ x)
                big = scale * (np.abs(k) @ np.abs(x)).max()
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                p = np.exp(s - s.max())
                p /= p.sum()
                o[cu[b] + i, h] = p @ v
                bound[cu[b] + i, h] = (2 * 2.0 ** -19 * big + 2.0 ** -19) * (p @ np.abs(v))
    return o, bound


def dev(*arrays):
    out = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]
    return out if len(out) > 1 else out[0]
