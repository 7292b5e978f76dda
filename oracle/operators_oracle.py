"""The operators around the cache, from their definitions in float64 (test infrastructure).

* ``attend``: attention of the newest tokens over the (dequantized) cache, with capped, biased and windowed scores;
* ``norm_rotary``: head norms and position rotation;
* ``reorder``: which history each sequence has after a reordering.
"""
from __future__ import annotations

import numpy as np

from oracle import kvq_oracle as o


def visible(n: int, n_q: int, window: int = 0, prefix: int = 0) -> np.ndarray:
    """[n_q, n] truth values: row i (at position n - n_q + i) sees key j."""
    p = n - n_q + np.arange(n_q)[:, None]
    j = np.arange(n)[None, :]
    seen = j <= p
    if window:
        seen &= p - j < window
    return seen | (j < prefix)


def scores(q, k, n: int, scale: float, cap: float = 0.0, slopes=None, gqa: int = 1):
    """[Hq, n_q, n] scores of q [n_q, Hq, d] against k [n, Hkv, d], before the mask."""
    n_q, hq, _ = q.shape
    kh = np.repeat(k.astype(np.float64), gqa, axis=1)
    s = scale * np.matmul(q.astype(np.float64).transpose(1, 0, 2), kh.transpose(1, 2, 0))
    if cap:
        s = cap * np.tanh(s / cap)
    if slopes is not None:
        p = n - n_q + np.arange(n_q)[:, None]
        s = s - np.asarray(slopes, np.float64)[:, None, None] * np.abs(p - np.arange(n)[None, :])
    return s


def cached(cfg: o.Config, k16, v16, chunks=None):
    """Dequantized keys and values [n, Hkv, d] (float64) as the cache holds them, rotated where it rotates."""
    if cfg.akvq_delta:
        kh, vh = (np.asarray(o.cache_tokens(cfg, x), np.float64) for x in (k16, v16))
        img = o.akvq_cache_image(cfg, kh, vh, chunks or [k16.shape[0]])
        G = cfg.group
        for i, (kc, ks, kz, vc, vs, vz) in enumerate(img["groups"]):
            kh[i * G:(i + 1) * G] = o.dequantize_keys(kc, ks, kz).transpose(1, 0, 2)
            vh[i * G:(i + 1) * G] = o.dequantize_values(vc, vs, vz, G).transpose(1, 0, 2)
        return kh, vh
    if cfg.rotate:
        k16, v16 = o.rotate_fp16(k16), o.rotate_fp16(v16)
    return o.dequantized_cache(cfg, k16, v16)


def attend(cfg: o.Config, k16, v16, q, scale: float = 0.0, cap: float = 0.0, window: int = 0, slopes=None, prefix: int = 0,
           chunks=None):
    """(out, tol): outputs [n_q, Hq, d] of one sequence and how far a correct fp16 result may be from them.

    tol per element, with A = sum_j alpha_j |v_j|, all roundings at most half a step (fp16: 2^-11 relative):
      2^-11 |out|     the result's rounding
      2^-11 (A + |out|) the weights' rounding to fp16, p_j (1 + d_j) with |d_j| <= 2^-11: where the sum is of the rounded weights
                      too, the result is off by sum_j alpha_j d_j (v_j - out), and sum_j alpha_j |v_j - out| <= A + |out|
      2^-11 A         the values' (s code + z) rounding to fp16
      n 2^-25 max|v|  weights below 2^-14 of the largest are subnormal in fp16: off by 2^-25 at most
      2 delta A       scores off by delta move the result by at most 2 delta A
      2^-24           the result's and the values' subnormal steps
    delta: 2^-17 times the absolute mass of the dot product (d + 2 fp32 additions of 2^-24 each, the query kept to 2^-22), 2^-25
    (an fp16 residual below the subnormals) per channel times the largest code, and 2^-20 of the largest of |score|, the cap (the
    exponent's, the tanh's and the bias's own roundings, 2^-24 to 2^-22 each).  A rotated cache adds fp32 butterflies on the
    query and the result: 2^-21 of the rows' norms.
    """
    kh, vh = cached(cfg, k16, v16, chunks)
    n, n_q = kh.shape[0], q.shape[0]
    d, gqa = cfg.head_dim, cfg.gqa
    q = q.astype(np.float64)
    if cfg.rotate:
        q = o.rotate_fp64(q)
    scale = scale or 1.0 / np.sqrt(d)
    s = scores(q, kh, n, scale, cap, slopes, gqa)
    seen = visible(n, n_q, window, prefix)[None]
    sm = np.where(seen, s, -np.inf)
    top = sm.max(-1, keepdims=True)
    e = np.where(seen, np.exp(sm - np.where(np.isfinite(top), top, 0.0)), 0.0)
    tot = e.sum(-1, keepdims=True)
    alpha = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
    v = np.repeat(vh.astype(np.float64), gqa, axis=1)
    v = v.transpose(1, 0, 2)
    out = np.matmul(alpha, v).transpose(1, 0, 2)
    A = np.matmul(alpha, np.abs(v)).transpose(1, 0, 2)
    # the dot product's mass: |q| (|s code| + |z|) <= |q| (|k| + 2 |z|), z at most the largest |k| of the channel
    kk = np.repeat(np.abs(kh).max(0)[None] * 3, gqa, axis=1)
    mass = (np.abs(q) * kk[0]).sum(-1)                                           # [n_q, Hq]
    big = np.where(seen & (alpha > 1e-9), np.abs(s), 0.0).max(-1).T + cap
    delta = scale * (2.0 ** -17 * mass + d * 15 * 2.0 ** -25) + 2.0 ** -20 * (1 + big)
    tol = 2.0 ** -11 * 2 * (np.abs(out) + A) + n * 2.0 ** -25 * np.abs(vh).max() + 2 * delta[..., None] * A + 2.0 ** -24
    if cfg.rotate:
        tol = np.sqrt((tol ** 2).sum(-1, keepdims=True)) + 2.0 ** -11 * np.abs(out).max(-1, keepdims=True)
        tol = np.broadcast_to(tol, out.shape) + 2.0 ** -21 * np.linalg.norm(out, axis=-1, keepdims=True)
        out = o.rotate_fp64(out)
    return out, tol


def norm_rotary(x, pos, inv_freq, sections=None, weight=None, eps: float = 0.0, interleaved: bool = False):
    """Rows x [n, heads, d] normed (where a weight is given) and rotated; pos [axes, n]."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    P = len(inv_freq)
    axis = np.repeat(np.arange(len(sections or [P])), sections or [P])
    t = pos[axis].T.astype(np.float64) * np.asarray(inv_freq, np.float64)        # [n, P]
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    a, b = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if interleaved else (slice(0, P), slice(P, 2 * P))
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def reorder(items, parent):
    """What each place holds after place b took over parent[b]'s, for all b < len(parent) at once."""
    return [items[parent[b]] if b < len(parent) else items[b] for b in range(len(items))]
