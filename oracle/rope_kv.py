"""fp64 CPU implementations of rotary positions, of rows written to and read
from a cache, and of tree attention over a cache of keys and values per head.
Plain loops and numpy, used by tests only; nothing here shares code with the
library or with the timed cases.
"""

from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, orig_ctx=0, beta_fast=32.0,
                     beta_slow=1.0, attn_factor=0.0):
    """Angle per position of each pair, and the factor on the rotated pair."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    amp, out = 1.0, []
    for j in range(rot_dim // 2):
        f = base ** (-2.0 * j / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            def pair_of(turns):
                return rot_dim * math.log(orig_ctx / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo = max(math.floor(pair_of(beta_fast)), 0)
            hi = min(math.ceil(pair_of(beta_slow)), rot_dim - 1)
            ramp = min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f / factor * ramp + f * (1.0 - ramp)
            amp = attn_factor if attn_factor > 0 else 0.1 * math.log(factor) + 1.0
        out.append(f)
    return np.array(out, dtype=np.float64), amp


def rope(x, pos, freq, amp, layout, off):
    """x [.., H, dim] float64, pos [..] positions of its rows: the same with the
    2 len(freq) elements from `off` on rotated."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    h = len(freq)
    ang = np.asarray(pos, dtype=np.float64)[..., None] * freq
    c, s = (np.cos(ang) * amp)[..., None, :], (np.sin(ang) * amp)[..., None, :]
    if layout == "half":
        iu, iv = off + np.arange(h), off + h + np.arange(h)
    else:
        iu, iv = off + 2 * np.arange(h), off + 2 * np.arange(h) + 1
    y[..., iu] = x[..., iu] * c - x[..., iv] * s
    y[..., iv] = x[..., iv] * c + x[..., iu] * s
    return y


def row_exponent(x):
    """Exponent e of each row of x [.., dim]: the smallest with max|x| <= 448 * 2^e
    over the finite elements, in [-117, 119]."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    m = np.max(np.where(np.isfinite(a), a, 0.0), axis=-1)
    e = np.full(m.shape, -117, dtype=np.int64)
    for idx in np.ndindex(m.shape):
        k = -117
        while k < 119 and m[idx] > 448.0 * 2.0 ** k:
            k += 1
        e[idx] = k
    return e


def gqa_attn(q, k, v, parent, prefix_len, scale, n_nodes=None):
    """q [B, N, H, d], k / v [B, T, H_kv, d] float64 (rows already gathered): out
    [B, N, H, d], NaN for rows behind n_nodes."""
    B, N, H, d = q.shape
    G = H // k.shape[2]
    out = np.full(q.shape, np.nan)
    for b in range(B):
        for i in range(N if n_nodes is None else int(n_nodes[b])):
            see = list(range(int(prefix_len[b])))
            path, j = [], i
            while j >= 0:
                path.append(int(prefix_len[b]) + j)
                j = int(parent[b][j])
            see += path[::-1]
            for h in range(H):
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (k[b, see, h // G] @ q[b, i, h])
                    p = np.exp(s - s.max())
                    out[b, i, h] = (p / p.sum()) @ v[b, see, h // G]
    return out
