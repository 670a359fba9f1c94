"""fp64 CPU implementations of the steps between the attention calls: the norm
with the residual's addition, one byte per element with an exponent per group,
the shared projection with adapters, block tables.  Plain loops and numpy,
used by tests only; nothing here shares code with the library or with the
timed cases.
"""

from __future__ import annotations

import numpy as np

from oracle.rope_kv import row_exponent

GROUP = 32


def rmsnorm(x, weight, eps, residual=None, weight_offset=0.0):
    """x [.., dim]: (y, h) with h = x + residual."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        y = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
        if weight is not None:
            y = y * (np.asarray(weight, dtype=np.float64) + weight_offset)
    return y, h


def group_exponent(y):
    """Exponent of each group of 32 of y [.., dim]."""
    y = np.asarray(y, dtype=np.float64)
    return row_exponent(y.reshape(y.shape[:-1] + (-1, GROUP)))


def e4m3(code):
    """Values of E4M3 bytes."""
    code = np.asarray(code, dtype=np.int64)
    s, e, m = code >> 7, (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


def widen(code, scale):
    """Values of codes [.., dim] with exponent bytes [.., dim / 32]."""
    v = e4m3(code)
    f = 2.0 ** (np.asarray(scale, dtype=np.float64) - 127)
    return v * np.repeat(f, GROUP, axis=-1)


def project(x, W, A=None, Bm=None, adapter=None, adapter_scale=None):
    """x [B, N, K], W [M, K], A [a, R, K], Bm [a, M, R]: y [B, N, M] and the sum of the magnitudes of
    its terms."""
    y, mag = x @ W.T, np.abs(x) @ np.abs(W).T
    for b in range(x.shape[0]):
        a = -1 if adapter is None else int(adapter[b])
        if a < 0:
            continue
        s = 1.0 if adapter_scale is None else float(adapter_scale[a])
        y[b] += s * ((x[b] @ A[a].T) @ Bm[a].T)
        mag[b] += abs(s) * ((np.abs(x[b]) @ np.abs(A[a]).T) @ np.abs(Bm[a]).T)
    return y, mag


def pages_resize(rows, page_size, max_pages, num_pages, free, n_pages, table):
    """One resize to `rows[b]` rows (None: a request that is refused).  free: the stack as a list, n_pages
    a list, table a list of lists; all changed in place.  Returns whether the free list ran out.  (A request that
    would get an id out of range stops the taking too.)"""
    B = len(rows)
    want = [n_pages[b] if r is None else -(-r // page_size) for b, r in enumerate(rows)]
    for b in reversed(range(B)):
        for p in reversed(range(want[b], n_pages[b])):
            free.append(table[b][p])
            table[b][p] = -1
        n_pages[b] = min(n_pages[b], want[b])
    short = False
    for b in range(B):
        need = want[b] - n_pages[b]
        if need <= 0:
            continue
        short = need > len(free)
        if short or not all(0 <= p < num_pages for p in free[len(free) - need:]):
            break
        for p in range(n_pages[b], want[b]):
            table[b][p] = free.pop()
        n_pages[b] = want[b]
    return short


def slots(prefix_len, n_live, N, page_size, num_pages, n_pages, table):
    out = np.full((len(prefix_len), N), -1, dtype=np.int64)
    for b, (L, n) in enumerate(zip(prefix_len, n_live)):
        if L < 0 or L + n > n_pages[b] * page_size:
            continue
        for i in range(n):
            page = table[b][(L + i) // page_size]
            if 0 <= page < num_pages:
                out[b, i] = page * page_size + (L + i) % page_size
    return out
