"""Rotary tables and the refusals of the rotary, cache-write and cache-read calls: host only."""

import ctypes
from fractions import Fraction

import numpy as np
import pytest

from oracle import rope_kv as O
from speculative_decoding_tree_mla_gb300 import kdtv

# 1 / (2 pi) to 40 digits
INV_2PI = Fraction(1591549430918953357688837633725143620344, 10 ** 40)


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_tree_mla_gb300 import build
    build.build()
    return kdtv.lib()


@pytest.mark.parametrize("kw", [
    dict(rot_dim=2), dict(rot_dim=64, base=500000.0), dict(rot_dim=256),
    dict(rot_dim=128, scaling="linear", factor=4.0),
    dict(rot_dim=96, scaling="ntk", factor=8.0),
    dict(rot_dim=64, scaling="yarn", factor=32.0, base=50000.0, orig_ctx=4096),
    dict(rot_dim=128, scaling="yarn", factor=1.0, orig_ctx=32),
    dict(rot_dim=64, scaling="yarn", factor=4.0, orig_ctx=8192, attn_factor=1.25),
])
def test_table_matches_the_definition(L, kw):
    """turn[j] is f_j / 2 pi in units of 2^-64 turns.  pow and log may differ from the
    oracle's by an ulp or two (2^-52 relative each; YARN mixes two of them): 2^-49."""
    t = kdtv.RopeTable(**kw)
    f, amp = O.rope_frequencies(**kw)
    for j, w in enumerate(f):
        want = Fraction(float(w)) * INV_2PI * 2 ** 64
        assert abs(t.c.turn[j] - want) <= want / 2 ** 49 + 1
    assert abs(t.amp - amp) <= 2.0 ** -23 * amp
    assert all(t.c.turn[j] == 0 for j in range(len(f), 128))


def test_first_pair_is_exact(L):
    """f_0 = 1: the table holds 1 / 2 pi to its last bit, so far positions stay exact."""
    t = kdtv.RopeTable(128)
    assert abs(t.c.turn[0] - INV_2PI * 2 ** 64) <= 1


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), "KDTV_ERR_INVALID_ARG"), (dict(rot_dim=7), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_dim=258), "KDTV_ERR_UNSUPPORTED"), (dict(rot_dim=64, base=1.0), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_dim=64, base=float("nan")), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="linear", factor=0.5), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="linear", factor=float("inf")), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_dim=2, scaling="ntk", factor=2.0), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="yarn", factor=2.0), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_dim=64, scaling="yarn", factor=2.0, orig_ctx=64, beta_fast=1.0, beta_slow=2.0),
     "KDTV_ERR_INVALID_ARG"),
])
def test_table_refusals(L, kw, code):
    with pytest.raises(kdtv.KdtvError, match=code):
        kdtv.RopeTable(**kw)
    assert L.kdtv_rope_init(None, None) == kdtv.STATUS_CODE["KDTV_ERR_INVALID_ARG"]


def _rope(L, table=None, x=256, y=512, rest=None, **fields):
    t = table or kdtv.RopeTable(64)
    a = kdtv.KdtvRopeArgs(2, 3, 4, 128, 0, kdtv.KDTV_BF16)
    for k, v in fields.items():
        setattr(a, k, v)
    return kdtv.STATUS[L.kdtv_rope(ctypes.byref(t.c), ctypes.byref(a), x, y, rest, None, None, None, None)]


@pytest.mark.parametrize("fields,code", [
    (dict(B=0), "KDTV_ERR_INVALID_ARG"), (dict(N=-1), "KDTV_ERR_INVALID_ARG"),
    (dict(H=0), "KDTV_ERR_INVALID_ARG"), (dict(dim=63), "KDTV_ERR_INVALID_ARG"),
    (dict(rot_off=-1), "KDTV_ERR_INVALID_ARG"), (dict(rot_off=65), "KDTV_ERR_INVALID_ARG"),
    (dict(dtype=kdtv.KDTV_BF16_FP8KV), "KDTV_ERR_INVALID_ARG"),
    (dict(x=None), "KDTV_ERR_INVALID_ARG"), (dict(y=None), "KDTV_ERR_INVALID_ARG"),
    (dict(rest=256), "KDTV_ERR_INVALID_ARG"), (dict(rest=512), "KDTV_ERR_INVALID_ARG"),
    (dict(x=256, y=256, rest=512), "KDTV_ERR_INVALID_ARG"),
    (dict(x=256, y=256, x_stride=(ctypes.c_int64 * 3)(2000, 600, 130)), "KDTV_ERR_INVALID_ARG"),
    (dict(dim=1 << 17), "KDTV_ERR_UNSUPPORTED"), (dict(B=1 << 20, N=1 << 20), "KDTV_ERR_UNSUPPORTED"),
    (dict(B=1 << 14, N=1 << 14, H=64), "KDTV_ERR_UNSUPPORTED"),
])
def test_rope_refusals(L, fields, code):
    assert _rope(L, **fields) == code


def _kv(L, which, rope=None, prefix=256, table=None, status=256, parts=1, part=None, **fields):
    d = kdtv.KdtvKvDims(2, 3, kdtv.KDTV_BF16, kdtv.KDTV_BF16, 0, 64, 0, 0, 0.0, parts)
    for k, v in fields.items():
        setattr(d, k, v)
    p = (kdtv.KdtvKvPart * 2)()
    for q in p:
        q.cache, q.src, q.out, q.heads, q.dim = 256, 256, 256, 2, 64
        for k, v in (part or {}).items():
            setattr(q, k, v)
    if which == "append":
        r = ctypes.byref(rope.c) if rope else None
        rc = L.kdtv_kv_append(ctypes.byref(d), p, r, prefix, None, None, table, status, None)
    else:
        rc = L.kdtv_kv_read(ctypes.byref(d), p, prefix, None, table, status, None)
    return kdtv.STATUS[rc]


@pytest.mark.parametrize("which", ["append", "read"])
@pytest.mark.parametrize("fields,code", [
    (dict(B=0), "KDTV_ERR_INVALID_ARG"), (dict(N=0), "KDTV_ERR_INVALID_ARG"),
    (dict(parts=0), "KDTV_ERR_INVALID_ARG"), (dict(parts=3), "KDTV_ERR_INVALID_ARG"),
    (dict(dtype=2), "KDTV_ERR_INVALID_ARG"), (dict(cache_dtype=3), "KDTV_ERR_INVALID_ARG"),
    (dict(page_size=64), "KDTV_ERR_INVALID_ARG"), (dict(table=256), "KDTV_ERR_INVALID_ARG"),
    (dict(page_size=-1), "KDTV_ERR_INVALID_ARG"), (dict(t_stride=0), "KDTV_ERR_INVALID_ARG"),
    (dict(page_size=64, table=256, max_pages=0, num_pages=4), "KDTV_ERR_INVALID_ARG"),
    (dict(page_size=64, table=256, max_pages=1 << 25, num_pages=4), "KDTV_ERR_INVALID_ARG"),
    (dict(status=None), "KDTV_ERR_INVALID_ARG"), (dict(part=dict(cache=None)), "KDTV_ERR_INVALID_ARG"),
    (dict(part=dict(src=None, out=None)), "KDTV_ERR_INVALID_ARG"),
    (dict(part=dict(scale=256)), "KDTV_ERR_INVALID_ARG"),
    (dict(part=dict(heads=0)), "KDTV_ERR_INVALID_ARG"), (dict(part=dict(dim=513)), "KDTV_ERR_UNSUPPORTED"),
    (dict(B=65536), "KDTV_ERR_UNSUPPORTED"), (dict(N=1 << 28), "KDTV_ERR_UNSUPPORTED"),
])
def test_kv_refusals(L, which, fields, code):
    assert _kv(L, which, **fields) == code


def test_append_rotation_refusals(L):
    assert _kv(L, "append", part=dict(rotate=1)) == "KDTV_ERR_INVALID_ARG"              # no table
    t = kdtv.RopeTable(64)
    for off in (-1, 1):
        assert _kv(L, "append", rope=t, part=dict(rotate=1, rot_off=off)) == "KDTV_ERR_INVALID_ARG"
    t.c.rot_dim = 300                                                                   # not from rope_init
    assert _kv(L, "append", rope=t, part=dict(rotate=1)) == "KDTV_ERR_INVALID_ARG"
    assert _rope(L, table=t) == "KDTV_ERR_INVALID_ARG"


def test_row_exponent_is_the_smallest():
    x = np.array([[0.0, 0.0], [448.0, 1.0], [448.5, 1.0], [-1.0, 0.5], [np.inf, 2.0], [np.nan, -900.0],
                  [1e-38, 0.0], [3e38, 0.0]])
    assert O.row_exponent(x).tolist() == [-117, 0, 1, -8, -7, 2, -117, 119]
