"""Refusals of the norm, projection and page-table calls: host only."""

import ctypes

import numpy as np
import pytest

from oracle import serve_ops as O
from speculative_decoding_tree_mla_gb300 import kdtv


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_tree_mla_gb300 import build
    build.build()
    return kdtv.lib()


def _fill(s, fields):
    for k, v in fields.items():
        if isinstance(v, tuple):
            v = (ctypes.c_int64 * len(v))(*v)
        setattr(s, k, v)


INVALID, UNSUPPORTED = "KDTV_ERR_INVALID_ARG", "KDTV_ERR_UNSUPPORTED"


@pytest.mark.parametrize("fields,ptr,code", [
    (dict(B=0), {}, INVALID), (dict(N=0), {}, INVALID), (dict(H=-1), {}, INVALID), (dict(dim=0), {}, INVALID),
    (dict(dtype=kdtv.KDTV_BF16_FP8KV), {}, INVALID), (dict(out_dtype=kdtv.KDTV_F32), {}, INVALID),
    (dict(out_dtype=kdtv.KDTV_BF16_FP8KV), {}, INVALID), ({}, dict(scale=256), INVALID),
    (dict(out_dtype=kdtv.KDTV_BF16_FP8KV, dim=100), dict(scale=256), INVALID),
    (dict(eps=-1.0), {}, INVALID), (dict(eps=float("nan")), {}, INVALID), (dict(weight_offset=float("inf")), {}, INVALID),
    ({}, dict(x=None), INVALID), ({}, dict(y=None), INVALID), ({}, dict(res=None), INVALID),
    ({}, dict(y=1536), INVALID), ({}, dict(y=1024), INVALID), ({}, dict(res_out=1536), INVALID),
    (dict(y_stride=(2000, 600, 130)), dict(y=256), INVALID),            # in place with other strides
    (dict(y_stride=(2000, 600, 130)), dict(y=512), INVALID),            # over the residual
    (dict(r_stride=(2000, 600, 130)), dict(res_out=512), INVALID),
    (dict(y_stride=(0, 512, 128)), {}, INVALID), (dict(y_stride=(1536, 0, 128)), {}, INVALID),
    (dict(ro_stride=(1536, 512, 0)), {}, INVALID),
    (dict(out_dtype=kdtv.KDTV_BF16_FP8KV), dict(y=256, scale=256), INVALID),
    (dict(dim=32769), {}, UNSUPPORTED), (dict(B=1 << 20, N=1 << 12), {}, UNSUPPORTED),
])
def test_norm_refusals(L, fields, ptr, code):
    a = kdtv.KdtvNormArgs(2, 3, 4, 128, kdtv.KDTV_BF16, kdtv.KDTV_BF16, 1e-6, 0.0)
    _fill(a, fields)
    p = dict(x=256, res=512, res_out=1024, weight=1536, y=2048, scale=None)
    p.update(ptr)
    rc = L.kdtv_rmsnorm(ctypes.byref(a), p["x"], p["res"], p["res_out"], p["weight"], p["y"], p["scale"], None, None)
    assert kdtv.STATUS[rc] == code


def test_null_structs(L):
    assert kdtv.STATUS[L.kdtv_rmsnorm(None, 256, None, None, None, 512, None, None, None)] == INVALID
    assert kdtv.STATUS[L.kdtv_project(None, *([256] * 11), None)] == INVALID
    assert kdtv.STATUS[L.kdtv_pages_resize(None, *([256] * 8), None)] == INVALID
    assert L.kdtv_project_workspace_size(None) == 0 and L.kdtv_project_launches_per_call(None) == -1


def _proj_dims(**fields):
    d = kdtv.KdtvProjectDims(2, 3, 128, 64, kdtv.KDTV_BF16, 4, 16, 0)
    _fill(d, fields)
    return d


@pytest.mark.parametrize("fields,code", [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(d_in=0), INVALID), (dict(d_out=-5), INVALID),
    (dict(dtype=5), INVALID), (dict(adapters=-1), INVALID), (dict(rank=0), INVALID),
    (dict(dtype=kdtv.KDTV_BF16_FP8KV, d_in=100), INVALID),
    (dict(adapters=4097), UNSUPPORTED), (dict(rank=257), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(d_in=(1 << 20) + 8), UNSUPPORTED), (dict(d_out=(1 << 20) + 1), UNSUPPORTED),
    (dict(B=4096, N=4096), UNSUPPORTED),
])
def test_projection_dims_refused(L, fields, code):
    d = _proj_dims(**fields)
    assert L.kdtv_project_workspace_size(ctypes.byref(d)) == 0 and L.kdtv_project_launches_per_call(ctypes.byref(d)) == -1
    rc = L.kdtv_project(ctypes.byref(d), 256, None, 512, None, 768, 1024, None, 256, None, 1280, 256, None)
    assert kdtv.STATUS[rc] == code


@pytest.mark.parametrize("fields,ptr", [
    ({}, dict(x=None)), ({}, dict(W=None)), ({}, dict(y=None)), ({}, dict(status=None)), ({}, dict(y=256)), ({}, dict(y=512)),
    ({}, dict(xs=256)), ({}, dict(ws=256)), (dict(dtype=kdtv.KDTV_BF16_FP8KV), dict(xs=256)),
    (dict(dtype=kdtv.KDTV_BF16_FP8KV), dict(ws=256)), ({}, dict(A=None)), ({}, dict(Bm=None)),
    ({}, dict(A=None, Bm=None)), (dict(adapters=0), {}), (dict(workspace=None), {}), (dict(workspace=4096 + 16), {}),
    (dict(workspace_bytes=1), {}),
    (dict(dtype=kdtv.KDTV_BF16_FP8KV, x_stride=(1000, 200)), dict(xs=256, ws=256)),
    (dict(y_stride=(0, 64)), {}), (dict(y_stride=(192, 0)), {}),
])
def test_projection_refusals(L, fields, ptr):
    d = _proj_dims(workspace=4096, workspace_bytes=1 << 40)
    _fill(d, fields)
    p = dict(x=256, xs=None, W=512, ws=None, A=768, Bm=1024, ad=256, y=1280, status=256)
    p.update(ptr)
    rc = L.kdtv_project(ctypes.byref(d), p["x"], p["xs"], p["W"], p["ws"], p["A"], p["Bm"], None, p["ad"], None, p["y"],
                        p["status"], None)
    assert kdtv.STATUS[rc] == INVALID


@pytest.mark.parametrize("fields", [{}, dict(dtype=kdtv.KDTV_F32), dict(dtype=kdtv.KDTV_BF16_FP8KV), dict(adapters=0, rank=0),
                                    dict(flags=kdtv.KDTV_FLAG_SIMT), dict(B=512, N=1, adapters=300, rank=64),
                                    dict(B=4, N=5000, d_in=8192, d_out=12288), dict(d_in=7, d_out=9, rank=3)])
def test_projection_workspace(L, fields):
    d = _proj_dims(**fields)
    n = L.kdtv_project_workspace_size(ctypes.byref(d))
    assert n > 0 and n % 256 == 0 and 1 <= L.kdtv_project_launches_per_call(ctypes.byref(d)) <= 3


@pytest.mark.parametrize("fields,ptr,code", [
    (dict(B=0), {}, INVALID), (dict(N=-1), {}, INVALID), (dict(page_size=0), {}, INVALID), (dict(max_pages=0), {}, INVALID),
    (dict(num_pages=0), {}, INVALID), (dict(max_pages=1 << 26, page_size=64), {}, INVALID),
    (dict(B=8193), {}, UNSUPPORTED), (dict(B=4096, N=1 << 20), {}, UNSUPPORTED), (dict(B=1, N=(1 << 30) + 1), {}, UNSUPPORTED),
    (dict(B=8192, max_pages=1 << 18), {}, UNSUPPORTED),
] + [({}, {k: None}, INVALID) for k in ("prefix", "free", "count", "held", "table", "status")])
def test_pages_refusals(L, fields, ptr, code):
    d = kdtv.KdtvPagesDims(2, 3, 16, 8, 32)
    _fill(d, fields)
    p = dict(prefix=256, live=None, free=256, count=256, held=256, table=256, slots=256, status=256)
    p.update(ptr)
    rc = L.kdtv_pages_resize(ctypes.byref(d), *p.values(), None)
    assert kdtv.STATUS[rc] == code


def test_oracle_pages_round_trip():
    """Growing and trimming back restores the stack, tables and counts."""
    rng = np.random.default_rng(3)
    free, held = [int(v) for v in rng.permutation(40)], [0, 0, 0]
    table = [[-1] * 16 for _ in range(3)]
    assert not O.pages_resize([30, 0, 65], 16, 16, 40, free, held, table)
    before = (list(free), list(held), [list(r) for r in table])
    assert held == [2, 0, 5]
    assert not O.pages_resize([47, 20, 120], 16, 16, 40, free, held, table)
    assert not O.pages_resize([30, 0, 65], 16, 16, 40, free, held, table)
    assert (free, held, table) == before
    assert O.pages_resize([30, 16 * 16, 16 * 16 + 0], 16, 16, 20, free[:], held[:], [list(r) for r in table]) is False
    assert O.pages_resize([30, 256, 65], 16, 16, 40, free[:5], held[:], [list(r) for r in table]) is True


def test_oracle_widen_matches_the_format():
    import torch
    codes = np.arange(256)
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.e4m3(codes), want)
    y = np.array([[448.0] + [0.0] * 31 + [449.0] + [1.0] * 31])
    assert O.group_exponent(y).tolist() == [[0, 1]]
