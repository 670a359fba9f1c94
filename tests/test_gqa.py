"""Refusals and plan of the GQA tree attention: host only."""

import ctypes

import pytest

from speculative_decoding_tree_mla_gb300 import kdtv


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_tree_mla_gb300 import build
    build.build()
    return kdtv.lib()


def dims(**kw):
    d = kdtv.KdtvGqaDims(2, 8, 16, 4, 128, kdtv.KDTV_BF16, 0, 512, 0, 0, 0.0, 0, 4096, 1 << 40)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def call(L, d, q=256, k=256, v=256, ks=None, vs=None, parent=256, prefix=256, table=None, out=256, status=256):
    return kdtv.STATUS[L.kdtv_gqa_verify_attn(ctypes.byref(d), q, k, v, ks, vs, parent, prefix, None, table, out,
                                              status, None)]


@pytest.mark.parametrize("flags", [0, kdtv.KDTV_FLAG_SIMT])
@pytest.mark.parametrize("fields,code", [
    (dict(B=0), "KDTV_ERR_INVALID_ARG"), (dict(N=0), "KDTV_ERR_INVALID_ARG"), (dict(N=129), "KDTV_ERR_UNSUPPORTED"),
    (dict(H=15), "KDTV_ERR_INVALID_ARG"), (dict(H_kv=0), "KDTV_ERR_INVALID_ARG"), (dict(d=0), "KDTV_ERR_INVALID_ARG"),
    (dict(d=257), "KDTV_ERR_UNSUPPORTED"), (dict(dtype=3), "KDTV_ERR_INVALID_ARG"),
    (dict(t_stride=0), "KDTV_ERR_INVALID_ARG"), (dict(page_size=-64), "KDTV_ERR_INVALID_ARG"),
    (dict(page_size=64, num_pages=9), "KDTV_ERR_INVALID_ARG"),
    (dict(page_size=64, max_pages=1 << 25, num_pages=9), "KDTV_ERR_INVALID_ARG"),
    (dict(B=1 << 14), "KDTV_ERR_UNSUPPORTED"), (dict(B=1 << 13, N=128, H=512, H_kv=4), "KDTV_ERR_UNSUPPORTED"),
])
def test_bad_dims(L, fields, code, flags):
    d = dims(flags=flags, **fields)
    assert L.kdtv_gqa_workspace_size(ctypes.byref(d)) == 0
    assert L.kdtv_gqa_launches_per_call(ctypes.byref(d)) == -1
    assert call(L, d) == code


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(parent=None), dict(prefix=None),
                                dict(out=None), dict(status=None), dict(table=256), dict(ks=256), dict(vs=256),
                                dict(q=264), dict(k=257), dict(v=258), dict(out=260)])
def test_bad_pointers(L, kw):
    assert call(L, dims(), **kw) == "KDTV_ERR_INVALID_ARG"


def test_one_byte_cache_needs_scales(L):
    d = dims(dtype=kdtv.KDTV_BF16_FP8KV)
    assert call(L, d, ks=256) == call(L, d, vs=256) == call(L, d) == "KDTV_ERR_INVALID_ARG"


def test_workspace(L):
    d = dims()
    n = L.kdtv_gqa_workspace_size(ctypes.byref(d))
    assert n > 0 and n % 256 == 0 and L.kdtv_gqa_launches_per_call(ctypes.byref(d)) >= 1
    for ws, size in ((None, 1 << 40), (4096 + 16, 1 << 40), (4096, n - 1)):
        assert call(L, dims(workspace=ws, workspace_bytes=size)) == "KDTV_ERR_INVALID_ARG"
    assert L.kdtv_gqa_workspace_size(None) == 0 and L.kdtv_gqa_launches_per_call(None) == -1


@pytest.mark.parametrize("flags", [0, kdtv.KDTV_FLAG_SIMT])
@pytest.mark.parametrize("fields", [dict(B=1, t_stride=(1 << 30) + 1), dict(B=1, N=128, H=1 << 15, H_kv=1, d=64)])
def test_sizes_beyond_the_grid(L, fields, flags):
    """Positions beyond 2^30, query rows of a head beyond 16 * 65535."""
    d = dims(flags=flags, **fields)
    assert L.kdtv_gqa_workspace_size(ctypes.byref(d)) == 0
    assert call(L, d) == "KDTV_ERR_UNSUPPORTED"


def test_compaction_of_rows_too_wide(L):
    """Rows whose accepted chunk does not fit a CTA's shared memory are refused before any launch."""
    d = kdtv.KdtvDims(2, 8, 8, 128, 64, 128, 1 << 17, kdtv.KDTV_BF16, 0, 512)
    assert kdtv.STATUS[L.kdtv_compact_kv(ctypes.byref(d), 256, 256, 256, 256, 256, None, 256, None)] == \
        "KDTV_ERR_UNSUPPORTED"
