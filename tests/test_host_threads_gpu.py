"""Calls of different sizes from four host threads, separate workspaces: kernels whose shared memory
depends on the size must launch whatever the other thread asked for in between."""

import ctypes
import threading

import pytest
import torch

from speculative_decoding_tree_mla_gb300 import kdtv, workloads as W
from tests.test_gqa_gpu import SIMT, Case

pytestmark = pytest.mark.gpu


def _compaction(width):
    """Rows whose chunk takes 64 * width bytes of shared memory; nothing moves."""
    spec = W.Spec("wide", 0, B=1, N=4, H=1, d_nope=width, d_rope=width, d_v=width, d_c=width, dtype="bf16",
                  prefix=("fixed", 0), tree=("chain",))
    d = kdtv.make_dims(spec, dtype="bf16", t_stride=8)
    K, V = (torch.zeros((1, 8, width), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    word = torch.zeros(8, dtype=torch.int32, device="cuda")
    path = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    plen = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    fn, ptrs = kdtv.lib().kdtv_compact_kv, [t.data_ptr() for t in (K, V, word[:1], path, plen)]

    def call(stream):
        return fn(ctypes.byref(d), *ptrs, None, word[4:].data_ptr(), stream)
    call.keep = (K, V, word, path, plen)
    return call


def _gqa(d):
    """CUDA cores, fp32: head dims 129 .. 256 share an instance and differ in shared memory."""
    op = Case(1, 2, 2, 1, d, "f32", 0, [40], seed=31).op(SIMT)

    def call(stream):
        return op._fn(*op._args, stream)
    call.keep = op
    return call


def _mla_simt(d_c):
    wl = W.make(W.small_spec("threads_simt", B=1, N=2, H=16, d_c=d_c, dtype="f32", prefix=("fixed", 40)))
    op = kdtv.for_workload(wl, "cuda")
    stream_call = type("S", (), {})

    def call(stream):
        s = stream_call()
        s.cuda_stream = stream
        op(stream=s)
        return 0
    call.keep = op
    return call


def _mla_absorb(d_nope):
    wl = W.make(W.small_spec("threads_absorb", B=1, N=2, H=16, d_nope=d_nope, prefix=("fixed", 40)))
    op = kdtv.for_workload(wl, "cuda")
    stream_call = type("S", (), {})

    def call(stream):
        s = stream_call()
        s.cuda_stream = stream
        op(stream=s)
        return 0
    call.keep = op
    return call


def _tree_build(N, K):
    lp = torch.zeros((1, 8, K), device="cuda")
    tok = torch.zeros((1, 8, K), dtype=torch.int32, device="cuda")
    root = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.zeros((1, N), dtype=torch.int32, device="cuda") for _ in range(5)]
    fn = kdtv.lib().kdtv_tree_build
    ptrs = [t.data_ptr() for t in (lp, tok, root, *out)]

    def call(stream):
        return fn(1, 8, K, N, *ptrs, stream)
    call.keep = (lp, tok, root, out)
    return call


PAIRS = {"compact": (_compaction, (1600,), (3400,)), "gqa": (_gqa, (160,), (256,)),
         "mla_simt": (_mla_simt, (256,), (512,)), "mla_absorb": (_mla_absorb, (64,), (256,)),
         "tree_build": (_tree_build, (110, 60), (128, 64))}


@pytest.mark.parametrize("what", list(PAIRS))
def test_sizes_beside_each_other(what):
    make, small, large = PAIRS[what]
    calls = [make(*size) for size in (small, large, small, large)]
    torch.cuda.synchronize()
    bad, begin = [], threading.Barrier(len(calls))

    def engine(call):
        stream = torch.cuda.Stream()
        begin.wait()
        for k in range(15000):
            try:
                rc = call(stream.cuda_stream)
            except kdtv.KdtvError as e:
                rc = e.code
            if rc:
                bad.append(kdtv.STATUS[rc])
            if k % 64 == 63:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=engine, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, (len(bad), bad[:3])
