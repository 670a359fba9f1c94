"""GQA tree attention at the edges of its types, errors and head counts.

Tolerance, fixed before the first run: that of bf16 caches, for one-byte caches too.  With delta =
(d + 4) * 2^-24 * scale * max_t sum_e |q_e k_te| bounding a score's fp32 error, the weights are off
by a factor of at most 1 + 2 delta + 2^-20, on tensor cores each is rounded to bf16 (2^-8), so with
A = sum_t p_t |v_t| the sum is off by (2 delta + 2^-20 + T 2^-24 [+ 2^-8]) * A, and the output's
rounding adds 2^-8 |o|.  Queries and keys count as they are: a query held in parts has to be their
exact sum, down to 2^-31 of its row's largest element.
"""

import numpy as np
import pytest
import torch

from oracle import rope_kv as O
from speculative_decoding_tree_mla_gb300 import kdtv
from tests.test_gqa_gpu import SIMT, Case

pytestmark = pytest.mark.gpu

BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def check(x, out, tensor_cores):
    k, v = x.gathered()
    v = np.where(np.abs(v) > BF16_MAX, np.copysign(np.inf, v), v)     # as widened
    q = x.q.float().cpu().double().numpy()
    scale, G, T = x.d ** -0.5, x.H // x.Hkv, k.shape[1]
    want = O.gqa_attn(q, k, v, x.parent, x.prefix, scale, x.n)
    A = O.gqa_attn(q, k, np.abs(v), x.parent, x.prefix, scale, x.n)
    got = out.float().cpu().double().numpy()
    for b in range(x.B):
        n = int(x.n[b])
        assert (got[b, n:] == 9.0).all()
        kk = np.repeat(np.abs(k[b]).max(0), G, axis=0)                # [H, d]
        delta = (x.d + 4) * 2.0 ** -24 * scale * (np.abs(q[b, :n]) * kk).sum(-1)[..., None]
        rel = 2 * delta + 2.0 ** -20 + T * 2.0 ** -24 + (2.0 ** -8 if tensor_cores else 0.0)
        w, g, a = want[b, :n], got[b, :n], A[b, :n]
        fin = np.isfinite(w)
        assert (np.isnan(g) == np.isnan(w)).all() and (g[np.isinf(w)] == w[np.isinf(w)]).all()
        with np.errstate(invalid="ignore"):
            err, tol = np.abs(g - w)[fin], (rel * a + 2.0 ** -8 * np.abs(w))[fin]
        assert (err <= tol).all(), (b, (err / tol).max())


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("times", [64, 1 << 10, 1 << 14], ids=lambda n: f"x{n}")
@pytest.mark.parametrize("channel", [0, 0x28], ids=["keys0", "keys_small"])
@pytest.mark.parametrize("N,H,Hkv,d,page", [(5, 16, 2, 128, 64), (3, 8, 2, 64, 0), (24, 16, 2, 128, 0),
                                            (70, 8, 2, 64, 16)])
def test_queries_with_an_outlier(N, H, Hkv, d, page, channel, times, flags):
    """One channel of every query is `times` the others, and the keys do not tell each other apart in
    it: the softmax follows the small elements alone.  (0x28 is E4M3's 0.25.)"""
    x = Case(2, N, H, Hkv, d, "fp8", page, [300, 90], seed=21, sharp=2.0)
    for s in x.scales:
        s.fill_(120)
    x.kv[0].view(-1, Hkv, d)[..., 5] = channel
    x.q[..., 5] = float(times)
    op = x.op(flags)
    check(x, op(), flags == 0)
    assert op.status() == 0


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("d,page", [(128, 0), (64, 16)])
def test_queries_over_a_wide_range(d, page, flags):
    """The elements of a query row spread over 2^14, the keys' over as much the other way, so that all
    count alike in a score."""
    x = Case(1, 9, 8, 2, d, "fp8", page, [500], seed=22)
    e = torch.arange(d, device="cuda") % 14
    x.q.copy_((x.q.float() * torch.exp2(7.0 - e)).to(x.q.dtype))
    for s in x.scales:
        s.fill_(127)
    k = x.kv[0].view(-1, 2, d)                     # E4M3 exponents 1 .. 14, signs and mantissas as they were
    k.copy_((k & 0x87) | (8 * (e + 1)).to(torch.uint8))
    op = x.op(flags)
    check(x, op(), flags == 0)
    assert op.status() == 0


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("byte", [247, 250, 254])
@pytest.mark.parametrize("d,page,prefix", [(128, 0, 20), (128, 16, 700), (64, 16, 61), (64, 0, 700)])
def test_values_that_overflow(d, page, prefix, byte, flags):
    """A node whose value row overflows when it is widened (scale bytes above 246) reaches itself and
    its descendants alone; in the prefix it reaches all."""
    for in_prefix in (False, True):
        x = Case(1, 14, 8, 2, d, "fp8", page, [prefix], seed=23, tree=(3, 3))
        nodes = (2, 5, 11) if not in_prefix else (-3,)
        for node, codes in zip(nodes, ((0x7E, 0x01, 0x02, 0xFE), (0xFE, 0x7E, 0x00, 0x01), (0x00, 0x81, 0xFE, 0x7F))):
            row = x.rows(0, prefix + node + 1)[-1].cuda()
            x.scales[1].view(-1, 2)[row, 0] = byte
            x.kv[1].view(-1, 2, d)[row, 0] = 0
            x.kv[1].view(-1, 2, d)[row, 0, 3:7] = torch.tensor(codes, dtype=torch.uint8, device="cuda")
        op = x.op(flags)
        check(x, op(), flags == 0)
        assert op.status() == 0


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_a_wait_that_runs_out_behind_another_error(cache, d):
    """The loads never start (a test flag; every wait has a limit) in a call whose batch has a bad
    prefix as well, or whose status word holds an earlier error: the timeout is reported and no row
    is written, whatever the workspace held."""
    for earlier in (0, kdtv.STATUS_CODE["KDTV_ERR_BAD_TREE"]):
        x = Case(3, 9, 8, 2, d, cache, 16, [700, 300, 20], seed=24)
        good = x.prefix.copy()
        if not earlier:
            x.prefix[1] = -1
        op = x.op(kdtv.KDTV_FLAG_TEST_STALL)
        op.workspace.zero_()                       # what was not written looks like partial rows
        op._status.fill_(earlier)
        out = op()
        assert kdtv.STATUS[op.status()] == "KDTV_ERR_DEVICE_TIMEOUT"
        assert (out == 9.0).all()
        assert op.status() == 0
        x.prefix = good
        again = x.op()
        x.check(again(), True)
        assert again.status() == 0


HEADS = [
    # B, N, H, Hkv, d, cache, page, prefix, n_nodes: blocks of 8, 6, 3 and 1 key heads
    (2, 5, 16, 16, 128, "bf16", 64, [300, 20], [5, 3]),
    (1, 1, 32, 32, 128, "bf16", 64, [700], None),
    (2, 20, 96, 12, 64, "bf16", 0, [129, 0], [20, 1]),
    (1, 40, 72, 9, 128, "bf16", 16, [250], None),
    (3, 3, 22, 11, 64, "bf16", 32, [5, 400, 60], [3, 0, 2]),
    (2, 5, 16, 16, 128, "fp8", 16, [300, 20], None),
    (1, 10, 48, 24, 64, "fp8", 0, [513], None),
    (35, 2, 32, 16, 128, "bf16", 16, list(range(0, 350, 10)), None),
]


@pytest.mark.parametrize("c", HEADS, ids=lambda c: "-".join(map(str, c[:7])))
def test_many_key_heads(c):
    """More key heads than a group of CTAs takes side by side: several blocks of heads per request."""
    x = Case(*c, seed=25)
    op = x.op()
    out = op()
    assert op.status() == 0
    check(x, out, True)


@pytest.mark.parametrize("cache,page", [("bf16", 0), ("bf16", 64), ("fp8", 64)])
@pytest.mark.parametrize("N,H,Hkv", [(1, 32, 32), (30, 48, 12), (7, 64, 16)])
def test_many_key_heads_in_long_ragged_batches(N, H, Hkv, cache, page):
    """The same, cut into many pieces: tensor cores against the CUDA cores.  Both round the output
    (2^-8 each); the weights' rounding, 2^-8, meets A = attention over |v|."""
    rng = np.random.default_rng([26, N, H])
    B = 7
    prefix, n = rng.integers(1, 4000, size=B), rng.integers(0, N + 1, size=B)
    n[0] = N
    x = Case(B, N, H, Hkv, 128, cache, page, prefix, n, seed=27, sharp=2.0, fill=float("nan"))
    got, want = x.op(), x.op(SIMT)
    g, w = got().float(), want().float()
    assert got.status() == 0 and want.status() == 0
    if cache == "fp8":
        x.kv[1] &= 0x7F
    else:
        x.kv[1].abs_()
    a = x.op(SIMT)().float()
    assert torch.isfinite(g).all() and torch.isfinite(w).all()
    tol = 2.0 ** -8 * (w.abs() * 2 + a * (1 + 2.0 ** -7)) + 2.0 ** -10 * a
    assert ((g - w).abs() <= tol).all(), ((g - w).abs() / tol).max()


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("kv_scale", [0.07, 2.0 ** -5])
def test_a_cache_written_with_one_scale(kv_scale, flags):
    """Per-head rows written without scale bytes: bytes of 127, the softmax scale and the result times
    kv_scale.  (fp32 products with kv_scale: 2^-24 more of a value, a key and the result each.)"""
    B, N, H, Hkv, d, T = 2, 6, 8, 2, 64, 200
    rng = np.random.default_rng(28)
    rows = [torch.from_numpy(rng.standard_normal((B, T, Hkv, d), dtype=np.float32)).cuda() for _ in range(2)]
    K, V = (torch.zeros((B, T, Hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    st = kdtv.kv_append([kdtv.KvPart(c, src=x) for c, x in zip((K, V), rows)], None, kv_scale=kv_scale)
    back = [torch.zeros_like(x) for x in rows]
    st2 = kdtv.kv_read([kdtv.KvPart(c, out=x) for c, x in zip((K, V), back)], kv_scale=kv_scale)
    assert int(st.item()) == int(st2.item()) == 0
    x = Case(B, N, H, Hkv, d, "fp8", 0, [T - N, 31], seed=29)
    one = torch.full((B, T, Hkv), 127, dtype=torch.uint8, device="cuda")
    out, status = kdtv.gqa_verify_attn(x.q, K, V, torch.from_numpy(x.parent).cuda(), torch.from_numpy(x.prefix).cuda(),
                                       k_scale=one, v_scale=one, scale=d ** -0.5 * kv_scale, flags=flags)
    assert int(status.item()) == 0
    x.gathered = lambda: [t.cpu().double().numpy() for t in back]
    check(x, out.float() * kv_scale, flags == 0)
