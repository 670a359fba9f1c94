"""GQA tree attention against the fp64 oracle.

Tolerance, fixed before the first run.  With delta = (d + 4) * 2^-24 * scale *
max_t sum_e |q_e k_te| bounding a score's fp32 error, the weights are off by a
factor of at most 1 + 2 delta + 2^-20 (the base-2 exponential and the sums),
and on tensor cores each weight is rounded to bf16 (2^-8) before it meets its
value.  With one-byte keys the tensor cores take a query row, scaled by a
power of two so that its largest element is at least 2^7, as two E4M3 parts:
an element's error is at most 2^-10 there (half of E4M3's smallest step), so
2^-17 of the row's largest, and delta grows by scale * 2^-17 * max|q| *
max_t sum_e |k_te|.  Against the oracle's A = sum_t p_t |v_t| this gives (2 delta + 2^-20
[+ 2^-8]) * A + T 2^-24 A for the sum, and the output's rounding, 2^-8 |o|
(bf16) or 2^-24 |o|.
"""


import numpy as np
import pytest
import torch

from oracle import rope_kv as O
from speculative_decoding_tree_mla_gb300 import kdtv, workloads as W

pytestmark = pytest.mark.gpu
SIMT = kdtv.KDTV_FLAG_SIMT


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Case:
    """Tensors of one call, and the gathered float64 rows for the oracle."""

    def __init__(self, B, N, H, Hkv, d, cache, page, prefix, n_nodes=None, seed=0, sharp=1.0, t_extra=5,
                 tree=(8, 8), fill=None):
        rng = np.random.default_rng([seed, B, N, H, d, page])
        self.B, self.N, self.H, self.Hkv, self.d, self.page, self.cache = B, N, H, Hkv, d, page, cache
        self.prefix = np.array(prefix, np.int32)
        self.n = np.full(B, N, np.int32) if n_nodes is None else np.array(n_nodes, np.int32)
        self.parent = np.stack([W.random_tree(rng, N, *tree) for _ in range(B)])
        for b in range(B):                            # what tree_build leaves behind the last node
            self.parent[b, self.n[b]:] = -1
        dt = torch.float32 if cache == "f32" else torch.bfloat16
        self.q = (dev(rng.standard_normal((B, N, H, d), dtype=np.float32)) * sharp).to(dt)
        T = int((self.prefix + self.n).max()) + t_extra
        if page:
            per = -(-T // page)
            num = B * per + 2
            self.table = rng.permutation(num)[:B * per].reshape(B, per).astype(np.int32)
            shape = (num, page, Hkv, d)
            self.T = per * page
        else:
            self.table, shape, self.T = None, (B, T, Hkv, d), T
        self.kv, self.scales = [], []
        for _ in range(2):
            x = dev(rng.standard_normal(shape, dtype=np.float32))
            if cache == "fp8":
                self.kv.append((x * 100.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
                self.scales.append(dev(rng.integers(119, 122, size=shape[:3]).astype(np.uint8)))
            else:
                self.kv.append(x.to(dt))
                self.scales.append(None)
        if fill is not None:                          # everything no node may see
            used = torch.zeros(shape[0] * shape[1], dtype=torch.bool)
            for b in range(B):
                used[self.rows(b, int(self.prefix[b] + self.n[b]))] = True
            for x in self.kv:
                flat = x.view(-1, Hkv * d)
                flat[~used.cuda()] = 0x7F if cache == "fp8" else fill

    def rows(self, b, count):
        t = np.arange(count)
        r = b * self.T + t if not self.page else self.table[b, t // self.page].astype(np.int64) * self.page + t % self.page
        return torch.from_numpy(np.asarray(r, np.int64))

    def op(self, flags=0, **kw):
        kw.setdefault("out", torch.full_like(self.q, 9.0))
        return kdtv.GqaVerifyAttn(self.q, *self.kv, dev(self.parent), dev(self.prefix), n_nodes=dev(self.n),
                                  page_table=None if self.table is None else dev(self.table),
                                  k_scale=self.scales[0], v_scale=self.scales[1], flags=flags, **kw)

    def gathered(self):
        out = []
        for x, s in zip(self.kv, self.scales):
            T = int((self.prefix + self.n).max())
            g = np.zeros((self.B, max(T, 1), self.Hkv, self.d))
            for b in range(self.B):
                c = int(self.prefix[b] + self.n[b])
                r = self.rows(b, c)
                v = x.reshape(-1, self.Hkv, self.d)[r.cuda()]
                if self.cache == "fp8":
                    v = W.fp8_e4m3_decode(v.cpu().numpy()).astype(np.float64)
                    v = v * 2.0 ** (s.reshape(-1, self.Hkv)[r.cuda()].cpu().numpy().astype(np.float64) - 127)[..., None]
                else:
                    v = v.float().cpu().double().numpy()
                g[b, :c] = v
            out.append(g)
        return out

    def check(self, out, tensor_cores, scale=None, rows=None):
        scale = scale or self.d ** -0.5
        k, v = self.gathered()
        q = self.q.float().cpu().double().numpy()
        want = O.gqa_attn(q, k, v, self.parent, self.prefix, scale, self.n)
        A = O.gqa_attn(q, k, np.abs(v), self.parent, self.prefix, scale, self.n)
        G = self.H // self.Hkv
        got = out.float().cpu().double().numpy()
        half = 2.0 ** -24 if self.cache == "f32" else 2.0 ** -8
        T = k.shape[1]
        for b in range(self.B):
            n = int(self.n[b])
            assert (got[b, n:] == 9.0).all()
            # finite keys only: a row that sees another has NaN for its weights, and the scores of
            # a row that does not are made of finite keys alone
            kk = np.repeat(np.where(np.isfinite(k[b]), np.abs(k[b]), 0.0).max(0), G, axis=0)   # [H, d]
            delta = (self.d + 4) * 2.0 ** -24 * scale * (np.abs(q[b, :n]) * kk).sum(-1)[..., None]
            if tensor_cores and self.cache == "fp8":
                delta = delta + scale * 2.0 ** -17 * np.abs(q[b, :n]).max(-1, keepdims=True) * kk.sum(-1)[:, None]
            rel = 2 * delta + 2.0 ** -20 + T * 2.0 ** -24 + (2.0 ** -8 if tensor_cores else 0.0)
            for i in range(n) if rows is None else rows(b):
                w, g, a = want[b, i], got[b, i], A[b, i]
                fin = np.isfinite(w)
                assert (np.isnan(g) == np.isnan(w)).all() and (g[np.isinf(w)] == w[np.isinf(w)]).all()
                err, tol = np.abs(g - w)[fin], (rel[i] * a + half * np.abs(w))[fin]
                assert (err <= tol).all(), (b, i, (err / tol).max())


CASES = [
    # B, N, H, Hkv, d, cache, page, prefix, n_nodes
    (1, 1, 1, 1, 64, "bf16", 0, [0], None),                       # one node, no prefix
    (1, 1, 8, 2, 128, "bf16", 64, [700], None),                   # single-token decode
    (2, 3, 4, 4, 128, "bf16", 16, [1, 126], None),                # one query head per key head
    (2, 13, 14, 2, 64, "bf16", 0, [129, 255], [13, 5]),           # G = 7: 126 rows a tile
    (3, 16, 16, 2, 128, "bf16", 64, [0, 64, 300], [16, 1, 0]),    # 128 rows; a request without nodes
    (1, 17, 16, 2, 128, "bf16", 128, [113], None),                # 136 rows: a second tile with 8
    (2, 33, 32, 4, 128, "bf16", 32, [511, 40], [33, 32]),         # 264 and 256 rows
    (1, 128, 8, 1, 64, "bf16", 0, [640], None),                   # 1024 rows
    (1, 128, 2, 2, 128, "bf16", 0, [1], None),                    # tree longer than the prefix
    (1, 2, 128, 1, 128, "bf16", 64, [257], None),                 # G = 128
    (1, 2, 130, 1, 64, "bf16", 64, [57], None),                   # G = 130: CUDA cores
    (2, 5, 6, 3, 128, "bf16", 24, [100, 3], None),                # page of 24 rows: CUDA cores
    (2, 5, 6, 2, 80, "bf16", 0, [100, 31], None),                 # head dim 80: CUDA cores
    (1, 4, 2, 1, 256, "bf16", 16, [65], None),
    (1, 1, 8, 2, 128, "fp8", 64, [700], None),
    (2, 16, 16, 2, 128, "fp8", 0, [1, 384], [16, 9]),
    (2, 40, 8, 1, 64, "fp8", 16, [200, 333], [40, 3]),
    (1, 70, 16, 2, 128, "fp8", 64, [250], None),
    (3, 9, 9, 3, 100, "fp8", 7, [20, 50, 0], [9, 0, 4]),
    (2, 7, 4, 2, 64, "f32", 0, [90, 33], [7, 2]),
    (1, 1, 4, 1, 128, "f32", 64, [1000], None),
    (2, 12, 6, 2, 33, "f32", 5, [47, 0], None),
]


def tc(c, flags):
    return c[5] != "f32" and not flags and c[4] in (64, 128) and c[2] // c[3] <= 128 and c[6] in (0, 16, 32, 64, 128)


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(map(str, c[:7])))
def test_against_oracle(c, flags):
    x = Case(*c)
    op = x.op(flags)
    out = op()
    assert op.status() == 0
    x.check(out, tc(c, flags))


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("cache", ["bf16", "fp8", "f32"])
def test_unseen_rows_may_hold_anything(cache, flags):
    """NaN in every row behind the tree, on pages of nobody and in the rest of the last page; sharp
    and flat softmaxes; a given scale."""
    for fill in (float("nan"), float("inf"), -3.0e38):
        for page in (0, 16):
            c = (2, 11, 8, 2, 64, cache, page, [117, 130], [11, 4])
            x = Case(*c, seed=3, sharp=8.0, fill=fill)
            op = x.op(flags, scale=0.3)
            x.check(op(), tc(c, flags), scale=0.3)
            assert op.status() == 0


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("cache,page", [("bf16", 0), ("bf16", 64), ("fp8", 16), ("f32", 0)])
def test_masked_nodes_with_infinities(cache, page, flags):
    """A node whose own key or value is not finite reaches itself and its descendants alone."""
    for B, N, H, Hkv, prefix in ((1, 20, 8, 1, [119]), (2, 50, 16, 2, [5, 250])):
        c = (B, N, H, Hkv, 128, cache, page, prefix, None)
        x = Case(*c, seed=4)
        bad = {3: (1, 0x7F, float("nan")), 7: (1, 0xFF, float("inf")), 9: (1, 0x7F, float("-inf")),
               12: (0, 0x7F, float("nan")), 15: (0, 0xFF, float("-inf"))}
        for b in range(B):
            for node, (which, code, value) in bad.items():
                row = int(x.rows(b, int(x.prefix[b]) + node + 1)[-1])
                flat = x.kv[which].view(-1, Hkv, 128)
                flat[row, 0, 5:40 + node] = code if cache == "fp8" else value
        op = x.op(flags)
        x.check(op(), tc(c, flags))
        assert op.status() == 0


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
def test_infinite_prefix(flags):
    """A value in the prefix that every node sees: the output's element is infinite or NaN."""
    c = (1, 6, 8, 2, 64, "bf16", 0, [300], None)
    x = Case(*c, seed=5)
    x.kv[1][0, 7, 0, 3] = float("inf")
    x.kv[1][0, 200, 1, 9] = float("nan")
    op = x.op(flags)
    x.check(op(), tc(c, flags))


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
def test_malformed_trees_leave_their_rows(flags):
    """Rows whose root path is malformed stay as they were; the others are right; the code is recorded."""
    c = (2, 12, 16, 2, 128, "bf16", 64, [200, 90], None)
    x = Case(*c, seed=6, tree=(1, 3))
    x.parent[0] = W.chain_tree(12)
    x.parent[0, 6] = 9                       # not before its child: 6 and what hangs from it
    x.parent[1] = W.star_tree(12)
    x.parent[1, 4] = -1                      # a second root
    op = x.op(flags)
    out = op()
    assert op.status() == kdtv.STATUS_CODE["KDTV_ERR_BAD_TREE"] and op.status() == 0
    good = [list(range(6)), [i for i in range(12) if i != 4]]
    for b in range(2):
        for i in range(12):
            if i not in good[b]:
                assert (out[b, i] == 9.0).all()
                x.parent[b, i] = 0           # the oracle walks every node
    x.check(out, tc(c, flags), rows=lambda b: good[b])
    x.parent[:, 0] = 3
    op = x.op(flags)
    assert (op() == 9.0).all() and op.status() == kdtv.STATUS_CODE["KDTV_ERR_BAD_TREE"]


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("page", [0, 16])
def test_bad_prefix_and_pages(flags, page):
    c = (3, 5, 8, 2, 64, "bf16", page, [200, 140, 3], None)
    x = Case(*c, seed=7)
    kinds = [("KDTV_ERR_BAD_PREFIX", -1, None), ("KDTV_ERR_BAD_PREFIX", x.T - 4, None),
             ("KDTV_ERR_BAD_PREFIX", (1 << 31) - 1, None)]
    if page:
        kinds += [("KDTV_ERR_BAD_PAGE", None, -1), ("KDTV_ERR_BAD_PAGE", None, 1 << 30)]
    for code, L, pg in kinds:
        prefix, table = x.prefix.copy(), None if x.table is None else x.table.copy()
        if L is not None:
            x.prefix[1] = L
        else:
            x.table[1, 8] = pg
        op = x.op(flags)
        out = op()
        assert op.status() == kdtv.STATUS_CODE[code]
        assert (out[1] == 9.0).all()
        x.prefix, x.table = prefix, table
        x.n[1] = 0                           # the oracle skips it
        x.check(out, tc(c, flags))
        x.n[1] = 5


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_long_cache(cache):
    """Offsets past 2^31 elements: the keys of a far request, and a prefix in many pieces."""
    B, T, Hkv, d = 3, 1 << 20, 8, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    dt = torch.uint8 if cache == "fp8" else torch.bfloat16
    k, v = (torch.zeros((B, T, Hkv, d), dtype=dt, device="cuda") for _ in range(2))
    sc = [torch.full((B, T, Hkv), 127, dtype=torch.uint8, device="cuda") for _ in range(2)] if cache == "fp8" else [None] * 2
    L = T - 3
    one = 0x38 if cache == "fp8" else 1.0               # E4M3 1.0
    v[2, L:] = one                                      # the three nodes' values
    k[2, 12345] = one
    v[2, 12345] = one
    q = torch.ones((B, 3, 16, d), dtype=torch.bfloat16, device="cuda")
    parent = torch.tensor([[-1, 0, 1]] * B, dtype=torch.int32, device="cuda")
    prefix = torch.tensor([5, 0, L], dtype=torch.int32, device="cuda")
    op = kdtv.GqaVerifyAttn(q, k, v, parent, prefix, k_scale=sc[0], v_scale=sc[1], scale=0.125)
    out = op()
    assert op.status() == 0
    w = np.exp(16.0)                                    # the marked key scores 128 / 8, the others 0
    for i in range(3):
        want = (w + i + 1) / (w + L - 1 + i + 1)
        assert abs(out[2, i].float() - want).max().item() <= 2.0 ** -7 * want
    assert (out[:2] == 0).all()


LONG = [
    # many key tiles a CTA, several pieces, requests with one and with two row tiles side by side
    (8, 32, 64, 8, 128, "bf16", 0, (300, 6000), (1, 32)),
    (8, 32, 64, 8, 128, "fp8", 64, (300, 6000), (1, 32)),
    (24, 8, 64, 8, 128, "bf16", 64, (1, 5000), (0, 8)),
    (24, 8, 64, 8, 64, "fp8", 16, (1, 5000), (0, 8)),
    (5, 60, 32, 8, 64, "bf16", 32, (100, 9000), (20, 60)),
    (40, 1, 32, 8, 128, "bf16", 64, (1, 9000), (1, 1)),
    (40, 1, 32, 8, 128, "fp8", 0, (1, 9000), (1, 1)),
    (1, 128, 64, 8, 128, "bf16", 64, (17000, 17000), (128, 128)),
    (1, 100, 28, 4, 128, "fp8", 64, (30000, 30000), (100, 100)),
]


@pytest.mark.parametrize("c", LONG, ids=lambda c: "-".join(map(str, c[:7])))
@pytest.mark.parametrize("seed", [0, 1])
def test_long_ragged_batches(c, seed):
    """Tensor cores against the CUDA cores (which the cases above hold to the oracle), NaN in every
    row that no node may see.  Both round the output (2^-8 each); the weights' rounding to bf16,
    2^-8, meets values of A = attention over |v|, which the CUDA cores give as well."""
    rng = np.random.default_rng([9, seed, c[0], c[1]])
    B, N = c[0], c[1]
    prefix = rng.integers(c[7][0], c[7][1] + 1, size=B)
    n = rng.integers(c[8][0], c[8][1] + 1, size=B)
    x = Case(*c[:7], prefix, n, seed=seed, sharp=2.0, fill=float("nan"))
    got, want = x.op(), x.op(SIMT)
    g, w = got().float(), want().float()
    assert got.status() == 0 and want.status() == 0
    if c[5] == "fp8":
        x.kv[1] &= 0x7F
    else:
        x.kv[1].abs_()
    a = x.op(SIMT)().float()
    assert torch.isfinite(g).all() and torch.isfinite(w).all()
    tol = 2.0 ** -8 * (w.abs() * 2 + a * (1 + 2.0 ** -7)) + 2.0 ** -10 * a
    if c[5] == "fp8":                 # the queries' two parts: 2 delta, scores of 448 * 2^-6 at most
        k = 448.0 * 2.0 ** -6 * x.d * x.d ** -0.5
        tol = tol + 2 * 2.0 ** -17 * x.q.float().abs().amax(-1, keepdim=True) * k * a
    assert ((g - w).abs() <= tol).all(), ((g - w).abs() / tol).max()


@pytest.mark.parametrize("c", [CASES[1], CASES[6], CASES[15], CASES[17]], ids=["one", "tree", "fp8", "fp8tree"])
def test_graph_streams_and_repeats(c):
    """Bitwise the same on repeats, from a captured graph with new inputs in the same buffers, on
    another stream, and from two objects at work at the same time."""
    x = Case(*c, seed=8)
    op, op2 = x.op(), x.op()
    first = op().clone()
    for _ in range(20):
        assert torch.equal(op(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op2(side)
    op()
    side.synchronize()
    assert torch.equal(op2.out, first) and torch.equal(op.out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op()
    x.q.copy_(torch.randn_like(x.q.float()).to(x.q.dtype))
    graph.replay()
    got = op.out.clone()
    assert not torch.equal(got, first)
    x.check(got, tc(c, 0))
    assert torch.equal(op2(), got)
    assert op.status() == 0 and op2.status() == 0


def test_function_form_and_checks():
    x = Case(1, 4, 8, 2, 64, "bf16", 0, [40])
    pa, pl = dev(x.parent), dev(x.prefix)
    out, status = kdtv.gqa_verify_attn(x.q, *x.kv, pa, pl)
    x.check(out, True)
    assert int(status.item()) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, _ = kdtv.gqa_verify_attn(x.q, *x.kv, pa, pl, stream=side)
    side.synchronize()
    assert torch.equal(out, out2)
    k, v = x.kv
    for args, kw in (((x.q.half(), k, v, pa, pl), {}), ((x.q, k, v[:, 1:], pa, pl), {}),
                     ((x.q, k.float(), v.float(), pa, pl), {}), ((x.q, k, v, pa.long(), pl), {}),
                     ((x.q, k, v, pa, None), {}), ((x.q[:, :, :7], k, v, pa, pl), {}),
                     ((x.q, k, v, pa, pl), dict(k_scale=k)), ((x.q, k, v, pa, pl), dict(out=x.q.float())),
                     ((x.q, k.view(torch.uint8)[..., :64].contiguous(), v.view(torch.uint8)[..., :64].contiguous(), pa, pl), {}),
                     ((x.q, k.cpu(), v.cpu(), pa, pl), {}), ((x.q, k, v, pa, pl), dict(page_table=pl))):
        with pytest.raises(ValueError):
            kdtv.gqa_verify_attn(*args, **kw)
    with pytest.raises(kdtv.KdtvError):
        kdtv.gqa_verify_attn(torch.zeros((1, 129, 8, 64), dtype=torch.bfloat16, device="cuda"), k, v,
                             torch.zeros((1, 129), dtype=torch.int32, device="cuda"), pl)


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("fp8", 128), ("fp8", 64)])
def test_a_wait_that_runs_out(cache, d):
    """The loads never start (a test flag; every wait has a limit): the status says so, and the next
    call is as if nothing had been."""
    x = Case(2, 9, 8, 2, d, cache, 16, [300, 20], seed=4)
    stalled, op = x.op(kdtv.KDTV_FLAG_TEST_STALL), x.op()
    stalled()
    assert kdtv.STATUS[stalled.status()] == "KDTV_ERR_DEVICE_TIMEOUT"
    assert stalled.status() == 0
    x.check(op(), True)
    assert op.status() == 0


def test_bound_on_one_stream_called_on_another():
    """The words and results that a caller allocates are cleared on the stream it was bound on; its
    first call elsewhere waits for that."""
    x = Case(2, 4, 8, 2, 64, "bf16", 0, [40, 7], seed=5)
    x.prefix[1] = -3                       # an error to be kept
    big = torch.empty(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        for _ in range(8):
            big.zero_()                    # the clearing of the status word lies behind these
        op = x.op()
        op(side)
        assert kdtv.STATUS[op.status()] == "KDTV_ERR_BAD_PREFIX"


def test_extreme_exponents():
    """Key and value scales from the smallest to 2^90, queries tiny and huge beside them: fp32
    attention and tensor cores agree with the oracle."""
    x = Case(1, 3, 4, 2, 64, "fp8", 0, [150], seed=6)
    for byte, q_scale in ((1, 2.0 ** 100), (40, 2.0 ** 60), (217, 2.0 ** -100)):
        x.scales[0].fill_(byte)
        x.scales[1].fill_(240 - byte)
        x.q.copy_((torch.randn(x.q.shape, device="cuda") * q_scale).to(x.q.dtype))
        for flags in (0, SIMT):
            op = x.op(flags)
            x.check(op(), flags == 0)
            assert op.status() == 0


@pytest.mark.parametrize("flags", [0, SIMT], ids=["auto", "simt"])
@pytest.mark.parametrize("d,page", [(128, 0), (64, 16)])
def test_every_code_and_scale(d, page, flags):
    """One node and nothing before it: its output is its own value row, every code at scales from
    2^-126 to 2^119 (exactly; below 2^-117 a code may not be exact in bf16), NaN included."""
    bytes_ = [1, 5, 10, 64, 120, 127, 133, 134, 135, 200, 246]
    Hkv = 256 // d
    x = Case(len(bytes_), 1, Hkv, Hkv, d, "fp8", page, [0] * len(bytes_), seed=7)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(Hkv, d)
    for b, byte in enumerate(bytes_):
        r = x.rows(b, 1).cuda()
        x.kv[1].view(-1, Hkv, d)[r] = codes
        x.scales[1].view(-1, Hkv)[r] = byte
    op = x.op(flags)
    got = op().float().cpu().double().numpy()
    assert op.status() == 0
    value = W.fp8_e4m3_decode(codes.cpu().numpy()).astype(np.float64)
    for b, byte in enumerate(bytes_):
        want = value * 2.0 ** (byte - 127)
        fin = np.isfinite(want)
        assert (np.isnan(got[b, 0]) == ~fin).all()
        assert (np.abs(got[b, 0] - want)[fin] <= (2.0 ** -134 if byte < 10 else 0.0)).all()


@pytest.mark.parametrize("cache,page", [("bf16", 0), ("fp8", 16)])
def test_many_requests_some_of_them_bad(cache, page):
    """More requests than a warp has lanes, some empty, some with a prefix that does not fit, one whose
    last nodes have no parent (31): those rows stay, all others are right."""
    rng = np.random.default_rng(10)
    B = 70
    prefix, n = rng.integers(0, 700, size=B), rng.integers(0, 6, size=B)
    x = Case(B, 5, 8, 2, 128, cache, page, prefix, n, seed=11)
    x.n[[33, 50]] = 0
    x.n[[31, 32, 69]] = 5
    good, known = x.prefix.copy(), n.copy()
    x.prefix[[32, 69]] = [-1, 1 << 20]
    got, want = x.op(), x.op(SIMT)
    g, w = got().float(), want().float()
    first = ("KDTV_ERR_BAD_PREFIX", "KDTV_ERR_BAD_TREE")
    assert kdtv.STATUS[got.status()] in first and kdtv.STATUS[want.status()] in first
    for out in (g, w):
        assert (out[[32, 33, 50, 69]] == 9.0).all() and (out[31, max(known[31], 1):] == 9.0).all()
    x.prefix, x.n[[32, 69]] = good, 0

    def whole(b):                             # nodes with a root path
        return range(min(int(x.n[b]), max(int(known[b]), 1)) if b == 31 else int(x.n[b]))

    x.parent[31, max(known[31], 1):] = 0      # (for the oracle, whose rows there are not looked at)
    x.check(got.out, True, rows=whole)
    x.check(want.out, False, rows=whole)
