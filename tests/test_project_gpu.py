"""kdtv_project against the fp64 oracle.

Tolerances.  With T the sum of the magnitudes of a sum's terms: CUDA cores, fp32: chains of 128 products,
their totals (at most d_in / 128 + 8 of them) and the adapter's R terms, each addition off by 2^-24 of at
most T, and the products' own rounding: (140 + d_in / 128 + R) 2^-24 T.  (The inner product A x has the same
chains, 16 to a lane and the lanes' totals.)  Tensor cores: products are exact, and each of at most (d_in + 2
R) additions may lose 2^-23 of T (truncated, not rounded); A x enters as two bf16 parts, 2^-16 of it.  Then
half a step of the output type, 2^-8 for bf16, relative to the value.  Whole-number cases, where every sum
is exact, are equal bit for bit."""

import numpy as np
import pytest

from oracle import serve_ops as O
from speculative_decoding_tree_mla_gb300 import kdtv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SIMT = kdtv.KDTV_FLAG_SIMT
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}


def f64(t):
    return t.float().cpu().double().numpy()


class Case:
    def __init__(self, B, N, K, M, dtype, adapters=0, rank=16, seed=0, whole=False, ids=None, n_live=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt = TYPE[dtype]

        def values(*shape, std=1.0):
            if whole:
                return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dt)
            return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

        self.B, self.N, self.K, self.M, self.dtype, self.rank = B, N, K, M, dtype, rank
        self.x, self.W = values(B, N, K), values(M, K, std=K ** -0.5)
        self.kw = {}
        if dtype == "fp8":
            self.W, ws = kdtv.quantise_weight(self.W)
            self.x, xs = kdtv.rmsnorm(self.x, one_byte=True) if not whole else self._codes(self.x)
            self.kw.update(x_scale=xs, W_scale=ws)
            self.x64 = O.widen(self.x.cpu().numpy(), xs.cpu().numpy())
            self.W64 = O.widen(self.W.cpu().numpy(), ws.cpu().numpy())
        else:
            self.x64, self.W64 = f64(self.x), f64(self.W)
        self.o = {}
        if adapters:
            A, Bm = values(adapters, rank, K, std=K ** -0.5), values(adapters, M, rank, std=0.5)
            s = torch.tensor([0.5, 1.0, 2.0, -1.0], device="cuda")[torch.arange(adapters, device="cuda") % 4]
            self.ids = np.asarray(ids if ids is not None else rng.integers(-1, adapters, B), dtype=np.int32)
            self.kw.update(A=A, Bm=Bm, adapter_scale=s, adapter=torch.tensor(self.ids, device="cuda"))
            self.o = dict(A=f64(A), Bm=f64(Bm), adapter=self.ids, adapter_scale=f64(s))
        self.n = np.full(B, N) if n_live is None else np.asarray(n_live)
        if n_live is not None:
            self.kw["n_live"] = torch.tensor(self.n, dtype=torch.int32, device="cuda")

    @staticmethod
    def _codes(x):
        B, N, K = x.shape
        c, s = kdtv.quantise_weight(x.reshape(B * N, K))
        return c.view(B, N, K), s.view(B, N, K // 32)

    def oracle(self):
        return O.project(self.x64, self.W64, **self.o)

    def check(self, out, flags=0, exact=False, before=7.0):
        y, mag = self.oracle()
        got = f64(out)
        for b in range(self.B):
            m = min(max(int(self.n[b]), 0), self.N)
            assert (got[b, m:] == before).all(), (b, "rows that are not live")
            if exact:
                want = f64(torch.tensor(y[b, :m]).to(TYPE[self.dtype]))
                assert np.array_equal(got[b, :m], want), (b, np.abs(got[b, :m] - want).max())
                continue
            R = self.rank if self.o else 0
            if self.dtype == "f32" or flags & SIMT:
                tol = (140 + self.K / 128 + R) * 2.0 ** -24
            else:
                tol = (self.K + 2 * R) * 2.0 ** -23 + (2.0 ** -16 if R else 0.0)
            step = 2.0 ** -24 if self.dtype == "f32" else 2.0 ** -8
            err = np.abs(got[b, :m] - y[b, :m])
            lim = tol * mag[b, :m] + step * np.abs(y[b, :m])
            assert (err <= lim).all(), (b, float((err / lim).max()), np.argwhere(err > lim)[:4])

    def run(self, flags=0, **kw):
        out = torch.full((self.B, self.N, self.M), 7.0, dtype=TYPE[self.dtype], device="cuda")
        got, st = kdtv.project(self.x, self.W, flags=flags, out=out, **self.kw, **kw)
        assert int(st) == 0
        return got


PATHS = [("f32", 0), ("bf16", 0), ("bf16", SIMT), ("fp8", 0), ("fp8", SIMT)]


@pytest.mark.parametrize("dtype,flags", PATHS)
@pytest.mark.parametrize("B,N,K,M,adapters,rank", [
    (1, 1, 32, 1, 0, 0), (1, 1, 64, 128, 1, 16), (3, 13, 96, 130, 2, 8), (1, 1, 2048, 640, 3, 16), (64, 1, 256, 384, 40, 16),
    (5, 33, 192, 100, 3, 24), (2, 300, 320, 256, 2, 64), (300, 1, 128, 200, 100, 8), (4, 128, 512, 1000, 4, 32),
    (1, 700, 224, 129, 1, 128), (17, 8, 1024, 72, 5, 40), (2, 129, 64, 64, 2, 16), (9, 100, 160, 257, 3, 256)])
def test_matches_oracle(dtype, flags, B, N, K, M, adapters, rank):
    c = Case(B, N, K, M, dtype, adapters, rank, seed=B + N)
    c.check(c.run(flags), flags)


@pytest.mark.parametrize("dtype,flags", PATHS)
@pytest.mark.parametrize("B,N,K,M,adapters,rank", [
    (1, 1, 64, 3, 1, 8), (64, 1, 64, 300, 20, 8), (7, 9, 96, 130, 3, 16), (2, 257, 128, 140, 2, 24), (33, 8, 160, 64, 33, 16),
    (3, 1030, 64, 260, 3, 8), (260, 1, 32, 40, 260, 8)])
def test_whole_numbers_are_exact(dtype, flags, B, N, K, M, adapters, rank):
    """Entries of -2 .. 2: every sum is a whole number below 2^24 (A x, up to 4 K, splits into two bf16 parts
    exactly), so each output is the correctly rounded sum, element by element."""
    c = Case(B, N, K, M, dtype, adapters, rank, seed=1, whole=True)
    c.check(c.run(flags), flags, exact=True)


@pytest.mark.parametrize("dtype,flags", PATHS)
@pytest.mark.parametrize("B,N,K,M", [(6, 20, 128, 96), (5, 300, 64, 130), (70, 5, 64, 64), (3, 2000, 64, 40)])
def test_ragged_rows(dtype, flags, B, N, K, M):
    rng = np.random.default_rng(5)
    n = rng.integers(0, N + 1, B)
    n[0], n[1], n[-1] = 0, N, N + 5 if B > 4 else 1
    c = Case(B, N, K, M, dtype, 3, 16, seed=2, whole=True, n_live=n)
    if dtype != "fp8":
        for b in range(B):
            c.x[b, max(0, int(n[b])):] = float("nan")          # rows that do not count may hold anything
            c.x64[b, max(0, int(n[b])):] = 0.0
    c.check(c.run(flags), flags, exact=True)
    n[:] = 0
    c.kw["n_live"].zero_()
    c.check(c.run(flags), flags, exact=True)


@pytest.mark.parametrize("B,N,K,M", [(3, 5, 96, 70), (2, 40, 160, 130), (1, 200, 1056, 300), (5, 1, 2080, 260), (2, 70, 416, 64),
                                     (1, 300, 2784, 100), (7, 3, 32, 9), (1, 1, 8160, 520)])
@pytest.mark.parametrize("flags", [0, SIMT])
def test_one_byte_exponents_at_any_address(flags, B, N, K, M):
    """d_in whose rows of exponent bytes (K / 32 of them) start off 4 and 16 bytes; the bytes behind the
    last group, which belong to other rows, are NaN's there and count for nothing."""
    c = Case(B, N, K, M, "fp8", 2, 16, seed=K)
    c.check(c.run(flags), flags)
    for name in ("x_scale", "W_scale"):                        # the same bytes at an odd address
        s = c.kw[name]
        wide = torch.full((s.numel() + 7,), 255, dtype=torch.uint8, device="cuda")
        wide[3:3 + s.numel()] = s.flatten()
        c.kw[name] = wide[3:3 + s.numel()].view(s.shape)
    c.check(c.run(flags), flags)


@pytest.mark.parametrize("B,N,K,M,adapters", [(9, 1, 5649, 256, 2), (25, 20, 1592, 1152, 7), (1, 1, 4096, 4100, 1), (40, 10, 777, 640, 3),
                                              (2, 300, 4099, 130, 2), (1, 16, 8191, 33, 1)])
def test_fp32_shares_d_in_between_ctas(B, N, K, M, adapters):
    c = Case(B, N, K, M, "f32", adapters, 5, seed=K)
    out = c.run()
    c.check(out)
    assert torch.equal(out, c.run())


@pytest.mark.parametrize("dtype,flags", [("f32", 0), ("bf16", SIMT), ("fp8", SIMT)])
@pytest.mark.parametrize("B,N,K,M,adapters", [(1, 1, 8192, 2100, 1), (1, 1, 32, 3, 0), (2, 1, 4128, 77, 2), (5, 3, 992, 70, 3),
                                              (16, 1, 4096, 33, 5), (2, 8, 64, 5000, 2), (9, 1, 544, 9, 3), (1, 16, 20000, 40, 1)])
def test_few_rows_on_cuda_cores(dtype, flags, B, N, K, M, adapters):
    """Weights streamed once per eight rows, one to eight warps along d_in; some of the rows not live; element by
    element where d_in or an address is odd."""
    n = np.random.default_rng(B + K).integers(0, N + 2, B)
    for live in (None, n):
        c = Case(B, N, K, M, dtype, adapters, 16, seed=K + M, n_live=live)
        c.check(c.run(flags), flags)
    if dtype != "fp8":
        c = Case(B, N, K + 3, M, dtype, adapters, 5, seed=K, whole=True)
        c.check(c.run(flags), flags, exact=True)


@pytest.mark.parametrize("B,N,K,M", [(60000, 1, 3, 2), (300, 200, 5, 1), (2, 3000, 1, 7), (700, 9, 40, 33)])
def test_many_small_rows_on_cuda_cores(B, N, K, M):
    c = Case(B, N, K, M, "f32", 4, 2, seed=B, whole=True)
    c.check(c.run(), exact=True)


@pytest.mark.parametrize("K,rank,dtype", [(7, 16, "bf16"), (100, 16, "bf16"), (64, 3, "bf16"), (33, 5, "f32"), (1, 1, "f32"),
                                          (64, 12, "fp8"), (1001, 5, "f32")])
def test_odd_sizes(K, rank, dtype):
    c = Case(3, 13, K, 51, dtype, 2, rank, seed=3)
    c.check(c.run(), SIMT)


@pytest.mark.parametrize("dtype,flags", [("f32", 0), ("bf16", 0), ("bf16", SIMT)])
@pytest.mark.parametrize("xpad,ypad,off", [(8, 0, 0), (0, 8, 0), (24, 3, 0), (3, 1, 0), (8, 8, 1), (64, 64, 8)])
def test_strided_rows(dtype, flags, xpad, ypad, off):
    """Rows that are parts of wider ones, at any alignment; what lies beside them stays."""
    c = Case(3, 50, 128, 72, dtype, 2, 16, seed=4, whole=True)
    wide = torch.zeros((3, 50, 128 + xpad + off), dtype=TYPE[dtype], device="cuda")
    wide[..., off:off + 128] = c.x
    c.x = wide[..., off:off + 128]
    out = torch.full((3, 50, 72 + ypad + off), 5.0, dtype=TYPE[dtype], device="cuda")
    got, st = kdtv.project(c.x, c.W, flags=flags, out=out[..., off:off + 72], **c.kw)
    assert int(st) == 0
    c.check(got.contiguous(), flags, exact=True)
    assert (out[..., :off] == 5.0).all() and (out[..., off + 72:] == 5.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("over", ["requests", "rows", "windows"])
def test_rows_that_share_memory(dtype, over):
    """One request's rows for all, one row for all of a request, and rows that overlap."""
    B, N, K = 5, 6, 64
    c = Case(B, N, K, 96, dtype, 3, 16, seed=8)
    if over == "windows":                     # row i of request b starts 8 elements behind the one before
        base = c.x.reshape(-1)[:8 * B * N + K]
        c.x = base.as_strided((B, N, K), (8 * N, 8, 1))
    else:
        c.x = c.x[:1].expand(B, N, K) if over == "requests" else c.x[:, :1].expand(B, N, K)
    c.x64 = f64(c.x)
    c.check(c.run(), flags=0 if over == "windows" else SIMT)          # (a stride of 0 runs on CUDA cores)


@pytest.mark.parametrize("dtype,flags", PATHS)
def test_permuted_requests(dtype, flags):
    """x [N, B, K] seen as [B, N, K], and requests in a buffer with gaps."""
    if dtype == "fp8":
        pytest.skip("one-byte rows are contiguous")
    c = Case(5, 12, 64, 64, dtype, 2, 16, seed=5, whole=True)
    c.x = c.x.transpose(0, 1).contiguous().transpose(0, 1)
    c.check(c.run(flags), flags, exact=True)


@pytest.mark.parametrize("dtype,flags", PATHS)
def test_adapters_keep_to_their_requests(dtype, flags):
    """Infinities and NaN in one adapter, or in one request's rows, reach no other request's output."""
    B, K, M = 40, 128, 200
    c = Case(B, 2, K, M, dtype, 5, 16, seed=6, whole=True, ids=np.arange(B) % 6 - 1)
    clean = f64(c.run(flags))
    for what in ("Bm", "A"):
        keep = c.kw[what].clone()
        c.kw[what][2, 3] = float("inf")
        c.kw[what][2, 7] = float("nan")
        c.kw[what][2, 9] = -float("inf")
        got = f64(c.run(flags))
        mine = c.ids == 2
        assert np.array_equal(got[~mine], clean[~mine])
        assert not np.isfinite(got[mine]).all()
        c.kw[what].copy_(keep)
    if dtype != "fp8":
        c.x[7, 1] = float("nan")
        got = f64(c.run(flags))
        assert np.isnan(got[7, 1]).all()
        got[7, 1] = clean[7, 1]
        assert np.array_equal(got, clean)


@pytest.mark.parametrize("dtype,flags", PATHS)
def test_adapter_index_out_of_range(dtype, flags):
    c = Case(9, 3, 64, 70, dtype, 2, 16, seed=7, whole=True, ids=[0, 1, -1, 2, 0, -2, 1, 2 ** 30, 0])
    out = torch.full((9, 3, 70), 7.0, dtype=TYPE[dtype], device="cuda")
    op = kdtv.Project(c.x, c.W, flags=flags, out=out, **c.kw)
    op()
    assert kdtv.STATUS[op.status()] == "KDTV_ERR_BAD_ADAPTER" and op.status() == 0
    c.n = np.where(np.isin(np.arange(9), (3, 5, 7)), 0, 3)
    c.o["adapter"] = np.where(c.n == 0, -1, c.ids)
    c.check(out, flags, exact=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_extreme_scales(dtype):
    """Sums far from 1, down to bf16's small values and up to its large ones, keep their relative error."""
    for e in (-60, 50):
        c = Case(2, 5, 128, 64, "bf16", 1, 16, seed=8, ids=[0, -1])
        if dtype == "fp8":
            c.dtype = "fp8"
            c.W, ws = kdtv.quantise_weight(c.W)
            c.x, xs = c._codes((c.x.float() * 2.0 ** e).to(torch.bfloat16))
            c.kw.update(x_scale=xs, W_scale=ws)
            c.x64, c.W64 = O.widen(c.x.cpu().numpy(), xs.cpu().numpy()), O.widen(c.W.cpu().numpy(), ws.cpu().numpy())
        else:
            c.x = (c.x.float() * 2.0 ** e).to(torch.bfloat16)
            c.x64 = f64(c.x)
        c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_deterministic_streams_and_capture(dtype):
    c = Case(24, 8, 1024, 520, dtype, 7, 16, seed=9)
    op = kdtv.Project(c.x, c.W, **c.kw)
    first = op().clone()
    for _ in range(20):
        assert torch.equal(op(), first)
    side = torch.cuda.Stream()
    op.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    op(side)
    side.synchronize()
    assert torch.equal(op.out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op()
    op.out.zero_()
    op.workspace.fill_(255)                                    # nothing in it outlives a call
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(op.out, first) and op.status() == 0
    ids = c.kw["adapter"]
    ids.copy_(ids.flip(0))
    c.ids = ids.cpu().numpy()
    c.o["adapter"] = c.ids
    g.replay()
    torch.cuda.synchronize()
    c.check(op.out, SIMT if dtype == "f32" else 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_wait_that_runs_out_is_reported(dtype):
    """A stalled pipeline ends within its limit, says so, and the next call works."""
    c = Case(6, 8, 512, 300, dtype, 3, 16, seed=11, whole=True)
    out = torch.full((6, 8, 300), 7.0, dtype=torch.bfloat16, device="cuda")
    op = kdtv.Project(c.x, c.W, flags=kdtv.KDTV_FLAG_TEST_STALL, out=out, **c.kw)
    op()
    assert kdtv.STATUS[op.status()] == "KDTV_ERR_DEVICE_TIMEOUT"
    assert (out == 7.0).all()
    c.check(c.run(), exact=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,N,K,M", [(1100, 130, 32, 24), (2500, 1, 2048, 40), (5, 64, 4096, 1280), (40, 1, 4096, 2560), (1, 1, 8192, 2000)])
def test_many_requests_and_cut_tiles(dtype, B, N, K, M):
    """More groups of requests than one launch plans; tiles whose d_in is shared by several CTAs."""
    c = Case(B, N, K, M, dtype, 6, 8, seed=12, whole=True)
    c.check(c.run(), exact=True)


def test_python_refusals():
    c = Case(2, 3, 64, 40, "bf16", 2, 16, seed=10)
    ok = dict(x=c.x, W=c.W, **c.kw)
    bad = [dict(x=c.x.float()), dict(x=c.x.transpose(1, 2)), dict(W=c.W.t()), dict(W=c.W[:, :32]), dict(A=None), dict(Bm=None),
           dict(A=c.kw["A"][:1]), dict(Bm=c.kw["Bm"].float()), dict(adapter=c.kw["adapter"].long()),
           dict(adapter_scale=c.kw["adapter_scale"].double()), dict(x_scale=torch.zeros(2, 3, 2, dtype=torch.uint8, device="cuda")),
           dict(out=torch.zeros(2, 3, 40, device="cuda")), dict(out=torch.zeros(2, 3, 1, dtype=torch.bfloat16, device="cuda").expand(2, 3, 40)),
           dict(n_live=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(x=c.x[:1, :1].expand(2, 3, 64))]
    for kw in bad:
        with pytest.raises(ValueError):
            kdtv.project(**{**ok, **kw})
    big = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kdtv.KdtvError, match="UNSUPPORTED"):
        kdtv.project(big, c.W, A=torch.zeros(1, 300, 64, dtype=torch.bfloat16, device="cuda"),
                     Bm=torch.zeros(1, 40, 300, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        kdtv.quantise_weight(c.W[:, :33])


@pytest.mark.parametrize("flags", [0, SIMT])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("part", ["first rows", "last row", "one row each", "one request"])
def test_strides_of_single_rows_and_requests(dtype, flags, part):
    """x and out where B or N is 1, as parts of larger buffers: what stands beside a dimension of one element, whatever
    its stride, does not matter (one byte: contiguous but for that)."""
    whole = Case(1, 6, 64, 40, dtype, 2, 16, seed=13, whole=True, ids=[1])
    scale = whole.kw.get("x_scale")
    c = Case(*{"first rows": (1, 4), "last row": (1, 1), "one row each": (6, 1), "one request": (1, 6)}[part], 64, 40, dtype, 2, 16,
             seed=14, whole=True)

    def inside(t):
        wide = t.new_zeros((2, 8, t.shape[2]))
        wide[1, 1:7] = t[0]
        return wide[1:, 1:7]

    cut = {"first rows": lambda t: t[:, :4], "last row": lambda t: t[:, -1:], "one row each": lambda t: t.transpose(0, 1),
           "one request": inside}[part]
    c.x, c.x64 = cut(whole.x), cut(torch.from_numpy(whole.x64)).numpy()
    if scale is not None:
        c.kw["x_scale"] = cut(scale).contiguous()
    c.W, c.W64 = whole.W, whole.W64
    if dtype == "fp8":
        c.kw["W_scale"] = whole.kw["W_scale"]
    out = torch.full((1, 6, 43), 7.0, dtype=TYPE[dtype], device="cuda")
    mine = cut(out[..., :40]) if part != "one request" else out[..., :40]
    got, st = kdtv.project(c.x, c.W, flags=flags, out=mine, **c.kw)
    assert int(st) == 0
    c.check(got, flags, exact=True)
    assert (out[..., 40:] == 7.0).all()
    if part == "first rows":
        assert (out[:, 4:] == 7.0).all()


def _by_definition(c):
    """c.oracle()'s y, product by product: 0 times an infinity is NaN, and nothing else is."""
    y = c.x64 @ c.W64.T
    for b in range(c.B):
        a = int(c.ids[b])
        if a >= 0:
            low = np.einsum("ik,rk->ir", c.x64[b], c.o["A"][a])
            Bm = f64(c.kw["Bm"][a])
            with np.errstate(invalid="ignore"):
                add = sum(low[:, r, None] * Bm[None, :, r] for r in range(c.rank))
                y[b] += c.o["adapter_scale"][a] * add
    return y


@pytest.mark.parametrize("dtype,flags", PATHS)
@pytest.mark.parametrize("B,N,K,M", [(1, 1, 128, 200), (1, 300, 128, 200), (2, 300, 64, 72), (1, 5, 2048, 640), (40, 2, 2048, 200),
                                     (3, 200, 2048, 129), (8, 64, 128, 12800), (1, 600, 128, 12800)])
def test_infinities_of_an_adapter(dtype, flags, B, N, K, M):
    """An infinity in Bm times a finite A x is that infinity, whatever the batch: one request's tile or
    several's, cut over several CTAs or whole.  (Whole numbers: everything else is exact.)"""
    if flags & SIMT and M > 10000:
        pytest.skip("a size for the tensor cores' tiles")
    c = Case(B, N, K, M, dtype, 3, 16, seed=15, whole=True, ids=(np.arange(B) + 2) % 4 - 1)
    Bm = c.kw["Bm"]
    Bm[1, 3, 4], Bm[1, 7, 0], Bm[1, M - 1, 15] = float("inf"), -float("inf"), float("inf")
    Bm[0, 5, 2] = float("nan")
    want = _by_definition(c)
    got = f64(c.run(flags))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isinf(want).any()
    far = np.isinf(want)
    assert np.array_equal(got[far], want[far])
    rest = np.isfinite(want)
    assert np.array_equal(got[rest], f64(torch.tensor(want[rest]).to(TYPE[dtype])))


@pytest.mark.parametrize("flags", [0, SIMT])
@pytest.mark.parametrize("B,N", [(1, 1), (1, 5), (1, 300), (40, 1)])
@pytest.mark.parametrize("rank", [8, 16, 24])
def test_infinite_rows_and_ranks(flags, B, N, rank):
    """An infinity in x, where every weight that it meets is positive, gives infinities, whether or not the ranks fill the
    products' sixteens."""
    c = Case(B, N, 128, 72, "bf16", 2, rank, seed=16, whole=True, ids=[0] * B)
    c.W[:, 3], c.kw["A"][:, :, 3] = 1.0, 1.0
    c.kw["Bm"].abs_().add_(1.0)
    other = c.x[..., 3].clone()
    c.x[0, N // 2, 3] = float("inf")
    got = f64(c.run(flags))
    assert (got[0, N // 2] == np.inf).all()
    c.x[..., 3] = other
    clean = f64(c.run(flags))
    got[0, N // 2] = clean[0, N // 2]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("flags", [0, SIMT])
@pytest.mark.parametrize("B,N", [(1, 1), (1, 20), (30, 1)])
def test_largest_inner_products(flags, B, N):
    """A x between bf16's largest value and fp32's, times 1 / 2: finite."""
    c = Case(B, N, 64, 72, "bf16", 2, 16, seed=17, ids=[1] * B)
    c.x.zero_()
    c.W.zero_()
    c.kw["A"].zero_()
    c.kw["Bm"].zero_()
    c.x[..., :2] = 2.0 ** 100
    c.kw["A"][1, 5, 0], c.kw["A"][1, 5, 1] = 1.9921875 * 2.0 ** 27, 0.75 * 2.0 ** 20
    c.kw["Bm"][1, :, 5] = torch.tensor([0.5, -0.5], dtype=torch.bfloat16, device="cuda").repeat(36)
    c.x64, c.W64 = f64(c.x), f64(c.W)
    c.o.update(A=f64(c.kw["A"]), Bm=f64(c.kw["Bm"]))
    c.check(c.run(flags), flags)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B,N,M", [(1, 1, 640), (64, 1, 384), (2, 150, 256), (6, 9, 130)])
def test_long_sums_of_ordinary_values(dtype, B, N, M):
    """d_in 8192.  An addition loses at most 2^-23 of the running sum or of what is added to it: with P the largest of an
    output's running sums in d_in's order, a sum that begins anywhere is at most 2 P, within 32 elements (whose order
    is the hardware's) at most G = their terms' magnitudes more; the adapter's terms U, all of them, may be added too.  So
    d_in + 2 R additions lose 2^-23 (2 P + G + U) each at most and, of what they add, 2^-23 T; A x enters as two bf16
    parts, 2^-16 of U.  Then half a step of bf16.  (A twentieth of the terms' magnitudes' bound.)"""
    K, R = 8192, 16
    c = Case(B, N, K, M, dtype, 3, R, seed=18)
    out = torch.full((B, N, M), 7.0, dtype=torch.bfloat16, device="cuda")
    got, st = kdtv.project(c.x, c.W, out=out, **c.kw)
    assert int(st) == 0
    y, mag = c.oracle()
    x, W = torch.from_numpy(c.x64).cuda().view(B * N, K), torch.from_numpy(c.W64).cuda()
    U = mag.reshape(B * N, M) - (np.abs(c.x64) @ np.abs(c.W64).T).reshape(B * N, M)
    y, got, T = y.reshape(B * N, M), f64(got).reshape(B * N, M), mag.reshape(B * N, M)
    worst = 0.0
    for t in range(0, B * N, 7):
        terms = x[t][None] * W
        P = terms.cumsum(1).abs().amax(1).cpu().numpy()
        G = terms.abs().view(M, K // 32, 32).sum(2).amax(1).cpu().numpy()
        lim = 2.0 ** -23 * ((K + 2 * R) * (2 * P + G + U[t]) + T[t]) + 2.0 ** -16 * U[t] + 2.0 ** -8 * np.abs(y[t])
        worst = max(worst, float((np.abs(got[t] - y[t]) / lim).max()))
    assert worst <= 1.0
