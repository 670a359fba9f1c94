"""The operators of a layer in a verify step, one after the other as an engine runs them.

Pages for the tree's rows -> residual and norm (to one byte with exponents) -> queries, keys and values by
one shared projection with each request's adapter -> norms of the heads, in place -> rotary positions -> the
keys and values to the paged cache -> tree attention -> output projection -> residual and norm -> accept ->
compaction -> the pages that the rejected nodes leave go back.  Every step is held to its 64-bit oracle over
what it was given; pages, slots and the cache's other rows are equal.
"""

import threading

import numpy as np
import pytest

from oracle import rope_kv as R
from oracle import serve_ops as O
from speculative_decoding_tree_mla_gb300 import kdtv, workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.test_gqa_gpu import Case as Attention          # noqa: E402
from tests.test_norm_gpu import ARITH, STEP, check_one_byte, f64, make, near    # noqa: E402
from tests.test_pages_gpu import Pool, dev                # noqa: E402
from tests.test_project_gpu import TYPE, Case as Projection    # noqa: E402
from tests.test_verify_steps_gpu import drafts            # noqa: E402

D, H, HKV, HEAD, ADAPTERS, RANK = 256, 8, 2, 64, 3, 16
QKV = (H + 2 * HKV) * HEAD


class Weights:
    def __init__(self, dtype, one_byte, seed):
        t = TYPE["f32" if dtype == "f32" else "bf16"]

        def mat(*shape, k, s):
            return (make(shape, "f32", seed + s) * k ** -0.5).to(t)

        self.norm, self.q_norm, self.k_norm, self.last = ((1 + 0.1 * make((n,), "f32", seed + k)).to(t)
                                                          for k, n in enumerate((D, HEAD, HEAD, D)))
        self.qkv, self.o = mat(QKV, D, k=D, s=10), mat(D, H * HEAD, k=H * HEAD, s=11)
        self.A, self.Bm = mat(ADAPTERS, RANK, D, k=D, s=12), mat(ADAPTERS, QKV, RANK, k=4 * RANK, s=13)
        self.scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
        self.qkv_scale = None
        if one_byte:
            self.qkv, self.qkv_scale = kdtv.quantise_weight(self.qkv)


def check_projection(out, x, W, n, dtype, before, **o):
    """out [B, N, M] against the oracle, with test_project_gpu's bounds; x, W: 64-bit values."""
    c = Projection.__new__(Projection)
    c.B, c.N, c.K = x.shape
    c.M, c.dtype, c.rank, c.n, c.o = W.shape[0], dtype, RANK, n, o
    live = np.arange(c.N)[None, :, None] < np.asarray(n)[:, None, None]
    c.x64, c.W64 = np.where(live, x, 0.0), W
    c.check(out, before=before)


@pytest.mark.parametrize("cache,one_byte,page", [("fp8", True, 16), ("fp8", False, 16), ("bf16", True, 64),
                                                 ("f32", False, 16)])
def test_layer_steps(cache, one_byte, page):
    B, N, T = 4, 12, 192
    dtype = "f32" if cache == "f32" else "bf16"
    dt, rng = TYPE[dtype], np.random.default_rng([7, page])
    w = Weights(dtype, one_byte, 100)
    width = T // page
    pool = Pool(B, width, B * width - 3, page, 5)              # (fewer pages than all requests could have)
    shape = (pool.num, page, HKV, HEAD)
    K, V = (torch.zeros(shape, dtype=torch.uint8 if cache == "fp8" else dt, device="cuda") for _ in range(2))
    ks, vs = ((torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)) if cache == "fp8"
              else (None, None))
    table = pool.gpu.page_table
    rope = kdtv.RopeTable(HEAD)
    spec = W_spec()
    kd = kdtv.make_dims(spec(HKV * HEAD), dtype={"f32": "f32", "bf16": "bf16", "fp8": "fp8kv"}[cache], page_size=page,
                        max_pages=width, num_pages=pool.num)
    sd = kdtv.make_dims(spec(HKV), dtype="fp8kv", page_size=page, max_pages=width, num_pages=pool.num)
    adapter = dev([2, -1, 0, 2])

    def cached(rows):
        out = [torch.zeros((B, T, HKV, HEAD), device="cuda") for _ in range(2)]
        st = kdtv.kv_read([kdtv.KvPart(K, out=out[0], scale=ks), kdtv.KvPart(V, out=out[1], scale=vs)],
                          n_live=dev(rows), page_table=table)
        assert int(st) == 0
        return [f64(o) for o in out]

    def append(k, v, at, n, depth=None):
        st = kdtv.kv_append([kdtv.KvPart(K, src=k, scale=ks, rot_off=0), kdtv.KvPart(V, src=v, scale=vs)], at,
                            rope=rope, depth=depth, n_live=n, page_table=table)
        assert int(st) == 0

    L = np.array([0, 5, 60, 33])
    assert pool.resize(L, [0] * B, N, slots=False) == (False, "KDTV_OK")
    append(*(make((B, 60, HKV, HEAD), dtype, 20 + k) for k in range(2)), dev([0] * B), dev(L))
    for step in range(4):
        prefix = dev(L)
        g, target, n = drafts(rng, B, N)
        if step == 2:                                          # a request that waits
            n[1] = 0
            g["n_nodes"][1] = 0
        live = g["n_nodes"]
        before = cached(L)
        short, st = pool.resize(L, [N] * B, N)                 # (compaction asks for the pages of all N rows)
        assert (short, st) == (False, "KDTV_OK")

        x, res = make((B, N, D), dtype, 40 + step), make((B, N, D), dtype, 50 + step, 2.0)
        res0 = f64(res)
        if one_byte:
            a, a_scale = kdtv.rmsnorm(x, w.norm, residual=res, n_live=live, one_byte=True)
        else:
            a, a_scale = kdtv.rmsnorm(x, w.norm, residual=res, n_live=live), None
        y, h = O.rmsnorm(f64(x), f64(w.norm), 1e-6, res0)
        for b in range(B):
            m = int(n[b])
            near(f64(res[b, :m]), h[b, :m], STEP[dtype])
            assert np.array_equal(f64(res[b, m:]), res0[b, m:])
            if m and one_byte:
                check_one_byte(a[b, :m], a_scale[b, :m], y[b, :m])
            elif m:
                near(f64(a[b, :m]), y[b, :m], ARITH + STEP[dtype])

        qkv, st = kdtv.project(a, w.qkv, x_scale=a_scale, W_scale=w.qkv_scale, A=w.A, Bm=w.Bm, adapter=adapter,
                               adapter_scale=w.scale, n_live=live, out=torch.full((B, N, QKV), 3.0, dtype=dt, device="cuda"))
        assert int(st) == 0
        a64 = O.widen(a.cpu().numpy(), a_scale.cpu().numpy()) if one_byte else f64(a)
        w64 = O.widen(w.qkv.cpu().numpy(), w.qkv_scale.cpu().numpy()) if one_byte else f64(w.qkv)
        check_projection(qkv, a64, w64, n, "fp8" if one_byte else dtype, 3.0, A=f64(w.A), Bm=f64(w.Bm),
                         adapter=adapter.tolist(), adapter_scale=w.scale.tolist())

        heads = qkv.unflatten(-1, (H + 2 * HKV, HEAD))
        q, k, v = heads[:, :, :H], heads[:, :, H:H + HKV], heads[:, :, H + HKV:]
        q0, k0, v0 = f64(q), f64(k), f64(v)
        kdtv.rmsnorm(q, w.q_norm, n_live=live, out=q)
        kdtv.rmsnorm(k, w.k_norm, n_live=live, out=k)
        for got, was, weight in ((q, q0, w.q_norm), (k, k0, w.k_norm)):
            want, _ = O.rmsnorm(was, f64(weight), 1e-6)
            for b in range(B):
                near(f64(got)[b, :n[b]], want[b, :n[b]], ARITH + STEP[dtype])
                assert (f64(got)[b, n[b]:] == 3.0).all()
        assert np.array_equal(f64(v), v0)

        qr = kdtv.rope(rope, q, prefix_len=prefix, depth=g["depth"], n_live=live,
                       out=torch.zeros((B, N, H, HEAD), dtype=dt, device="cuda"))
        append(k, v, prefix, live, g["depth"])
        out, st = kdtv.gqa_verify_attn(qr, K, V, g["parent"], prefix, n_nodes=live, page_table=table, k_scale=ks,
                                       v_scale=vs, out=torch.full_like(qr, 9.0))
        assert int(st) == 0
        after = cached(L + n)
        for which in range(2):
            for b in range(B):
                assert np.array_equal(after[which][b, :L[b]], before[which][b, :L[b]])
        c = Attention.__new__(Attention)                       # (its bounds, over the rows as cached)
        c.B, c.N, c.H, c.Hkv, c.d, c.page, c.cache = B, N, H, HKV, HEAD, page, cache
        c.prefix, c.n, c.parent, c.q, c.gathered = L.astype(np.int32), n, g["parent"].cpu().numpy(), qr, lambda: after
        c.check(out, tensor_cores=cache != "f32")

        attn = out.view(B, N, H * HEAD)
        o, st = kdtv.project(attn, w.o, n_live=live, out=torch.full((B, N, D), 4.0, dtype=dt, device="cuda"))
        assert int(st) == 0
        check_projection(o, f64(attn), f64(w.o), n, dtype, 4.0)
        was, res0 = f64(o), f64(res)
        kdtv.rmsnorm(o, w.last, residual=res, n_live=live, out=o)
        y, h = O.rmsnorm(was, f64(w.last), 1e-6, res0)
        for b in range(B):
            near(f64(o)[b, :n[b]], y[b, :n[b]], ARITH + STEP[dtype])
            near(f64(res)[b, :n[b]], h[b, :n[b]], STEP[dtype])
            assert (f64(o)[b, n[b]:] == 4.0).all() and np.array_equal(f64(res)[b, n[b]:], res0[b, n[b]:])

        path, plen, _ = kdtv.tree_accept(g["parent"], g["token"], target)
        keep = np.where(n > 0, plen.cpu().numpy(), 0)
        assert int(kdtv.compact_kv(kd, K, V, prefix, path, plen, table)) == 0
        if cache == "fp8":
            assert int(kdtv.compact_kv(sd, ks, vs, prefix, path, plen, table)) == 0
        kept, pa = cached(L + keep), path.cpu().numpy()
        for b in range(B):
            rows = np.concatenate([np.arange(L[b]), L[b] + pa[b, :keep[b]]])
            for which in range(2):
                assert np.array_equal(kept[which][b, :L[b] + keep[b]], after[which][b, rows])
        L = L + keep
        if step == 1:
            L[2] = 0                                           # a request ends, another takes its place
        assert pool.resize(L, [0] * B, 0, slots=False) == (False, "KDTV_OK")
        final = cached(L)
        for which in range(2):
            for b in range(B):
                assert np.array_equal(final[which][b, :L[b]], kept[which][b, :L[b]])
    assert pool.resize([0] * B, [0] * B, 0, slots=False) == (False, "KDTV_OK") and len(pool.free) == pool.num


def W_spec():
    def spec(width):
        return W.Spec("layer_rows", 0, B=4, N=12, H=1, d_nope=width, d_rope=width, d_v=width, d_c=width, dtype="bf16",
                      prefix=("fixed", 0), tree=("chain",))
    return spec


@pytest.mark.parametrize("one_byte", [True, False])
def test_captured_layer(one_byte):
    """The same layer as one graph, replayed over other lengths, trees, adapters and inputs: the same bits as the calls
    one by one; pages grow and go back inside the graph."""
    B, N, page, width = 3, 9, 16, 20
    rng = np.random.default_rng(11)
    w = Weights("bf16", one_byte, 200)
    x, res = make((B, N, D), "bf16", 60), make((B, N, D), "bf16", 61)
    prefix, live, adapter = dev([100, 0, 17]), dev([9, 4, 9]), dev([1, -1, 0])
    parent = dev(np.stack([W.random_tree(rng, N, 8, 8) for _ in range(B)]))
    rope = kdtv.RopeTable(HEAD)

    def bound():
        pool = kdtv.PagePool.empty(B, width, 2 * width + 5, page)
        K, V = (torch.full((pool.num_pages, page, HKV, HEAD), 0x30, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.full(K.shape[:3], 120, dtype=torch.uint8, device="cuda") for _ in range(2))
        mine = res.clone()
        pages = kdtv.PagesResize(pool, prefix, n_live=live, N=N, slots=True)
        norm = kdtv.RmsNorm(x, w.norm, residual=mine, n_live=live, one_byte=one_byte)
        for t in (norm.out, norm.out_scale) if one_byte else (norm.out,):
            t.zero_()
        qkv = kdtv.Project(norm.out, w.qkv, x_scale=norm.out_scale, W_scale=w.qkv_scale, A=w.A, Bm=w.Bm, adapter=adapter,
                           adapter_scale=w.scale, n_live=live, out=torch.zeros((B, N, QKV), dtype=torch.bfloat16, device="cuda"))
        heads = qkv.out.unflatten(-1, (H + 2 * HKV, HEAD))
        q, k, v = heads[:, :, :H], heads[:, :, H:H + HKV], heads[:, :, H + HKV:]
        qn, kn = kdtv.RmsNorm(q, w.q_norm, n_live=live, out=q), kdtv.RmsNorm(k, w.k_norm, n_live=live, out=k)
        qr = torch.zeros((B, N, H, HEAD), dtype=torch.bfloat16, device="cuda")
        rot = kdtv.Rope(rope, q, prefix_len=prefix, n_live=live, out=qr)
        app = kdtv.KvAppend([kdtv.KvPart(K, src=k, scale=ks, rot_off=0), kdtv.KvPart(V, src=v, scale=vs)], prefix,
                            rope=rope, n_live=live, page_table=pool.page_table)
        att = kdtv.GqaVerifyAttn(qr, K, V, parent, prefix, n_nodes=live, page_table=pool.page_table, k_scale=ks, v_scale=vs,
                                 out=torch.zeros_like(qr))
        o = kdtv.Project(att.out.view(B, N, H * HEAD), w.o, n_live=live,
                         out=torch.zeros((B, N, D), dtype=torch.bfloat16, device="cuda"))
        last = kdtv.RmsNorm(o.out, w.last, residual=mine, n_live=live, out=o.out)
        trim = kdtv.PagesResize(pool, prefix, N=0)
        steps = [pages, norm, qkv, qn, kn, rot, app, att, o, last, trim]
        state = [pool.page_table, pool.n_pages, pool.free_count, pages.slots, K, V, ks, vs, mine, qkv.out, qr, att.out, o.out]
        words = [pages.status, app.status, trim.status, qkv._status, att._status, o._status]
        return steps, state, words, mine

    (a, sa, wa, ma), (b, sb, wb, mb) = bound(), bound()
    for op in a + b:
        op()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for op in a:
            op()
    for step in range(5):
        x.copy_(make((B, N, D), "bf16", 70 + step))
        ma.copy_(res)
        mb.copy_(res)
        prefix.copy_(dev([100 - 25 * step, 33 * step, 17 + 64 * (step % 2)]))
        live.copy_(dev([9, 4 + step, 0 if step == 3 else 7]))
        adapter.copy_(dev(rng.integers(-1, ADAPTERS, B)))
        graph.replay()
        for op in b:
            op()
        for s, t in zip(sa, sb):
            assert torch.equal(s, t)
        assert torch.isfinite(sa[-1].float()).all()
    assert all(int(s) == 0 for s in wa + wb)


def test_host_threads():
    """Projections (both paths, several sizes of shared memory and tiles), norms and page tables from six host
    threads at once, each on a stream of its own: the same bits as alone."""
    def projection(dtype, B, N, K, M, flags=0):
        c = Projection(B, N, K, M, dtype, 3, 16, seed=B + K)
        op = kdtv.Project(c.x, c.W, flags=flags, **c.kw)
        return op, lambda: [op.out]

    def norm(shape, one_byte):
        op = kdtv.RmsNorm(make(shape, "bf16", 90), make(shape[-1:], "bf16", 91), one_byte=one_byte)
        return op, lambda: [op.out] + ([op.out_scale] if one_byte else [])

    def pages(B, N):
        pool = kdtv.PagePool.empty(B, 40, 40 * B, 16)
        there, back = kdtv.PagesResize(pool, dev(np.arange(B) % 500), N=N, slots=True), kdtv.PagesResize(pool, dev([0] * B), N=0)

        def op(stream=None):
            back(stream)
            there(stream)
        return op, lambda: [there.slots, pool.page_table, pool.free_count]

    work = [[lambda: projection("bf16", 64, 1, 1024, 768), lambda: norm((64, 1, 1024), True)],
            [lambda: projection("fp8", 8, 8, 512, 640), lambda: pages(8, 8)],
            [lambda: projection("bf16", 1, 600, 512, 1000), lambda: norm((5, 9, 4, 64), False)],
            [lambda: projection("fp8", 2, 300, 1024, 384), lambda: pages(600, 4)],
            [lambda: projection("f32", 9, 5, 777, 300), lambda: norm((300, 2, 2048), True)],
            [lambda: projection("bf16", 3, 20, 100, 200), lambda: projection("fp8", 1, 1, 4096, 256)]]
    made = [[f() for f in engine] for engine in work]
    want = []
    for engine in made:
        for op, _ in engine:
            op()
        want.append([[t.clone() for t in results()] for _, results in engine])
    torch.cuda.synchronize()
    bad, begin = [], threading.Barrier(len(made))

    def run(engine, expected):
        stream = torch.cuda.Stream()
        begin.wait()
        with torch.cuda.stream(stream):
            for _ in range(40):
                for op, _ in engine:
                    for _ in range(5):
                        op()
                for (_, results), e in zip(engine, expected):
                    if not all(torch.equal(s, t) for s, t in zip(results(), e)):
                        bad.append(1)

    threads = [threading.Thread(target=run, args=p) for p in zip(made, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
