"""The operators of a verify step, one after the other as an engine runs them.

A step: draft tree -> rotary positions of the queries -> the nodes' rows,
rotated, to the cache -> tree attention -> accept -> compaction.  After every
step the cache's rows are read back: the rows that stay must be, bit for bit,
the accepted nodes' rows in path order behind the old prefix; new rows are held
to the fp64 rotation (and the quantiser's half step); the attention to the fp64
oracle over the rows as cached.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import rope_kv as O
from speculative_decoding_tree_mla_gb300 import kdtv, workloads as W
from tests.test_gqa_gpu import Case

pytestmark = pytest.mark.gpu


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.float().cpu().double().numpy()


def drafts(rng, B, N, depth=6, k=4):
    """A tree per request by kdtv_tree_build, and target tokens that follow some of its paths."""
    lp = np.sort(-rng.exponential(1.0, size=(B, depth, k)).astype(np.float32), axis=2)[:, :, ::-1]
    tok = rng.integers(0, 50, size=(B, depth, k)).astype(np.int32)
    g = kdtv.tree_build(dev(lp), dev(tok), dev(rng.integers(0, 50, size=B).astype(np.int32)), N)
    parent, token = g["parent"].cpu().numpy(), g["token"].cpu().numpy()
    n = g["n_nodes"].cpu().numpy()
    target = rng.integers(50, 60, size=(B, N)).astype(np.int32)
    for b in range(B):
        for j in range(1, int(n[b])):
            if rng.random() < 0.7:
                target[b, parent[b, j]] = token[b, j]
    return g, dev(target), n


def rotated(x, pos, freq, layout, off=0):
    """fp64 rotation of x [N, H, dim] and a bound on the kernel's error before the result is rounded:
    an angle is off by 2^-31 turns or less, 2^-28 of angle; cos and sin by 2^-27 in all with the
    polynomials; two products and a sum, 2^-23 of their size."""
    y = O.rope(x, pos, freq, 1.0, layout, off)
    mate = np.abs(x).max(-1, keepdims=True)
    return y, 2 * mate * (2.0 ** -26 + 2.0 ** -23)


@pytest.mark.parametrize("cache,page,layout", [("fp8", 16, "half"), ("bf16", 0, "interleaved"), ("fp8", 0, "half"),
                                               ("f32", 16, "half")])
def test_gqa_steps(cache, page, layout):
    B, N, H, Hkv, d, T = 3, 12, 8, 2, 64, 192
    rng = np.random.default_rng([1, page])
    dt = torch.float32 if cache == "f32" else torch.bfloat16
    ct = torch.uint8 if cache == "fp8" else dt
    shape = (B * T // page + 1, page, Hkv, d) if page else (B, T, Hkv, d)
    table = dev(rng.permutation(shape[0])[:B * T // page].reshape(B, -1).astype(np.int32)) if page else None
    K, V = (torch.zeros(shape, dtype=ct, device="cuda") for _ in range(2))
    ks, vs = ((torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)) if cache == "fp8"
              else (None, None))
    prefix = dev(np.array([0, 5, 60], np.int32))
    rope = kdtv.RopeTable(d, layout=layout)
    freq, _ = O.rope_frequencies(d)

    def to_dims(dtype, width):
        spec = W.Spec("gqa_rows", 0, B=B, N=N, H=1, d_nope=width, d_rope=width, d_v=width, d_c=width, dtype=dtype,
                      prefix=("fixed", 0), tree=("chain",))
        return kdtv.make_dims(spec, dtype=dtype, page_size=page, t_stride=0 if page else T,
                              max_pages=T // page if page else 0, num_pages=shape[0] if page else 0)

    kd = to_dims({"f32": "f32", "bf16": "bf16", "fp8": "fp8kv"}[cache], Hkv * d)
    sd = to_dims("fp8kv", Hkv)

    def cached():
        """Rows 0 .. T of every request, as values (float32: exact)."""
        out = [torch.zeros((B, T, Hkv, d), device="cuda") for _ in range(2)]
        st = kdtv.kv_read([kdtv.KvPart(K, out=out[0], scale=ks), kdtv.KvPart(V, out=out[1], scale=vs)],
                          page_table=table)
        assert int(st.item()) == 0
        return [f64(o) for o in out]

    # what the prefixes hold
    first = [dev(rng.standard_normal((B, 60, Hkv, d), dtype=np.float32), dt) for _ in range(2)]
    st = kdtv.kv_append([kdtv.KvPart(K, src=first[0], scale=ks), kdtv.KvPart(V, src=first[1], scale=vs)],
                        torch.zeros_like(prefix), n_live=prefix, page_table=table)
    assert int(st.item()) == 0
    for step in range(4):
        before = cached()
        L = prefix.cpu().numpy().astype(np.int64)
        g, target, n = drafts(rng, B, N)
        assert n.min() >= 1
        q = dev(rng.standard_normal((B, N, H, d), dtype=np.float32), dt)
        new = [dev(rng.standard_normal((B, N, Hkv, d), dtype=np.float32), dt) for _ in range(2)]

        qr = kdtv.rope(rope, q, prefix_len=prefix, depth=g["depth"], n_live=g["n_nodes"], out=torch.zeros_like(q))
        st = kdtv.kv_append([kdtv.KvPart(K, src=new[0], scale=ks, rot_off=0), kdtv.KvPart(V, src=new[1], scale=vs)],
                            prefix, rope=rope, depth=g["depth"], n_live=g["n_nodes"], page_table=table)
        out, gst = kdtv.gqa_verify_attn(qr, K, V, g["parent"], prefix, n_nodes=g["n_nodes"], page_table=table,
                                        k_scale=ks, v_scale=vs, out=torch.full_like(q, 9.0))
        assert int(st.item()) == 0 and int(gst.item()) == 0

        after = cached()
        depth = g["depth"].cpu().numpy()
        half = 2.0 ** -24 if cache == "f32" else 2.0 ** -8
        for b in range(B):
            nb, Lb = int(n[b]), int(L[b])
            pos = Lb + depth[b, :nb]
            want, err = rotated(f64(q)[b, :nb], pos, freq, layout)
            assert (np.abs(f64(qr)[b, :nb] - want) <= err + half * np.abs(want)).all()
            for which in range(2):
                assert np.array_equal(after[which][b, :Lb], before[which][b, :Lb])
                assert np.array_equal(after[which][b, Lb + nb:], before[which][b, Lb + nb:])
                want, err = f64(new[which])[b, :nb], 0.0
                if which == 0:
                    want, err = rotated(want, pos, freq, layout)
                tol = half * np.abs(want) + err
                if cache == "fp8":       # half a step of the code, or of the smallest one
                    s = 2.0 ** O.row_exponent(want)[..., None]
                    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s) + err * (1 + 2.0 ** -4)
                assert (np.abs(after[which][b, Lb:Lb + nb] - want) <= tol).all()

        x = Case.__new__(Case)           # the oracle's view: rows as cached
        x.B, x.N, x.H, x.Hkv, x.d, x.page, x.cache = B, N, H, Hkv, d, page, cache
        x.prefix, x.n, x.parent, x.q = L.astype(np.int32), n, g["parent"].cpu().numpy(), qr
        x.gathered = lambda: after
        x.check(out, tensor_cores=cache != "f32")

        path, plen, bonus = kdtv.tree_accept(g["parent"], g["token"], target)
        st = kdtv.compact_kv(kd, K, V, prefix, path, plen, table)
        assert int(st.item()) == 0
        if cache == "fp8":
            st = kdtv.compact_kv(sd, ks, vs, prefix, path, plen, table)
            assert int(st.item()) == 0
        kept = cached()
        pl, pa = plen.cpu().numpy(), path.cpu().numpy()
        for b in range(B):
            rows = np.concatenate([np.arange(L[b]), L[b] + pa[b, :pl[b]]])
            for which in range(2):
                assert np.array_equal(kept[which][b, :L[b] + pl[b]], after[which][b, rows])
        prefix += plen
    assert int(plen.max()) > 1               # (some path was longer than its root)


@pytest.mark.parametrize("dtype,page", [("bf16", 0), ("fp8kv", 64), ("f32", 64)])
def test_mla_steps(dtype, page):
    """The latent cache: the query projection's rows split and rotated, c_kv and the rotated k_rope
    appended (one-byte caches with one scale), then verify, accept and compaction."""
    B, N, H, T = 2, 8, 8, 256
    spec = W.Spec("mla_steps", 0, B=B, N=N, H=H, d_nope=128, d_rope=64, d_v=128, d_c=512, dtype=dtype,
                  prefix=("fixed", 0), tree=("chain",))
    kv_scale = 2.0 ** -6
    rng = np.random.default_rng([2, page])
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    ct = torch.uint8 if dtype == "fp8kv" else dt
    lead = (B * T // page + 1, page) if page else (B, T)
    table = dev(rng.permutation(lead[0])[:B * T // page].reshape(B, -1).astype(np.int32)) if page else None
    c_kv, k_rope = torch.zeros(lead + (512,), dtype=ct, device="cuda"), torch.zeros(lead + (64,), dtype=ct, device="cuda")
    prefix = dev(np.array([3, 130], np.int32))
    rope = kdtv.RopeTable(64, layout="interleaved")
    freq, _ = O.rope_frequencies(64)
    W_UK = dev(rng.standard_normal((H, 128, 512), dtype=np.float32) * 0.05, dt)
    W_UV = dev(rng.standard_normal((H, 128, 512), dtype=np.float32) * 0.05, dt)
    scale = kv_scale if dtype == "fp8kv" else 0.0

    def cached():
        out = [torch.zeros((B, T, w), device="cuda") for w in (512, 64)]
        st = kdtv.kv_read([kdtv.KvPart(c_kv, out=out[0]), kdtv.KvPart(k_rope, out=out[1])], page_table=table,
                          kv_scale=scale)
        assert int(st.item()) == 0
        return [f64(o) for o in out]

    first = [dev(rng.standard_normal((B, 130, w), dtype=np.float32), dt) for w in (512, 64)]
    st = kdtv.kv_append([kdtv.KvPart(c_kv, src=first[0]), kdtv.KvPart(k_rope, src=first[1])], torch.zeros_like(prefix),
                        n_live=prefix, page_table=table, kv_scale=scale)
    assert int(st.item()) == 0
    for step in range(3):
        L = prefix.cpu().numpy().astype(np.int64)
        g, target, n = drafts(rng, B, N)
        assert (n == N).all()
        q = dev(rng.standard_normal((B, N, H, 192), dtype=np.float32), dt)      # [nope | rope]
        lat = dev(rng.standard_normal((B, N, 512), dtype=np.float32), dt)
        kr = dev(rng.standard_normal((B, N, 1, 64), dtype=np.float32), dt)
        q_rope, q_nope = kdtv.rope(rope, q, prefix_len=prefix, depth=g["depth"], rot_off=128, split=True)
        assert torch.equal(q_nope, q[..., :128])
        st = kdtv.kv_append([kdtv.KvPart(c_kv, src=lat), kdtv.KvPart(k_rope, src=kr, rot_off=0)], prefix, rope=rope,
                            depth=g["depth"], page_table=table, kv_scale=scale)
        assert int(st.item()) == 0
        tens = dict(q_nope=q_nope, q_rope=q_rope, W_UK=W_UK, W_UV=W_UV, c_kv=c_kv, k_rope=k_rope,
                    parent=g["parent"], prefix_len=prefix, page_table=table)
        op = kdtv.VerifyAttn(spec, tens, t_stride=0 if page else T, max_pages=T // page if page else 0,
                             num_pages=lead[0] if page else 0, page_size=page, kv_scale=scale)
        out = op()
        assert op.status() == 0

        after = cached()
        depth = g["depth"].cpu().numpy()
        for b in range(B):
            pos = L[b] + depth[b]
            want, err = rotated(f64(q)[b][..., 128:], pos, freq, "interleaved")
            half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
            assert (np.abs(f64(q_rope)[b] - want) <= err + half * np.abs(want)).all()
            for got, want, err in ((after[0][b, L[b]:L[b] + N], f64(lat)[b], 0.0),
                                   (after[1][b, L[b]:L[b] + N], *[x[:, 0] for x in rotated(f64(kr)[b], pos, freq, "interleaved")])):
                tol = half * np.abs(want) + err
                if dtype == "fp8kv":
                    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * kv_scale) + err * (1 + 2.0 ** -4)
                assert (np.abs(got - want) <= tol).all()
        ref = oracle.verify_attn(f64(q_nope), f64(q_rope), f64(W_UK), f64(W_UV), after[0], after[1],
                                 g["parent"].cpu().numpy(), L, spec.scale)
        rel = np.linalg.norm(f64(out) - ref) / np.linalg.norm(ref)
        assert rel <= (1e-5 if dtype == "f32" else 5e-3)      # the attention's own bars

        path, plen, _ = kdtv.tree_accept(g["parent"], g["token"], target)
        assert int(kdtv.compact_kv(op.dims, c_kv, k_rope, prefix, path, plen, table).item()) == 0
        kept = cached()
        pl, pa = plen.cpu().numpy(), path.cpu().numpy()
        for b in range(B):
            rows = np.concatenate([np.arange(L[b]), L[b] + pa[b, :pl[b]]])
            for which in range(2):
                assert np.array_equal(kept[which][b, :L[b] + pl[b]], after[which][b, rows])
        prefix += plen


def test_captured_gqa_step():
    """Rotation, append and attention captured as one graph, replayed over changed inputs: the same
    bits as the calls one by one."""
    B, N, H, Hkv, d, T = 2, 7, 8, 4, 128, 300
    rng = np.random.default_rng(3)
    q, k, v = (dev(rng.standard_normal((B, N, h, d), dtype=np.float32), torch.bfloat16) for h in (H, Hkv, Hkv))
    prefix = dev(np.array([128, 250], np.int32))
    parent = dev(np.stack([W.random_tree(rng, N, 8, 8) for _ in range(B)]).astype(np.int32))
    fill = torch.randint(0, 0x78, (B, T, Hkv, d), dtype=torch.uint8, device="cuda")
    rope = kdtv.RopeTable(d)

    def bound():
        K, V = fill.clone(), fill.clone()
        ks, vs = (torch.full((B, T, Hkv), 118, dtype=torch.uint8, device="cuda") for _ in range(2))
        qr = torch.zeros_like(q)
        steps = [kdtv.Rope(rope, q, prefix_len=prefix, out=qr),
                 kdtv.KvAppend([kdtv.KvPart(K, src=k, scale=ks, rot_off=0), kdtv.KvPart(V, src=v, scale=vs)], prefix,
                               rope=rope),
                 kdtv.GqaVerifyAttn(qr, K, V, parent, prefix, k_scale=ks, v_scale=vs)]
        return steps, (K, V, ks, vs)

    (a, ka), (b, kb) = bound(), bound()
    for op in a + b:
        op()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for op in a:
            op()
    for step in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn_like(t.float()).to(t.dtype))
        prefix.copy_(dev(np.array([128 - 40 * step, 250 + 7 * step], np.int32)))
        graph.replay()
        for op in b:
            op()
        assert torch.equal(a[2].out, b[2].out)
        for x, y in zip(ka, kb):
            assert torch.equal(x, y)
    assert a[2].status() == 0 and b[2].status() == 0 and int(a[1].status.item()) == 0


def test_two_host_threads():
    """Two engines in two host threads, each with a stream of its own: the same bits as alone."""
    import threading
    cases = [Case(2, 12, 16, 4, 128, "fp8", 16, [400, 33], [12, 9], seed=1),
             Case(3, 5, 16, 2, 64, "bf16", 0, [700, 0, 129], seed=2)]
    rope = kdtv.RopeTable(64)
    want = []
    for x in cases:
        qr = kdtv.rope(rope, x.q, prefix_len=dev(x.prefix))
        want.append((qr.clone(), x.op()().clone()))
    torch.cuda.synchronize()
    bad = []

    def engine(x, w):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            op, qr = x.op(), torch.zeros_like(x.q)
            rot = kdtv.Rope(rope, x.q, prefix_len=dev(x.prefix), out=qr)
            for _ in range(50):
                out = op()
                rot()
                if not (torch.equal(out, w[1]) and torch.equal(qr, w[0])):
                    bad.append(1)

    threads = [threading.Thread(target=engine, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8], ids=["bf16", "f32", "bytes"])
@pytest.mark.parametrize("page", [0, 16])
def test_compaction_of_wide_rows(dtype, page):
    """A per-head cache's keys and values as the two tensors: rows whose chunk passes the 48 KiB of
    shared memory that need no opt-in."""
    B, N, T, width = 3, 40, 96, 1024 if dtype != torch.uint8 else 2048
    rng = np.random.default_rng([4, page])
    shape = (B * T // page, page, width) if page else (B, T, width)
    table = rng.permutation(shape[0]).reshape(B, -1).astype(np.int32) if page else None
    K, V = (dev(rng.integers(0, 200, size=shape)).to(dtype) for _ in range(2))
    prefix, plen = np.array([0, 17, 50], np.int32), np.array([40, 1, 9], np.int32)
    path = np.full((B, N), -1, np.int32)
    for b in range(B):
        path[b, :plen[b]] = [0] + sorted(rng.choice(np.arange(1, N), size=plen[b] - 1, replace=False))
    name = {torch.bfloat16: "bf16", torch.float32: "f32", torch.uint8: "fp8kv"}[dtype]
    spec = W.Spec("wide", 0, B=B, N=N, H=1, d_nope=width, d_rope=width, d_v=width, d_c=width, dtype=name,
                  prefix=("fixed", 0), tree=("chain",))
    d = kdtv.make_dims(spec, dtype=name, page_size=page, t_stride=0 if page else T,
                       max_pages=T // page if page else 0, num_pages=shape[0] if page else 0)

    def rows(x, b):
        return x[torch.from_numpy(table[b]).long().cuda()].view(T, width) if page else x[b]

    before = [[rows(x, b).clone() for b in range(B)] for x in (K, V)]
    st = kdtv.compact_kv(d, K, V, dev(prefix), dev(path), dev(plen), dev(table) if page else None)
    assert int(st.item()) == 0
    for x, old in zip((K, V), before):
        for b in range(B):
            want = old[b].clone()
            for k in range(plen[b]):
                want[prefix[b] + k] = old[b][prefix[b] + path[b, k]]
            assert torch.equal(rows(x, b), want)
