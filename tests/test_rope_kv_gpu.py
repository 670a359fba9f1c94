"""Rotary positions and cache writes / reads against the fp64 oracle.

Tolerances, fixed before the first run.  Rotation: cos and sin are off by at
most 2^-23 (the angle is exact to 2^-32 turns and 2^-24 of itself, below pi / 4
after the reduction; the polynomials' steps add less than that again), each of the two products and the sum rounds
once: 8 * 2^-24 * amp * (|u| + |v|) covers it, then one rounding to the output
type, at most half a step (bf16 2^-8 of the value with its eps of 2^-7, fp32
2^-24).  E4M3: half a step is 2^-4 of the value, or 2^-10 of the scale among
subnormals.  What is only moved or widened is compared bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import rope_kv as O
from speculative_decoding_tree_mla_gb300 import kdtv, workloads as W

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def rng_for(*key):
    return np.random.default_rng([int(k) for k in key])


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def f64(t):
    return t.detach().float().cpu().double().numpy()


def rot_tol(x, freq_count, amp, layout, off):
    """8 * 2^-24 * amp * (|u| + |v|) at each rotated element, 0 elsewhere."""
    a = np.abs(x)
    t = np.zeros_like(a)
    h = freq_count
    iu = off + (np.arange(h) if layout == "half" else 2 * np.arange(h))
    iv = off + (h + np.arange(h) if layout == "half" else 2 * np.arange(h) + 1)
    t[..., iu] = t[..., iv] = 8 * 2.0 ** -24 * amp * (a[..., iu] + a[..., iv])
    return t


ROPES = [
    # B, N, H, dim, rot, off, layout, dtype, table
    (1, 1, 1, 2, 2, 0, "half", "f32", {}),
    (1, 1, 32, 128, 128, 0, "half", "bf16", {}),
    (2, 5, 3, 128, 64, 0, "half", "bf16", dict(scaling="linear", factor=4.0)),
    (2, 7, 4, 192, 64, 128, "interleaved", "bf16", dict(scaling="yarn", factor=32.0, base=50000.0, orig_ctx=4096)),
    (3, 4, 5, 80, 80, 0, "half", "bf16", dict(scaling="ntk", factor=8.0)),
    (2, 3, 9, 66, 34, 13, "half", "bf16", {}),          # scalar accesses
    (2, 3, 9, 67, 34, 13, "interleaved", "f32", {}),
    (1, 2, 3, 256, 256, 0, "interleaved", "f32", {}),
    (5, 130, 17, 128, 32, 96, "half", "f32", {}),
    (2, 600, 64, 128, 64, 32, "interleaved", "bf16", {}),   # several heads per thread
]


@pytest.mark.parametrize("case", ROPES, ids=lambda c: "-".join(map(str, c[:8])))
@pytest.mark.parametrize("mode", ["out", "in_place", "split", "strided"])
def test_rope(case, mode):
    B, N, H, dim, rot, off, layout, dtype, kw = case
    rng = rng_for(B, N, H, dim, rot, off)
    if mode == "strided":      # heads of a fused projection: rows wider than the heads, heads apart
        base = dev(rng.standard_normal((B, N, 2 * H + 1, dim + 8), dtype=np.float32), DT[dtype])
        x = base[:, :, 1::2, :dim]
    else:
        x = dev(rng.standard_normal((B, N, H, dim), dtype=np.float32), DT[dtype])
    prefix = rng.integers(0, 200000, size=B).astype(np.int32)
    prefix[0] = (1 << 31) - 200
    depth = rng.integers(0, 100, size=(B, N)).astype(np.int32)
    live = rng.integers(0, N + 1, size=B).astype(np.int32)
    live[0] = N
    t = kdtv.RopeTable(rot, layout=layout, **kw)
    want_args = {k: v for k, v in kw.items()}
    freq, amp = O.rope_frequencies(rot, **want_args)
    xs = f64(x)
    pos = prefix[:, None].astype(np.int64) + depth
    want = O.rope(xs, pos, freq, amp, layout, off)
    # the oracle's angle is a double: at positions near 2^31 it is itself off by 2^-22
    tol = rot_tol(xs, rot // 2, amp, layout, off) * (1 + (pos > 1 << 24)[..., None, None] * 8) + HALF[dtype] * np.abs(want)
    ix = dict(prefix_len=dev(prefix), depth=dev(depth), n_live=dev(live), rot_off=off)
    if mode == "split":
        y, rest = kdtv.rope(t, x, split=True, **ix)
        got = np.empty_like(want)
        got[..., off:off + rot] = f64(y)
        got[..., :off], got[..., off + rot:] = f64(rest)[..., :off], f64(rest)[..., off:]
    elif mode == "in_place":
        y = kdtv.rope(t, x, out=x, **ix)
        assert y is x
        got = f64(y)
    else:
        out = torch.full((B, N, H, dim), 7.0, dtype=DT[dtype], device="cuda")
        got = f64(kdtv.rope(t, x, out=out, **ix))
    for b in range(B):
        n = live[b]
        assert (np.abs(got[b, :n] - want[b, :n]) <= tol[b, :n]).all()
        keep = np.ones(dim, bool)
        keep[off:off + rot] = False
        assert (got[b, :n][..., keep] == xs[b, :n][..., keep]).all()
        if mode == "in_place":
            assert (got[b, n:] == xs[b, n:]).all()
        elif mode in ("out", "strided"):
            assert (got[b, n:] == 7.0).all()


def test_rope_default_positions_and_clamped_counts():
    """No prefix: positions 0, 1, ..; n_live beyond [0, N] is clamped; position 0 is the identity."""
    x = dev(np.random.default_rng(1).standard_normal((3, 4, 2, 64), dtype=np.float32))
    t = kdtv.RopeTable(64)
    freq, amp = O.rope_frequencies(64)
    y = kdtv.rope(t, x, n_live=dev(np.array([9, -3, 2], np.int32)), out=torch.zeros_like(x))
    want = O.rope(f64(x), np.arange(4)[None].repeat(3, 0), freq, amp, "half", 0)
    assert np.abs(f64(y)[0] - want[0]).max() <= 1e-5
    assert (f64(y)[1] == 0).all() and (f64(y)[2, 2:] == 0).all()
    assert (f64(y)[[0, 2], 0] == f64(x)[[0, 2], 0]).all()


def test_rope_keeps_relative_scores():
    """q.k of rotated pairs depends on the distance alone, also a billion positions out."""
    rng = np.random.default_rng(3)
    q, k = (dev(rng.standard_normal((1, 1, 4, 128), dtype=np.float32)) for _ in range(2))
    t = kdtv.RopeTable(128)
    at = lambda x, p: kdtv.rope(t, x, prefix_len=dev(np.array([p], np.int32)))     # noqa: E731
    s = [(at(q, p + 37).double() * at(k, p).double()).sum(-1) for p in (0, 5, 1 << 20, 1 << 30)]
    norm = (q.double().norm(dim=-1) * k.double().norm(dim=-1)).max().item()
    for v in s[1:]:
        assert (v - s[0]).abs().max().item() <= 32 * 2.0 ** -24 * norm


# ---- cache rows ---------------------------------------------------------------------------

def make_cache(rng, cache, B, T, heads, dim, page, per_row):
    """A cache with values everywhere, its page table, and (b, t) -> flat row."""
    if page:
        per = -(-T // page)
        num = B * per + 3
        table = rng.permutation(num)[:B * per].reshape(B, per).astype(np.int32)
        shape, rows = (num, page, heads, dim), num * page
        at = lambda b, t: int(table[b, t // page]) * page + t % page       # noqa: E731
    else:
        table, shape, rows = None, (B, T, heads, dim), B * T
        at = lambda b, t: b * T + t                                         # noqa: E731
    if cache == "fp8":
        c = torch.from_numpy(rng.integers(0, 256, size=shape).astype(np.uint8)).cuda()
        s = torch.from_numpy(rng.integers(100, 150, size=shape[:3]).astype(np.uint8)).cuda() if per_row else None
    else:
        c = dev(rng.standard_normal(shape, dtype=np.float32), DT[cache])
        s = None
    return c, s, table, at, rows


KVS = [
    # B, N, (heads, dim) of the parts, src, cache, page, per row
    (2, 5, [(1, 512), (1, 64)], "bf16", "fp8", 64, False),
    (1, 1, [(1, 512), (1, 64)], "bf16", "bf16", 0, False),
    (3, 130, [(8, 128), (8, 128)], "bf16", "fp8", 16, True),
    (2, 300, [(4, 64), (4, 64)], "f32", "fp8", 0, True),
    (2, 9, [(2, 80), (2, 80)], "bf16", "fp8", 7, True),
    (2, 9, [(3, 36), (3, 36)], "f32", "fp8", 5, True),           # scalar accesses
    (1, 4, [(1, 500)], "bf16", "fp8", 0, True),
    (2, 7, [(5, 128), (5, 128)], "f32", "f32", 64, False),
    (2, 7, [(5, 33), (5, 33)], "f32", "bf16", 64, False),
    (2, 7, [(2, 256)], "bf16", "f32", 0, False),
    (2, 2100, [(8, 128), (8, 128)], "bf16", "fp8", 64, True),    # several heads per group
]


@pytest.mark.parametrize("case", KVS, ids=lambda c: "-".join(map(str, (c[0], c[1], c[2][0], *c[3:]))))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_and_read(case, layout):
    B, N, parts, src_t, cache_t, page, per_row = case
    rng = rng_for(B, N, parts[0][0], parts[0][1], page, layout == "half")
    live = rng.integers(0, N + 1, size=B).astype(np.int32)
    live[0] = N
    prefix = rng.integers(0, 70, size=B).astype(np.int32)
    depth = rng.integers(0, 9, size=(B, N)).astype(np.int32)
    T = int((prefix + live).max())
    kv_scale = 0.0625 if cache_t == "fp8" and not per_row else 0.0
    made, objs, args, state = None, [], [], []
    for k, (heads, dim) in enumerate(parts):
        seeded = np.random.default_rng([7, B, N, page])         # both parts share the page table
        c, s, table, at, _ = make_cache(seeded, cache_t, B, T, heads, dim, page, per_row)
        x = rng.standard_normal((B, N, heads, dim), dtype=np.float32) * np.exp(rng.normal(0, 4, (B, N, heads, 1))).astype(np.float32)
        if k == 0:
            x[0, 0, 0, :] = 0.0                                  # a row of zeros
        src = dev(x, DT[src_t])
        if k == len(parts) - 1:                                  # from a wider projection
            wide = torch.zeros((B, N, heads + 2, dim), dtype=src.dtype, device="cuda")
            wide[:, :, 1:-1] = src
            src = wide[:, :, 1:-1]
        rot = min(64, dim // 4 * 2) if k == len(parts) - 1 else None
        off = 0 if rot is None or dim - rot < 8 else 8
        objs.append(kdtv.KvPart(c, src=src, scale=s, rot_off=None if rot is None else off))
        args.append((heads, dim, rot, off, at))
        state.append((c.clone(), None if s is None else s.clone()))
    t = kdtv.RopeTable(args[-1][2], layout=layout, base=500.0)
    freq, amp = O.rope_frequencies(args[-1][2], base=500.0)
    pt = None if table is None else dev(table)
    st = kdtv.kv_append(objs, dev(prefix), rope=t, depth=dev(depth), n_live=dev(live), page_table=pt, kv_scale=kv_scale)
    assert int(st.item()) == 0
    pos = prefix[:, None].astype(np.int64) + depth
    for p, (heads, dim, rot, off, at), (c0, s0) in zip(objs, args, state):
        x = f64(p.src)
        y, tol = x, np.zeros_like(x)
        if rot is not None:
            y = O.rope(x, pos, freq, amp, layout, off)
            tol = rot_tol(x, rot // 2, amp, layout, off)
        flat = p.cache.reshape(-1, heads, dim)
        flat0 = c0.reshape(-1, heads, dim)
        touched = np.zeros(flat.shape[0], bool)
        rows = [(b, i, at(b, int(prefix[b]) + i)) for b in range(B) for i in range(live[b])]
        idx = np.array([r for _, _, r in rows])
        sel = (np.array([b for b, _, _ in rows]), np.array([i for _, i, _ in rows]))
        touched[idx] = True
        assert torch.equal(flat[torch.from_numpy(~touched).cuda()], flat0[torch.from_numpy(~touched).cuda()])
        got, want, slack = flat[torch.from_numpy(idx).cuda()], y[sel], tol[sel]
        if cache_t != "fp8":
            assert (np.abs(f64(got) - want) <= slack + HALF[cache_t] * np.abs(want)).all()
            continue
        code = got.cpu().numpy()
        if per_row:
            e = p.scale.reshape(-1, heads)[torch.from_numpy(idx).cuda()].cpu().numpy().astype(np.int64) - 127
            s = p.scale.reshape(-1, heads).cpu().numpy()
            assert (s[~touched] == s0.reshape(-1, heads).cpu().numpy()[~touched]).all()
            exact_e = O.row_exponent(want)
            if rot is None:
                assert (e == exact_e).all()
            else:      # a largest magnitude within the rotation's error of a border may fall on either side
                assert ((e == exact_e) | (e == O.row_exponent(want * (1 + 2.0 ** -20))) | (e == O.row_exponent(want * (1 - 2.0 ** -20)))).all()
            s = 2.0 ** e[..., None]
        else:
            s = kv_scale
        if rot is None:
            assert (code == W.fp8_e4m3_encode((want / s).astype(np.float32))).all()
        val = W.fp8_e4m3_decode(code).astype(np.float64) * s
        sat = np.clip(want, -448.0 * s, 448.0 * s)
        assert (np.abs(val - sat) <= slack + np.maximum(2.0 ** -4 * np.abs(sat), 2.0 ** -10 * s)).all()
    # read back, in both types, into rows that stay as they were behind the live ones
    for out_t in ("bf16", "f32"):
        rd = []
        for p, (heads, dim, *_) in zip(objs, args):
            rd.append(kdtv.KvPart(p.cache, scale=p.scale,
                                  out=torch.full((B, N, heads, dim), 3.0, dtype=DT[out_t], device="cuda")))
        st = kdtv.kv_read(rd, dev(prefix), dev(live), page_table=pt, kv_scale=kv_scale)
        assert int(st.item()) == 0
        for p, (heads, dim, rot, off, at) in zip(rd, args):
            flat = p.cache.reshape(-1, heads, dim)
            for b in range(B):
                assert (p.out[b, live[b]:] == 3.0).all()
                if live[b] == 0:
                    continue
                r = torch.tensor([at(b, int(prefix[b]) + i) for i in range(live[b])]).cuda()
                x = flat[r]
                if cache_t == "fp8":
                    v = W.fp8_e4m3_decode(x.cpu().numpy()).astype(np.float64)
                    v = v * (2.0 ** (p.scale.reshape(-1, heads)[r].cpu().numpy().astype(np.float64) - 127)[..., None]
                             if per_row else kv_scale)
                    want = torch.from_numpy(v).to(DT[out_t])     # exact in both types
                else:
                    want = x.to(DT[out_t]).cpu()
                assert torch.equal(p.out[b, :live[b]].cpu(), want)


def test_append_special_values():
    """Infinities saturate at the exponent of the finite elements, NaN stays, extremes clamp, a
    value that fp8 cannot tell from zero is zero, ties go to even."""
    inf, nan = float("inf"), float("nan")
    x = np.zeros((1, 8, 1, 8), np.float32)
    x[0, 0, 0, :4] = [inf, 1.0, -inf, 0.5]
    x[0, 1, 0, :3] = [nan, 2.0, -900.0]
    x[0, 2, 0, :2] = [3.0e38, -1.0]
    x[0, 3, 0, :2] = [1e-44, 0.0]
    x[0, 4, 0, :3] = [448.0, 17.0, 19.0]          # ties between 16 and 18, 18 and 20: the even code
    x[0, 5, 0, :2] = [-0.0, 448.0]
    x[0, 6, 0, :3] = [448.0, 2.0 ** -10, 3 * 2.0 ** -10]      # ties among subnormals
    x[0, 7, 0, :] = inf
    cache = torch.full((1, 8, 1, 8), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.zeros((1, 8, 1), dtype=torch.uint8, device="cuda")
    assert int(kdtv.kv_append([kdtv.KvPart(cache, src=dev(x), scale=scale)], dev(np.zeros(1, np.int32))).item()) == 0
    e = scale.cpu().numpy()[0, :, 0].astype(int) - 127
    assert e.tolist() == O.row_exponent(x)[0, :, 0].tolist()
    v = W.fp8_e4m3_decode(cache.cpu().numpy())[0, :, 0].astype(np.float64) * 2.0 ** e[:, None]
    assert v[0, :4].tolist() == [448 * 2.0 ** -8, 1.0, -448 * 2.0 ** -8, 0.5]
    assert np.isnan(v[1, 0]) and v[1, 1] == 2.0 and v[1, 2] == -896.0
    assert v[2, 0] == 448.0 * 2.0 ** 119 and v[2, 1] == 0.0
    assert v[3, 0] == 0.0 and e[3] == -117
    assert v[4, :3].tolist() == [448.0, 16.0, 20.0]
    assert np.signbit(v[5, 0]) and v[5, 1] == 448.0
    assert v[6, :3].tolist() == [448.0, 0.0, 2.0 ** -8]
    assert (v[7] == 448 * 2.0 ** -117).all()


@pytest.mark.parametrize("page", [0, 4])
def test_bad_requests_are_left_unwritten(page):
    """A prefix that is negative or does not fit, or a page out of range: that request's rows stay,
    the others are written, the status word holds the first code until it is cleared."""
    B, N, T = 4, 3, 16
    rng = np.random.default_rng(4)
    x = dev(rng.standard_normal((B, N, 2, 16), dtype=np.float32), torch.bfloat16)
    shape = (B * T // 4, 4, 2, 16) if page else (B, T, 2, 16)
    table = np.arange(B * T // 4, dtype=np.int32).reshape(B, -1)
    good = [6, 13, 0, 5]
    for b, L, pg, code in ((1, -1, None, 6), (1, T - N + 1, None, 6), (0, 1 << 30, None, 6),
                           (0, 6, -1, 7), (0, 6, B * T // 4, 7)):
        if pg is not None and not page:
            continue
        prefix = np.array(good, np.int32)
        prefix[b] = L
        tb = table.copy()
        if pg is not None:
            tb[b, 2] = pg
        for which in ("append", "read"):
            cache = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
            out = torch.full((B, N, 2, 16), 5.0, dtype=torch.bfloat16, device="cuda")
            pt = dev(tb) if page else None
            if which == "append":
                st = kdtv.kv_append([kdtv.KvPart(cache, src=x)], dev(prefix), page_table=pt)
                flat = cache.reshape(B, T, 2, 16)
                for r in range(B):
                    want = torch.zeros((T, 2, 16), dtype=torch.bfloat16, device="cuda")
                    if r != b:
                        want[good[r]:good[r] + N] = x[r]
                    assert torch.equal(flat[r], want)
            else:
                st = kdtv.kv_read([kdtv.KvPart(cache, out=out)], dev(prefix), page_table=pt)
                for r in range(B):
                    assert (out[r] == (5.0 if r == b else 0.0)).all()
            assert int(st.item()) == code


def test_far_rows():
    """Rows of a cache beyond 2^31 bytes and 2^31 elements."""
    T, dim = (1 << 23) + 1000, 512                      # 4.3e9 elements of one byte
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    cache = torch.zeros((1, T, 1, dim), dtype=torch.uint8, device="cuda")
    L = (1 << 23) + 300
    x = dev(np.random.default_rng(5).standard_normal((1, 9, 1, dim), dtype=np.float32))
    scale = torch.zeros((1, T, 1), dtype=torch.uint8, device="cuda")
    out = torch.zeros((1, 9, 1, dim), device="cuda")
    at = dev(np.array([L], np.int32))
    assert int(kdtv.kv_append([kdtv.KvPart(cache, src=x, scale=scale)], at).item()) == 0
    assert int(kdtv.kv_read([kdtv.KvPart(cache, out=out, scale=scale)], at).item()) == 0
    want = f64(x)
    s = 2.0 ** O.row_exponent(want)[..., None]
    assert (np.abs(f64(out) - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s)).all()
    assert int(cache[0, :L].max()) == 0 and int(cache[0, L + 9:].max()) == 0


def test_graph_and_other_stream():
    """Captured and replayed with new values in the same buffers; called on a stream of its own."""
    rng = np.random.default_rng(6)
    x = dev(rng.standard_normal((2, 6, 4, 64), dtype=np.float32), torch.bfloat16)
    cache = torch.zeros((2, 40, 4, 64), dtype=torch.uint8, device="cuda")
    scale = torch.zeros((2, 40, 4), dtype=torch.uint8, device="cuda")
    y = torch.zeros_like(x)
    back = torch.zeros_like(x)
    prefix = dev(np.array([3, 30], np.int32))
    t = kdtv.RopeTable(64)
    ops = [kdtv.Rope(t, x, prefix_len=prefix, out=y),
           kdtv.KvAppend([kdtv.KvPart(cache, src=x, scale=scale, rot_off=0)], prefix, rope=t),
           kdtv.KvRead([kdtv.KvPart(cache, out=back, scale=scale)], prefix)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for op in ops:
        op(side)
    side.synchronize()
    first = (y.clone(), back.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for op in ops:
            op()
    for k in range(3):
        x.copy_(dev(rng.standard_normal((2, 6, 4, 64), dtype=np.float32), torch.bfloat16))
        prefix.copy_(dev(np.array([k, 20 + k], np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        got = (y.clone(), back.clone())
        assert not torch.equal(got[0], first[0])
        for op in ops:
            op()
        assert torch.equal(y, got[0]) and torch.equal(back, got[1])
    assert ops[1].status.item() == 0 and ops[2].status.item() == 0


def test_python_checks():
    x = torch.zeros((2, 3, 4, 64), device="cuda")
    t = kdtv.RopeTable(64)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(prefix_len=i.long()), dict(prefix_len=i.cpu()), dict(prefix_len=i[:1]),
                dict(depth=i), dict(rot_off=1), dict(out=x.bfloat16()), dict(out=x[:1]),
                dict(rest=x), dict(out=x[:, :, :1].expand(2, 3, 4, 64)),
                dict(out=x.as_strided((2, 3, 4, 64), (768, 256, 32, 1)))):
        with pytest.raises(ValueError):
            kdtv.rope(t, x, **bad)
    for bad in (x.half(), x.cpu(), x.transpose(2, 3), x[:0], x[0], x[0, 0, 0].expand(2, 3, 4, 64)):
        with pytest.raises(ValueError):
            kdtv.rope(t, bad)
    cache = torch.zeros((2, 8, 4, 64), dtype=torch.uint8, device="cuda")
    s = torch.zeros((2, 8, 4), dtype=torch.uint8, device="cuda")
    for part, kw in ((kdtv.KvPart(cache[:, ::2], src=x), {}), (kdtv.KvPart(cache, src=x[:1]), {}),
                     (kdtv.KvPart(cache, src=x, scale=s[:, :4]), {}), (kdtv.KvPart(cache, src=x, rot_off=0), {}),
                     (kdtv.KvPart(cache.float(), src=x, scale=s), {}), (kdtv.KvPart(cache.int(), src=x), {}),
                     (kdtv.KvPart(cache[..., :32].contiguous(), src=x), {}), (kdtv.KvPart(cache, src=None), {}),
                     (kdtv.KvPart(cache, src=x), dict(page_table=i)),
                     (kdtv.KvPart(cache, src=x[0, 0, 0].expand(2, 3, 4, 64)), {})):
        with pytest.raises(ValueError):
            kdtv.kv_append([part], i, **kw)


def test_broadcast_rows():
    """One row for all heads, or all requests: strides of 0 beside others."""
    rng = np.random.default_rng(7)
    t = kdtv.RopeTable(64)
    base = dev(rng.standard_normal((1, 3, 1, 64), dtype=np.float32))
    x = base.expand(2, 3, 4, 64)
    assert torch.equal(kdtv.rope(t, x), kdtv.rope(t, x.contiguous()))
    a, b = (torch.zeros((2, 8, 4, 64), device="cuda") for _ in range(2))
    at = dev(np.array([1, 5], np.int32))
    for cache, src in ((a, x), (b, x.contiguous())):
        assert int(kdtv.kv_append([kdtv.KvPart(cache, src=src, rot_off=0)], at, rope=t).item()) == 0
    assert torch.equal(a, b) and not torch.equal(a, torch.zeros_like(a))
    one = base[:, :1]                                  # one row: any strides
    assert torch.equal(kdtv.rope(t, one), kdtv.rope(t, one.clone()))


@pytest.mark.parametrize("kv_scale", [0.07, 3e-3, 1.75, 2.0 ** -9])
@pytest.mark.parametrize("heads,dim", [(1, 512), (1, 64), (6, 128), (3, 33)])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_static_scales_bit_by_bit(kv_scale, heads, dim, src):
    """The code nearest x / kv_scale in fp32 (a division, also where a product would do), and the
    code times kv_scale, rounded once."""
    x = dev(np.random.default_rng(8).standard_normal((2, 19, heads, dim), dtype=np.float32), DT[src])
    cache = torch.zeros((2, 30, heads, dim), dtype=torch.uint8, device="cuda")
    at = dev(np.array([3, 11], np.int32))
    assert int(kdtv.kv_append([kdtv.KvPart(cache, src=x)], at, kv_scale=kv_scale).item()) == 0
    s = np.float32(kv_scale)
    codes = torch.from_numpy(np.clip(x.float().cpu().numpy() / s, -448, 448)).to(torch.float8_e4m3fn)
    back = torch.zeros_like(x)
    assert int(kdtv.kv_read([kdtv.KvPart(cache, out=back)], at, dev(np.array([19, 19], np.int32)),
                            kv_scale=kv_scale).item()) == 0
    value = torch.from_numpy(codes.float().numpy() * s).to(DT[src])
    for b, L in enumerate((3, 11)):
        assert torch.equal(cache[b, L:L + 19].cpu(), codes[b].view(torch.uint8))
        assert torch.equal(back[b].cpu(), value[b])
