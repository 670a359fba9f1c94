"""kdtv_rmsnorm against the fp64 oracle.

Tolerances.  fp32: a thread's sum of squares is a chain of at most 40 terms, the reduction adds 11: the
sum is within 51 * 2^-24, its root's reciprocal within 26 * 2^-24 plus three roundings (mean, root,
reciprocal), the two products add two more, and h itself one: 2^-19 covers it.  Then half a step of the
output type relative to the value (bf16 2^-8).  One byte: half a step of E4M3, 2^-4 of the value, or 2^-10 of
the exponent's unit below the smallest normal."""

import numpy as np
import pytest

from oracle import serve_ops as O
from speculative_decoding_tree_mla_gb300 import kdtv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ARITH = 2.0 ** -19
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.float().cpu().double().numpy()


def make(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(TYPE[dtype])


def near(got, want, tol, floor=0.0):
    err = np.abs(got - want)
    assert (err <= tol * np.abs(want) + floor).all(), float((err / (np.abs(want) + 1e-30)).max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,dim", [
    (1, 1, 1, 8192), (1, 1, 1, 1), (3, 5, 1, 7), (2, 3, 4, 128), (5, 70, 8, 64), (1, 2, 1, 32768), (1, 3, 1, 32767),
    (400, 1, 1, 576), (3, 200, 1, 1536), (2, 300, 1, 8192), (2, 200, 1, 20000), (7, 60, 3, 80), (2, 400, 1, 1001),
    (700, 1, 2, 8), (330, 1, 1, 9000)])
def test_matches_oracle(dtype, B, N, H, dim):
    x, r, w = make((B, N, H, dim), dtype, 1, 2.0), make((B, N, H, dim), dtype, 2, 5.0), make((dim,), dtype, 3)
    out, kept = torch.zeros_like(x), torch.zeros_like(x)
    kdtv.rmsnorm(x, w, residual=r, residual_out=kept, eps=1e-5, out=out)
    y, h = O.rmsnorm(f64(x), f64(w), 1e-5, f64(r))
    near(f64(out), y, ARITH + STEP[dtype])
    near(f64(kept), h, STEP[dtype])
    plain = kdtv.rmsnorm(x, w, eps=1e-5)                       # without a residual
    near(f64(plain), O.rmsnorm(f64(x), f64(w), 1e-5)[0], ARITH + STEP[dtype])
    bare = kdtv.rmsnorm(x, eps=0.0)
    near(f64(bare), O.rmsnorm(f64(x), None, 0.0)[0], ARITH + STEP[dtype])
    shifted = kdtv.rmsnorm(x, w, weight_offset=1.0)            # (w + 1 is rounded to fp32, relative to its terms)
    near(f64(shifted), O.rmsnorm(f64(x), f64(w), 1e-6, weight_offset=1.0)[0], ARITH + STEP[dtype],
         2.0 ** -24 * 4 * float(x.float().abs().max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,dim", [(1, 1, 1, 8192), (1, 1, 1, 32), (2, 3, 4, 64), (3, 150, 1, 4096), (500, 1, 1, 96),
                                       (1, 2, 1, 32768), (350, 1, 1, 1056), (2, 3, 1, 9984)])
def test_one_byte(dtype, B, N, H, dim):
    x, r, w = make((B, N, H, dim), dtype, 4, 2.0), make((B, N, H, dim), dtype, 5, 4.0), make((dim,), dtype, 6)
    x[0, 0, 0, : min(dim, 40)] *= 0.0                          # a group that is all zero
    r[0, 0, 0, : min(dim, 40)] *= 0.0
    codes, scale = kdtv.rmsnorm(x, w, residual=r, residual_out=False, one_byte=True)
    assert codes.dtype == torch.uint8 and scale.shape == (B, N, H, dim // 32)
    y, _ = O.rmsnorm(f64(x), f64(w), 1e-6, f64(r))
    check_one_byte(codes, scale, y)


def check_one_byte(codes, scale, y):
    s = scale.cpu().numpy().astype(np.int64) - 127
    want = O.group_exponent(y)
    top = np.abs(y).reshape(want.shape + (32,)).max(-1)
    border = np.abs(top / (448.0 * 2.0 ** np.minimum(s, want)) - 1.0) < 2 * ARITH
    assert ((s == want) | (border & (np.abs(s - want) == 1))).all()
    got = O.widen(codes.cpu().numpy(), scale.cpu().numpy())
    unit = np.repeat(2.0 ** s.astype(np.float64), 32, axis=-1)
    assert (np.abs(got - y) <= np.maximum((2.0 ** -4 + ARITH) * np.abs(y), 2.0 ** -10 * unit)).all()


def test_one_byte_odd_addresses():
    """Rows that start off 16 bytes take the element-wise instance."""
    base = make((3, 40, 321), "bf16", 7)
    x = base[:, :, 1:]
    codes, scale = kdtv.rmsnorm(x, one_byte=True)
    check_one_byte(codes, scale, O.rmsnorm(f64(x), None, 1e-6)[0])


@pytest.mark.parametrize("one_byte", [False, True])
def test_strides_and_live_rows(one_byte):
    """Parts of wider rows, ragged live rows: what is not live, and what lies beside the part, stays."""
    B, N, H, dim = 4, 9, 3, 64
    wide = make((B, N, H * dim + 40), "bf16", 8)
    x = wide[..., 16:16 + H * dim].unflatten(-1, (H, dim))
    res_wide = make((B, N, H, dim + 8), "bf16", 9)
    res = res_wide[..., :dim]
    before = res_wide.clone()
    n = torch.tensor([9, 0, 4, 100], dtype=torch.int32, device="cuda")
    w = make((dim,), "bf16", 10)
    y, h = O.rmsnorm(f64(x), f64(w), 1e-6, f64(res))
    if one_byte:
        out = torch.full((B, N, H, dim), 77, dtype=torch.uint8, device="cuda")
        scale = torch.full((B, N, H, dim // 32), 78, dtype=torch.uint8, device="cuda")
        kdtv.rmsnorm(x, w, residual=res, n_live=n, out=out, out_scale=scale)
    else:
        out_wide = torch.full((B, N, H * dim + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        out = out_wide[..., 8:8 + H * dim].unflatten(-1, (H, dim))
        kdtv.rmsnorm(x, w, residual=res, n_live=n, out=out)
        assert (out_wide[..., :8] == 7.0).all() and (out_wide[..., 8 + H * dim:] == 7.0).all()
    assert torch.equal(res_wide[..., dim:], before[..., dim:])
    for b, m in enumerate([9, 0, 4, 9]):
        if m:
            near(f64(res[b, :m]), h[b, :m], STEP["bf16"])
            if one_byte:
                check_one_byte(out[b, :m], scale[b, :m], y[b, :m])
            else:
                near(f64(out[b, :m]), y[b, :m], ARITH + STEP["bf16"])
        assert torch.equal(res[b, m:], before[b, m:, :, :dim])
        assert (out[b, m:] == (77 if one_byte else 7.0)).all()
        if one_byte:
            assert (scale[b, m:] == 78).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,pad,off", [(64, 1, 0), (65, 0, 0), (66, 3, 5), (100, 7, 3), (333, 0, 0), (858, 0, 2), (4365, 4, 1),
                                         (8191, 2, 7), (16383, 0, 0), (32750, 1, 1), (72, 9, 4)])
def test_rows_that_start_anywhere(dtype, dim, pad, off):
    """All of a row's tensors the same distance behind 16 bytes (or not: the last run); what lies beside the rows stays."""
    B, N = 3, (200 if dim < 1000 else 7)

    def part(seed, shift=off):
        wide = make((B * N * (dim + pad) + 64,), dtype, seed)
        return wide, wide[shift:].as_strided((B, N, dim), (N * (dim + pad), dim + pad, 1))

    w = make((dim,), dtype, 43)
    n = torch.tensor([N, 3, 0], dtype=torch.int32, device="cuda")
    for shifts in ((off,) * 4, (off, off + 1, off, off + 2)):
        (_, x), (rw, r), (kw, kept), (ow, out) = (part(40 + k, s) for k, s in enumerate(shifts))
        before = rw.clone(), kw.clone(), ow.clone()
        y, h = O.rmsnorm(f64(x), f64(w), 1e-6, f64(r))
        kdtv.rmsnorm(x, w, residual=r, residual_out=kept, out=out, n_live=n)
        for b, m in enumerate((N, 3, 0)):
            near(f64(out[b, :m]), y[b, :m], ARITH + STEP[dtype])
            near(f64(kept[b, :m]), h[b, :m], STEP[dtype])
        assert torch.equal(rw, before[0])
        for wide, was, t in ((kw, before[1], kept), (ow, before[2], out)):
            for b, m in enumerate((N, 3, 0)):
                t[b, :m] = 0
            s = shifts[2] if t is kept else shifts[3]
            mine = was[s:].as_strided((B, N, dim), (N * (dim + pad), dim + pad, 1))
            for b, m in enumerate((N, 3, 0)):
                mine[b, :m] = 0
            assert torch.equal(wide, was)
    _, x = part(44)
    y, _ = O.rmsnorm(f64(x), f64(w), 1e-6)
    kdtv.rmsnorm(x, w, out=x)                                  # in place
    near(f64(x), y, ARITH + STEP[dtype])


@pytest.mark.parametrize("dim", [64, 1000, 8192])
def test_in_place(dim):
    for where in ("x", "residual"):
        x, r, w = make((3, 5, dim), "bf16", 11), make((3, 5, dim), "bf16", 12), make((dim,), "bf16", 13)
        y, h = O.rmsnorm(f64(x), f64(w), 1e-6, f64(r))
        if where == "x":
            kdtv.rmsnorm(x, w, residual=r, out=x)
            near(f64(x), y, ARITH + STEP["bf16"])
            near(f64(r), h, STEP["bf16"])
        else:
            kdtv.rmsnorm(x, w, residual=r, residual_out=x, out=r)
            near(f64(r), y, ARITH + STEP["bf16"])
            near(f64(x), h, STEP["bf16"])


def test_values_that_are_not_finite():
    """A row with an infinity or NaN keeps to itself; in one byte infinities saturate, NaN stays NaN."""
    x = make((4, 1, 256), "bf16", 14)
    x[1, 0, 5] = float("inf")
    x[2, 0, 70] = float("nan")
    out = kdtv.rmsnorm(x)
    y, _ = O.rmsnorm(f64(x), None, 1e-6)
    got = f64(out)
    near(got[[0, 3]], y[[0, 3]], ARITH + STEP["bf16"])
    assert np.isnan(got[1, 0, 5]) and (got[1, 0, np.arange(256) != 5] == 0).all() and np.isnan(got[2]).all()
    codes, scale = kdtv.rmsnorm(x, one_byte=True)
    v = O.widen(codes.cpu().numpy(), scale.cpu().numpy())
    assert np.isnan(v[1, 0, 5]) and (v[1, 0, np.arange(256) != 5] == 0).all() and np.isnan(v[2]).all()
    check_one_byte(codes[[0, 3]], scale[[0, 3]], y[[0, 3]])
    zero = kdtv.rmsnorm(torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda"))
    assert (zero == 0).all()
    w = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    w[7] = float("inf")                                        # an infinite value beside finite ones
    x = make((1, 1, 256), "bf16", 15)
    codes, scale = kdtv.rmsnorm(x, w, one_byte=True)
    v = O.widen(codes.cpu().numpy(), scale.cpu().numpy())[0, 0]
    assert abs(v[7]) == 448.0 * 2.0 ** (int(scale[0, 0, 0]) - 127) and np.isfinite(v).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [8, 64, 333, 8192])
def test_squares_beyond_fp32(dtype, dim):
    """Rows times 2^100 and 2^-100 (and up to the type's largest) beside ordinary ones."""
    x = make((6, 5, 3, dim), dtype, 30)
    for k, f in enumerate((2.0 ** 100, 2.0 ** -100, 2.0 ** 62, 2.0 ** -66)):
        x[k] = (x[k].double() * f).to(x.dtype)
    x[4, 0, 0, 0] = 3.0e38
    x[4, 1, 2, dim - 1] = 2.0 ** -120
    for eps in (0.0, 1e-6, 3.0):
        near(f64(kdtv.rmsnorm(x, eps=eps)), O.rmsnorm(f64(x), None, eps)[0], ARITH + STEP[dtype], 2.0 ** -133)
    if dim % 32 == 0:
        check_one_byte(*kdtv.rmsnorm(x, eps=0.0, one_byte=True), O.rmsnorm(f64(x), None, 0.0)[0])


def test_deterministic_streams_and_capture():
    x, r, w = make((64, 8, 4096), "bf16", 16), make((64, 8, 4096), "bf16", 17), make((4096,), "bf16", 18)
    op = kdtv.RmsNorm(x, w, residual=r, residual_out=torch.empty_like(r), one_byte=True)
    codes, scale = (t.clone() for t in op())
    side = torch.cuda.Stream()
    again = op(side)
    side.synchronize()
    assert torch.equal(again[0], codes) and torch.equal(again[1], scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op()
    x.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    y, _ = O.rmsnorm(f64(x[:2]), f64(w), 1e-6, f64(r[:2]))
    check_one_byte(op.out[:2], op.out_scale[:2], y)


def test_python_refusals():
    x = make((2, 3, 64), "bf16", 19)
    for kw in (dict(weight=x[0, 0].float()), dict(weight=x[0, 0, :32]), dict(residual=x.float()), dict(residual_out=x),
               dict(out=x.float()), dict(out=x.expand(2, 3, 64)[:1].expand(2, 3, 64)), dict(n_live=torch.zeros(2, device="cuda")),
               dict(one_byte=True, out_scale=torch.zeros(2, 3, 3, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            kdtv.rmsnorm(x, **kw)
    with pytest.raises(ValueError):
        kdtv.rmsnorm(x[..., :40].contiguous(), one_byte=True)
    with pytest.raises(ValueError):
        kdtv.rmsnorm(x.cpu())
    with pytest.raises(kdtv.KdtvError, match="UNSUPPORTED"):
        kdtv.rmsnorm(make((1, 1, 32776), "bf16", 20))


def test_strides_of_single_rows():
    """A dimension of one element may have any stride: in place by two views of the same row, and rows of 16-byte
    words whatever lies beside them."""
    buf, w = make((1, 6, 64), "bf16", 45), make((64,), "bf16", 46)
    x = buf[:, 2:3]
    y, _ = O.rmsnorm(f64(x), f64(w), 1e-6)
    before = buf.clone()
    kdtv.rmsnorm(x, w, out=x.as_strided((1, 1, 64), (64, 64, 1), x.storage_offset()))
    near(f64(x), y, ARITH + STEP["bf16"])
    assert torch.equal(buf[:, :2], before[:, :2]) and torch.equal(buf[:, 3:], before[:, 3:])
    res = buf[:, 4:5]
    y, h = O.rmsnorm(f64(x), f64(w), 1e-6, f64(res))
    kdtv.rmsnorm(x, w, residual=res, residual_out=res.as_strided((1, 1, 64), (1, 3, 1), res.storage_offset()), out=x)
    near(f64(x), y, ARITH + STEP["bf16"])
    near(f64(res), h, STEP["bf16"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [8, 64, 333, 8190, 8192, 32768])
def test_rows_of_subnormals(dtype, dim):
    """No eps, rows down to the type's smallest values: one such element among zeros, several, a row full of them,
    and such elements beside larger ones.  (The elements and their sums are exact, as everywhere; the statistic is of the row
    scaled by a power of two, so the bounds are those of ordinary rows.)"""
    least = 2.0 ** -149 if dtype == "f32" else 2.0 ** -133
    x = torch.zeros((12, 1, dim), dtype=torch.float64)
    x[0, 0, dim // 2] = 2.0 ** -145 if dtype == "f32" else least
    x[1, 0, 0] = -least
    x[2, 0, ::3] = 3 * least
    x[3] = least
    x[4] = 2.0 ** -126
    x[5, 0, : dim // 2] = least
    x[5, 0, dim - 1] = 2.0 ** -118
    x[6, 0, 1] = 2.0 ** -106
    x[7, 0, ::2] = -5 * 2.0 ** -109
    x[8, 0, ::5] = 2.0 ** -103
    x[9, 0, 3] = 1.75 * 2.0 ** -90
    x[10, 0, dim - 1] = 2.0 ** -31
    x[11] = torch.linspace(-40, 40, dim).round().double() * least
    x[11, 0, 0] = 40 * least
    x = x.to("cuda", TYPE[dtype])
    y, _ = O.rmsnorm(f64(x), None, 0.0)
    near(f64(kdtv.rmsnorm(x, eps=0.0)), y, ARITH + STEP[dtype])
    ordinary = make((1, 1, dim), dtype, 47)                    # beside an ordinary row, and with a residual that takes all away
    both = torch.cat((ordinary, x, -x, ordinary))
    near(f64(kdtv.rmsnorm(both, eps=0.0)), O.rmsnorm(f64(both), None, 0.0)[0], ARITH + STEP[dtype])
    near(f64(kdtv.rmsnorm(x, eps=0.0, residual=x.clone())), O.rmsnorm(f64(x), None, 0.0, f64(x))[0], ARITH + STEP[dtype])
    if dim % 32 == 0:
        check_one_byte(*kdtv.rmsnorm(x, eps=0.0, one_byte=True), y)
    tiny = float(np.float32(2.0 ** -140))                      # an eps of that size counts
    x = torch.full((1, 1, dim), 2.0 ** -70, dtype=TYPE[dtype], device="cuda")
    near(f64(kdtv.rmsnorm(x, eps=tiny)), O.rmsnorm(f64(x), None, tiny)[0], ARITH + STEP[dtype])


@pytest.mark.parametrize("where", ["whole", "any address"])
def test_largest_rows_keep_their_bits(where):
    """Rows of +-m / 128 * 2^127: squares, their sum and its root are exact in fp32 once a power of two is taken out, so
    1 is off by the reciprocal's rounding and the product's: 2^-23."""
    m = torch.tensor([129, 200, 216, 217, 222, 231, 244, 253, 255], dtype=torch.float64)
    x = ((m / 128)[:, None, None] * 2.0 ** 127 * torch.tensor([1.0, -1.0], dtype=torch.float64).repeat(256)[None, None]).float().cuda()
    if where != "whole":
        wide = torch.zeros((9, 1, 515), device="cuda")
        wide[..., 3:] = x
        x = wide[..., 3:]
    got = f64(kdtv.rmsnorm(x, eps=0.0))
    near(got, np.sign(f64(x)), 2.0 ** -23)
    codes, scale = kdtv.rmsnorm(x, eps=0.0, one_byte=True)
    assert np.array_equal(O.widen(codes.cpu().numpy(), scale.cpu().numpy()), np.sign(f64(x)))
