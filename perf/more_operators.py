"""Timed cases of the operators of kdtv that stand between the attention calls of a served step.

  norm   the residual's addition and a root-mean-square norm (kdtv.RmsNorm), to the inputs' type or
         to one byte per element with an exponent byte per 32; one-byte rows are widened behind it
         (kdtv.KvRead, the groups as heads), so that what comes out are the values the codes stand for
  proj   a projection that all requests share, with a low-rank adapter per request (kdtv.Project);
         float32, bfloat16, or one-byte inputs and weights with exponent bytes per 32
  pages  a paged cache's block tables and slot map from the requests' lengths, and the drafts'
         pages given back (kdtv.PagesResize)

``run`` computes each either in elementary torch operations (``own`` false) or with the library's
kernels (``own`` true); ``exact`` is the definition in 64 bits.  Lengths, live row counts and the
requests' adapters follow from the case alone, values and page ids from the seed.
"""

import math

import torch

own = False

DEV = "cuda"
FP8_MAX = 448.0                      # largest E4M3 value
GROUP = 32                           # elements that share an exponent byte
E_MIN, E_MAX = -117, 119             # range of the exponents
EPS = 1e-6


# ---- the cases ----------------------------------------------------------------------------

def _norm(name, B, N, H, dim, dtype, residual=True, one_byte=False, ragged=False, pad=0):
    """pad: elements between the rows of x (a part of a wider row)."""
    return dict(name=name, op="norm", B=B, N=N, H=H, dim=dim, dtype=dtype, residual=residual,
                one_byte=one_byte, ragged=ragged, pad=pad)


def _proj(name, B, N, K, M, dtype, adapters, rank, ragged=False):
    return dict(name=name, op="proj", B=B, N=N, K=K, M=M, dtype=dtype, adapters=adapters, rank=rank,
                ragged=ragged)


def _pages(name, B, N, page, Lmin, Lmax, ragged=False):
    return dict(name=name, op="pages", B=B, N=N, page=page, Lmin=Lmin, Lmax=Lmax, ragged=ragged)


def listed():
    return [
        # one decoded token of one request: pure latency
        _norm("norm_one_token", 1, 1, 1, 8192, "bf16"),
        # query heads of 64 chain drafts normed inside their wider rows (64 heads and 2 x 8 behind them)
        _norm("norm_heads_drafts", 64, 8, 64, 128, "bf16", residual=False, pad=2048),
        # a ragged prompt chunk normed to one byte, for the one-byte projection
        _norm("norm_prompt_one_byte", 4, 2000, 1, 8192, "bf16", one_byte=True, ragged=True),
        # a small fp32 drafter, odd everywhere
        _norm("norm_f32_odd", 3, 13, 1, 1001, "f32", ragged=True),
        # one decoded token of one request, with its adapter: the weights' bytes
        _proj("proj_one_token", 1, 1, 8192, 10240, "bf16", 8, 16),
        # one decoded token each of 64 requests with 40 adapters among them
        _proj("proj_decode_64", 64, 1, 8192, 8192, "bf16", 40, 16),
        # 64 chain drafts of 8 nodes, one-byte weights
        _proj("proj_drafts_one_byte", 64, 8, 8192, 8192, "fp8", 16, 32),
        # a ragged prompt chunk of four requests
        _proj("proj_prompt", 4, 2000, 4096, 12288, "bf16", 3, 64, ragged=True),
        # long prompts, one-byte weights: the largest
        _proj("proj_prompt_one_byte", 2, 4096, 8192, 8192, "fp8", 4, 16),
        # an fp32 drafter with sizes that are multiples of nothing
        _proj("proj_f32_odd", 3, 13, 1001, 515, "f32", 2, 5, ragged=True),
        # pages for 64 chain drafts, their slots, and the pages given back
        _pages("pages_drafts", 64, 8, 64, 1024, 32768),
        # ragged prompts of 512 new requests
        _pages("pages_prompts", 512, 6000, 16, 0, 0, ragged=True),
    ]


def draw(rng):
    def logu(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm", "proj", "proj", "proj", "pages"])
    if op == "norm":
        heads = rng.random() < 0.4
        H, dim = (rng.choice([1, 8, 14, 64]), rng.choice([64, 80, 128, 192])) if heads else (1, logu(256, 16384))
        one_byte = not heads and rng.random() < 0.5
        if one_byte:
            dim = -(-dim // GROUP) * GROUP
        elif not heads and rng.random() < 0.7:
            dim = -(-dim // 8) * 8
        B, N = logu(1, 64), logu(1, 4000)
        while B * N * H * dim > 60 * 10 ** 6:
            N, B = max(1, N * 2 // 3), max(1, B * 2 // 3)
        c = _norm("", B, N, H, dim, "bf16" if one_byte else rng.choice(["bf16", "bf16", "f32"]),
                  residual=not heads, one_byte=one_byte, ragged=rng.random() < 0.5,
                  pad=0 if rng.random() < 0.5 else 8 * rng.randint(1, 200))
    elif op == "proj":
        dtype = rng.choice(["bf16", "bf16", "fp8", "fp8", "f32"])
        K, M = logu(256, 8192), logu(64, 16384)
        K = K if dtype == "f32" else -(-K // 8) * 8 if dtype == "bf16" else -(-K // GROUP) * GROUP
        if rng.random() < 0.7:
            M = -(-M // 64) * 64
        B, N = (logu(1, 256), rng.choice([1, 1, 8, logu(2, 128)])) if rng.random() < 0.6 else (logu(1, 8), logu(64, 5000))
        rank = rng.choice([3, 8, 20]) if dtype == "f32" else rng.choice([8, 16, 16, 32, 64])
        while B * N * K * M > (6 * 10 ** 9 if dtype == "f32" else 5 * 10 ** 11) or B * rank * K > 10 ** 8:
            N, B = max(1, N * 2 // 3), max(1, B * 2 // 3)
        c = _proj("", B, N, K, M, dtype, min(B + 3, logu(1, 64)), rank, ragged=rng.random() < 0.5)
    else:
        B = logu(1, 512)
        lo = rng.choice([0, logu(1, 20000)])
        N = rng.choice([1, 8, logu(2, 128)]) if lo else logu(16, 6000)
        page = rng.choice([16, 32, 64, 100, 128])
        c = _pages("", B, N, page, lo, 2 * lo, ragged=rng.random() < 0.5)
    del c["name"]
    return c


# ---- lengths and adapters (from the case alone) -----------------------------------------------

def _spread(lo, hi, count, phase):
    """`count` whole numbers of [lo, hi], evenly spread over their logarithm."""
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    return [min(hi, max(lo, int(round(math.exp(a + (b - a) * ((0.61803398875 * (i + 1) + phase) % 1.0)) - 1))))
            for i in range(count)]


def _live(c):
    n = _spread(max(1, c["N"] // 4), c["N"], c["B"], 0.43) if c["ragged"] else [c["N"]] * c["B"]
    if c["ragged"]:
        n[0] = c["N"]
    return n


def _lengths(c):
    return _spread(c["Lmin"], c["Lmax"], c["B"], 0.17) if c["Lmax"] > c["Lmin"] else [c["Lmin"]] * c["B"]


def _adapters(c):
    """Adapter of each request: every ninth has none, the others are spread unevenly."""
    return [-1 if b % 9 == 8 else (b * b + 3 * b) % c["adapters"] for b in range(c["B"])]


def work(c):
    n = _live(c)
    live = sum(n)
    if c["op"] == "norm":
        e = 4 if c["dtype"] == "f32" else 2
        elems = live * c["H"] * c["dim"]
        out = elems * (1 + e) + 2 * elems // GROUP + elems if c["one_byte"] else elems * e
        return {"bytes": elems * e * (3 if c["residual"] else 1) + out + c["dim"] * e, "flops": 5 * elems}
    if c["op"] == "proj":
        K, M, R = c["K"], c["M"], c["rank"]
        e = {"f32": 4.0, "bf16": 2.0, "fp8": 1.0 + 1.0 / GROUP}[c["dtype"]]
        w = 4 if c["dtype"] == "f32" else 2
        ids = _adapters(c)
        used = len({a for a in ids if a >= 0})
        turned = sum(m for m, a in zip(n, ids) if a >= 0)
        return {"bytes": int(K * M * e + live * K * e) + live * M * w + used * R * (K + M) * w,
                "flops": 2 * live * K * M + 2 * turned * R * (K + M)}
    moved = sum(-(-(l + m) // c["page"]) + -(-l // c["page"]) * -1 for l, m in zip(_lengths(c), n))
    return {"bytes": 8 * c["B"] * c["N"] + 4 * live // c["page"] + 16 * moved + 32 * c["B"], "flops": 2 * live}


# ---- inputs ------------------------------------------------------------------------------

def _pow2(e):
    """2^e in float32, e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x):
    """Codes (float8_e4m3fn) like x, and exponent bytes [.., dim / GROUP]."""
    g = x.unflatten(-1, (-1, GROUP))
    m, k = torch.frexp(g.abs().amax(-1))
    e = (k - 9 + (m > 0.875).to(k.dtype)).clamp(E_MIN, E_MAX)
    y = (g * _pow2(-e)[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return y.flatten(-2), (e + 127).to(torch.uint8)


def _widened(codes, scale):
    return (codes.float().unflatten(-1, (-1, GROUP)) * _pow2(scale.int() - 127)[..., None]).flatten(-2)


def prepare(c, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)

    def normal(shape, dtype, std=1.0):
        return (torch.randn(shape, generator=gd, device=DEV, dtype=torch.float32) * std).to(dtype)

    B, N = c["B"], c["N"]
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    s = {"c": c, "n_live": torch.tensor(_live(c), dtype=torch.int32, device=DEV)}
    if c["op"] == "norm":
        H, dim = c["H"], c["dim"]
        wide = normal((B, N, H * dim + c["pad"]), dt, 2.0)
        s["x"] = wide[..., :H * dim].view(B, N, H, dim)
        s["weight"] = (1.0 + 0.2 * normal((dim,), torch.float32)).to(dt)
        s["residual"] = s["residual_out"] = None
        if c["residual"]:
            s["residual"] = normal((B, N, H, dim), dt, 5.0)
            s["residual"][..., :3] *= 30.0                     # a few channels carry most of the stream
            s["residual_out"] = torch.zeros_like(s["residual"])
        s["y"] = torch.zeros((B, N, H, dim), dtype=dt, device=DEV)
        if c["one_byte"]:
            s["codes"] = torch.zeros((B, N, H, dim), dtype=torch.uint8, device=DEV)
            s["scale"] = torch.zeros((B, N, H, dim // GROUP), dtype=torch.uint8, device=DEV)
        return s
    if c["op"] == "proj":
        K, M, R, A = c["K"], c["M"], c["rank"], c["adapters"]
        x = normal((B, N, K), dt)
        x[..., ::97] *= 8.0
        W = normal((M, K), dt, 1.0 / math.sqrt(K))
        s["x_scale"] = s["W_scale"] = None
        if c["dtype"] == "fp8":
            x, s["x_scale"] = _quantised(x.float())
            W, s["W_scale"] = _quantised(W.float())
        s["x"], s["W"] = x, W
        s["A"] = normal((A, R, K), dt, 1.0 / math.sqrt(K))
        s["Bm"] = normal((A, M, R), dt, 0.5 / math.sqrt(R))
        s["adapter_scale"] = torch.linspace(0.5, 2.0, A, device=DEV)
        s["adapter"] = torch.tensor(_adapters(c), dtype=torch.int32, device=DEV)
        s["y"] = torch.zeros((B, N, M), dtype=dt, device=DEV)
        return s
    # pages: requests that hold the pages of their prefix, the other pages free, in any order
    L, n, page = _lengths(c), _live(c), c["page"]
    held = [-(-l // page) for l in L]
    need = sum(-(-(l + m) // page) for l, m in zip(L, n))
    num = need + 7
    perm = torch.randperm(num, generator=g).to(torch.int32)
    width = max(-(-(l + c["N"]) // page) for l in L) + 1
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = perm[at:at + k]
        at += k
    free = torch.full((num,), -1, dtype=torch.int32)
    free[:num - at] = perm[at:]
    s["L"] = torch.tensor(L, dtype=torch.int32, device=DEV)
    s["page_table"], s["free"] = table.to(DEV), free.to(DEV)
    s["free_count"] = torch.tensor([num - at], dtype=torch.int32, device=DEV)
    s["n_pages"] = torch.tensor(held, dtype=torch.int32, device=DEV)
    s["slots"] = torch.zeros((B, N), dtype=torch.int64, device=DEV)
    s["none"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    return s


# ---- one pass --------------------------------------------------------------------------------

def _handle(s):
    """The library's callers over this state's tensors, made on the state's first pass."""
    if "op" not in s:
        from speculative_decoding_tree_mla_gb300 import kdtv
        c = s["c"]
        if c["op"] == "norm":
            kw = dict(residual=s["residual"], residual_out=s["residual_out"], n_live=s["n_live"], eps=EPS)
            if c["one_byte"]:
                B, N, H, dim = s["x"].shape
                groups = (B, N, H * dim // GROUP, GROUP)
                s["op"] = [kdtv.RmsNorm(s["x"], s["weight"], out=s["codes"], out_scale=s["scale"], **kw),
                           kdtv.KvRead([kdtv.KvPart(s["codes"].view(groups), scale=s["scale"].view(groups[:3]),
                                                    out=s["y"].view(groups))], None, s["n_live"])]
            else:
                s["op"] = [kdtv.RmsNorm(s["x"], s["weight"], out=s["y"], **kw)]
        elif c["op"] == "proj":
            s["op"] = [kdtv.Project(s["x"], s["W"], x_scale=s["x_scale"], W_scale=s["W_scale"], A=s["A"],
                                    Bm=s["Bm"], adapter=s["adapter"], adapter_scale=s["adapter_scale"],
                                    n_live=s["n_live"], out=s["y"])]
        else:
            pool = kdtv.PagePool(s["page_table"], s["n_pages"], s["free"], s["free_count"], c["page"])
            s["op"] = [kdtv.PagesResize(pool, s["L"], n_live=s["n_live"], slots=s["slots"]),
                       kdtv.PagesResize(pool, s["L"], N=0)]
    return s["op"]


def _outputs(s):
    c = s["c"]
    if c["op"] == "norm":
        return {"y": s["y"], "residual": s["residual_out"]} if c["residual"] else {"y": s["y"]}
    if c["op"] == "proj":
        return {"y": s["y"]}
    return {k: s[k] for k in ("slots", "page_table", "n_pages", "free", "free_count")}


def run(s):
    c = s["c"]
    if own:
        for call in _handle(s):
            call()
        return _outputs(s)
    if c["op"] == "norm":
        _plain_norm(s)
    elif c["op"] == "proj":
        _plain_proj(s)
    else:
        rows = s["n_live"].long()
        s["slots"].copy_(_plain_resize(s, s["L"].long() + rows))
        _plain_resize(s, s["L"].long())
    return _outputs(s)


def _alive(s):
    return torch.arange(s["c"]["N"], device=DEV)[None] < s["n_live"][:, None]


def _plain_norm(s):
    c = s["c"]
    live = _alive(s)[:, :, None, None]
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
        s["residual_out"].copy_(torch.where(live, h.to(s["x"].dtype), s["residual_out"]))
    y = h * (1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)) * s["weight"].float()
    if c["one_byte"]:
        y = _widened(*_quantised(y))
    s["y"].copy_(torch.where(live, y.to(s["y"].dtype), s["y"]))


def _plain_proj(s):
    c = s["c"]
    if c["dtype"] == "fp8":
        x, W = _widened(s["x"], s["x_scale"]), _widened(s["W"], s["W_scale"])
    else:
        x, W = s["x"].float(), s["W"].float()
    y = x @ W.t()
    a = s["adapter"].long()
    has = (a >= 0).float() * s["adapter_scale"][a.clamp_min(0)]
    a = a.clamp_min(0)
    low = torch.bmm(x, s["A"][a].float().transpose(1, 2)) * has[:, None, None]
    y = torch.baddbmm(y, low, s["Bm"][a].float().transpose(1, 2))
    s["y"].copy_(torch.where(_alive(s)[:, :, None], y.to(s["y"].dtype), s["y"]))


def _plain_resize(s, rows):
    """Tables, counts and free pages for `rows` rows of each request; the slots of the rows from
    the prefix on.  Pages go back from the last request to the first, each from its end."""
    c = s["c"]
    page, table = c["page"], s["page_table"]
    have, want = s["n_pages"].long(), (rows + page - 1) // page
    give, take = (have - want).clamp_min(0), (want - have).clamp_min(0)
    i = torch.arange(table.shape[1], device=DEV)[None]
    top = s["free_count"].long()
    back = (i >= want[:, None]) & (i < have[:, None])
    behind = give.sum() - give.cumsum(0)                       # pages of the requests behind
    at = torch.where(back, top + behind[:, None] + have[:, None] - 1 - i, s["free"].numel())
    free = torch.cat((s["free"], s["free"].new_zeros(1))).scatter_(0, at.flatten(), table.flatten())[:-1]
    top = top + give.sum()
    new = (i >= have[:, None]) & (i < want[:, None])
    at = top - 1 - (take.cumsum(0) - take)[:, None] - (i - have[:, None])
    table.copy_(torch.where(new, free[at.clamp(0, free.numel() - 1)], torch.where(back, -1, table)))
    s["free"].copy_(free)
    s["free_count"].copy_(top - take.sum())
    s["n_pages"].copy_(want)
    t = s["L"].long()[:, None] + torch.arange(c["N"], device=DEV)[None]
    live = t < rows[:, None]
    p = table.gather(1, (t // page).clamp_max(table.shape[1] - 1)).long()
    return torch.where(live, p * page + t % page, -1)


# ---- the definition in 64 bits ---------------------------------------------------------------

def _nearest_codes(x):
    """Values [.., groups, GROUP] as one byte with an exponent per group holds them, in 64 bits."""
    e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / FP8_MAX)).clamp(E_MIN, E_MAX)
    x = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.round(x / step) * step * torch.exp2(e)


def _values(x, scale):
    if scale is None:
        return x.double()
    return x.double() * torch.exp2(scale.double() - 127.0).repeat_interleave(GROUP, -1)


def exact(c, seed):
    if c["op"] == "pages":
        return None
    s = prepare(c, seed)
    n = _live(c)
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    if c["op"] == "norm":
        res = torch.zeros_like(y) if c["residual"] else None
        w = s["weight"].double()
        for b, m in enumerate(n):
            h = s["x"][b, :m].double()
            if res is not None:
                h += s["residual"][b, :m]
                res[b, :m] = h
            v = h / (h.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * w
            y[b, :m] = _nearest_codes(v.unflatten(-1, (-1, GROUP))).flatten(-2) if c["one_byte"] else v
        return {"y": y} if res is None else {"y": y, "residual": res}
    if 2 * sum(n) * c["K"] * c["M"] > 4e12:
        return None
    W = _values(s["W"], s["W_scale"])
    for b, (m, a) in enumerate(zip(n, _adapters(c))):
        x = _values(s["x"][b, :m], None if s["x_scale"] is None else s["x_scale"][b, :m])
        y[b, :m] = torch.einsum("ik,mk->im", x, W)
        if a >= 0:
            low = torch.einsum("ik,rk->ir", x, s["A"][a].double())
            y[b, :m] += float(s["adapter_scale"][a]) * torch.einsum("ir,mr->im", low, s["Bm"][a].double())
    return {"y": y}
