"""Timed cases of the rotary, cache and grouped-query attention operators of kdtv.

Three groups of calls that a serving step makes around a tree-verify attention:

  rope   rotary positions applied to queries (kdtv.Rope)
  kv     new rows rotated, quantised and written into a latent (MLA) or a
         key/value (GQA) cache (kdtv.KvAppend); for a one-byte cache the rows
         are read back in bf16 (kdtv.KvRead), so that what comes out are the
         values the codes stand for
  read   a span of a cache read back into contiguous rows (kdtv.KvRead)
  attn   attention of a draft tree over a paged or contiguous GQA cache
         (kdtv.GqaVerifyAttn)

``run`` computes each either in elementary torch operations (``own`` false) or
with the library's kernels (``own`` true); ``exact`` is the definition in 64
bits.  Prefix lengths and live row counts follow from the case alone, values
and trees from the seed.
"""

import math

import torch

own = False

DEV = "cuda"
FP8_MAX = 448.0                      # largest E4M3 value
MLA_SCALE = 0.125                    # static scale of the one-byte latent cache
E_MIN, E_MAX = -117, 119             # range of the per-row exponents of a one-byte GQA cache


# ---- the cases ----------------------------------------------------------------------------

def _rope(name, B, N, H, dim, rot, off, layout, scaling, dtype, Lmin, Lmax, tree=False,
          split=False, ragged=False, base=10000.0, factor=1.0, orig=4096):
    return dict(name=name, op="rope", B=B, N=N, H=H, dim=dim, rot=rot, off=off, layout=layout,
                scaling=scaling, dtype=dtype, Lmin=Lmin, Lmax=Lmax, tree=tree, split=split,
                ragged=ragged, base=base, factor=factor, orig=orig)


def _kv(name, op, kind, B, N, Hkv, D, dtype, cache, page, Lmin, Lmax, tree=False, ragged=False):
    return dict(name=name, op=op, kind=kind, B=B, N=N, Hkv=Hkv, D=D, dtype=dtype, cache=cache,
                page=page, Lmin=Lmin, Lmax=Lmax, tree=tree, ragged=ragged)


def _attn(name, B, N, Hq, Hkv, D, cache, page, Lmin, Lmax, ragged=False):
    return dict(name=name, op="attn", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, cache=cache, page=page,
                Lmin=Lmin, Lmax=Lmax, ragged=ragged)


def listed():
    return [
        # one decoded token of one request: pure latency
        _rope("rope_one_token", 1, 1, 32, 128, 128, 0, "half", "none", "bf16", 4096, 4096),
        # the MLA query of a 64-node draft tree: the last 64 of 192 dims rotated at
        # prefix + depth (long-context scaling), both parts laid out for the verify call
        _rope("rope_mla_tree_split", 1, 64, 64, 192, 64, 128, "interleaved", "yarn", "bf16",
              65536, 65536, tree=True, split=True, base=50000.0, factor=32.0),
        # queries of a long prompt chunk, ragged, half of each head rotated
        _rope("rope_prompt_partial", 4, 2000, 64, 128, 64, 0, "half", "linear", "bf16", 1, 30000,
              ragged=True, factor=4.0),
        # latent rows of 64 chain drafts into a paged one-byte MLA cache, and back
        _kv("kv_mla_fp8_drafts", "kv", "mla", 64, 8, 1, 512, "bf16", "fp8", 64, 1024, 32768),
        # a prompt chunk of odd length into a one-byte GQA cache with a scale per row and head
        _kv("kv_gqa_fp8_prompt", "kv", "gqa", 2, 8191, 8, 128, "bf16", "fp8", 64, 1, 4000, ragged=True),
        # a long cached prefix read back in bf16
        _kv("read_gqa_fp8_prefix", "read", "gqa", 1, 65536, 8, 128, "bf16", "fp8", 64, 0, 0),
        # ragged latent prefixes read back from a contiguous one-byte cache
        _kv("read_mla_fp8_ragged", "read", "mla", 8, 8192, 1, 512, "bf16", "fp8", 0, 0, 100, ragged=True),
        # one decoded token over a few thousand keys
        _attn("attn_one_token", 1, 1, 32, 8, 128, "bf16", 64, 4096, 4096),
        # an fp32 tree of a small drafter, odd sizes everywhere
        _attn("attn_f32_odd", 3, 13, 14, 2, 80, "f32", 0, 5, 1500, ragged=True),
        # a batch of draft trees over a contiguous cache
        _attn("attn_tree_batched", 8, 32, 64, 8, 128, "bf16", 0, 2048, 8192, ragged=True),
        # a served batch of chain drafts over a paged one-byte cache
        _attn("attn_paged_fp8", 64, 8, 64, 8, 128, "fp8", 64, 1024, 32768),
        # a large tree over a long prefix: the tensor cores' case
        _attn("attn_tree_long", 1, 128, 64, 8, 128, "bf16", 64, 65536, 65536),
    ]


def draw(rng):
    def logu(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "rope", "kv", "read", "attn", "attn", "attn"])
    if op == "rope":
        B, N = logu(1, 64), logu(1, 4000)
        H = rng.choice([1, 4, 7, 16, 32, 64])
        while B * N * H > 500000:
            N = max(1, N // 2)
            H = max(1, H // 2)
        split = rng.random() < 0.3
        rot = rng.choice([32, 64, 128])
        dim, off = (192, 128) if split else (128, 0)
        rot = 64 if split else rot
        lo = logu(1, 60000)
        c = _rope("", B, N, H, dim, rot, off, rng.choice(["half", "interleaved"]),
                  rng.choice(["none", "linear", "ntk", "yarn"]),
                  rng.choice(["bf16", "bf16", "f32"]), lo, lo * 2, tree=N <= 128, split=split,
                  ragged=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                  factor=rng.choice([2.0, 8.0, 32.0]))
    elif op in ("kv", "read"):
        kind = rng.choice(["mla", "gqa"])
        Hkv, D = (1, 512) if kind == "mla" else rng.choice([(8, 128), (4, 64), (2, 128), (8, 80)])
        B = logu(1, 32)
        N = max(1, min(logu(1, 16000), 65536 // B))
        lo = logu(1, 8000) if op == "kv" else 0
        c = _kv("", op, kind, B, N, Hkv, D, "bf16", rng.choice(["bf16", "fp8", "fp8"]),
                rng.choice([0, 64]), lo, 2 * lo if op == "kv" else logu(1, 200),
                tree=op == "kv" and N <= 128, ragged=rng.random() < 0.5)
    else:
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 7, 8, 16])
        D = rng.choice([64, 128, 128])
        cache = rng.choice(["bf16", "bf16", "fp8", "fp8", "f32"])
        B, N = logu(1, 48), logu(1, 128)
        lo = logu(16, 20000)
        while B * N * Hkv * G * lo > (4 if cache == "f32" else 120) * 10 ** 7:
            lo = max(16, lo // 2)
            N = max(1, N * 2 // 3)
            B = max(1, B * 2 // 3)
        c = _attn("", B, N, Hkv * G, Hkv, D, cache, rng.choice([0, 64]), lo, 2 * lo,
                  ragged=rng.random() < 0.5)
    del c["name"]
    return c


# ---- lengths (from the case alone) ----------------------------------------------------------

def _spread(lo, hi, count, phase):
    """`count` whole numbers of [lo, hi], evenly spread over their logarithm."""
    a, b = math.log(lo + 1.0), math.log(hi + 1.0)
    return [min(hi, max(lo, int(round(math.exp(a + (b - a) * ((0.61803398875 * (i + 1) + phase) % 1.0)) - 1))))
            for i in range(count)]


def _lengths(c):
    """Prefix (or first row) and live rows of each request."""
    L = _spread(c["Lmin"], c["Lmax"], c["B"], 0.17) if c["Lmax"] > c["Lmin"] else [c["Lmin"]] * c["B"]
    n = _spread(max(1, c["N"] // 4), c["N"], c["B"], 0.43) if c["ragged"] else [c["N"]] * c["B"]
    if c["ragged"]:
        n[0] = c["N"]
    return L, n


def work(c):
    L, n = _lengths(c)
    live = sum(n)
    if c["op"] == "rope":
        e = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * live * c["H"] * c["dim"] * e + 8 * c["B"] * c["N"],
                "flops": 3 * live * c["H"] * c["rot"]}
    if c["op"] in ("kv", "read"):
        width = c["D"] + 64 if c["kind"] == "mla" else 2 * c["Hkv"] * c["D"]
        scales = 2 * c["Hkv"] if c["kind"] == "gqa" and c["cache"] == "fp8" else 0
        row = width * (1 if c["cache"] == "fp8" else 2) + scales      # one cached row
        wide = width * 2
        if c["op"] == "read":
            return {"bytes": live * (row + wide), "flops": live * width}
        back = wide if c["cache"] == "fp8" else 0
        return {"bytes": live * (wide + row + back), "flops": 4 * live * width}
    D, rows = c["D"], 0
    e = {"f32": 4, "bf16": 2, "fp8": 1}[c["cache"]]
    io = 4 if c["cache"] == "f32" else 2
    per_row = 2 * c["Hkv"] * (D * e + (1 if c["cache"] == "fp8" else 0))
    b = sum((l + m) * per_row for l, m in zip(L, n)) + 2 * live * c["Hq"] * D * io
    rows = sum((l + 1) * m for l, m in zip(L, n)) * c["Hq"]
    return {"bytes": b, "flops": 4 * D * rows}


# ---- inputs ------------------------------------------------------------------------------

def _trees(c, g):
    """parent and depth [B, N] of random draft trees (each node hangs from one of the 8 before it)."""
    B, N = c["B"], c["N"]
    parent = torch.full((B, N), -1, dtype=torch.int64)
    depth = torch.zeros((B, N), dtype=torch.int64)
    pick = torch.rand((B, N), generator=g)
    for i in range(1, N):
        lo = max(0, i - 8)
        p = lo + (pick[:, i] * (i - lo)).long().clamp_(max=i - lo - 1)
        parent[:, i] = p
        depth[:, i] = depth.gather(1, p[:, None])[:, 0] + 1
    return parent, depth


def _cache_shape(c, L, n, g):
    """Rows of the cache and the page table (None: contiguous [B, T])."""
    T = [l + m for l, m in zip(L, n)]
    if c["page"] == 0:
        return (c["B"], -(-max(T) // 64) * 64), None
    per = [-(-t // c["page"]) for t in T]
    perm = torch.randperm(sum(per), generator=g)
    table = torch.full((c["B"], max(per)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = perm[at:at + k]
        at += k
    return (sum(per), c["page"]), table


def _rows(s, start, count):
    """Index of row start[b] + i of request b in the cache's flat rows, and the live ones [B, count];
    the others have the index of row start[b]."""
    i = torch.arange(count, device=DEV)[None]
    live = i < s["n_live"].long()[:, None]
    t = start.long()[:, None] + torch.where(live, i, torch.zeros_like(i))
    if s["page_table"] is None:
        return torch.arange(t.shape[0], device=DEV)[:, None] * s["t_stride"] + t, live
    page = s["page_table"].long().gather(1, t // s["page"])
    return page * s["page"] + t % s["page"], live


def _pow2(e):
    """2^e in float32, e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantised(x, per_row):
    """Codes (float8_e4m3fn), and exponent bytes for each row where asked."""
    if not per_row:
        return (x / MLA_SCALE).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), None
    m, k = torch.frexp(x.abs().amax(-1))
    e = (k - 9 + (m > 0.875).to(k.dtype)).clamp(E_MIN, E_MAX)
    y = (x * _pow2(-e)[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return y, (e + 127).to(torch.uint8)


def prepare(c, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)

    def normal(shape, dtype):
        return torch.randn(shape, generator=gd, device=DEV, dtype=torch.float32).to(dtype)

    L, n = _lengths(c)
    s = {"c": c, "B": c["B"], "N": c["N"], "prefix_len": torch.tensor(L, dtype=torch.int32, device=DEV),
         "n_live": torch.tensor(n, dtype=torch.int32, device=DEV), "page_table": None, "page": c.get("page", 0),
         "t_stride": 0, "depth": None, "parent": None}
    if c.get("tree") or c["op"] == "attn":
        parent, depth = _trees(c, g)
        s["parent"], s["depth"] = parent.int().to(DEV), depth.int().to(DEV)
    if c["op"] == "rope":
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        s["x"] = normal((c["B"], c["N"], c["H"], c["dim"]), dt)
        if c["split"]:
            s["y"] = torch.zeros((c["B"], c["N"], c["H"], c["rot"]), dtype=dt, device=DEV)
            s["rest"] = torch.zeros((c["B"], c["N"], c["H"], c["dim"] - c["rot"]), dtype=dt, device=DEV)
        else:
            s["y"], s["rest"] = torch.zeros_like(s["x"]), None
        return s

    shape, table = _cache_shape(c, L, n, g)
    if table is None:
        s["t_stride"] = shape[1]
    else:
        s["page_table"] = table.to(DEV)
    if c["op"] == "attn":
        dt = torch.float32 if c["cache"] == "f32" else torch.bfloat16
        s["q"] = normal((c["B"], c["N"], c["Hq"], c["D"]), torch.float32)
        s["q"] *= torch.linspace(0.5, 3.0, c["Hq"], device=DEV)[:, None]      # some heads attend sharply
        s["q"] = s["q"].to(dt)
        s["out"] = torch.zeros_like(s["q"])
        for name in ("k", "v"):
            x = normal((*shape, c["Hkv"], c["D"]), dt)
            if name == "k":
                x[..., :4] *= 4.0                                              # a few strong channels
            s[name + "_scale"] = None
            if c["cache"] == "fp8":
                x, s[name + "_scale"] = _quantised(x.float(), True)
            s[name] = x
        return s

    # kv, read: the parts of a row, each [.., heads, dim]
    heads = [(1, c["D"]), (1, 64)] if c["kind"] == "mla" else [(c["Hkv"], c["D"])] * 2
    s["parts"] = []
    for k, (h, d) in enumerate(heads):
        p = {"heads": h, "dim": d, "scale": None}
        rotated = k == (1 if c["kind"] == "mla" else 0)
        per_row = c["kind"] == "gqa"
        x = normal((*shape, h, d), torch.bfloat16)
        if c["cache"] == "fp8":
            x, p["scale"] = _quantised(x.float(), per_row)
        p["cache"] = x
        if c["op"] == "kv":
            p["src"] = normal((c["B"], c["N"], h, d), torch.bfloat16)
            p["rotated"] = rotated
        if c["op"] == "read" or c["cache"] == "fp8":
            p["out"] = torch.zeros((c["B"], c["N"], h, d), dtype=torch.bfloat16, device=DEV)
        s["parts"].append(p)
    return s


# ---- rotary frequencies ----------------------------------------------------------------------

def _frequencies(rot, base, scaling, factor, orig):
    """Angle per position of each pair (float64), and the factor on cos and sin."""
    j = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * j / rot)
    amp = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        # pairs that turn more than beta_fast = 32 times over the original context keep
        # their frequency, those below beta_slow = 1 turn are interpolated, a ramp between
        def at(turns):
            return rot * math.log(orig / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((j - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = f / factor * ramp + f * (1.0 - ramp)
        amp = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    return f, amp


def _rope_args(c):
    """Rotary settings of a case: the cached keys of the kv cases use plain half rotation."""
    if c["op"] == "rope":
        return c["rot"], c["layout"], c["base"], c["scaling"], c["factor"], c["orig"]
    return (64, "interleaved", 50000.0, "yarn", 32.0, 4096) if c["kind"] == "mla" else \
        (c["D"], "half", 10000.0, "none", 1.0, 4096)


def _rotate(x, pos, off, args):
    """x [B, N, H, dim] with dims off .. off + rot rotated by pos [B, N]; angles in 64 bits."""
    rot, layout, base, scaling, factor, orig = args
    f, amp = _frequencies(rot, base, scaling, factor, orig)
    angle = pos.double()[:, :, None] * f.to(DEV)
    cos = (torch.cos(angle) * amp).to(x.dtype)[:, :, None]
    sin = (torch.sin(angle) * amp).to(x.dtype)[:, :, None]
    r = x[..., off:off + rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = x.clone()
    y[..., off:off + rot] = torch.stack((u, v), -1).flatten(-2) if layout == "interleaved" else torch.cat((u, v), -1)
    return y


def _positions(s):
    step = s["depth"].long() if s["depth"] is not None else torch.arange(s["N"], device=DEV)[None]
    return s["prefix_len"].long()[:, None] + step


# ---- one pass --------------------------------------------------------------------------------

def _handle(s):
    """The library's callers over this state's tensors, made on the state's first pass."""
    if "op" not in s:
        from speculative_decoding_tree_mla_gb300 import kdtv
        c = s["c"]
        if c["op"] == "rope":
            rot, layout, base, scaling, factor, orig = _rope_args(c)
            t = kdtv.RopeTable(rot, layout=layout, base=base, scaling=scaling, factor=factor, orig_ctx=orig)
            s["op"] = [kdtv.Rope(t, s["x"], prefix_len=s["prefix_len"], depth=s["depth"], n_live=s["n_live"],
                                 rot_off=c["off"], out=s["y"], rest=s["rest"])]
        elif c["op"] == "attn":
            s["op"] = [kdtv.GqaVerifyAttn(s["q"], s["k"], s["v"], s["parent"], s["prefix_len"],
                                          n_nodes=s["n_live"], page_table=s["page_table"],
                                          k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])]
        else:
            scale = MLA_SCALE if c["kind"] == "mla" else 0.0
            s["op"] = []
            if c["op"] == "kv":
                rot, layout, base, scaling, factor, orig = _rope_args(c)
                t = kdtv.RopeTable(rot, layout=layout, base=base, scaling=scaling, factor=factor, orig_ctx=orig)
                s["op"].append(kdtv.KvAppend(
                    [kdtv.KvPart(p["cache"], src=p["src"], scale=p["scale"], rot_off=0 if p["rotated"] else None)
                     for p in s["parts"]], s["prefix_len"], rope=t, depth=s["depth"], n_live=s["n_live"],
                    page_table=s["page_table"], kv_scale=scale))
            if "out" in s["parts"][0]:
                s["op"].append(kdtv.KvRead(
                    [kdtv.KvPart(p["cache"], out=p["out"], scale=p["scale"]) for p in s["parts"]],
                    s["prefix_len"], s["n_live"], page_table=s["page_table"], kv_scale=scale))
    return s["op"]


def _outputs(s):
    c = s["c"]
    if c["op"] == "rope":
        return {"y": s["y"]} if s["rest"] is None else {"y": s["y"], "rest": s["rest"]}
    if c["op"] == "attn":
        return {"out": s["out"]}
    return {"part%d" % k: p["out"] if "out" in p else p["cache"] for k, p in enumerate(s["parts"])}


def run(s):
    if own:
        for call in _handle(s):
            call()
        return _outputs(s)
    c = s["c"]
    if c["op"] == "rope":
        y = _rotate(s["x"].float(), _positions(s), c["off"], _rope_args(c)).to(s["x"].dtype)
        live = (torch.arange(s["N"], device=DEV)[None] < s["n_live"][:, None])[:, :, None, None]
        if c["split"]:
            s["rest"].copy_(torch.where(live, y[..., :c["off"]], s["rest"]))
            y = y[..., c["off"]:]
        s["y"].copy_(torch.where(live, y, s["y"]))
    elif c["op"] == "attn":
        _plain_attn(s)
    else:
        rows, live = _rows(s, s["prefix_len"], s["N"])
        wide = live[:, :, None, None]
        for p in s["parts"]:
            flat = p["cache"].view(-1, p["heads"], p["dim"])
            if c["op"] == "kv":
                x = p["src"].float()
                if p["rotated"]:
                    x = _rotate(x, _positions(s), 0, _rope_args(c))
                x = torch.where(wide, x, x[:, :1])          # rows without a place repeat row 0
                if c["cache"] == "fp8":
                    code, scale = _quantised(x, c["kind"] == "gqa")
                    flat.view(torch.uint8)[rows] = code.view(torch.uint8)
                    if scale is not None:
                        p["scale"].view(-1, p["heads"])[rows] = scale
                else:
                    flat[rows] = x.to(flat.dtype)
            if "out" in p:
                p["out"].copy_(torch.where(wide, _values(c, p, rows).to(p["out"].dtype), p["out"]))
    return _outputs(s)


def _values(c, p, rows):
    """The cached rows in 32 bits."""
    x = p["cache"].view(-1, p["heads"], p["dim"])
    if c["cache"] != "fp8":
        return x[rows].float()
    x = x.view(torch.uint8)[rows].view(torch.float8_e4m3fn).float()
    if p["scale"] is None:
        return x * MLA_SCALE
    return x * _pow2(p["scale"].view(-1, p["heads"])[rows].int() - 127)[..., None]


def _visible(s, T):
    """[B, N, T]: node i sees the prefix and its own root path, itself included."""
    B, N = s["B"], s["N"]
    me = torch.arange(N, device=DEV)
    hop = (s["parent"].long()[:, :, None] == me[None, None]).float()           # [B, N, N]: i to its parent
    up, k = hop + torch.eye(N, device=DEV), 1
    while k < N:                                             # paths of up to 2k hops
        up = (torch.bmm(up, up) > 0).float()
        k *= 2
    reach = up > 0
    live = me[None] < s["n_live"][:, None]
    reach = reach & live[:, :, None] & live[:, None, :]
    t = torch.arange(T, device=DEV)[None]
    L = s["prefix_len"].long()[:, None]
    node = (t - L).clamp(0, N - 1)[:, None].expand(B, N, T)
    inside = ((t >= L) & (t < L + N))[:, None]
    return ((t < L)[:, None] & live[:, :, None]) | (inside & reach.gather(2, node))


def _attn_rows(s, T):
    t = torch.arange(T, device=DEV)[None].expand(s["B"], T)
    have = t < (s["prefix_len"] + s["n_live"]).long()[:, None]
    t = torch.where(have, t, torch.zeros_like(t))
    if s["page_table"] is None:
        return torch.arange(s["B"], device=DEV)[:, None] * s["t_stride"] + t, have
    return s["page_table"].long().gather(1, t // s["page"]) * s["page"] + t % s["page"], have


def _attn_values(s, name, rows, dtype):
    c = s["c"]
    x = s[name].view(-1, c["Hkv"], c["D"])
    if c["cache"] != "fp8":
        return x[rows].to(dtype)
    x = x.view(torch.uint8)[rows].view(torch.float8_e4m3fn).to(dtype)
    return x * _pow2(s[name + "_scale"].view(-1, c["Hkv"])[rows].int() - 127)[..., None].to(dtype)


def _plain_attn(s):
    c = s["c"]
    B, N, Hq, Hkv, D = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"]
    L, n = _lengths(c)
    T = max(l + m for l, m in zip(L, n))
    rows, have = _attn_rows(s, T)
    k = _attn_values(s, "k", rows, torch.float32).permute(0, 2, 3, 1)          # [B, Hkv, D, T]
    v = _attn_values(s, "v", rows, torch.float32)
    v = torch.where(have[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)        # [B, Hkv, T, D]
    q = s["q"].float().view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    a = (q @ k).mul_(1.0 / math.sqrt(D)).view(B, Hkv, N, Hq // Hkv, T)
    a.masked_fill_(~_visible(s, T)[:, None, :, None], float("-inf"))
    m = a.amax(-1, keepdim=True)
    a.sub_(torch.where(m > float("-inf"), m, torch.zeros_like(m))).exp_()
    l = a.sum(-1, keepdim=True)
    o = (a.view(B, Hkv, -1, T) @ v).view(B, Hkv, N, Hq // Hkv, D) / l
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    live = (torch.arange(N, device=DEV)[None] < s["n_live"][:, None])[:, :, None, None]
    s["out"].copy_(torch.where(live, o.to(s["out"].dtype), s["out"]))


# ---- the definition in 64 bits ---------------------------------------------------------------

def _e4m3(x):
    """Nearest E4M3 value (ties to the even code, saturating) of each float64."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=FP8_MAX)


def _turned(c, x, pos):
    """One row's heads [H, dim] of the rotated part, rotated by `pos` in 64 bits through complex numbers."""
    rot, layout, base, scaling, factor, orig = _rope_args(c)
    amp, f = 1.0, []
    for j in range(rot // 2):
        b = base * factor ** (rot / (rot - 2.0)) if scaling == "ntk" else base
        w = math.exp(-2.0 * j / rot * math.log(b))
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            pair = [rot / 2.0 * math.log(orig / (2.0 * math.pi * turns), base) for turns in (32.0, 1.0)]
            lo, hi = max(0, math.floor(pair[0])), min(rot - 1, math.ceil(pair[1]))
            mix = min(1.0, max(0.0, (j - lo) / (hi - lo if hi > lo else 0.001)))
            w = w * (1.0 - mix) + w / factor * mix
            amp = 1.0 + 0.1 * math.log(factor)
        f.append(w)
    f = torch.tensor(f, dtype=torch.float64, device=DEV)
    w = torch.polar(torch.full_like(f, amp)[None], pos.double()[:, None] * f)[:, None]
    if layout == "interleaved":
        z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * w
        return torch.view_as_real(z).flatten(-2)
    z = torch.complex(x[..., :rot // 2].double(), x[..., rot // 2:].double()) * w
    return torch.cat((z.real, z.imag), -1)


def exact(c, seed):
    s = prepare(c, seed)
    L, n = _lengths(c)
    pos = _positions(s)
    if c["op"] == "rope":
        y = s["x"].double()
        lo, hi = c["off"], c["off"] + c["rot"]
        for b, m in enumerate(n):
            y[b, :m, :, lo:hi] = _turned(c, s["x"][b, :m, :, lo:hi], pos[b, :m])
            y[b, m:] = 0.0
        return {"y": y[..., lo:hi], "rest": y[..., :lo]} if c["split"] else {"y": y}
    if c["op"] == "attn":
        return {"out": _exact_attn(s, L, n)}
    got = {}
    for k, p in enumerate(s["parts"]):
        cache = p["cache"].view(-1, p["heads"], p["dim"])
        back = torch.zeros((c["B"], c["N"], p["heads"], p["dim"]), dtype=torch.float64, device=DEV)
        whole = None if "out" in p else cache.double()
        for b, (l, m) in enumerate(zip(L, n)):
            t = torch.arange(l, l + m, device=DEV)
            if s["page_table"] is None:
                r = b * s["t_stride"] + t
            else:
                r = s["page_table"][b].long()[t // c["page"]] * c["page"] + t % c["page"]
            if c["op"] == "kv":
                x = p["src"][b, :m]
                x = _turned(c, x, pos[b, :m]) if p["rotated"] else x.double()
                if c["cache"] == "fp8" and c["kind"] == "gqa":
                    e = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / FP8_MAX)).clamp(E_MIN, E_MAX)
                    x = _e4m3(x / torch.exp2(e)) * torch.exp2(e)
                elif c["cache"] == "fp8":
                    x = _e4m3(x / MLA_SCALE) * MLA_SCALE
            elif c["cache"] == "fp8":
                x = cache.view(torch.uint8)[r].view(torch.float8_e4m3fn).double()
                x = x * MLA_SCALE if p["scale"] is None else \
                    x * torch.exp2(p["scale"].view(-1, p["heads"])[r].double() - 127)[..., None]
            else:
                x = cache[r].double()
            back[b, :m] = x
            if whole is not None:
                whole[r] = x
        got["part%d" % k] = back if whole is None else whole.view(p["cache"].shape)
    return got


def _exact_attn(s, L, n):
    """Node by node groups: the visible rows of each request gathered, softmax and sum in 64 bits."""
    c = s["c"]
    if 4 * c["D"] * c["Hq"] * sum((l + m) * m for l, m in zip(L, n)) > 8e11:
        return None
    G, D = c["Hq"] // c["Hkv"], c["D"]
    out = torch.zeros((c["B"], c["N"], c["Hq"], D), dtype=torch.float64, device=DEV)
    parent = s["parent"].tolist()
    for b, (l, m) in enumerate(zip(L, n)):
        t = torch.arange(l + m, device=DEV)
        if s["page_table"] is None:
            r = b * s["t_stride"] + t
        else:
            r = s["page_table"][b].long()[t // c["page"]] * c["page"] + t % c["page"]
        see = torch.zeros((m, l + m), dtype=torch.bool)
        see[:, :l] = True
        for i in range(m):
            j = i
            while j >= 0:
                see[i, l + j] = True
                j = parent[b][j]
        see = see.to(DEV)
        k, v = (s[name].view(-1, c["Hkv"], D) for name in ("k", "v"))
        if c["cache"] == "fp8":
            k, v = (x.view(torch.uint8)[r].view(torch.float8_e4m3fn).double()
                    * torch.exp2(e.view(-1, c["Hkv"])[r].double() - 127.0)[..., None]
                    for x, e in ((k, s["k_scale"]), (v, s["v_scale"])))
        else:
            k, v = k[r].double(), v[r].double()
        q = s["q"][b, :m].double().view(m, c["Hkv"], G, D)
        for h in range(c["Hkv"]):
            a = torch.einsum("igd,td->igt", q[:, h], k[:, h]) / math.sqrt(D)
            a = torch.softmax(a.masked_fill(~see[:, None], float("-inf")), -1)
            out[b, :m, h * G:(h + 1) * G] = torch.einsum("igt,td->igd", a, v[:, h])
    return out
