"""ctypes binding of libkdtv.so (include/kdtv.h), plus a torch-side caller.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  ``torch`` supplies device memory and the stream.  There is no CPU
fallback: if the library was not built, every call raises.
"""

from __future__ import annotations

import ctypes
import math
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkdtv.so")

KDTV_F32, KDTV_BF16, KDTV_BF16_FP8KV = 0, 1, 2
KDTV_FLAG_SIMT = 0x1
KDTV_FLAG_SIMT_PROJ = 0x2
KDTV_FLAG_TEST_STALL = 0x100
STATUS = {0: "KDTV_OK", 1: "KDTV_ERR_INVALID_ARG", 2: "KDTV_ERR_UNSUPPORTED",
          3: "KDTV_ERR_CUDA", 4: "KDTV_ERR_BAD_TREE", 5: "KDTV_ERR_DEVICE_TIMEOUT",
          6: "KDTV_ERR_BAD_PREFIX", 7: "KDTV_ERR_BAD_PAGE"}
STATUS_CODE = {v: k for k, v in STATUS.items()}

# Every symbol include/kdtv.h declares (checked by the CPU tests).
EXPORTS = ("kdtv_workspace_size", "kdtv_verify_attn", "kdtv_get_device_status",
           "kdtv_strerror", "kdtv_launches_per_call", "kdtv_tree_accept", "kdtv_compact_kv",
           "kdtv_tree_build", "kdtv_verify_attn_noalloc", "kdtv_rope_init", "kdtv_rope",
           "kdtv_kv_append", "kdtv_kv_read", "kdtv_gqa_workspace_size",
           "kdtv_gqa_launches_per_call", "kdtv_gqa_verify_attn")


class KdtvDims(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("N", ctypes.c_int32), ("H", ctypes.c_int32),
        ("d_nope", ctypes.c_int32), ("d_rope", ctypes.c_int32),
        ("d_v", ctypes.c_int32), ("d_c", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("t_stride", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("num_pages", ctypes.c_int32), ("scale", ctypes.c_float),
        ("flags", ctypes.c_uint32), ("kv_chunk", ctypes.c_int32),
        ("kv_scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("phase_events", ctypes.c_void_p),
    ]


ROPE_MAX_DIM = 256
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class KdtvRopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("orig_ctx", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("attn_factor", ctypes.c_double)]


class KdtvRopeTable(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("amp", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turn", ctypes.c_uint64 * (ROPE_MAX_DIM // 2))]


class KdtvRopeArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("H", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("rot_off", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("x_stride", ctypes.c_int64 * 3),
                ("y_stride", ctypes.c_int64 * 3), ("rest_stride", ctypes.c_int64 * 3)]


class KdtvKvPart(ctypes.Structure):
    _fields_ = [("cache", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("src", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("src_stride", ctypes.c_int64 * 3), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("rotate", ctypes.c_int32),
                ("rot_off", ctypes.c_int32)]


class KdtvKvDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("cache_dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("t_stride", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("kv_scale", ctypes.c_float),
                ("parts", ctypes.c_int32)]


class KdtvGqaDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("H", ctypes.c_int32),
                ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("t_stride", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("scale", ctypes.c_float), ("flags", ctypes.c_uint32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class KdtvError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


_lib = None


def lib():
    """Loads libkdtv.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m speculative_decoding_tree_mla_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(KdtvDims)
        vp = ctypes.c_void_p
        L.kdtv_workspace_size.argtypes = [P]
        L.kdtv_workspace_size.restype = ctypes.c_size_t
        L.kdtv_verify_attn.argtypes = [P] + [vp] * 10 + [vp]
        L.kdtv_verify_attn.restype = ctypes.c_int
        L.kdtv_get_device_status.argtypes = [P, vp]
        L.kdtv_get_device_status.restype = ctypes.c_int
        L.kdtv_strerror.argtypes = [ctypes.c_int]
        L.kdtv_strerror.restype = ctypes.c_char_p
        L.kdtv_launches_per_call.argtypes = [P]
        L.kdtv_launches_per_call.restype = ctypes.c_int
        i32 = ctypes.c_int
        L.kdtv_tree_accept.argtypes = [i32, i32] + [vp] * 6 + [vp]
        L.kdtv_tree_accept.restype = ctypes.c_int
        L.kdtv_compact_kv.argtypes = [P] + [vp] * 7 + [vp]
        L.kdtv_compact_kv.restype = ctypes.c_int
        L.kdtv_tree_build.argtypes = [i32, i32, i32, i32] + [vp] * 8 + [vp]
        L.kdtv_tree_build.restype = ctypes.c_int
        L.kdtv_verify_attn_noalloc.argtypes = [P] + [vp] * 11 + [vp]
        L.kdtv_verify_attn_noalloc.restype = ctypes.c_int
        L.kdtv_rope_init.argtypes = [ctypes.POINTER(KdtvRopeConfig), ctypes.POINTER(KdtvRopeTable)]
        L.kdtv_rope_init.restype = ctypes.c_int
        L.kdtv_rope.argtypes = [ctypes.POINTER(KdtvRopeTable), ctypes.POINTER(KdtvRopeArgs)] + [vp] * 6 + [vp]
        L.kdtv_rope.restype = ctypes.c_int
        KP = [ctypes.POINTER(KdtvKvDims), ctypes.POINTER(KdtvKvPart)]
        L.kdtv_kv_append.argtypes = KP + [ctypes.POINTER(KdtvRopeTable)] + [vp] * 5 + [vp]
        L.kdtv_kv_append.restype = ctypes.c_int
        L.kdtv_kv_read.argtypes = KP + [vp] * 4 + [vp]
        L.kdtv_kv_read.restype = ctypes.c_int
        G = ctypes.POINTER(KdtvGqaDims)
        L.kdtv_gqa_workspace_size.argtypes = [G]
        L.kdtv_gqa_workspace_size.restype = ctypes.c_size_t
        L.kdtv_gqa_launches_per_call.argtypes = [G]
        L.kdtv_gqa_launches_per_call.restype = ctypes.c_int
        L.kdtv_gqa_verify_attn.argtypes = [G] + [vp] * 11 + [vp]
        L.kdtv_gqa_verify_attn.restype = ctypes.c_int
        _lib = L
    return _lib


def strerror(code):
    return lib().kdtv_strerror(int(code)).decode()


DTYPE_CODE = {"f32": KDTV_F32, "bf16": KDTV_BF16, "fp8kv": KDTV_BF16_FP8KV}


def make_dims(spec_or_shape, *, dtype, page_size=0, t_stride=0, max_pages=0,
              num_pages=0, scale=0.0, flags=0, kv_chunk=0, kv_scale=0.0):
    s = spec_or_shape
    d = KdtvDims()
    d.B, d.N, d.H = s.B, s.N, s.H
    d.d_nope, d.d_rope, d.d_v, d.d_c = s.d_nope, s.d_rope, s.d_v, s.d_c
    d.dtype = DTYPE_CODE.get(dtype, dtype if isinstance(dtype, int) else KDTV_F32)
    d.kv_scale = kv_scale
    d.page_size, d.t_stride = page_size, t_stride
    d.max_pages, d.num_pages = max_pages, num_pages
    d.scale, d.flags, d.kv_chunk = scale, flags, kv_chunk
    return d


def workspace_size(dims):
    return int(lib().kdtv_workspace_size(ctypes.byref(dims)))


def launches_per_call(dims):
    return int(lib().kdtv_launches_per_call(ctypes.byref(dims)))


def verify_attn_raw(dims, q_nope, q_rope, W_UK, W_UV, c_kv, k_rope, parent,
                    prefix_len, page_table, out, stream):
    """Direct C-ABI call with integer device pointers; returns the status."""
    return int(lib().kdtv_verify_attn(ctypes.byref(dims), q_nope, q_rope, W_UK, W_UV,
                                      c_kv, k_rope, parent, prefix_len,
                                      page_table or None, out, stream or None))


def get_device_status(dims, stream=0):
    return int(lib().kdtv_get_device_status(ctypes.byref(dims), stream or None))


class VerifyAttn:
    """Torch-side caller: holds the dims, the workspace and the output buffer.

    ``tensors`` maps q_nope, q_rope, W_UK, W_UV, c_kv, k_rope, parent,
    prefix_len and (paged) page_table to contiguous CUDA tensors.
    """

    def __init__(self, spec, tensors, *, t_stride=0, max_pages=0, num_pages=0,
                 page_size=0, flags=0, kv_chunk=0, scale=0.0, kv_scale=0.0):
        import torch
        self.torch = torch
        self.t = tensors
        dev = tensors["c_kv"].device
        self.dims = make_dims(spec, dtype=spec.dtype, page_size=page_size,
                              t_stride=t_stride, max_pages=max_pages,
                              num_pages=num_pages, scale=scale or spec.scale,
                              flags=flags, kv_chunk=kv_chunk, kv_scale=kv_scale)
        nbytes = workspace_size(self.dims)
        if nbytes == 0:
            raise KdtvError(STATUS_CODE["KDTV_ERR_UNSUPPORTED"], "workspace size")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        self.dims.workspace = self.workspace.data_ptr()
        self.dims.workspace_bytes = nbytes
        self.out = torch.empty((spec.B, spec.N, spec.H, spec.d_v), dtype=torch.float32,
                               device=dev)
        self._ev = None

    def set_phase_events(self, events):
        """events: list of 5 torch.cuda.Event (created with enable_timing)."""
        if events is None:
            self.dims.phase_events = None
            self._ev = None
            return
        for e in events:             # torch creates the CUDA event lazily
            if not e.cuda_event:
                e.record()
        handles = (ctypes.c_void_p * 5)(*[e.cuda_event for e in events])
        if not all(handles):
            raise RuntimeError("phase events could not be created")
        self._ev = handles
        self.dims.phase_events = ctypes.cast(handles, ctypes.c_void_p)

    def __call__(self, stream=None, out=None):
        t = self.t
        s = stream if stream is not None else self.torch.cuda.current_stream()
        o = self.out if out is None else out
        pt = t.get("page_table")
        code = verify_attn_raw(self.dims, t["q_nope"].data_ptr(), t["q_rope"].data_ptr(),
                               t["W_UK"].data_ptr(), t["W_UV"].data_ptr(),
                               t["c_kv"].data_ptr(), t["k_rope"].data_ptr(),
                               t["parent"].data_ptr(), t["prefix_len"].data_ptr(),
                               pt.data_ptr() if pt is not None else 0, o.data_ptr(),
                               s.cuda_stream)
        if code != 0:
            raise KdtvError(code, "kdtv_verify_attn")
        return o

    def status(self, stream=None):
        s = stream if stream is not None else self.torch.cuda.current_stream()
        return get_device_status(self.dims, s.cuda_stream)

    def launches(self):
        return launches_per_call(self.dims)


def for_workload(wl, device="cuda", **kw):
    """VerifyAttn over a ``workloads.Workload`` moved to ``device``."""
    names = ["q_nope", "q_rope", "W_UK", "W_UV", "c_kv", "k_rope", "parent", "prefix_len"]
    if wl.page_size:
        names.append("page_table")
    tens = {n: wl.t[n].to(device).contiguous() for n in names}
    kw.setdefault("kv_scale", wl.kv_scale)
    return VerifyAttn(wl.spec, tens, t_stride=wl.t_stride, max_pages=wl.max_pages,
                      num_pages=wl.num_pages, page_size=wl.page_size, **kw)


def default_scale(d_nope, d_rope):
    return 1.0 / math.sqrt(d_nope + d_rope)


def _p(t):
    return t.data_ptr() if t is not None else None


def _s(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def tree_accept(parent, draft_tok, target_argmax, stream=None):
    """Torch caller of kdtv_tree_accept; returns (path, path_len, bonus)."""
    import torch
    B, N = parent.shape
    dev = parent.device
    path = torch.empty((B, N), dtype=torch.int32, device=dev)
    plen = torch.empty(B, dtype=torch.int32, device=dev)
    bonus = torch.empty(B, dtype=torch.int32, device=dev)
    code = lib().kdtv_tree_accept(B, N, _p(parent), _p(draft_tok), _p(target_argmax),
                                  _p(path), _p(plen), _p(bonus), _s(stream))
    if code:
        raise KdtvError(code, "kdtv_tree_accept")
    return path, plen, bonus


def compact_kv(dims, c_kv, k_rope, prefix_len, path, path_len, page_table=None,
               status=None, stream=None):
    """Torch caller of kdtv_compact_kv (in place); returns the status tensor."""
    import torch
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=c_kv.device)
    code = lib().kdtv_compact_kv(ctypes.byref(dims), _p(c_kv), _p(k_rope), _p(prefix_len),
                                 _p(path), _p(path_len), _p(page_table), _p(status),
                                 _s(stream))
    if code:
        raise KdtvError(code, "kdtv_compact_kv")
    return status


def tree_build(logp, tokens, root_token, n_nodes, stream=None):
    """Torch caller of kdtv_tree_build; returns dict(parent, token, depth,
    score, n_nodes)."""
    import torch
    B, D, K = logp.shape
    dev = logp.device
    N = n_nodes
    out = {k: torch.empty((B, N), dtype=torch.int32, device=dev)
           for k in ("parent", "token", "depth")}
    out["score"] = torch.empty((B, N), dtype=torch.float32, device=dev)
    out["n_nodes"] = torch.empty(B, dtype=torch.int32, device=dev)
    code = lib().kdtv_tree_build(B, D, K, N, _p(logp), _p(tokens), _p(root_token),
                                 _p(out["parent"]), _p(out["token"]), _p(out["depth"]),
                                 _p(out["score"]), _p(out["n_nodes"]), _s(stream))
    if code:
        raise KdtvError(code, "kdtv_tree_build")
    return out


# ---- rotary positions, cache writes and reads -----------------------------------------
# Each caller below binds its tensors once, as VerifyAttn does, checks them, and launches on
# their device when called; the functions of the same names in lower case bind and call.

def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _index(t, shape, device, name):
    """An int32 index tensor of one of the calls (None passes)."""
    import torch
    if t is None:
        return None
    _need(t.dtype == torch.int32 and tuple(t.shape) == tuple(shape) and t.is_contiguous()
          and t.device == device, f"{name}: contiguous int32 {list(shape)} on {device}")
    return t


def _strides(t):
    """Strides of [B, N, H, ..] for the library, where all zero means contiguous."""
    s = t.stride()[:3]
    _need(any(s) or t.shape[:3].numel() == 1, "a tensor that repeats one row: make it contiguous")
    return (ctypes.c_int64 * 3)(*s)


def _apart(t):
    """Whether no two elements of a result share memory."""
    reach = 0
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
        if stride <= reach:
            return False
        reach += stride * (size - 1)
    return True


class _Bound:
    """A library call over bound tensors, launched on their device."""

    def _bind(self, name, device, args, keep, own=()):
        import torch
        self.torch, self._name, self.device = torch, name, device
        self._fn, self._args, self._keep = getattr(lib(), name), tuple(args), keep
        # what was allocated here belongs to the stream that is current now
        self._own, self._home = own, torch.cuda.current_stream(device)
        self._streams = {self._home.cuda_stream}

    def _join(self, s):
        """First launch on another stream than the one that was current at binding: behind what
        that one has under way (a word being cleared, the memory's last user), and what was
        allocated here stays until this stream is done with it."""
        torch = self.torch
        with torch.cuda.stream(s):
            if not torch.cuda.is_current_stream_capturing():
                s.wait_stream(self._home)
        for t in self._own:
            t.record_stream(s)
        self._streams.add(s.cuda_stream)

    def _launch(self, stream):
        torch = self.torch
        # (a Stream object for the current stream takes 2 us, a third of a small call)
        s = torch._C._cuda_getCurrentRawStream(self.device.index) if stream is None else stream.cuda_stream
        if s not in self._streams:
            self._join(torch.cuda.current_stream(self.device) if stream is None else stream)
        if torch.cuda.current_device() == self.device.index:
            code = self._fn(*self._args, s)
        else:
            with torch.cuda.device(self.device):
                code = self._fn(*self._args, s)
        if code:
            raise KdtvError(code, self._name)


def _on(stream):
    """What a call allocates belongs to the stream that it runs on."""
    import contextlib
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class RopeTable:
    """Rotary frequencies (kdtv_rope_init): `rot_dim` rotated elements per head, pairs
    (j, j + rot_dim / 2) ("half") or (2j, 2j + 1) ("interleaved"); `scaling` "none", "linear",
    "ntk" or "yarn" for long contexts.

    "yarn" also multiplies what it rotates by attn_factor, 0.1 ln(factor) + 1 unless given.  Give 1
    where the model puts its factor into the softmax scale (DeepSeek and Kimi models do)."""

    def __init__(self, rot_dim, *, layout="half", base=10000.0, scaling="none", factor=1.0,
                 orig_ctx=0, beta_fast=0.0, beta_slow=0.0, attn_factor=0.0):
        _need(layout in ROPE_LAYOUT, f"layout: one of {list(ROPE_LAYOUT)}")
        _need(scaling in ROPE_SCALING, f"scaling: one of {list(ROPE_SCALING)}")
        c = KdtvRopeConfig(rot_dim, ROPE_LAYOUT[layout], ROPE_SCALING[scaling], orig_ctx, base,
                           factor, beta_fast, beta_slow, attn_factor)
        self.c = KdtvRopeTable()
        code = lib().kdtv_rope_init(ctypes.byref(c), ctypes.byref(self.c))
        if code:
            raise KdtvError(code, "kdtv_rope_init")
        self.rot_dim, self.layout, self.amp = rot_dim, layout, self.c.amp


class Rope(_Bound):
    """Caller of kdtv_rope.  x: [B, N, H, dim], last dimension contiguous, float32 or bfloat16.

    Without `split`, out is like x with elements rot_off .. rot_off + rot_dim of every head
    rotated (out=x: in place).  With `split` (or a `rest` tensor), out holds the rotated part
    alone and rest the other elements: what VerifyAttn takes as q_rope and q_nope.
    """

    def __init__(self, table, x, *, prefix_len=None, depth=None, n_live=None, rot_off=0, out=None,
                 rest=None, split=False):
        import torch
        _need(isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 4 and x.numel() > 0
              and x.dtype in (torch.float32, torch.bfloat16) and x.stride(3) == 1,
              "x: a float32 or bfloat16 CUDA tensor [B, N, H, dim] with a contiguous last dimension")
        B, N, H, dim = x.shape
        split = split or rest is not None
        _need(0 <= rot_off and rot_off + table.rot_dim <= dim, "the rotated part lies outside the head")

        def result(t, d, name):
            if t is None:
                return torch.empty((B, N, H, d), dtype=x.dtype, device=x.device)
            _need(tuple(t.shape) == (B, N, H, d) and t.dtype == x.dtype and t.device == x.device
                  and (d == 0 or t.stride(3) == 1 and _apart(t)),
                  f"{name}: {[B, N, H, d]} like x, no two elements in one place")
            return t

        self.out = result(out, table.rot_dim if split else dim, "out")
        self.rest = result(rest, dim - table.rot_dim, "rest") if split else None
        # a head that is rotated whole has nothing left to copy: plain rotation
        copied = self.rest if self.rest is not None and self.rest.numel() else None
        a = KdtvRopeArgs(B, N, H, dim, rot_off, KDTV_F32 if x.dtype == torch.float32 else KDTV_BF16)
        for name, t in (("x_stride", x), ("y_stride", self.out), ("rest_stride", copied)):
            if t is not None:
                setattr(a, name, _strides(t))
        pl = _index(prefix_len, (B,), x.device, "prefix_len")
        dp = _index(depth, (B, N), x.device, "depth")
        nl = _index(n_live, (B,), x.device, "n_live")
        self._bind("kdtv_rope", x.device,
                   (ctypes.byref(table.c), ctypes.byref(a), _p(x), _p(self.out), _p(copied), _p(pl),
                    _p(dp), _p(nl)), (table, a, x, self.out, self.rest, pl, dp, nl),
                   [t for t in (self.out, self.rest) if t is not None])

    def __call__(self, stream=None):
        self._launch(stream)
        return self.out if self.rest is None else (self.out, self.rest)


def rope(table, x, *, stream=None, **kw):
    """Rotates x (see Rope); returns out, or (out, rest) when split.  Rows that are not live
    are left as they were in a given out, and undefined in a new one."""
    with _on(stream):
        return Rope(table, x, **kw)(stream)


class KvPart:
    """One tensor of a cache: [B, T, heads, dim] or [num_pages, page_size, heads, dim] (or
    without `heads`), float32, bfloat16, or one byte per element (uint8 or float8_e4m3fn);
    `scale`, for one-byte caches: exponent bytes, the cache's shape without dim, uint8.

    append: `src` [B, N, heads, dim] (last dimension contiguous), rotated from `rot_off` on
    unless that is None.  read: `out` [B, N, heads, dim], contiguous.
    """

    def __init__(self, cache, *, src=None, out=None, scale=None, rot_off=None):
        self.cache, self.src, self.out, self.scale, self.rot_off = cache, src, out, scale, rot_off


def _kv_setup(parts, which, page_table, kv_scale):
    """kdtv_kv_dims and kdtv_kv_part[] of KvPart objects; the rows come from their `which`."""
    import torch
    _need(1 <= len(parts) <= 2, "one or two parts")
    one_byte = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))
    d, cp, first, keep = KdtvKvDims(), (KdtvKvPart * len(parts))(), None, [page_table]
    for k, part in enumerate(parts):
        x, cache, scale = getattr(part, which), part.cache, part.scale
        _need(isinstance(x, torch.Tensor) and isinstance(cache, torch.Tensor) and x.is_cuda
              and cache.device == x.device, f"cache and {which}: CUDA tensors of one device")
        if cache.dim() == 3:
            cache = cache.unsqueeze(2)
            scale = scale.unsqueeze(2) if scale is not None and scale.dim() == 2 else scale
        if x.dim() == 3:
            x = x.unsqueeze(2)
        _need(x.dim() == 4 and cache.dim() == 4 and x.numel() > 0 and cache.numel() > 0
              and x.shape[2:] == cache.shape[2:], f"{which}: [B, N, heads, dim] with the cache's heads and dim")
        _need(cache.is_contiguous(), "cache: contiguous")
        _need(x.dtype in (torch.float32, torch.bfloat16), f"{which}: float32 or bfloat16")
        _need(x.stride(3) == 1 if which == "src" else x.is_contiguous(),
              f"{which}: " + ("last dimension contiguous" if which == "src" else "contiguous"))
        _need(cache.dtype in (torch.float32, torch.bfloat16) + one_byte,
              "cache: float32, bfloat16, uint8 or float8_e4m3fn")
        if scale is not None:
            _need(cache.dtype in one_byte and scale.dtype == torch.uint8 and scale.is_contiguous()
                  and scale.device == x.device and scale.shape == cache.shape[:3],
                  "scale: contiguous uint8, one byte per row and head of a one-byte cache")
        kind = (x.shape[:2], x.dtype, x.device, cache.dtype in one_byte or cache.dtype, cache.shape[:2])
        first = first or kind
        _need(kind == first, "the parts differ in rows, types or cache extent")
        cp[k].cache, cp[k].scale = _p(cache), _p(scale)
        setattr(cp[k], which, _p(x))
        if which == "src":
            cp[k].src_stride = _strides(x)
            cp[k].rotate, cp[k].rot_off = part.rot_off is not None, part.rot_off or 0
        cp[k].heads, cp[k].dim = x.shape[2], x.shape[3]
        keep += [x, cache, scale]
    (B, N), dtype, device, cdtype, extent = first
    d.B, d.N, d.parts, d.kv_scale = B, N, len(parts), kv_scale
    d.dtype = KDTV_F32 if dtype == torch.float32 else KDTV_BF16
    d.cache_dtype = KDTV_BF16_FP8KV if cdtype is True else KDTV_F32 if cdtype == torch.float32 else KDTV_BF16
    if page_table is None:
        _need(extent[0] == B, "a contiguous cache has one row block per request")
        d.t_stride = extent[1]
    else:
        _need(page_table.dim() == 2, "page_table: [B, max_pages]")
        _index(page_table, (B, page_table.shape[1]), device, "page_table")
        d.num_pages, d.page_size, d.max_pages = extent[0], extent[1], page_table.shape[1]
    return d, cp, device, B, N, keep


def _status_word(status, device):
    import torch
    if status is None:
        return torch.zeros(1, dtype=torch.int32, device=device)
    return _index(status, (1,), device, "status")


class KvAppend(_Bound):
    """Caller of kdtv_kv_append: the live rows of every part's src, rotated and quantised, to
    cache rows prefix_len[b] + i.  Calling it returns the status word (a tensor, 0 if all is
    well; it keeps the first error until it is cleared)."""

    def __init__(self, parts, prefix_len, *, rope=None, depth=None, n_live=None, page_table=None,
                 kv_scale=0.0, status=None):
        d, cp, device, B, N, keep = _kv_setup(parts, "src", page_table, kv_scale)
        _need(rope is not None or all(p.rot_off is None for p in parts), "a part rotates: rope is missing")
        pl = _index(prefix_len, (B,), device, "prefix_len")
        dp = _index(depth, (B, N), device, "depth")
        nl = _index(n_live, (B,), device, "n_live")
        self.status = _status_word(status, device)
        self._bind("kdtv_kv_append", device,
                   (ctypes.byref(d), cp, ctypes.byref(rope.c) if rope is not None else None, _p(pl), _p(dp),
                    _p(nl), _p(page_table), _p(self.status)), (d, cp, rope, pl, dp, nl, keep), [self.status])

    def __call__(self, stream=None):
        self._launch(stream)
        return self.status


class KvRead(_Bound):
    """Caller of kdtv_kv_read: cache rows start[b] .. start[b] + n_live[b] - 1 into every part's
    out[b].  Calling it returns the status word."""

    def __init__(self, parts, start=None, n_live=None, *, page_table=None, kv_scale=0.0, status=None):
        d, cp, device, B, N, keep = _kv_setup(parts, "out", page_table, kv_scale)
        st = _index(start, (B,), device, "start")
        nl = _index(n_live, (B,), device, "n_live")
        self.status = _status_word(status, device)
        self._bind("kdtv_kv_read", device, (ctypes.byref(d), cp, _p(st), _p(nl), _p(page_table),
                                            _p(self.status)), (d, cp, st, nl, keep), [self.status])

    def __call__(self, stream=None):
        self._launch(stream)
        return self.status


def kv_append(parts, prefix_len, *, stream=None, **kw):
    """Writes rows to a cache (see KvAppend); returns the status word."""
    with _on(stream):
        return KvAppend(parts, prefix_len, **kw)(stream)


def kv_read(parts, start=None, n_live=None, *, stream=None, **kw):
    """Reads rows of a cache (see KvRead); returns the status word."""
    with _on(stream):
        return KvRead(parts, start, n_live, **kw)(stream)


class GqaVerifyAttn(_Bound):
    """Caller of kdtv_gqa_verify_attn: a draft tree over a cache of keys and values per head.

    q, out: [B, N, H, d]; k, v: the caches, [B, T, H_kv, d] or (with page_table [B, max_pages])
    [num_pages, page_size, H_kv, d]; float32 or bfloat16, the caches also one byte per element
    with exponent bytes k_scale, v_scale (the caches' shape without d; for a cache that was written
    with one kv_scale: bytes of 127, `scale` times kv_scale, and the result times kv_scale).  Holds
    the workspace: calls of one object must not overlap on the GPU.  status() reads the status word.
    """

    def __init__(self, q, k, v, parent, prefix_len, *, n_nodes=None, page_table=None, k_scale=None,
                 v_scale=None, scale=0.0, flags=0, out=None):
        import torch
        one_byte = (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8))
        _need(isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 4 and q.is_contiguous()
              and q.numel() > 0 and q.dtype in (torch.float32, torch.bfloat16),
              "q: a contiguous float32 or bfloat16 CUDA tensor [B, N, H, d]")
        B, N, H, d = q.shape
        for t in (k, v):
            _need(isinstance(t, torch.Tensor) and t.device == q.device and t.dim() == 4 and t.is_contiguous()
                  and t.shape == k.shape and t.dtype == k.dtype and t.shape[3] == d and t.numel() > 0
                  and H % t.shape[2] == 0, "k, v: contiguous caches of one shape, [.., .., H_kv, d], on q's device")
        fp8 = k.dtype in one_byte
        _need(q.dtype == (torch.bfloat16 if fp8 else k.dtype), "q: the cache's type, bfloat16 for a one-byte cache")
        for t in (k_scale, v_scale):
            _need((t is not None) == fp8, "k_scale, v_scale: with a one-byte cache, and only there")
            _need(t is None or (t.dtype == torch.uint8 and t.is_contiguous() and t.device == q.device
                                and t.shape == k.shape[:3]), "k_scale, v_scale: contiguous uint8 [.., .., H_kv]")
        pa = _index(parent, (B, N), q.device, "parent")
        pl = _index(prefix_len, (B,), q.device, "prefix_len")
        _need(pa is not None and pl is not None, "parent and prefix_len")
        nn = _index(n_nodes, (B,), q.device, "n_nodes")
        D = KdtvGqaDims(B, N, H, k.shape[2], d)
        D.dtype = KDTV_BF16_FP8KV if fp8 else KDTV_F32 if q.dtype == torch.float32 else KDTV_BF16
        if page_table is None:
            _need(k.shape[0] == B, "a contiguous cache has one row block per request")
            D.t_stride = k.shape[1]
        else:
            _need(page_table.dim() == 2, "page_table: [B, max_pages]")
            _index(page_table, (B, page_table.shape[1]), q.device, "page_table")
            D.num_pages, D.page_size, D.max_pages = k.shape[0], k.shape[1], page_table.shape[1]
        D.scale, D.flags = scale, flags
        self.out = torch.empty_like(q) if out is None else out
        _need(self.out.shape == q.shape and self.out.dtype == q.dtype and self.out.device == q.device
              and self.out.is_contiguous(), "out: like q")
        with torch.cuda.device(q.device):
            nbytes = int(lib().kdtv_gqa_workspace_size(ctypes.byref(D)))
        if nbytes == 0:
            raise KdtvError(STATUS_CODE["KDTV_ERR_UNSUPPORTED"], "workspace size")
        self.dims = D
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        D.workspace, D.workspace_bytes = self.workspace.data_ptr(), nbytes
        self._status = torch.zeros(1, dtype=torch.int32, device=q.device)
        self._bind("kdtv_gqa_verify_attn", q.device,
                   (ctypes.byref(D), _p(q), _p(k), _p(v), _p(k_scale), _p(v_scale), _p(pa), _p(pl), _p(nn),
                    _p(page_table), _p(self.out), _p(self._status)),
                   (q, k, v, k_scale, v_scale, pa, pl, nn, page_table), [self.out, self.workspace, self._status])

    def __call__(self, stream=None):
        self._launch(stream)
        return self.out

    def status(self):
        """First device-side error since it was last read (0: none), or the timeout of a wait, which
        replaces any other; waits for the device, clears it."""
        self.torch.cuda.synchronize(self.device)
        code = int(self._status.item())
        if code:
            self._status.zero_()
            self.torch.cuda.synchronize(self.device)
        return code

    def launches(self):
        return int(lib().kdtv_gqa_launches_per_call(ctypes.byref(self.dims)))


def gqa_verify_attn(q, k, v, parent, prefix_len, *, stream=None, **kw):
    """Tree attention over a GQA cache (see GqaVerifyAttn); returns (out, status word)."""
    with _on(stream):
        op = GqaVerifyAttn(q, k, v, parent, prefix_len, **kw)
        return op(stream), op._status
