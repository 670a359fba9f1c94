"""kdtv_pages_resize against plain loops: everything is whole numbers, and equal."""

import numpy as np
import pytest

from oracle import serve_ops as O
from speculative_decoding_tree_mla_gb300 import kdtv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dev(a, dtype=torch.int32):
    return torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


class Pool:
    """A pool on the GPU and the same one in plain lists."""

    def __init__(self, B, max_pages, num, page, seed):
        perm = np.random.default_rng(seed).permutation(num).astype(np.int32)
        self.page, self.num, self.max_pages = page, num, max_pages
        self.free, self.held, self.table = [int(p) for p in perm], [0] * B, [[-1] * max_pages for _ in range(B)]
        self.gpu = kdtv.PagePool(dev(self.table), dev(self.held), dev(perm), dev([num]), page)
        self.stack = perm.copy()

    def resize(self, L, n, N, slots=True):
        B = len(L)
        full = [min(max(int(v), 0), N) for v in n]
        rows = [None if l < 0 or l + m > self.max_pages * self.page else l + m for l, m in zip(L, full)]
        short = O.pages_resize(rows, self.page, self.max_pages, self.num, self.free, self.held, self.table)
        r = kdtv.pages_resize(self.gpu, dev(L), N=N, n_live=dev(n), slots=True if slots else None)
        got, st = r if slots else (None, r)
        self.same()
        if slots:
            want = O.slots(L, full, N, self.page, self.num, self.held, self.table)
            assert np.array_equal(got.cpu().numpy(), want)
        return short, kdtv.STATUS[int(st)]

    def same(self):
        g = self.gpu
        assert g.n_pages.tolist() == self.held and g.page_table.tolist() == self.table
        k = int(g.free_count)
        assert k == len(self.free) and g.free_pages[:k].tolist() == self.free


@pytest.mark.parametrize("B,N,page,lo,hi", [(1, 1, 64, 0, 1), (1, 1, 1, 5, 6), (64, 8, 64, 0, 3000), (7, 33, 5, 0, 400),
                                            (300, 4, 16, 0, 500), (1024, 8, 64, 0, 2000), (3, 6000, 128, 0, 50),
                                            (512, 100, 16, 0, 90), (2, 20000, 3, 0, 100), (8192, 1, 4, 0, 9)])
def test_grow_trim_and_slots(B, N, page, lo, hi):
    rng = np.random.default_rng(B + N)
    width = -(-(hi + N) // page) + 2
    P = Pool(B, width, B * width, page, 1)
    L = rng.integers(lo, hi, B)
    assert P.resize(L, [0] * B, N) == (False, "KDTV_OK")                       # the prefixes
    for step in range(3):
        n = rng.integers(0, N + 1, B)
        assert P.resize(L, n, N) == (False, "KDTV_OK")                         # rows behind them
        keep = np.array([rng.integers(0, m + 1) for m in n])
        assert P.resize(L + keep, [0] * B, 0, slots=False) == (False, "KDTV_OK")
        L = np.where(rng.random(B) < 0.2, 0, np.minimum(L + keep, hi))         # some end, others go on
    assert P.resize([0] * B, [0] * B, 0, slots=False) == (False, "KDTV_OK")
    assert len(P.free) == B * width


def test_round_trip_restores_the_stack():
    P = Pool(40, 64, 40 * 20, 16, 2)
    L = np.arange(40) * 5
    P.resize(L, [0] * 40, 0, slots=False)
    before = P.gpu.free_pages.clone(), P.gpu.page_table.clone()
    P.resize(L, [100] * 40, 100)
    P.resize(L, [0] * 40, 0, slots=False)
    assert torch.equal(before[0], P.gpu.free_pages) and torch.equal(before[1], P.gpu.page_table)


@pytest.mark.parametrize("num", [1, 10, 37, 90])
def test_free_list_runs_out(num):
    """The first request that it does not suffice for, and those behind it that need pages, get none."""
    B, N, page = 30, 50, 16
    P = Pool(B, 8, num, page, 3)
    L = np.arange(B) * 2
    short, st = P.resize(L, [N] * B, N)
    assert short and st == "KDTV_ERR_NO_PAGES" and 0 <= len(P.free) < 8
    short, st = P.resize(L, [0] * B, N)                                        # what some hold is enough for others
    P.resize([0] * B, [0] * B, 0, slots=False)
    assert len(P.free) == num


@pytest.mark.parametrize("N", [5, 5000])
def test_rows_that_do_not_fit(N):
    P = Pool(4, N // 16 + 3, 4 * (N // 16 + 3), 16, 4)
    assert P.resize([3, 0, 7, 40], [N] * 4, N)[1] == "KDTV_ERR_BAD_PREFIX" if N + 40 > (N // 16 + 3) * 16 else True
    assert P.resize([3, -1, 7, 2 ** 31 - 1], [N] * 4, N)[1] == "KDTV_ERR_BAD_PREFIX"


@pytest.mark.parametrize("B,N", [(6, 4), (600, 4)])
def test_wrong_state_is_reported(B, N):
    """Counts and page ids out of range: those requests keep what they have, the others go on."""
    P = Pool(B, 8, B * 8, 16, 5)
    L = np.full(B, 40)
    P.resize(L, [N] * B, N)
    g = P.gpu
    g.page_table[2, 2] = B * 8                                                 # would be given back
    g.page_table[4, 1] = -7                                                    # would stay
    g.n_pages[5] = 9
    table, held, count = g.page_table.clone(), g.n_pages.clone(), int(g.free_count)
    L0 = np.full(B, 20)
    slots, st = kdtv.pages_resize(g, dev(L0), N=N, n_live=dev([N] * B), slots=True)
    assert kdtv.STATUS[int(st)] == "KDTV_ERR_BAD_PAGE"
    assert torch.equal(g.page_table[2], table[2]) and torch.equal(g.page_table[5], table[5])
    assert int(g.n_pages[2]) == 3 and int(g.n_pages[5]) == 9
    rest = [b for b in range(B) if b not in (2, 5)]
    assert all(int(g.n_pages[b]) == 2 for b in rest) and int(g.free_count) == count + len(rest)
    assert (slots[4] == -1).all() and (slots[5] == -1).all() and (slots[0] >= 0).all() and (slots[2] >= 0).all()
    for bad in (-1, B * 8 + 1):
        before = g.page_table.clone(), g.n_pages.clone(), g.free_pages.clone()
        g.free_count[0] = bad
        st = kdtv.pages_resize(g, dev(np.full(B, 90)), N=0)
        assert kdtv.STATUS[int(st)] == "KDTV_ERR_BAD_PAGE" and int(g.free_count) == bad
        assert all(torch.equal(a, b) for a, b in zip(before, (g.page_table, g.n_pages, g.free_pages)))
    g.free_count[0] = B * 8                                                    # with pages that requests hold
    st = kdtv.pages_resize(g, dev(np.zeros(B)), N=0)
    assert kdtv.STATUS[int(st)] == "KDTV_ERR_BAD_PAGE" and int(g.free_count) == B * 8
    assert torch.equal(before[0], g.page_table)


def test_far_slots_and_status_stays():
    """Slots beyond 32 bits; the first error stays in the word."""
    page = 1 << 20
    P = kdtv.PagePool(dev([[-1] * 4]), dev([0]), dev(np.arange(8192)), dev([8192]), page)
    slots, st = kdtv.pages_resize(P, dev([0]), N=3, slots=True)
    assert slots[0].tolist() == [8191 * page + i for i in range(3)] and int(st) == 0
    word = dev([7])
    st = kdtv.pages_resize(P, dev([-5]), N=3, status=word)
    assert st is word and int(word) == 7


def test_capture_and_side_stream():
    P = Pool(64, 40, 64 * 40, 16, 6)
    L = dev(np.arange(64) * 7)
    grow, trim = kdtv.PagesResize(P.gpu, L, N=8, slots=True), kdtv.PagesResize(P.gpu, L, N=0)
    side = torch.cuda.Stream()
    slots = grow(side)[0]
    trim(side)
    side.synchronize()
    first = slots.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grow()
        trim()
    slots.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert int(grow.status) == 0 and int(trim.status) == 0
    P.resize(np.arange(64) * 7, [8] * 64, 8)
    assert torch.equal(slots >= 0, torch.ones_like(slots, dtype=torch.bool)) and slots.shape == first.shape


def test_python_refusals():
    P = Pool(4, 8, 32, 16, 7).gpu
    L = dev([0] * 4)
    for kw in (dict(), dict(N=4, n_live=dev([1] * 3)), dict(N=4, slots=torch.zeros(4, 5, dtype=torch.int64, device="cuda")),
               dict(N=4, slots=torch.zeros(4, 4, dtype=torch.int32, device="cuda")), dict(N=4, status=dev([0, 0]))):
        with pytest.raises(ValueError):
            kdtv.pages_resize(P, L, **kw)
    with pytest.raises(ValueError):
        kdtv.PagePool(dev([[0]]), dev([0, 0]), dev([0]), dev([1]), 16)


@pytest.mark.parametrize("N", [5, 5000])
def test_one_row_too_many(N):
    """A request whose rows fill its row of the table to the last place, and one that has one row more."""
    width = (N + 40) // 16
    room = width * 16
    P = Pool(4, width, 4 * width, 16, 9)
    assert P.resize([3, 0, room - N, 7], [N] * 4, N) == (False, "KDTV_OK")
    assert P.held[2] == width
    held = list(P.held)
    short, st = P.resize([0, 0, room - N + 1, 0], [0, 0, N, 0], N)
    assert not short and st == "KDTV_ERR_BAD_PREFIX" and P.held == [0, 0, held[2], 0]
    assert P.resize([0, 0, room, 0], [N, N, 0, N], N) == (False, "KDTV_OK")
    assert P.resize([room, 0, 0, 0], [1, 0, 0, 0], N)[1] == "KDTV_ERR_BAD_PREFIX"


@pytest.mark.parametrize("B,N", [(64, 8), (300, 40), (64, 1000)])
def test_replays_give_the_same_slots(B, N):
    """Growing and trimming back leaves the stack as it was, so every replay of the two gives the first call's slots."""
    P = Pool(B, 80, B * 80, 16, 10)
    L = dev(np.arange(B) % 97 * 2)
    grow, trim = kdtv.PagesResize(P.gpu, L, N=N, slots=True), kdtv.PagesResize(P.gpu, L, N=0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots = grow(side)[0]
    trim(side)
    side.synchronize()
    first = slots.clone()
    assert (first >= 0).all() and len(torch.unique(first)) == B * N
    state = [t.clone() for t in (P.gpu.free_pages, P.gpu.free_count, P.gpu.n_pages, P.gpu.page_table)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grow()
        trim()
    for _ in range(3):
        slots.zero_()
        g.replay()
        assert torch.equal(slots, first)
    assert all(torch.equal(a, b) for a, b in zip(state, (P.gpu.free_pages, P.gpu.free_count, P.gpu.n_pages, P.gpu.page_table)))
    assert int(grow.status) == 0 and int(trim.status) == 0


@pytest.mark.parametrize("bad", [-1, "num", 2 ** 31 - 1])
@pytest.mark.parametrize("B,N,page", [(30, 50, 16), (600, 50, 16), (30, 3000, 64)])
def test_bad_ids_on_the_free_stack(bad, B, N, page):
    """The request that would get an id out of range, and those behind it that need pages, keep what they have; nothing
    of the bad id leaves the stack, and once it is mended the pool goes on."""
    need = -(-N // page)
    P = Pool(B, need + 5, B * (need + 5), page, 11)
    assert P.resize([page] * B, [0] * B, N) == (False, "KDTV_OK")             # a page each
    for where in (0, need, 7 * need + 1, B * need - 1, B * need):              # places from the top; the last one is not taken
        at = len(P.free) - 1 - where
        was = P.free[at]
        P.free[at] = P.num if bad == "num" else bad
        P.gpu.free_pages[at] = P.free[at]
        short, st = P.resize([page] * B, [N] * B, N)                           # (tables, counts, stack and slots as the oracle's)
        assert not short and st == ("KDTV_ERR_BAD_PAGE" if where < B * need else "KDTV_OK")
        assert P.held == [1 + (need if b < where // need or where == B * need else 0) for b in range(B)]
        assert P.resize([page] * B, [0] * B, N) == (False, "KDTV_OK")
        P.free[at] = was
        P.gpu.free_pages[at] = was
    # some give back, some need: pages that went back are on top of the bad id
    P.resize([page] * B, [N if b < B // 2 else 0 for b in range(B)], N)
    at = len(P.free) - 1
    was, P.free[at] = P.free[at], -5
    P.gpu.free_pages[at] = -5
    short, st = P.resize([page] * B, [0 if b < B // 2 else N for b in range(B)], N)
    assert not short and st == "KDTV_OK"
    short, st = P.resize([page] * B, [page if b < B // 2 else N for b in range(B)], N)
    assert not short and st == "KDTV_ERR_BAD_PAGE" and P.held[0] == 1
    assert P.free[at] == -5


def test_nearly_two_to_the_31_entries():
    """All that the table may hold: counters that run past the last entry by whole runs stay unsigned.  (26 GB.)"""
    B, width, page = 8192, (1 << 18) - 1, 4096
    num = B * width
    ids = torch.arange(num, dtype=torch.int32, device="cuda")
    P = kdtv.PagePool(torch.full((B, width), -1, dtype=torch.int32, device="cuda"), dev(np.zeros(B)), ids.flip(0), dev([num]), page)
    full = dev(np.full(B, width * page))
    assert kdtv.STATUS[int(kdtv.pages_resize(P, full, N=0))] == "KDTV_OK"
    assert int(P.free_count) == 0 and (P.n_pages == width).all() and torch.equal(P.page_table.view(-1), ids)
    assert kdtv.STATUS[int(kdtv.pages_resize(P, dev(np.zeros(B)), N=0))] == "KDTV_OK"
    assert int(P.free_count) == num and (P.n_pages == 0).all() and (P.page_table == -1).all()
    assert torch.equal(P.free_pages.flip(0), ids)
    del P, ids, full
    torch.cuda.empty_cache()
