"""The pages' book (fork, reserve, free, compact) against lists, entry by entry, the
moves of their contents, and a run of all of it around paged attention."""

import math
import random

import pytest
import torch

import draft_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_attention_layout_gb300 import build
    build.build()
    from sparse_attention_layout_gb300 import bsp as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Device:
    """A book on the device beside one of lists."""

    def __init__(self, bsp, n_pages, n_seq, max_pages, page):
        self.bsp, self.page = bsp, page
        self.W = bsp.bsp_window_create()
        self.book = ref.Book(n_pages, n_seq, max_pages, page)
        self.pull()

    def pull(self):
        """The device's book from the lists'."""
        b = self.book
        self.refs, self.table, self.kv = ints(b.refs), ints(b.table), ints(b.kv)

    def same(self):
        b = self.book
        assert b.agrees()
        assert self.refs.tolist() == b.refs
        assert self.table.tolist() == b.table
        assert self.kv.tolist() == b.kv

    def status(self):
        return self.bsp.bsp_window_status(self.W)

    def free(self):
        self.bsp.bsp_pages_free(self.W, self.refs, self.table, self.kv, self.page)
        self.book.free()
        self.same()

    def fork(self, parent):
        self.bsp.bsp_pages_fork(self.W, self.refs, self.table, self.kv, ints(parent), self.page)
        self.book.fork(parent)
        self.same()

    def reserve(self, want):
        src, dst = self.bsp.bsp_pages_reserve(self.W, self.refs, self.table, self.kv, ints(want), self.page)
        s, d, enough = self.book.reserve(want)
        self.same()
        assert src.tolist() == s and dst.tolist() == d
        assert self.status() == (0 if enough else -4)
        return src, dst

    def compact(self, in_place):
        out = (self.refs, self.table) if in_place else (None, None)
        keep = self.refs.clone(), self.table.clone()
        refs, table, src, dst = self.bsp.bsp_pages_compact(self.W, self.refs, self.table, *out)
        assert in_place or (torch.equal(self.refs, keep[0]) and torch.equal(self.table, keep[1]))
        s, d = self.book.compact()
        self.refs, self.table = refs, table
        self.same()
        assert src.tolist() == s and dst.tolist() == d
        return src, dst

    def grow(self, want):
        """Lengths up to what was reserved."""
        for i, w in enumerate(want):
            if w > self.book.kv[i]:
                self.book.kv[i] = w
        self.kv = ints(self.book.kv)


# (n_pages, n_seq, max_pages, page, turns)
BOOKS = [(1, 1, 1, 16, 10), (7, 3, 4, 16, 60), (200, 12, 30, 16, 40), (5000, 60, 90, 32, 15), (3000, 1500, 8, 16, 8),
         (20000, 5, 4000, 16, 6), (70000, 40, 1024, 64, 4),
         (16384, 30, 500, 16, 4), (16385, 30, 500, 16, 4), (65537, 30, 500, 16, 3),
         (100000, 300, 400, 16, 3)]


@pytest.mark.parametrize("case", BOOKS, ids=str)
def test_turns(bsp, case):
    """Turns of everything, at random, until pages run out now and then."""
    n_pages, n_seq, max_pages, page, turns = case
    r = random.Random(n_pages)
    d = Device(bsp, n_pages, n_seq, max_pages, page)
    most = max_pages * page
    for turn in range(turns):
        lens = d.book.kv
        want = [min(most, n + r.choice((0, 1, page, r.randint(1, 3 * page + 1), r.randint(1, max(1, most // 3))))) for n in lens]
        before = [list(x) for x in d.book.table]
        d.reserve(want)
        if all(x >= 0 for i, row in enumerate(d.book.table) for x in row[:d.book.held(want[i])]) and \
                not any(n > 1 for i, row in enumerate(d.book.table) for j in range(lens[i] // page, d.book.held(want[i]))
                        if want[i] > lens[i] for n in (d.book.refs[row[j]],)):
            d.grow(want)
        else:  # not enough: some sequences end
            for i in r.sample(range(n_seq), max(1, n_seq // 3)):
                d.book.kv[i] = 0
            d.kv = ints(d.book.kv)
        if r.random() < 0.5:
            d.free()
        if r.random() < 0.7:
            d.fork([r.choice((i, i, r.randrange(n_seq), r.randrange(max(0, i - 2), i + 1), -1 if r.random() < 0.3 else i))
                    for i in range(n_seq)])
        if r.random() < 0.3:  # lengths fall back into pages that others share
            d.book.kv = [r.randint(n // 2, n) for n in d.book.kv]
            d.kv = ints(d.book.kv)
        if r.random() < 0.5:
            d.compact(r.random() < 0.5)
        assert d.status() == 0
    d.book.kv = [0] * n_seq
    d.kv = ints(d.book.kv)
    d.free()
    assert d.book.refs == [0] * n_pages


@pytest.mark.parametrize("n_pages", [4096, 4097, 16385, 65536, 200001])
def test_compaction_of_far_pages(bsp, n_pages):
    """Whole scans of pages that are free, or in use, or all of them."""
    W = bsp.bsp_window_create()
    g = torch.Generator(device="cuda").manual_seed(n_pages)
    half = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    half[n_pages - n_pages // 2:] = 1  # the last half: every page moves, or nearly
    last = torch.zeros_like(half)
    last[-1] = 3
    for refs in (half, last, torch.zeros_like(half), torch.ones_like(half), 1 - half,
                 torch.randint(0, 3, (n_pages,), generator=g, device="cuda", dtype=torch.int32)):
        table = refs.nonzero()[:, 0].to(torch.int32)
        table = torch.cat([table, table.new_full((7,), -1)]).flip(0)[None].contiguous()
        live = int((refs > 0).sum())
        high, low = (refs[live:] > 0).nonzero()[:, 0] + live, (refs[:live] == 0).nonzero()[:, 0]
        place = torch.arange(n_pages, device="cuda")
        place[high] = low
        want = refs.clone()
        want[low], want[high] = refs[high], 0
        out, moved, src, dst = bsp.bsp_pages_compact(W, refs, table)
        assert torch.equal(out, want) and torch.equal(moved, torch.where(table >= 0, place[table.clamp(min=0).long()].to(torch.int32), table))
        n = len(high)
        assert torch.equal(src[:n].long(), high) and torch.equal(dst[:n].long(), low)
        assert bool((src[n:] == -1).all()) and bool((dst[n:] == -1).all())
    assert bsp.bsp_window_status(W) == 0


def test_reordered_sequences(bsp):
    """Rows that all read one another's."""
    d = Device(bsp, 100, 8, 6, 16)
    d.reserve([10 * i for i in range(8)])
    d.grow([10 * i for i in range(8)])
    for parent in ([1, 2, 3, 4, 5, 6, 7, 0], [7, 6, 5, 4, 3, 2, 1, 0], [3] * 8, [0, 0, 2, 2, 2, 5, 5, -1], [-1] * 8):
        d.fork(parent)
        assert d.status() == 0


def test_shared_pages_are_copied_once_written(bsp):
    """Three forks of one sequence: the first of those that write keeps the page
    when all who hold it write, else nobody does."""
    for writers, keeps in (([0, 1, 2], 0), ([1, 2], None), ([2], None)):
        d = Device(bsp, 20, 3, 4, 16)
        d.reserve([20, 0, 0])
        d.grow([20, 0, 0])
        d.fork([0, 0, 0])
        page = d.book.table[0][1]
        src, dst = d.reserve([21 if i in writers else 0 for i in range(3)])
        for i in range(3):
            moved = i in writers and i != keeps
            assert (src[i].item() == page) == moved and (d.book.table[i][1] != page) == moved
            assert d.book.table[i][0] == d.book.table[0][0]
    # nothing to write: nothing to copy, not even beside a full page
    d = Device(bsp, 20, 2, 4, 16)
    d.reserve([32, 0])
    d.grow([32, 0])
    d.fork([0, 0])
    src, _ = d.reserve([32, 32])
    assert src.tolist() == [-1, -1]
    src, _ = d.reserve([33, 40])
    assert src.tolist() == [-1, -1]


def test_contents_follow_the_book(bsp):
    """Sequences that fork, write and move: each reads its own tokens back."""
    r = random.Random(3)
    for dtype, slots_first in ((torch.float32, False), (torch.bfloat16, True)):
        n_pages, n_seq, page, H, D = 150, 10, 16, 2, 16
        d = Device(bsp, n_pages, n_seq, 12, page)
        shape = (n_pages, page, H, D) if slots_first else (n_pages, H, page, D)
        K, V = torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(shape, dtype=dtype, device="cuda")
        if slots_first:
            K, V = K.transpose(1, 2), V.transpose(1, 2)
        text, token = [[] for _ in range(n_seq)], 0
        for turn in range(25):
            grow = [r.choice((0, 1, r.randint(1, 20))) if len(t) < 150 else 0 for t in text]
            want = [len(t) + g for t, g in zip(text, grow)]
            src, dst = d.reserve(want)
            bsp.bsp_paged_copy(d.W, K, V, src, dst)
            new = []
            for t, g in zip(text, grow):
                ids = [(token + i) % 251 for i in range(g)]
                token += g
                t += ids
                new += ids
            d.grow(want)
            rows = torch.tensor(new, device="cuda", dtype=dtype)[:, None, None].expand(len(new), H, D).contiguous()
            starts = ints([sum(grow[:i]) for i in range(n_seq + 1)])
            bsp.bsp_paged_append(d.W, rows, -rows, K, V, starts, d.kv, d.table)
            if r.random() < 0.6:
                parent = [r.choice((i, r.randrange(n_seq))) for i in range(n_seq)]
                d.fork(parent)
                text = [list(text[p]) for p in parent]
            if r.random() < 0.5:
                src, dst = d.compact(True)
                bsp.bsp_paged_copy(d.W, K, V, src, dst)
                live = sum(n > 0 for n in d.book.refs)
                K.transpose(1, 2)[live:] = math.nan  # nobody reads what lies behind
            for i, t in enumerate(text):
                at = torch.arange(len(t), device="cuda")
                pg, sl = d.table[i][at // page].long(), at % page
                want_k = torch.tensor(t, device="cuda", dtype=dtype)[:, None, None].expand(len(t), H, D)
                assert torch.equal(K[pg, :, sl], want_k) and torch.equal(V[pg, :, sl], -want_k)
        assert d.status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n_pages,H,page,D,slots_first", [(9, 1, 16, 16, False), (40, 3, 32, 80, True), (64, 8, 128, 128, False), (3000, 2, 16, 48, False)])
def test_copy(bsp, n_pages, H, page, D, slots_first, dtype):
    g = torch.Generator(device="cuda").manual_seed(n_pages)
    shape = (n_pages, page, H, D) if slots_first else (n_pages, H, page, D)
    K, V = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    if slots_first:
        K, V = K.transpose(1, 2), V.transpose(1, 2)
    order = torch.randperm(n_pages).tolist()
    n = n_pages // 2
    src, dst = order[:n], order[n:2 * n]
    src[0], dst[0] = -1, 3  # left out
    if n > 3:
        src[1] = src[2]  # one page to two
        src[3] = dst[3] = order[-1]
    k, v = K.clone(), V.clone()
    for a, b in zip(src, dst):
        if a >= 0:
            k[b], v[b] = K[a], V[a]
    W = bsp.bsp_window_create()
    bsp.bsp_paged_copy(W, K, V, ints(src), ints(dst))
    assert torch.equal(K, k) and torch.equal(V, v) and bsp.bsp_window_status(W) == 0
    for pair in ((n_pages, 0), (0, n_pages), (2 ** 31 - 1, 1), (1, 2 ** 31 - 1)):
        bsp.bsp_paged_copy(W, K, V, ints([pair[0], -5]), ints([pair[1], 0]))
        assert bsp.bsp_window_status(W) == -7 and torch.equal(K, k) and torch.equal(V, v)
    bsp.bsp_paged_copy(W, K, V, ints([]), ints([]))


def test_both_caches_in_one_tensor(bsp):
    """K and V of a page side by side; rows that the accepted ones move along too."""
    both = torch.randn(30, 2, 3, 32, 48, device="cuda", dtype=torch.float32).to(torch.float16)
    W, want = bsp.bsp_window_create(), both.clone()
    want[[4, 9]] = both[[20, 2]]
    bsp.bsp_paged_copy(W, both[:, 0], both[:, 1], ints([20, 2]), ints([4, 9]))
    assert torch.equal(both, want)
    table, kv, starts = ints([[7, 3]]), ints([40]), ints([0, 12])  # nodes at 28 .. 39
    for to, at in ((28, 28), (29, 31), (30, 39)):
        want[[7, 3][to // 32], :, :, to % 32] = both[[7, 3][at // 32], :, :, at % 32]
    bsp.bsp_paged_keep(W, both[:, 0], both[:, 1], starts, kv, table, ints([0, 3, 11] + [-1] * 9), ints([3]))
    assert torch.equal(both, want) and bsp.bsp_window_status(W) == 0


def test_copy_beyond_32_bit_offsets(bsp):
    K = torch.zeros(16500, 8, 128, 128, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros(16500, 8, 128, 128, dtype=torch.bfloat16, device="cuda")
    K[16499], V[16499] = torch.randn(2, 8, 128, 128, device="cuda").to(torch.bfloat16)
    W = bsp.bsp_window_create()
    bsp.bsp_paged_copy(W, K, V, ints([16499, 16499]), ints([16498, 0]))
    assert torch.equal(K[16498], K[16499]) and torch.equal(V[0], V[16499]) and not bool(K[16497].any())


def test_bad_books_are_reported(bsp):
    W = bsp.bsp_window_create()
    page = 16

    def fresh():
        d = Device(bsp, 20, 3, 4, page)
        d.reserve([20, 33, 5])
        d.grow([20, 33, 5])
        return d

    # lengths out of range: the sequence is left out
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        d = fresh()
        d.kv[1] = bad
        was = d.table.clone(), d.refs.clone()
        bsp.bsp_pages_free(W, d.refs, d.table, d.kv, page)
        assert bsp.bsp_window_status(W) == -7 and torch.equal(d.table, was[0]) and torch.equal(d.refs, was[1])
        bsp.bsp_pages_reserve(W, d.refs, d.table, d.kv, ints([20, 64, 5]), page)
        assert bsp.bsp_window_status(W) == -7 and torch.equal(d.table, was[0]) and torch.equal(d.refs, was[1])
        bsp.bsp_pages_fork(W, d.refs, d.table, d.kv, ints([0, 1, 1]), page)
        assert bsp.bsp_window_status(W) == -7 and torch.equal(d.table, was[0]) and torch.equal(d.refs, was[1])
        d = fresh()
        bsp.bsp_pages_reserve(W, d.refs, d.table, d.kv, ints([20, bad, 5]), page)
        assert bsp.bsp_window_status(W) == -7 and torch.equal(d.table, was[0]) and torch.equal(d.refs, was[1])
    for bad in (3, -2, 2 ** 31 - 1, -2 ** 31):
        d = fresh()
        was = d.table.clone(), d.refs.clone(), d.kv.clone()
        bsp.bsp_pages_fork(W, d.refs, d.table, d.kv, ints([0, bad, 2]), page)
        assert bsp.bsp_window_status(W) == -7
        assert torch.equal(d.table, was[0]) and torch.equal(d.refs, was[1]) and torch.equal(d.kv, was[2])
    # entries out of range count as none, and are never looked up
    for bad in (20, 2 ** 31 - 1):
        d = fresh()
        d.table[1, 2] = bad
        bsp.bsp_pages_fork(W, d.refs, d.table, d.kv, ints([0, 1, 1]), page)
        assert bsp.bsp_window_status(W) == -7 and d.table[2].tolist() == d.book.table[1][:2] + [-1, -1]
        d = fresh()
        d.table[1, 3] = bad
        bsp.bsp_pages_free(W, d.refs, d.table, d.kv, page)
        assert bsp.bsp_window_status(W) == -7 and d.table.tolist() == d.book.table and d.refs.tolist() == d.book.refs
        d.table[1, 2] = bad
        bsp.bsp_pages_reserve(W, d.refs, d.table, d.kv, ints([20, 40, 5]), page)
        assert bsp.bsp_window_status(W) == -7 and d.table[1, 2].item() == bad
        bsp.bsp_pages_compact(W, d.refs, d.table)
        assert bsp.bsp_window_status(W) == -7
    # no page left: what can be had is given, in order
    d = fresh()
    src, dst = bsp.bsp_pages_reserve(W, d.refs[:7], d.table, d.kv, ints([64, 64, 64]), page)
    assert bsp.bsp_window_status(W) == -4
    s, t, enough = d.book.reserve([64, 64, 64])
    first = [x if x < 7 else -1 for row in d.book.table for x in row]
    assert not any(x >= 0 for x in s) and [x for row in d.table.tolist() for x in row] == first


def test_refusals(bsp):
    W = bsp.bsp_window_create()
    d = Device(bsp, 20, 3, 4, 16)
    K = torch.zeros(20, 2, 16, 32, device="cuda")
    good = {
        "bsp_pages_free": [d.refs, d.table, d.kv, 16],
        "bsp_pages_fork": [d.refs, d.table, d.kv, ints([0, 1, 2]), 16],
        "bsp_pages_reserve": [d.refs, d.table, d.kv, ints([0, 0, 0]), 16],
        "bsp_pages_compact": [d.refs, d.table, d.refs, d.table],
        "bsp_paged_copy": [K, K.clone(), ints([0, 1]), ints([2, 3])],
    }
    for name, args in good.items():
        getattr(bsp, name)(W, *args)
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            for bad in (a.cpu(), a.double() if a.is_floating_point() else a.long(), a[None]):
                with pytest.raises((ValueError, TypeError)):
                    getattr(bsp, name)(W, *args[:i], bad, *args[i + 1:])
            if a is d.kv or i > 1:
                with pytest.raises(ValueError):
                    getattr(bsp, name)(W, *args[:i], a[:-1], *args[i + 1:])

    def code(name, *args):
        with pytest.raises(bsp.BspError) as e:
            getattr(bsp, name)(W, *args)
        return e.value.code

    for page in (0, 8, 17, 256, -16):
        assert code("bsp_pages_free", d.refs, d.table, d.kv, page) == -1
        assert code("bsp_pages_fork", d.refs, d.table, d.kv, ints([0, 1, 2]), page) == -1
        assert code("bsp_pages_reserve", d.refs, d.table, d.kv, d.kv, page) == -1
    assert code("bsp_paged_copy", K, K, ints([0]), ints([1])) == -1
    assert code("bsp_paged_copy", K[..., :24], K[..., :24].clone(), ints([0]), ints([1])) == -1
    assert code("bsp_paged_copy", K[:1].expand(20, 2, 16, 32), K, ints([0]), ints([1])) == -1
    lib, n = bsp.lib(), bsp._pages_bytes(3, 4, 20)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for at, size, want in ((ws.data_ptr(), n, 0), (ws.data_ptr(), n - 1, -1), (ws.data_ptr() + 4, n, -3), (None, n, -1)):
        p = [t.data_ptr() for t in (d.refs, d.table, d.kv, d.kv)]
        out = [torch.empty(20, dtype=torch.int32, device="cuda") for _ in range(2)]
        q = [t.data_ptr() for t in out]
        assert lib.bsp_pages_fork(W.handle, *p[:3], ints([0, 1, 2]).data_ptr(), 3, 4, 20, 16, at, size, stream) == want
        assert lib.bsp_pages_reserve(W.handle, *p, *q, 3, 4, 20, 16, at, size, stream) == want
        assert lib.bsp_pages_compact(W.handle, *p[:2], *p[:2], *q, 3, 4, 20, at, size, stream) == want
    assert lib.bsp_pages_workspace(3, 4, 0) == 0 and lib.bsp_pages_workspace(-1, 4, 4) == 0
    none = ints([])
    bsp.bsp_pages_free(W, d.refs, none.view(0, 4), none, 16)
    bsp.bsp_pages_fork(W, d.refs, none.view(0, 4), none, none, 16)
    assert bsp.bsp_pages_reserve(W, d.refs, none.view(0, 4), none, none, 16)[0].shape == (0,)
    assert bsp.bsp_pages_compact(W, d.refs, none.view(0, 4))[2].shape == (10,)
    assert bsp.bsp_window_status(W) == 0


# ------------------------------------------------------------ run together --

class Model:
    """One layer of attention over a small vocabulary, in fp32: embeddings, rotary
    positions, paged attention and an output row per token."""

    def __init__(self, bsp, V, Hq, Hkv, D, window, sinks, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bsp, self.V, self.D = bsp, V, D
        self.q, self.k, self.v = (torch.randn(V, H, D, generator=g, device="cuda") for H in (Hq, Hkv, Hkv))
        self.out = torch.randn(Hq * D, V, generator=g, device="cuda")
        self.W = bsp.bsp_window_create(window, sinks)
        self.R = bsp.bsp_rotary_create(*bsp.rotary_frequencies(D))

    def rows(self, tokens, positions):
        t = tokens.long()
        q, k = self.bsp.bsp_rotary(self.R, self.q[t], self.k[t], positions)
        return q, k, self.v[t]

    def logits(self, O):
        return (O.flatten(1) @ self.out) / math.sqrt(self.out.shape[0])


@pytest.mark.parametrize("window,sinks", [(0, 0), (12, 2)])
@pytest.mark.parametrize("greedy", [True, False])
def test_drafted_decoding(bsp, greedy, window, sinks):
    """Steps that reserve pages, turn, append, attend to trees of drafted tokens,
    verify them, keep the accepted rows and give pages back.  Greedy: the text is
    that of decoding one token after the other.  Drawn: what the cache holds in the
    end is what the text's tokens give, and a captured step does the same."""
    V, n_seq, page, steps, nodes = 8, 3, 16, 20, 7
    m = Model(bsp, V, 4, 2, 32, window, sinks, 1)
    W = m.W
    parent = [-1, 0, 0, 1, 1, 3, 5]
    n_pages, max_pages = 60, 16
    refs, table = torch.zeros(n_pages, dtype=torch.int32, device="cuda"), torch.full((n_seq, max_pages), -1, dtype=torch.int32, device="cuda")
    kv = ints([0] * n_seq)
    K, V_ = (torch.zeros(n_pages, 2, page, 32, device="cuda") for _ in range(2))
    last = ints([5, 1, 3])
    text = [[5], [1], [3]]
    starts, parents = ints([nodes * i for i in range(n_seq + 1)]), ints(parent * n_seq)
    g = torch.Generator(device="cuda").manual_seed(4)
    draft_p = torch.softmax(torch.randn(V, V, generator=g, device="cuda") * 2, -1)

    def step(last, kv, tokens, draft, accept, sample):
        """One step on given tokens; the pages are reserved already."""
        full = kv + nodes
        pos, bits = bsp.bsp_draft_tree(W, starts, full, parents, nodes)
        q, k, v = m.rows(tokens, pos)
        bsp.bsp_paged_append(W, k, v, K, V_, starts, full, table)
        O, _ = bsp.bsp_paged_tree_attention(W, q, K, V_, starts, full, table, pos, bits, scale=0.2)
        logits = m.logits(O)
        target = (logits.argmax(-1)[:, None] == torch.arange(V, device="cuda")).float() if greedy else torch.softmax(logits, -1)
        path, count, token = bsp.bsp_draft_verify(W, target, draft, tokens, starts, parents, accept, sample)
        bsp.bsp_paged_keep(W, K, V_, starts, full, table, path, count)
        return path, count, token

    def drafted(last):
        """Tokens of the trees, drawn from a row of the draft per token (or its
        likeliest ones)."""
        tok, rows = torch.zeros(n_seq, nodes, dtype=torch.int64, device="cuda"), []
        tok[:, 0] = last
        for a in range(1, nodes):
            p = draft_p[tok[:, parent[a]]]
            tok[:, a] = p.argsort(-1, descending=True)[:, parent[:a].count(parent[a])] if greedy else \
                torch.multinomial(p, 1, generator=g)[:, 0]
        return tok.flatten().to(torch.int32), None if greedy else draft_p[tok.flatten()].contiguous()

    for it in range(steps):
        src, dst = bsp.bsp_pages_reserve(W, refs, table, kv, kv + nodes, page)
        bsp.bsp_paged_copy(W, K, V_, src, dst)
        tokens, draft = drafted(last)
        accept, sample = torch.rand(n_seq * nodes, generator=g, device="cuda"), torch.rand(n_seq, generator=g, device="cuda")
        if it == steps - 1:
            # the last one captured, on the side as graphs are, and replayed
            before = [t.clone() for t in (K, V_)]
            want = step(last, kv, tokens, draft, accept, sample)
            after = [t.clone() for t in (K, V_)]
            K.copy_(before[0]), V_.copy_(before[1])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = step(last, kv, tokens, draft, accept, sample)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert torch.equal(K, after[0]) and torch.equal(V_, after[1])
            path, count, token = got
        else:
            path, count, token = step(last, kv, tokens, draft, accept, sample)
        for i in range(n_seq):
            took = path[nodes * i:nodes * i + count[i].item()].tolist()
            text[i] += [tokens[nodes * i + x].item() for x in took[1:]] + [token[i].item()]
        kv, last = kv + count, token
        bsp.bsp_pages_free(W, refs, table, kv, page)
        assert bsp.bsp_window_status(W) == 0
    assert refs.sum().item() == sum(-(-n // page) for n in kv.tolist())
    assert sum(len(t) for t in text) > n_seq * (steps + 1)  # something was accepted
    for i in range(n_seq):
        assert kv[i].item() == len(text[i]) - 1
    if greedy:
        # one token after the other, over a cache of its own
        refs2, table2 = torch.zeros_like(refs), torch.full_like(table, -1)
        kv2, now = ints([0] * n_seq), ints([5, 1, 3])
        K2, V2 = torch.zeros_like(K), torch.zeros_like(V_)
        ones = ints([0, 1, 2, 3])
        plain = [[t[0]] for t in text]
        for _ in range(max(len(t) for t in text) - 1):
            bsp.bsp_pages_reserve(W, refs2, table2, kv2, kv2 + 1, page)
            q, k, v = m.rows(now, kv2)
            kv2 = kv2 + 1
            bsp.bsp_paged_append(W, k, v, K2, V2, ones, kv2, table2)
            O, _ = bsp.bsp_paged_attention(W, q, K2, V2, ones, kv2, table2, scale=0.2)
            now = m.logits(O).argmax(-1).to(torch.int32)
            for i in range(n_seq):
                plain[i].append(now[i].item())
        assert [p[:len(t)] for p, t in zip(plain, text)] == text
    # the cache holds the text's own rows
    for i in range(n_seq):
        n = kv[i].item()
        at = torch.arange(n, device="cuda")
        _, k, v = m.rows(torch.tensor(text[i][:n], device="cuda"), at.to(torch.int32))
        pg, sl = table[i][at // page].long(), at % page
        assert torch.equal(K[pg, :, sl], k) and torch.equal(V_[pg, :, sl], v)


def test_a_captured_turn_follows_the_book(bsp):
    """Free, fork, reserve and copy in a graph, replayed on other lengths and parents."""
    d = Device(bsp, 80, 6, 8, 16)
    K, V = (torch.randn(80, 2, 16, 32, device="cuda") for _ in range(2))
    want, parent = ints([0] * 6), ints(list(range(6)))

    def turn():
        bsp.bsp_pages_free(d.W, d.refs, d.table, d.kv, 16)
        bsp.bsp_pages_fork(d.W, d.refs, d.table, d.kv, parent, 16)
        src, dst = bsp.bsp_pages_reserve(d.W, d.refs, d.table, d.kv, want, 16)
        bsp.bsp_paged_copy(d.W, K, V, src, dst)
        return src, dst

    turn()  # (nothing held, nothing wanted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        src, dst = turn()
    r = random.Random(5)
    for _ in range(12):
        d.book.free()
        p = [r.choice((i, r.randrange(6), -1)) for i in range(6)]
        d.book.fork(p)
        w = [min(128, n + r.randint(0, 30)) for n in d.book.kv]
        s, t, enough = d.book.reserve(w)
        assert enough
        k = K.clone()
        for a, b in zip(s, t):
            if a >= 0:
                k[b] = K[a]
        parent.copy_(ints(p))
        want.copy_(ints(w))
        graph.replay()
        torch.cuda.synchronize()
        d.same()
        assert src.tolist() == s and dst.tolist() == t and torch.equal(K, k) and d.status() == 0
        d.book.kv = w
        d.kv.copy_(ints(w))


def test_two_streams(bsp):
    """Books and caches of their own on two streams at once."""
    side = torch.cuda.Stream()
    W = bsp.bsp_window_create()
    state = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        K, V = (torch.randn(400, 4, 64, 64, generator=g, device="cuda") for _ in range(2))
        refs = torch.ones(400, dtype=torch.int32, device="cuda")
        refs[torch.randperm(400)[:130].cuda()] = 0
        table = refs.nonzero()[:, 0].to(torch.int32).view(10, 27).contiguous()
        state.append((K, V, refs, table))
    want = []
    for K, V, refs, table in state:
        r, t, src, dst = bsp.bsp_pages_compact(W, refs, table)
        k, v = K.clone(), V.clone()
        bsp.bsp_paged_copy(W, k, v, src, dst)
        want.append((k, v, r, t))
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for (K, V, refs, table), stream in zip(state, (None, side)):
            with torch.cuda.stream(stream) if stream else torch.cuda.stream(torch.cuda.current_stream()):
                k, v = K.clone(), V.clone()
            r, t, src, dst = bsp.bsp_pages_compact(W, refs, table, stream=stream)
            bsp.bsp_paged_copy(W, k, v, src, dst, stream=stream)
            got.append((k, v, r, t))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
