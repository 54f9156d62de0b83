"""Trees of drafted tokens over the paged cache, their verification and the rows
that stay, against plain forms in fp64, on the tensor-core and CUDA-core kernels."""

import math
import random

import numpy as np
import pytest
import torch

import draft_ref as ref
from window_ref import check, keep_mask

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def bsp():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_attention_layout_gb300 import build
    build.build()
    from sparse_attention_layout_gb300 import bsp as m
    return m


@pytest.fixture(params=["tc", "simt"])
def path(request, monkeypatch):
    if request.param == "simt":
        monkeypatch.setenv("BSP_FORCE_SIMT", "1")
    else:
        monkeypatch.delenv("BSP_FORCE_SIMT", raising=False)
    return request.param


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def grown(n, r, wide=6, roots=1):
    """A tree of n nodes; `roots` of them without a parent."""
    return [-1 if i < roots else r.randrange(max(0, i - wide), i) for i in range(n)]


SHAPES = {
    "chain": lambda n, r: [i - 1 for i in range(n)],
    "star": lambda n, r: [-1] + [0] * (n - 1),
    "tree": grown,
    "forest": lambda n, r: grown(n, r, 20, 3),
    "wide": lambda n, r: grown(n, r, n),
}


class Trees:
    """A ragged batch of trees over a paged cache with pages in random order."""

    def __init__(self, nodes, kv, Hq, Hkv, D, page, dtype, seed, shape="tree", slots_first=False, extra_tokens=0, fill=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = random.Random(seed)
        self.nodes, self.kv, self.page, self.Hkv = nodes, kv, page, Hkv
        self.parents = [SHAPES[shape](n, r) if n else [] for n in nodes]
        used = [-(-n // page) for n in kv]
        self.n_pages = sum(used) + 2
        order = list(range(self.n_pages))
        r.shuffle(order)
        table = torch.full((len(nodes), max(used + [1]) + 1), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table = table.cuda()
        dims = (self.n_pages, page, Hkv, D) if slots_first else (self.n_pages, Hkv, page, D)
        caches = [torch.randn(*dims, generator=g, device="cuda").to(dtype) for _ in range(2)]
        self.Kc, self.Vc = [c.transpose(1, 2) if slots_first else c for c in caches]
        if fill is not None:  # slots no sequence holds
            held = torch.zeros(self.n_pages, page, dtype=torch.bool, device="cuda")
            for i, n in enumerate(kv):
                held[self.slots(i, torch.arange(n, device="cuda"))] = True
            for c in (self.Kc, self.Vc):
                c.transpose(1, 2)[~held] = fill
        self.starts = [0]
        for n in nodes:
            self.starts.append(self.starts[-1] + n)
        self.T = self.starts[-1] + extra_tokens
        self.Q = torch.randn(self.T, Hq, D, generator=g, device="cuda").to(dtype)
        self.q_start, self.kv_len = ints(self.starts), ints(kv)
        self.parent = ints([p for t in self.parents for p in t] + [-1] * extra_tokens)

    def slots(self, i, pos):
        return self.table[i][pos // self.page].long(), pos % self.page

    def plan(self, bsp, W, **kw):
        return bsp.bsp_draft_tree(W, self.q_start, self.kv_len, self.parent, max(self.nodes), **kw)

    def attend(self, bsp, W, pos, bits, **kw):
        return bsp.bsp_paged_tree_attention(W, self.Q, self.Kc, self.Vc, self.q_start, self.kv_len, self.table, pos, bits, **kw)

    def check(self, O, lse, scale, window, sinks, masks=None, positions=None):
        G = self.Q.shape[1] // self.Hkv
        for i, (n, kv) in enumerate(zip(self.nodes, self.kv)):
            if n == 0:
                continue
            ctx, a, b = kv - n, self.starts[i], self.starts[i + 1]
            tree = ref.tree_mask(self.parents[i], ctx, window, sinks) if masks is None else masks[i]
            p = torch.tensor(ref.depths(self.parents[i]), device="cuda") + ctx if positions is None else positions[i]
            keep = torch.cat([keep_mask(p, torch.arange(ctx, device="cuda"), window, sinks),
                              torch.from_numpy(tree).cuda()], 1)
            pg, sl = self.slots(i, torch.arange(kv, device="cuda"))
            K, V = self.Kc[pg, :, sl].double(), self.Vc[pg, :, sl].double()
            for h in range(self.Q.shape[1]):
                want = ref.masked(self.Q[a:b, h].double(), K[:, h // G], V[:, h // G], keep, scale, self.Q.dtype)
                check(O[a:b, h], want[0], want[1], f"O of sequence {i}, head {h}")
                check(lse[a:b, h], want[2], want[3], f"lse of sequence {i}, head {h}")


# (nodes, kv, Hq, Hkv, D, page, window, sinks, shape)
CASES = [
    ([1], [1], 1, 1, 64, 16, 0, 0, "chain"),
    ([5], [5], 4, 2, 128, 16, 0, 0, "tree"),                              # no context
    ([13], [1000], 8, 2, 128, 16, 0, 0, "tree"),
    ([1, 3, 64, 2], [5, 129, 700, 2000], 4, 4, 64, 32, 0, 0, "star"),
    ([24] * 9, [24, 130, 137, 152, 255, 256, 257, 280, 900], 6, 2, 128, 64, 100, 3, "tree"),
    ([5, 0, 1, 130], [5, 40, 77, 600], 6, 2, 80, 16, 0, 0, "wide"),        # a sequence without nodes
    ([64, 300, 1], [64, 1100, 900], 10, 2, 96, 128, 64, 130, "tree"),      # several tiles of nodes, wide sinks
    ([17, 31, 40], [2000, 1500, 41], 3, 1, 48, 32, 5, 1, "chain"),         # deeper than the window
    ([33, 40], [90, 3000], 2, 1, 112, 32, 1, 0, "forest"),                 # each sees itself alone
    ([1000], [1300], 2, 1, 64, 128, 0, 0, "chain"),
    ([1024, 7], [1030, 50], 1, 1, 16, 16, 300, 8, "wide"),
    ([3] * 33, [300 + 7 * i for i in range(33)], 64, 1, 16, 16, 0, 0, "tree"),
    ([2] * 300, [2 + 3 * i for i in range(300)], 2, 2, 64, 16, 200, 5, "chain"),
    ([29], [9000], 4, 1, 128, 64, 0, 0, "tree"),                           # shared by many SMs
    ([100, 3], [12345, 9999], 3, 3, 64, 16, 0, 0, "forest"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"n{len(c[0])}_{c[0][0]}kv{c[1][-1]}H{c[2]}_{c[3]}D{c[4]}p{c[5]}w{c[6]}s{c[7]}{c[8]}")
def test_trees(bsp, path, case, dtype):
    nodes, kv, Hq, Hkv, D, page, window, sinks, shape = case
    b = Trees(nodes, kv, Hq, Hkv, D, page, DT[dtype], len(nodes) + D, shape, slots_first=bool(len(nodes) % 2), extra_tokens=3,
              fill=float("nan"))
    W = bsp.bsp_window_create(window, sinks)
    scale = 1.0 / math.sqrt(D)
    words = -(-max(nodes) // 32)
    pos, bits = torch.full((b.T,), 77, dtype=torch.int32, device="cuda"), torch.full((b.T, words), 77, dtype=torch.int32, device="cuda")
    b.plan(bsp, W, positions=pos, bits=bits)
    for i, (n, t) in enumerate(zip(kv, b.parents)):
        if t:
            rows = slice(b.starts[i], b.starts[i + 1])
            assert pos[rows].tolist() == [n - len(t) + d for d in ref.depths(t)]
            assert (bits[rows].cpu().numpy() == ref.pack(ref.tree_mask(t, n - len(t), window, sinks), words)).all()
    assert bool((pos[-3:] == 77).all()) and bool((bits[-3:] == 77).all())
    O = torch.full_like(b.Q, 7.0)
    lse = torch.full(b.Q.shape[:2], 7.0, device="cuda")
    b.attend(bsp, W, pos, bits, O=O, lse=lse, scale=scale)
    assert bsp.bsp_window_status(W) == 0
    b.check(O, lse, scale, window, sinks)
    assert bool((O[-3:] == 7.0).all()) and bool((lse[-3:] == 7.0).all())
    O2, lse2 = b.attend(bsp, W, pos, bits, scale=scale)
    assert torch.equal(O2[:-3], O[:-3]) and torch.equal(lse2[:-3], lse[:-3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_any_bits_and_positions(bsp, path, dtype):
    """Bits that are no tree's, words beyond the nodes, rows that see nothing."""
    for nodes, kv, words, window in (([40, 9], [40, 200], 2, 0), ([70, 33], [70, 500], 5, 50)):
        b = Trees(nodes, kv, 4, 2, 64, 16, DT[dtype], 3)
        g = np.random.default_rng(words)
        bits = g.integers(-2 ** 31, 2 ** 31, (b.T, words)).astype(np.int32)
        bits[3] = 0  # without a context: sees nothing
        masks = [np.unpackbits(bits[b.starts[i]:b.starts[i + 1]].view("u1"), axis=1, bitorder="little")[:, :n].astype(bool)
                 for i, n in enumerate(nodes)]
        positions = [torch.from_numpy(g.integers(n - m, n + 40, m)).cuda() for n, m in zip(kv, nodes)]
        pos = torch.cat(positions).to(torch.int32)
        pos[0] = kv[0] - nodes[0] - 5  # counts as the context's end
        positions[0][0] = kv[0] - nodes[0]
        W = bsp.bsp_window_create(window, 2)
        O, lse = b.attend(bsp, W, pos, torch.from_numpy(bits).cuda(), scale=0.125)
        assert bsp.bsp_window_status(W) == 0
        b.check(O, lse, 0.125, window, 2, masks, positions)
        assert bool((O[3] == 0).all()) and bool((lse[3] == -math.inf).all())


def test_a_chain_is_what_new_tokens_are(bsp, path):
    """Trees without branches, and new tokens of the paged attention: the same rows."""
    b = Trees([7, 20, 1], [300, 77, 513], 8, 2, 128, 64, torch.bfloat16, 5, "chain")
    W = bsp.bsp_window_create(90, 2)
    pos, bits = b.plan(bsp, W)
    O, lse = b.attend(bsp, W, pos, bits, scale=0.1)
    P, pl = bsp.bsp_paged_attention(W, b.Q, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, scale=0.1)
    b.check(P, pl, 0.1, 90, 2)
    b.check(O, lse, 0.1, 90, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nodes", [[1] * 40, [0, 2, 0, 1, 0], [0, 0, 3]], ids=str)
def test_no_more_nodes_than_sequences(bsp, path, nodes, dtype):
    """Tiles are single nodes then."""
    b = Trees(nodes, [n + 37 * (i + 1) for i, n in enumerate(nodes)], 6, 2, 96, 16, DT[dtype], 8, "tree")
    W = bsp.bsp_window_create(300, 1)
    pos, bits = b.plan(bsp, W)
    O, lse = b.attend(bsp, W, pos, bits, scale=0.1)
    assert bsp.bsp_window_status(W) == 0
    b.check(O, lse, 0.1, 300, 1)


def test_positions_out_of_range(bsp, path):
    """Positions are taken as at least the first node's and at most 2^30 - 1."""
    b = Trees([4], [300], 2, 1, 64, 16, torch.bfloat16, 8, "star")
    for window in (0, 50):
        W = bsp.bsp_window_create(window, 3)
        pos, bits = b.plan(bsp, W)
        wild = pos.clone()
        wild[1:] = ints([2 ** 31 - 1, -2 ** 31, -1])
        tame = pos.clone()
        tame[1:] = ints([2 ** 30 - 1, 296, 296])
        got, want = (b.attend(bsp, W, x, bits, scale=0.1) for x in (wild, tame))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bsp.bsp_window_status(W) == 0
        b.check(*want, 0.1, window, 3, None, [tame])


@pytest.mark.parametrize("limit", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_a_wait_that_runs_out_is_reported(bsp, monkeypatch, D, limit):
    """Tiles of 48 steps take tens of microseconds, the limits are 1.4 to 4: the call
    ends with its status, and the next one is right."""
    monkeypatch.delenv("BSP_FORCE_SIMT", raising=False)
    b = Trees([30, 1] * 75, [6144] * 150, 4, 2, D, 64, torch.bfloat16, 165)
    W = bsp.bsp_window_create()
    pos, bits = b.plan(bsp, W)
    want = b.attend(bsp, W, pos, bits, scale=0.1)
    assert bsp.bsp_window_status(W) == 0
    bsp.bsp_diag_window_wait_limit(W, limit)
    b.attend(bsp, W, pos, bits, scale=0.1)
    assert bsp.bsp_window_status(W) == -6 and bsp.bsp_window_status(W) == 0
    bsp.bsp_diag_window_wait_limit(W)
    for _ in range(2):
        assert all(torch.equal(a, c) for a, c in zip(b.attend(bsp, W, pos, bits, scale=0.1), want))
    assert bsp.bsp_window_status(W) == 0


def test_two_streams_at_once(bsp, path):
    """One handle's trees and verifications on two streams."""
    W = bsp.bsp_window_create(500, 4)
    batches = [Trees([20, 40, 7] * 8, [900 + 50 * i for i in range(24)], 8, 2, 128, 32, torch.bfloat16, s) for s in (1, 2)]
    rows = [rows_of(b.T, 3001, i) for i, b in enumerate(batches)]
    u = torch.rand(batches[0].T, device="cuda")

    def run(b, pq, stream):
        pos, bits = b.plan(bsp, W, stream=stream)
        O = b.attend(bsp, W, pos, bits, scale=0.09, stream=stream)
        return (pos, *O, *bsp.bsp_draft_verify(W, *pq, b.parent.clamp(min=0), b.q_start, b.parent, u, u[:24].contiguous(), stream=stream))

    want = [run(b, pq, None) for b, pq in zip(batches, rows)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, b, pq in zip(streams, batches, rows):
            with torch.cuda.stream(s):
                got.append(run(b, pq, s))
        torch.cuda.synchronize()
        for a, c in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, c))
    assert bsp.bsp_window_status(W) == 0


def test_hidden_nodes_of_infinite_score(bsp, path):
    """A node's keys of +inf or NaN reach nobody but those that see it."""
    b = Trees([20], [200], 4, 1, 64, 16, torch.bfloat16, 9, "star")
    W = bsp.bsp_window_create()
    pos, bits = b.plan(bsp, W)
    want, _ = b.attend(bsp, W, pos, bits, scale=0.125)
    pg, sl = b.slots(0, torch.tensor([187], device="cuda"))  # node 7, a leaf
    for bad in (math.inf, math.nan):
        b.Kc[pg, :, sl] = bad
        O, _ = b.attend(bsp, W, pos, bits, scale=0.125)
        rest = [i for i in range(20) if i != 7]
        assert torch.equal(O[rest], want[rest])


def test_cache_beyond_32_bit_offsets(bsp, path):
    n_pages, Hkv, page, D = 16500, 8, 128, 128  # 2.16e9 elements a cache
    dt = torch.bfloat16
    K = torch.zeros(n_pages, Hkv, page, D, dtype=dt, device="cuda")
    V = torch.zeros(n_pages, Hkv, page, D, dtype=dt, device="cuda")
    b = Trees([9], [300], 16, Hkv, D, page, dt, 2)
    for i, x in enumerate((n_pages - 1, n_pages - 2, 3)):
        K[x], V[x] = b.Kc[b.table[0, i].item()], b.Vc[b.table[0, i].item()]
    W = bsp.bsp_window_create()
    pos, bits = b.plan(bsp, W)
    want, _ = b.attend(bsp, W, pos, bits, scale=0.1)
    b.Kc, b.Vc, b.table = K, V, ints([[n_pages - 1, n_pages - 2, 3]])
    got, _ = b.attend(bsp, W, pos, bits, scale=0.1)
    assert torch.equal(got, want)
    # and the accepted rows
    kept = [0, 2, 5, 8]
    before = [(c[n_pages - 2 if 291 + x < 256 else 3, :, (291 + x) % 128].clone()) for c in (K, V) for x in kept]
    bsp.bsp_paged_keep(W, K, V, b.q_start, b.kv_len, b.table, ints(kept + [-1] * 5), ints([4]))
    after = [c[3, :, (291 + d) % 128] for c in (K, V) for d in range(4)]
    assert all(torch.equal(x, y) for x, y in zip(before, after)) and bsp.bsp_window_status(W) == 0


def test_bad_trees_are_reported(bsp, path):
    b = Trees([5, 4, 6], [40, 50, 60], 2, 1, 64, 16, torch.bfloat16, 4)
    W = bsp.bsp_window_create()
    pos, bits = b.plan(bsp, W)
    O, _ = b.attend(bsp, W, pos, bits)
    assert bsp.bsp_window_status(W) == 0
    good = b.parent.clone()
    for bad in (3, 7, -2, 2 ** 31 - 1, -2 ** 31):  # node 3 of the second sequence
        b.parent[5 + 3] = bad
        p2, b2 = b.plan(bsp, W)
        assert bsp.bsp_window_status(W) == -7
        t = [b.parents[0], b.parents[1][:3] + [-1], b.parents[2]]
        assert p2.tolist() == [kv - n + d for kv, n, x in zip(b.kv, b.nodes, t) for d in ref.depths(x)]
    b.parent.copy_(good)
    cases = [("kv_len", 1, -1), ("kv_len", 1, 3), ("kv_len", 1, b.table.shape[1] * 16 + 1), ("kv_len", 1, 2 ** 31 - 1),
             ("q_start", 3, 99), ("q_start", 0, -1), ("q_start", 3, 2 ** 31 - 1), ("q_start", 0, -2 ** 31)]
    for arr, at, bad in cases:
        t = getattr(b, arr)
        keep = t.clone()
        t[at] = bad
        p2, b2 = torch.full_like(pos, 77), torch.full_like(bits, 77)
        if (arr, bad) != ("kv_len", b.table.shape[1] * 16 + 1):  # (the plan knows no table)
            b.plan(bsp, W, positions=p2, bits=b2)
            assert bsp.bsp_window_status(W) == -7, (arr, bad)
            hit = slice(5, 9) if arr == "kv_len" else slice(9, 15) if at == 3 else slice(0, 5)
            want = pos.clone()
            want[hit] = 77
            assert torch.equal(p2, want)
        out = torch.full_like(b.Q, 7.0)
        b.attend(bsp, W, pos, bits, O=out)
        assert bsp.bsp_window_status(W) == -7, (arr, bad)
        if arr == "kv_len":
            assert torch.equal(out[:5], O[:5]) and torch.equal(out[9:], O[9:]) and bool((out[5:9] == 7.0).all())
        t.copy_(keep)
    # more nodes than the bits have words for
    c = Trees([40, 3], [90, 30], 2, 1, 64, 16, torch.bfloat16, 4)
    p2, b2 = bsp.bsp_draft_tree(W, c.q_start, c.kv_len, c.parent, 32)
    assert bsp.bsp_window_status(W) == -7
    out = torch.full_like(c.Q, 7.0)
    c.attend(bsp, W, p2, b2, O=out)
    assert bsp.bsp_window_status(W) == -7 and bool((out[:40] == 7.0).all()) and bool((out[40:] != 7.0).any())
    # a page of a visible key out of range
    keep = b.table.clone()
    for bad in (b.n_pages, -1, 2 ** 31 - 1):
        b.table[1, 2] = bad
        b.attend(bsp, W, pos, bits)
        assert bsp.bsp_window_status(W) == -7
    b.table.copy_(keep)
    # offsets that descend: no row is attended to
    b.q_start[2] = 2
    out = torch.full_like(b.Q, 7.0)
    b.attend(bsp, W, pos, bits, O=out)
    assert bsp.bsp_window_status(W) == -7 and bool((out == 7.0).all())


# ----------------------------------------------------------- verification --

def rows_of(T, V, seed, sharp=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, V, generator=g, device="cuda") * sharp
    return torch.softmax(x, -1), torch.softmax(x + 0.8 * torch.randn(T, V, generator=g, device="cuda"), -1)


def tokens_for(draft, parents, starts, seed, chosen):
    """Tokens of the nodes from their parents' rows of the draft."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    tok = torch.zeros(draft.shape[0], dtype=torch.int64, device="cuda")
    for s, t in zip(starts, parents):
        for a in range(1, len(t)):
            p = s + max(t[a], 0)
            if chosen:
                rank = t[:a].count(t[a])
                tok[s + a] = draft[p].float().argsort(descending=True, stable=True)[rank % draft.shape[1]]
            else:
                tok[s + a] = torch.multinomial(draft[p].float(), 1, generator=g)[0]
    return tok.to(torch.int32)


def verify(bsp, W, nodes, parents, target, draft, tok, accept, sample, q_start=None):
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    got = bsp.bsp_draft_verify(W, target, draft, tok, ints(starts), ints([p for t in parents for p in t]), accept, sample)
    path, count, token = (x.tolist() for x in got)
    t64 = target.double().cpu().numpy()
    d64 = None if draft is None else draft.double().cpu().numpy()
    tl, al, sl = tok.tolist(), accept.double().tolist(), sample.double().tolist()
    for i, (a, n) in enumerate(zip(starts, nodes)):
        if n == 0:
            assert count[i] == 0 and token[i] == -1
            continue
        b = a + n
        want, nxt = ref.verify(t64[a:b], None if draft is None else d64[a:b], tl[a:b], parents[i], al[a:b], sl[i])
        assert (count[i], path[a:b], token[i]) == (len(want), want + [-1] * (n - len(want)), nxt), i
    return got


@pytest.mark.parametrize("chosen", [False, True], ids=["drawn", "chosen"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4097, 32000, 50001])
def test_verification(bsp, V, dtype, chosen):
    r = random.Random(V)
    nodes = [1, 2, 5, 0, 9, 24, 40, 3]
    parents = [grown(n, r, 3) if i % 2 else grown(n, r, n) for i, n in enumerate(nodes)]
    starts = np.concatenate([[0], np.cumsum(nodes)]).tolist()
    p, q = rows_of(sum(nodes), V, V)
    p, q = p.to(DT[dtype]), q.to(DT[dtype])
    tok = tokens_for(q, parents, starts, V, chosen)
    W = bsp.bsp_window_create()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        accept = torch.rand(sum(nodes), generator=g, device="cuda")
        if seed == 1:
            accept.mul_(0.3).add_(0.7)  # mostly rejected
        sample = torch.rand(len(nodes), generator=g, device="cuda")
        got = verify(bsp, W, nodes, parents, p, None if chosen else q, tok, accept, sample)
    assert bsp.bsp_window_status(W) == 0
    again = bsp.bsp_draft_verify(W, p, None if chosen else q, tok, ints(starts), ints([x for t in parents for x in t]), accept, sample)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("n_seq", [1, 3, 700, 3000])
def test_verification_of_many(bsp, n_seq):
    r = random.Random(n_seq)
    nodes = [r.randint(1, 4) for _ in range(n_seq)]
    parents = [grown(n, r, 2) for n in nodes]
    starts = np.concatenate([[0], np.cumsum(nodes)]).tolist()
    p, q = rows_of(sum(nodes), 257, n_seq, 1.0)
    g = torch.Generator(device="cuda").manual_seed(n_seq)
    row = torch.tensor([s + max(a, 0) for s, t in zip(starts, parents) for a in t], device="cuda")
    tok = torch.multinomial(q[row], 1, generator=g)[:, 0].to(torch.int32)
    W = bsp.bsp_window_create()
    verify(bsp, W, nodes, parents, p, q, tok, torch.rand(sum(nodes), generator=g, device="cuda"),
           torch.rand(n_seq, generator=g, device="cuda"))
    assert bsp.bsp_window_status(W) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_any_stride(bsp, dtype):
    """Rows that begin anywhere in a wider tensor, the two tensors' differently."""
    r = random.Random(8)
    nodes, V = [7, 12], 5003
    parents = [grown(n, r, 4) for n in nodes]
    p, q = (x.to(DT[dtype]) for x in rows_of(sum(nodes), V, 8))
    tok = tokens_for(q, parents, [0, 7], 8, False)
    W = bsp.bsp_window_create()
    accept, sample = torch.rand(19, device="cuda"), torch.rand(2, device="cuda")
    for a, b in ((0, 0), (1, 1), (1, 2), (3, 0)):
        P, Q = torch.full((19, V + 9), math.nan, device="cuda", dtype=DT[dtype]), torch.full((19, V + 6), math.nan, device="cuda", dtype=DT[dtype])
        P[:, a:a + V], Q[:, b:b + V] = p, q
        verify(bsp, W, nodes, parents, P[:, a:a + V], Q[:, b:b + V], tok, accept, sample)
        verify(bsp, W, nodes, parents, P[:, a:a + V], None, tok, accept, sample)


def test_a_large_vocabulary_and_far_rows(bsp):
    """A million entries, and rows behind 2^31 elements."""
    W = bsp.bsp_window_create()
    r = random.Random(2)
    nodes, V = [6, 9], 1000003
    parents = [grown(n, r, 3) for n in nodes]
    p, q = (x.to(torch.bfloat16) for x in rows_of(15, V, 2, 1.0))
    tok = tokens_for(q, parents, [0, 6], 2, False)
    accept, sample = torch.rand(15, device="cuda"), torch.rand(2, device="cuda")
    for draft in (q, None):
        want = verify(bsp, W, nodes, parents, p, draft, tok, accept, sample)
        shift = 2200  # rows in front: the trees' begin at 2.2e9 elements
        far = [torch.cat([torch.empty(shift, V, dtype=x.dtype, device="cuda"), x]) for x in (p, q)]

        def behind(x):
            return torch.cat([torch.zeros(shift, dtype=x.dtype, device="cuda"), x])

        got = bsp.bsp_draft_verify(W, far[0], None if draft is None else far[1], behind(tok), ints([shift, shift + 6, shift + 15]),
                                   behind(ints([x for t in parents for x in t])), behind(accept), sample)
        assert torch.equal(got[0][shift:], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert bsp.bsp_window_status(W) == 0


def test_borders(bsp):
    """Numbers on a border go to the entry behind it; entries of 0 are never taken."""
    W = bsp.bsp_window_create()
    V = 4096
    flat = torch.zeros(1, V, device="cuda")
    flat[0, 100:116] = 1 / 16
    one = torch.zeros(1, device="cuda")
    for u in range(16):
        got = bsp.bsp_draft_verify(W, flat, None, ints([0]), ints([0, 1]), ints([-1]), one, one + u / 16)
        assert got[2].item() == 100 + u
        got = bsp.bsp_draft_verify(W, flat, None, ints([0]), ints([0, 1]), ints([-1]), one, one + (u + 1) / 16 - 2.0 ** -24)
        assert got[2].item() == 100 + u
    for bad in (1.0, 2.0, math.inf):  # no number below 1: the last entry
        assert bsp.bsp_draft_verify(W, flat, None, ints([0]), ints([0, 1]), ints([-1]), one, one + bad)[2].item() == 115
    for row in (torch.zeros(1, V), torch.full((1, V), -1.0), torch.full((1, V), math.nan)):  # nothing to take
        assert bsp.bsp_draft_verify(W, row.cuda(), None, ints([0]), ints([0, 1]), ints([-1]), one, one)[2].item() == -1
    flat[0, 3] = math.nan  # counts as 0
    flat[0, 4] = -5.0
    assert bsp.bsp_draft_verify(W, flat, None, ints([0]), ints([0, 1]), ints([-1]), one, one + 0.5)[2].item() == 108
    # equal rows: everything stays; rows apart: nothing does, and the next token is the target's
    same, _ = rows_of(5, 1000, 3)
    tok = tokens_for(same, [[-1, 0, 1, 2, 3]], [0], 3, False)
    chain, top = ints([-1, 0, 1, 2, 3]), torch.full((5,), 1 - 2.0 ** -24, device="cuda")
    path, count, _ = bsp.bsp_draft_verify(W, same, same, tok, ints([0, 5]), chain, top, one)
    assert count.item() == 5 and path.tolist() == [0, 1, 2, 3, 4]
    p, q = torch.zeros(5, 1000, device="cuda"), torch.zeros(5, 1000, device="cuda")
    p[:, 7], q[:, 8] = 1, 1
    path, count, token = bsp.bsp_draft_verify(W, p, q, ints([8] * 5), ints([0, 5]), chain, torch.zeros(5, device="cuda"), one)
    assert count.item() == 1 and path.tolist() == [0, -1, -1, -1, -1] and token.item() == 7
    # rejected where the target lies below the draft everywhere: the target's own row
    path, count, token = bsp.bsp_draft_verify(W, p / 2, p, ints([7] * 5), ints([0, 5]), chain, torch.full((5,), 0.75, device="cuda"), one)
    assert count.item() == 1 and token.item() == 7
    # the same token twice among the children: taken out once
    t = torch.zeros(3, 10, device="cuda")
    t[:, 2], t[:, 5] = 0.25, 0.75
    for draft in (None, t):
        path, count, token = bsp.bsp_draft_verify(W, t, draft, ints([0, 2, 2]), ints([0, 3]), ints([-1, 0, 0]),
                                                  torch.full((3,), 0.9, device="cuda"), one)
        want = ref.verify(t.double().cpu().numpy(), None if draft is None else t.double().cpu().numpy(), [0, 2, 2], [-1, 0, 0],
                          [0.9] * 3, 0.0)
        assert (path.tolist()[:count.item()], token.item()) == want


def test_distribution_of_the_tokens(bsp):
    """What comes out behind the first node is distributed as the target's row,
    whatever the draft: counts of N trials lie within 6 sqrt(N p (1 - p)) + 1 of
    N p (a normal variable leaves 6 deviations once in 10^9)."""
    N, V = 16384, 6
    W = bsp.bsp_window_create()
    p = torch.tensor([0.3, 0.05, 0.25, 0.2, 0.0, 0.2], device="cuda")
    q = torch.tensor([0.1, 0.4, 0.05, 0.2, 0.15, 0.1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for parent, draft in (([-1, 0], q), ([-1, 0, 0, 0], q), ([-1, 0, 0], None)):
        n = len(parent)
        target = p.expand(N * n, V).contiguous()
        tok = torch.multinomial(q.expand(N * n, V), 1, generator=g)[:, 0]
        if draft is None:
            tok = torch.tensor([0, 1, 2], device="cuda").repeat(N)  # any choice will do
        path, count, token = bsp.bsp_draft_verify(W, target, None if draft is None else draft.expand(N * n, V).contiguous(),
                                                  tok.to(torch.int32), ints([n * i for i in range(N + 1)]), ints(parent * N),
                                                  torch.rand(N * n, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda"))
        second = path.view(N, n)[:, 1].long()
        first = torch.where(count >= 2, tok.view(N, n).gather(1, second.clamp(min=0)[:, None])[:, 0], token.long())
        hits = torch.bincount(first, minlength=V).double().cpu().numpy()
        for x in range(V):
            e = float(p[x])
            assert abs(hits[x] - N * e) <= 6 * math.sqrt(N * e * (1 - e)) + 1, (parent, x, hits)


def test_bad_drafts_are_reported(bsp):
    W = bsp.bsp_window_create()
    p, q = rows_of(10, 50, 4)
    tok = tokens_for(q, [[-1, 0, 1, 2, 3]] * 2, [0, 5], 4, False)
    starts, parent = ints([0, 5, 10]), ints([-1, 0, 1, 2, 3] * 2)
    accept, sample = torch.zeros(10, device="cuda"), torch.full((2,), 0.5, device="cuda")

    def call():
        path = torch.full((10,), 77, dtype=torch.int32, device="cuda")
        _, count, token = bsp.bsp_draft_verify(W, p, q, tok, starts, parent, accept, sample, path=path)
        return path.tolist(), count.tolist(), token.tolist()

    path, count, token = call()
    assert count == [5, 5] and bsp.bsp_window_status(W) == 0
    for what, at, bad in ((tok, 7, 50), (tok, 7, -1), (tok, 7, 2 ** 31 - 1), (parent, 7, 2), (parent, 7, 4), (parent, 7, -2),
                          (parent, 7, 2 ** 31 - 1)):
        keep = what.clone()
        what[at] = bad  # node 2 of the second sequence falls away, and what is below it
        got = call()
        assert bsp.bsp_window_status(W) == -7
        assert got[0] == [0, 1, 2, 3, 4, 0, 1, -1, -1, -1] and got[1] == [5, 2] and got[2][0] == token[0]
        what.copy_(keep)
    parent[7] = -1  # a place without a token: nothing to report
    assert call()[1] == [5, 2] and bsp.bsp_window_status(W) == 0
    parent[7] = 1
    for at, bad in ((0, -1), (2, 11), (2, 2 ** 31 - 1), (2, -2 ** 31), (2, 4)):
        keep = starts.clone()
        starts[at] = bad
        got = call()
        assert bsp.bsp_window_status(W) == -7
        i = 0 if at == 0 else 1
        assert got[1][i] == 0 and got[2][i] == -1 and got[0][5 * i:5 * i + 5] == [77] * 5 and got[1][1 - i] == 5
        starts.copy_(keep)
    T = 1025  # one more than a sequence may have
    big, _ = rows_of(T, 3, 1)
    path, count, token = bsp.bsp_draft_verify(W, big, None, ints([0] * T), ints([0, T]), ints([-1] + [0] * (T - 1)),
                                              torch.zeros(T, device="cuda"), torch.zeros(1, device="cuda"))
    assert bsp.bsp_window_status(W) == -7 and count.item() == 0
    path, count, token = bsp.bsp_draft_verify(W, big[1:], None, ints([2] * (T - 1)), ints([0, T - 1]), ints(list(range(-1, T - 2))),
                                              torch.zeros(T - 1, device="cuda"), torch.zeros(1, device="cuda"))
    assert bsp.bsp_window_status(W) == 0 and count.item() == 1024 and path.tolist() == list(range(1024))


# ----------------------------------------------------------- rows that stay --

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slots_first", [False, True])
@pytest.mark.parametrize("nodes,kv,page,D", [([1], [1], 16, 16), ([9], [9], 16, 128), ([24, 0, 5, 60], [100, 40, 77, 600], 32, 80),
                                             ([1024], [1500], 128, 32), ([40] * 70, [40 + 13 * i for i in range(70)], 16, 64)])
def test_keep(bsp, nodes, kv, page, D, slots_first, dtype):
    b = Trees(nodes, kv, 2, 2, D, page, DT[dtype], 6, slots_first=slots_first, extra_tokens=2)
    r = random.Random(len(nodes))
    W = bsp.bsp_window_create()
    kept = [sorted(r.sample(range(n), r.randint(0, n))) for n in nodes]
    kept[0] = list(range(nodes[0])) if nodes[0] % 2 else kept[0]  # all of them: nothing moves
    path = ints([x for k, n in zip(kept, nodes) for x in k + [-5] * (n - len(k))] + [9, 9])
    K, V = b.Kc.clone(), b.Vc.clone()
    for i, k in enumerate(kept):
        if k:
            to = b.slots(i, torch.arange(len(k), device="cuda") + kv[i] - nodes[i])
            at = b.slots(i, torch.tensor(k, device="cuda") + kv[i] - nodes[i])
            for c, old in ((K, b.Kc), (V, b.Vc)):
                c[to[0], :, to[1]] = old[at[0], :, at[1]]
    bsp.bsp_paged_keep(W, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, path, ints([len(k) for k in kept]))
    assert bsp.bsp_window_status(W) == 0
    assert torch.equal(b.Kc, K) and torch.equal(b.Vc, V)


def test_bad_paths_are_reported(bsp):
    b = Trees([5, 6], [40, 50], 2, 1, 64, 16, torch.bfloat16, 4)
    W = bsp.bsp_window_create()
    K, V = b.Kc.clone(), b.Vc.clone()
    for path, count in (([0, 2, 1], 3), ([0, 0], 2), ([0, 5], 2), ([0, 2 ** 31 - 1], 2), ([-1], 1), ([-2 ** 31], 1), ([0, 1], 6), ([0, 1], -1)):
        bsp.bsp_paged_keep(W, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, ints(path + [4] * (5 - len(path)) + list(range(6))),
                           ints([count, 6]))
        assert bsp.bsp_window_status(W) == -7, (path, count)
        assert torch.equal(b.Kc, K) and torch.equal(b.Vc, V)
    good, path, count = b.table.clone(), ints([0, 3, 4, 0, 0] + list(range(6))), ints([3, 6])
    for bad in (-1, b.n_pages, 2 ** 31 - 1):
        b.table[0, 2] = bad  # positions 35 .. 39 all lie there
        bsp.bsp_paged_keep(W, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, path, count)
        assert bsp.bsp_window_status(W) == -7
        assert torch.equal(b.Kc, K) and torch.equal(b.Vc, V)
    b.table.copy_(good)
    for arr, at, bad in (("kv_len", 0, 4), ("kv_len", 0, -1), ("kv_len", 0, 2 ** 31 - 1), ("q_start", 0, -3), ("q_start", 1, 12)):
        t = getattr(b, arr)
        keep = t.clone()
        t[at] = bad
        bsp.bsp_paged_keep(W, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, path, ints([3, 0]))
        assert bsp.bsp_window_status(W) == -7, (arr, bad)
        assert torch.equal(b.Kc, K) and torch.equal(b.Vc, V)
        t.copy_(keep)


# ----------------------------------------------------------------- refusals --

def test_refusals(bsp):
    W = bsp.bsp_window_create()
    b = Trees([3, 2], [20, 30], 4, 2, 64, 16, torch.bfloat16, 1)
    pos, bits = b.plan(bsp, W)
    p, q = rows_of(5, 20, 1)
    tok, u, s = ints([0] * 5), torch.zeros(5, device="cuda"), torch.zeros(2, device="cuda")
    count = ints([1, 1])
    good = {
        "bsp_draft_tree": [b.q_start, b.kv_len, b.parent, 3],
        "bsp_paged_tree_attention": [b.Q, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, pos, bits],
        "bsp_draft_verify": [p, q, tok, b.q_start, b.parent, u, s],
        "bsp_paged_keep": [b.Kc, b.Vc, b.q_start, b.kv_len, b.table, b.parent, count],
    }
    for name, args in good.items():
        getattr(bsp, name)(W, *args)
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            sizes = a is b.parent and name != "bsp_draft_verify"  # (it is what says how many rows there are)
            for bad in (a.cpu(), a[None] if sizes else a[:-1], a.double() if a.is_floating_point() else a.long(), a[None]):
                with pytest.raises((ValueError, TypeError)):
                    getattr(bsp, name)(W, *args[:i], bad, *args[i + 1:])
    bsp.bsp_window_status(W)

    def code(name, *args, **kw):
        with pytest.raises(bsp.BspError) as e:
            getattr(bsp, name)(W, *args, **kw)
        return e.value.code

    assert code("bsp_draft_tree", b.q_start, b.kv_len, b.parent, 1025) == -2
    wide = torch.zeros(5, 33, dtype=torch.int32, device="cuda")
    assert code("bsp_paged_tree_attention", b.Q, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, pos, wide) == -2
    assert code("bsp_paged_tree_attention", b.Q, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, pos, wide[:, :0].contiguous()) == -1
    for scale in (0.0, -1.0, math.nan, math.inf):
        assert code("bsp_paged_tree_attention", b.Q, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, pos, bits, scale=scale) == -1
    assert code("bsp_paged_tree_attention", b.Q, b.Kc, b.Vc, b.q_start, b.kv_len, b.table, pos, bits, O=b.Q) == -1
    odd = [c[:, :, :8] for c in (b.Kc, b.Vc)]  # pages of 8 slots
    assert code("bsp_paged_tree_attention", b.Q, *odd, b.q_start, b.kv_len, b.table, pos, bits) == -1
    assert code("bsp_paged_keep", *odd, b.q_start, b.kv_len, b.table, b.parent, count) == -1
    assert code("bsp_paged_keep", b.Kc, b.Kc, b.q_start, b.kv_len, b.table, b.parent, count) == -1
    assert code("bsp_draft_verify", torch.zeros(1, 20, device="cuda").expand(5, 20), None, tok, b.q_start, b.parent, u, s) == -1
    with pytest.raises(ValueError):
        bsp.bsp_draft_verify(W, p.t().contiguous().t(), None, tok, b.q_start, b.parent, u, s)
    n = bsp._paged_workspace(W.device)
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    O, lse = torch.empty_like(b.Q), torch.empty(5, 4, device="cuda")

    def raw(at, size):
        return bsp.lib().bsp_paged_tree_attention(W.handle, 1, bsp._rows(b.Q), bsp._heads(b.Kc), bsp._heads(b.Vc), bsp._rows(O),
                                                  lse.data_ptr(), b.q_start.data_ptr(), b.kv_len.data_ptr(), b.table.data_ptr(),
                                                  pos.data_ptr(), bits.data_ptr(), 5, 2, b.table.shape[1], b.n_pages, 16, 4, 2, 64,
                                                  1, 1.0, at, size, torch.cuda.current_stream().cuda_stream)

    assert raw(ws.data_ptr(), n) == 0
    assert raw(ws.data_ptr(), n - 1) == -1 and raw(ws.data_ptr() + 16, n) == -3 and raw(None, n) == -1
    torch.cuda.synchronize()


def test_no_tokens(bsp, path):
    W = bsp.bsp_window_create()
    none, zero = ints([]), ints([0])
    K = torch.zeros(2, 1, 16, 64, device="cuda")
    pos, bits = bsp.bsp_draft_tree(W, zero, none, none, 4)
    assert pos.shape == (0,) and bits.shape == (0, 1)
    O, _ = bsp.bsp_paged_tree_attention(W, torch.zeros(0, 2, 64, device="cuda"), K, K.clone(), zero, none, none.view(0, 1).expand(0, 3),
                                        pos, bits)
    assert O.shape == (0, 2, 64)
    path_, count, token = bsp.bsp_draft_verify(W, torch.zeros(0, 5, device="cuda"), None, none, ints([0, 0, 0]), none,
                                               torch.zeros(0, device="cuda"), torch.zeros(2, device="cuda"))
    assert count.tolist() == [0, 0] and token.tolist() == [-1, -1]
    bsp.bsp_paged_keep(W, K, K.clone(), zero, none, none.view(0, 1), none, none)
    assert bsp.bsp_window_status(W) == 0
