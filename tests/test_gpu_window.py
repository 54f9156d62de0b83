"""Windowed attention, its gradient and the paged cache against fp64, entry by
entry within window_ref's bounds, on the tensor-core and CUDA-core kernels."""

import ctypes
import math

import pytest
import torch

import window_ref as ref
from window_ref import check

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


def randn(shape, dtype, seed, order="heads"):
    """[Z, H, S, D] values; order "rows": stored [Z, S, H, D], "fused": a slice
    of a wider row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    Z, H, S, D = shape
    if order == "rows":
        return torch.randn(Z, S, H, D, generator=g, device="cuda").to(dtype).transpose(1, 2)
    if order == "fused":
        return torch.randn(Z, S, H, 2 * D, generator=g, device="cuda").to(dtype)[..., :D].transpose(1, 2)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# (Z, Hq, Hkv, Sq, Sk, D, window, sinks)
DENSE = [
    (1, 1, 1, 1, 1, 16, 0, 0),        # one token
    (1, 1, 1, 128, 128, 128, 0, 0),   # one whole tile
    (2, 2, 2, 129, 129, 64, 1, 0),    # every row sees itself only
    (1, 4, 2, 200, 333, 64, 50, 3),   # fewer queries than keys
    (1, 2, 1, 300, 170, 32, 40, 2),   # more queries than keys: empty rows
    (1, 3, 1, 150, 150, 48, 64, 130), # three heads a group, sinks wider than a tile
    (2, 5, 5, 257, 257, 80, 100, 1),
    (1, 10, 2, 77, 400, 96, 0, 5),    # five heads a group, no limit
    (1, 64, 1, 9, 500, 112, 128, 4),  # the largest group
    (1, 7, 1, 131, 640, 128, 129, 17),
    (1, 8, 2, 1, 1000, 128, 256, 4),  # a single token
    (1, 2, 2, 1100, 1100, 128, 300, 4),
    (3, 4, 1, 1500, 1500, 64, 257, 64),
    (1, 1, 1, 4500, 4500, 64, 200, 4),  # the sinks' tile has many more queries than the others
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", DENSE, ids=str)
def test_dense(bsp, path, shape, dtype):
    Z, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    dt = DT[dtype]
    seed = sum(shape)
    order = ("heads", "rows", "fused")[seed % 3]
    Q, dO = randn((Z, Hq, Sq, D), dt, seed, order), randn((Z, Hq, Sq, D), dt, seed + 3, order)
    K, V = randn((Z, Hkv, Sk, D), dt, seed + 1, order), randn((Z, Hkv, Sk, D), dt, seed + 2)
    scale = 1.0 / math.sqrt(D)
    W = bsp.bsp_window_create(window, sinks)
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=scale)
    dQ, dK, dV = bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, scale=scale)
    assert bsp.bsp_window_status(W) == 0
    r = ref.dense(Q, K, V, scale, window, sinks, dO)
    check(O, r["O"], r["eO"], "O")
    check(lse, r["lse"], r["else_"], "lse")
    check(dQ, r["dQ"], r["eQ"], "dQ")
    check(dK, r["dK"], r["eK"], "dK")
    check(dV, r["dV"], r["eV"], "dV")
    # the same call again gives the same bits
    O2, _ = bsp.bsp_window_attention(W, Q, K, V, scale=scale)
    again = bsp.bsp_window_attention_backward(W, Q, K, V, O2, dO, lse, scale=scale)
    for a, b in zip((O, dQ, dK, dV), (O2, *again)):
        assert torch.equal(a, b)


# few to many rows over a history that many CTAs share; the last: ten keys whose
# queries many CTAs share
JOINED = [(1, 1, 1, Sq, 9000, D, 0, 0) for Sq, D in ((1, 64), (20, 16), (31, 128), (33, 64), (40, 48), (100, 128))]
JOINED += [(1, 6, 2, 7, 12345, 80, 0, 0), (1, 64, 1, 400, 394, 64, 0, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", JOINED, ids=str)
def test_tiles_of_many_pieces(bsp, path, shape, dtype):
    test_dense(bsp, path, shape, dtype)


def test_large_scores(bsp, path):
    """Scores of +-1000 with a moving maximum: no overflow, one key takes all."""
    Z, H, S, D = 1, 2, 400, 64
    Q, K, V = (randn((Z, H, S, D), torch.bfloat16, 5 + i) for i in range(3))
    K = K * torch.linspace(1, 16, S, device="cuda").to(K.dtype)[:, None]
    W = bsp.bsp_window_create(100, 2)
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=8.0)
    r = ref.dense(Q, K, V, 8.0, 100, 2)
    assert torch.isfinite(O).all()
    check(O, r["O"], r["eO"], "O")
    check(lse, r["lse"], r["else_"], "lse")


def test_gradient_by_differences(bsp):
    """fp32 gradients against central differences of the operator's own
    forward.  f = sum(O * dO) is evaluated from fp32 outputs: its error is at
    most N 2^-24 |O||dO| sums, and the difference's truncation h^2 f'''/6; both
    stay below 2 % of the direction's derivative here, h = 2^-6."""
    W = bsp.bsp_window_create(20, 2)
    Q, K, V, dO = (randn((1, H, 70, 32), torch.float32, 40 + i) for i, H in enumerate((4, 2, 2, 4)))
    scale = 0.2
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=scale)
    grads = bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, scale=scale)
    h = 2.0 ** -6
    for i, g in enumerate(grads):
        d = randn(tuple(g.shape), torch.float32, 50 + i)
        f = []
        for sgn in (1, -1):
            x = [Q, K, V]
            x[i] = x[i] + sgn * h * d
            f.append((bsp.bsp_window_attention(W, *x, scale=scale)[0].double() * dO.double()).sum())
        num = ((f[0] - f[1]) / (2 * h)).item()
        ana = (g.double() * d.double()).sum().item()
        norm = (g.double().norm() * d.double().norm()).item() / math.sqrt(g.numel())
        assert abs(num - ana) <= 0.02 * max(abs(ana), norm), (i, num, ana)


# ------------------------------------------------------------------- paged --

class Paged:
    """A ragged batch over a paged cache with pages in random order."""

    def __init__(self, new, kv, Hq, Hkv, D, page, dtype, seed, slots_first=False, extra_tokens=0, fill=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cg = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.page, self.Hkv = new, kv, page, Hkv
        used = [-(-n // page) for n in kv]
        self.n_pages = sum(used) + 2
        order = torch.randperm(self.n_pages, generator=cg).to(torch.int32)
        self.table = torch.full((len(new), max(used + [1]) + 1), -7, dtype=torch.int32)  # unused entries are rubbish
        at = 0
        for i, n in enumerate(used):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.table = self.table.cuda()
        shape = (self.n_pages, page, Hkv, D) if slots_first else (self.n_pages, Hkv, page, D)
        caches = [torch.randn(*shape, generator=g, device="cuda").to(dtype) for _ in range(2)]
        self.Kc, self.Vc = [c.transpose(1, 2) if slots_first else c for c in caches]
        if fill is not None:  # slots no sequence holds
            held = torch.zeros(self.n_pages, page, dtype=torch.bool, device="cuda")
            for i, n in enumerate(kv):
                pg, sl = self.slots(i, torch.arange(n, device="cuda"))
                held[pg, sl] = True
            for c in (self.Kc, self.Vc):
                c.transpose(1, 2)[~held] = fill
        T = sum(new) + extra_tokens
        self.Q = torch.randn(T, Hq, D, generator=g, device="cuda").to(dtype)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")

    def slots(self, i, pos):
        return self.table[i][pos // self.page].long(), pos % self.page

    def rows(self, cache, i):
        """Keys (or values) of sequence i, [1, Hkv, kv, D]."""
        pg, sl = self.slots(i, torch.arange(self.kv[i], device="cuda"))
        return cache[pg, :, sl].transpose(0, 1)[None]

    def attend(self, bsp, W, **kw):
        return bsp.bsp_paged_attention(W, self.Q, self.Kc, self.Vc, self.q_start, self.kv_len, self.table, **kw)

    def check(self, O, lse, scale, window, sinks):
        for i, (n, kv) in enumerate(zip(self.new, self.kv)):
            if n == 0:
                continue
            a, b = self.starts[i], self.starts[i + 1]
            r = ref.dense(self.Q[a:b].transpose(0, 1)[None], self.rows(self.Kc, i), self.rows(self.Vc, i), scale, window,
                          sinks)
            check(O[a:b], r["O"][0].transpose(0, 1), r["eO"][0].transpose(0, 1), f"O of sequence {i}")
            check(lse[a:b], r["lse"][0].T, r["else_"][0].T, f"lse of sequence {i}")


# (new, kv, Hq, Hkv, D, page, window, sinks)
PAGED = [
    ([1], [1], 1, 1, 64, 16, 0, 0),
    ([1], [1000], 8, 2, 128, 16, 0, 0),
    ([1, 1, 1, 1], [5, 129, 700, 2000], 4, 4, 64, 32, 0, 0),
    ([1] * 9, [1, 16, 17, 128, 130, 255, 256, 257, 900], 6, 2, 128, 64, 100, 3),
    ([5, 0, 1, 130], [5, 40, 77, 600], 6, 2, 80, 16, 0, 0),          # a sequence without new tokens
    ([3, 2], [0, 1], 2, 1, 32, 16, 0, 0),                             # fewer positions than tokens: empty rows
    ([64, 300, 1], [64, 1100, 900], 10, 2, 96, 128, 64, 130),
    ([17, 1, 40], [2000, 1500, 41], 3, 1, 48, 32, 33, 1),
    ([260], [260], 4, 1, 128, 128, 0, 0),                             # a first chunk
    ([2] * 33, [300 + 7 * i for i in range(33)], 64, 1, 16, 16, 0, 0),
    ([1] * 300, [1 + 3 * i for i in range(300)], 2, 2, 64, 16, 200, 5),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", PAGED, ids=lambda c: f"n{len(c[0])}kv{c[1][-1]}H{c[2]}_{c[3]}D{c[4]}p{c[5]}w{c[6]}s{c[7]}")
def test_paged(bsp, path, case, dtype):
    new, kv, Hq, Hkv, D, page, window, sinks = case
    # NaN in every slot that no sequence holds
    b = Paged(new, kv, Hq, Hkv, D, page, DT[dtype], len(new) + D, slots_first=bool(len(new) % 2), extra_tokens=3,
              fill=float("nan"))
    W = bsp.bsp_window_create(window, sinks)
    scale = 1.0 / math.sqrt(D)
    O = torch.full_like(b.Q, 7.0)
    lse = torch.full(b.Q.shape[:2], 7.0, device="cuda")
    b.attend(bsp, W, O=O, lse=lse, scale=scale)
    assert bsp.bsp_window_status(W) == 0
    b.check(O, lse, scale, window, sinks)
    assert bool((O[b.starts[-1]:] == 7.0).all()) and bool((lse[b.starts[-1]:] == 7.0).all())
    O2, lse2 = b.attend(bsp, W, scale=scale)
    assert torch.equal(O2[:b.starts[-1]], O[:b.starts[-1]]) and torch.equal(lse2[:b.starts[-1]], lse[:b.starts[-1]])


@pytest.mark.parametrize("new,kv", [
    ([1] * 700, [1 + i % 97 for i in range(700)]),           # more sequences than threads of a block
    ([2, 0, 0, 1, 3, 0, 0, 0], [300, 5, 0, 700, 3, 9, 9, 9]),  # as few tokens as sequences, but not one each
    ([0, 0, 0], [10, 0, 5]),                                  # no new token at all, rows of nobody
], ids=["700", "uneven", "none"])
def test_batches_of_few_tokens(bsp, path, new, kv):
    b = Paged(new, kv, 4, 2, 64, 16, torch.float16, 70 + len(new), extra_tokens=2)
    W = bsp.bsp_window_create(250, 3)
    O, lse = torch.full_like(b.Q, 7.0), torch.full(b.Q.shape[:2], 7.0, device="cuda")
    b.attend(bsp, W, O=O, lse=lse, scale=0.125)
    assert bsp.bsp_window_status(W) == 0
    b.check(O, lse, 0.125, 250, 3)
    assert bool((O[b.starts[-1]:] == 7.0).all()) and bool((lse[b.starts[-1]:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_history_of_one_sequence(bsp, path, dtype):
    """One token, and a short chunk, over a history cut into many pieces."""
    for new, G in ((1, 4), (3, 5)):
        b = Paged([new], [9000], 2 * G, 2, 128, 64, DT[dtype], 17 + G)
        W = bsp.bsp_window_create()
        O, lse = b.attend(bsp, W, scale=0.09)
        assert bsp.bsp_window_status(W) == 0
        b.check(O, lse, 0.09, 0, 0)
        assert torch.equal(O, b.attend(bsp, W, scale=0.09)[0])


def test_cache_beyond_32_bit_offsets(bsp, path):
    """Pages whose elements lie past 2^31 of the cache."""
    n_pages, Hkv, page, D = 2 ** 31 // (2 * 16 * 128) + 40, 2, 16, 128
    W = bsp.bsp_window_create()
    Kc, Vc = (torch.empty(n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[n_pages - 1, 3, n_pages - 30, n_pages - 2]], dtype=torch.int32, device="cuda")
    S = 61
    Q, K, V = (randn((1, H, S, D), torch.bfloat16, 90 + i) for i, H in enumerate((4, 2, 2)))
    rows = [t[0].transpose(0, 1) for t in (Q, K, V)]
    qs = torch.tensor([0, S], dtype=torch.int32, device="cuda")
    kl = torch.tensor([S], dtype=torch.int32, device="cuda")
    bsp.bsp_paged_append(W, rows[1], rows[2], Kc, Vc, qs, kl, table)
    O, lse = bsp.bsp_paged_attention(W, rows[0], Kc, Vc, qs, kl, table, scale=0.09)
    assert bsp.bsp_window_status(W) == 0
    r = ref.dense(Q, K, V, 0.09, 0, 0)
    check(O.transpose(0, 1)[None], r["O"], r["eO"], "O")
    check(lse.T[None], r["lse"], r["else_"], "lse")


def test_dense_beyond_32_bit_offsets(bsp):
    """Batch entries and rows whose elements lie past 2^31 of their tensors."""
    W = bsp.bsp_window_create(40, 1)
    Z, H, S, D = 2, 2, 150, 64
    wide = 2 ** 31 // (S * 2) // 8 * 8 + 64  # row stride: the second batch entry starts past 2^31
    def far(seed):
        t = torch.empty(Z * S * wide, dtype=torch.bfloat16, device="cuda").as_strided((Z, H, S, D), (S * wide, D, wide, 1))
        return t.copy_(randn((Z, H, S, D), torch.bfloat16, seed))
    Q, K, V, dO = (far(95 + i) for i in range(4))
    O, dQ, dK, dV = (far(0) for _ in range(4))
    _, lse = bsp.bsp_window_attention(W, Q, K, V, O=O, scale=0.125)
    bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, dQ, dK, dV, scale=0.125)
    r = ref.dense(Q.contiguous(), K.contiguous(), V.contiguous(), 0.125, 40, 1, dO.contiguous())
    for name, got in (("O", O), ("dQ", dQ), ("dK", dK), ("dV", dV)):
        check(got.contiguous(), r[name], r["e" + name[-1]], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_freed_pages_before_the_window(bsp, path, dtype):
    """Pages wholly between the sinks and every row's window may be given away:
    their table entries are never followed, their slots never read."""
    b = Paged([3, 1], [900, 500], 4, 2, 64, 16, DT[dtype], 3)
    window, sinks = 50, 5
    W = bsp.bsp_window_create(window, sinks)
    O, lse = b.attend(bsp, W, scale=0.1)
    for i, (n, kv) in enumerate(zip(b.new, b.kv)):
        low = kv - n - window + 1
        for pg in range(1, low // 16):
            phys = int(b.table[i, pg])
            b.Kc[phys], b.Vc[phys] = float("nan"), float("inf")
            b.table[i, pg] = 10 ** 6
    O2, lse2 = b.attend(bsp, W, scale=0.1)
    assert bsp.bsp_window_status(W) == 0
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_hidden_keys_of_infinite_score(bsp, path):
    """A hidden K row of inf or NaN changes nothing for the rows before it."""
    Q, K, V = (randn((1, 2, 200, 64), torch.float16, 60 + i) for i in range(3))
    W = bsp.bsp_window_create(0, 0)
    O, _ = bsp.bsp_window_attention(W, Q, K, V, scale=0.125)
    K2 = K.clone()
    K2[:, :, 150] = float("inf")
    K2[:, :, 151] = float("nan")
    O2, _ = bsp.bsp_window_attention(W, Q, K2, V, scale=0.125)
    assert torch.equal(O[:, :, :150], O2[:, :, :150])


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("Sq,Sk", [(300, 300), (2, 9000)])  # whole tiles; pieces that are joined
def test_rows_of_no_number_stay_so(bsp, path, Sq, Sk, value):
    """A row that is no number, or that sees a key of infinite score, gets NaN,
    not zeros as if it saw nothing; the other rows keep their values."""
    Q, K, V = randn((1, 4, Sq, 64), torch.bfloat16, 70), *(randn((1, 2, Sk, 64), torch.bfloat16, 71 + i) for i in range(2))
    W = bsp.bsp_window_create(0, 0)
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=0.125)
    Q2 = Q.clone()
    Q2[0, 1, 1] = math.nan
    O2, lse2 = bsp.bsp_window_attention(W, Q2, K, V, scale=0.125)
    assert bool(O2[0, 1, 1].isnan().all()) and bool(lse2[0, 1, 1].isnan())
    O2[0, 1, 1], lse2[0, 1, 1] = O[0, 1, 1], lse[0, 1, 1]
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    # one element: the scores' signs are the queries', +inf in some rows and heads, -inf (no weight) in others
    K2 = K.clone()
    K2[0, 0, Sk - 1, 5] = value
    O3, lse3 = bsp.bsp_window_attention(W, Q, K2, V, scale=0.125)
    none = (Q[0, :2, Sq - 1, 5] * value > 0) | torch.tensor(math.isnan(value), device="cuda")
    assert torch.equal(O3[0, :2, Sq - 1].isnan().all(-1), none) and torch.equal(lse3[0, :2, Sq - 1].isnan(), none)
    assert torch.equal(O3[:, :, :Sq - 1], O[:, :, :Sq - 1]) and torch.equal(O3[:, 2:], O[:, 2:])
    # one token over pages
    b = Paged([1, 1], [40, 5000], 4, 2, 64, 16, torch.bfloat16, 5)
    b.Q[1, 2] = math.nan
    O, lse = b.attend(bsp, W, scale=0.125)
    want = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    want[1, 2] = True
    assert torch.equal(O.isnan().all(-1), want) and torch.equal(O.isnan().any(-1), want)
    assert torch.equal(lse.isnan(), want) and bsp.bsp_window_status(W) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new,kv,page,D", [([1], [1], 16, 16), ([5, 0, 1, 130], [5, 40, 77, 600], 32, 80),
                                           ([3, 2], [1, 1], 16, 128), ([1] * 70, [1 + 9 * i for i in range(70)], 64, 64),
                                           ([700, 40], [700, 1000], 128, 128)], ids=str)
def test_append(bsp, new, kv, page, D, dtype):
    b = Paged(new, kv, 3, 3, D, page, DT[dtype], 9, slots_first=len(new) == 1, extra_tokens=2)
    W = bsp.bsp_window_create()
    K, V = b.Q, (b.Q * 3).transpose(0, 1).contiguous().transpose(0, 1)
    wantK, wantV = b.Kc.clone(), b.Vc.clone()
    for i, (n, m) in enumerate(zip(new, kv)):
        for t in range(n):
            pos = m - n + t
            if pos >= 0:
                pg, sl = int(b.table[i, pos // page]), pos % page
                wantK[pg, :, sl], wantV[pg, :, sl] = K[b.starts[i] + t], V[b.starts[i] + t]
    bsp.bsp_paged_append(W, K, V, b.Kc, b.Vc, b.q_start, b.kv_len, b.table)
    assert bsp.bsp_window_status(W) == 0
    assert torch.equal(b.Kc, wantK) and torch.equal(b.Vc, wantV)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_in_chunks_then_single_tokens_equals_dense(bsp, path, dtype):
    """Append + attention chunk by chunk, then token by token, as a server runs
    them, against the whole sequence at once in fp64."""
    dt, Hq, Hkv, D, page, S, window, sinks = DT[dtype], 6, 2, 64, 32, 333, 90, 4
    Q, K, V = (randn((1, H, S, D), dt, 80 + i) for i, H in enumerate((Hq, Hkv, Hkv)))
    W = bsp.bsp_window_create(window, sinks)
    n_pages = -(-S // page)
    Kc, Vc = (torch.full((n_pages, Hkv, page, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    got, lses, at = [], [], 0
    for n in [100, 1, 200, 17] + [1] * 15:
        r = slice(at, at + n)
        at += n
        qs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        kl = torch.tensor([at], dtype=torch.int32, device="cuda")
        rows = [t[0, :, r].transpose(0, 1) for t in (Q, K, V)]
        bsp.bsp_paged_append(W, rows[1], rows[2], Kc, Vc, qs, kl, table)
        o, l = bsp.bsp_paged_attention(W, rows[0], Kc, Vc, qs, kl, table, scale=0.125)
        got.append(o)
        lses.append(l)
    assert at == S and bsp.bsp_window_status(W) == 0
    ref_ = ref.dense(Q, K, V, 0.125, window, sinks)
    check(torch.cat(got).transpose(0, 1)[None], ref_["O"], ref_["eO"], "O")
    check(torch.cat(lses).T[None], ref_["lse"], ref_["else_"], "lse")


def test_decode_step_in_a_graph(bsp, path):
    """A captured append + attention follows the lengths and the table."""
    b = Paged([1, 1, 1], [40, 300, 130], 8, 2, 128, 16, torch.bfloat16, 21)
    W = bsp.bsp_window_create(200, 2)
    K, V = (torch.randn(3, 2, 128, device="cuda").to(torch.bfloat16) for _ in range(2))

    def step():
        bsp.bsp_paged_append(W, K, V, b.Kc, b.Vc, b.q_start, b.kv_len, b.table)
        return b.attend(bsp, W, scale=0.1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lse = step()
    for kv in ([41, 301, 131], [42, 9, 144]):
        b.kv = kv
        b.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        b.Q.normal_()
        K.normal_()
        graph.replay()
        torch.cuda.synchronize()
        b.check(O, lse, 0.1, 200, 2)
        for i, n in enumerate(kv):
            pg, sl = b.slots(i, torch.tensor([n - 1], device="cuda"))
            assert torch.equal(b.Kc[pg, :, sl][0], K[i])


def test_autograd_and_shared_heads(bsp):
    """The differentiable form: strided, expanded and shared leaves."""
    W = bsp.bsp_window_create(64, 2)
    Q = randn((2, 6, 150, 64), torch.bfloat16, 1, "rows").requires_grad_()
    KV = randn((1, 2, 150, 64), torch.bfloat16, 2).requires_grad_()
    both = KV.expand(2, 2, 150, 64)  # one prompt's keys for both batch entries, K = V
    dO = randn((2, 6, 150, 64), torch.bfloat16, 3, "fused")
    bsp.window_attention(W, Q, both, both, 0.125).backward(dO)
    r = ref.dense(Q.detach(), both.detach(), both.detach(), 0.125, 64, 2, dO)
    check(Q.grad, r["dQ"], r["eQ"], "dQ")
    u = 2.0 ** -8
    want = (r["dK"] + r["dV"]).sum(0, keepdim=True)
    # each gradient is rounded once more when autograd adds them, in bf16
    parts = (r["dK"].abs() + r["dV"].abs() + r["eK"] + r["eV"]).sum(0, keepdim=True)
    check(KV.grad, want, (r["eK"] + r["eV"]).sum(0, keepdim=True) + 3 * u * parts, "dK + dV")
    # an output gradient without strides of its own
    Q.grad = None
    bsp.window_attention(W, Q, both, both, 0.125).sum().backward()
    r = ref.dense(Q.detach(), both.detach(), both.detach(), 0.125, 64, 2, torch.ones_like(dO))
    check(Q.grad, r["dQ"], r["eQ"], "dQ of a sum")


def test_backward_in_a_graph(bsp):
    W = bsp.bsp_window_create(100, 4)
    Q, K, V, dO = (randn((1, H, 400, 64), torch.float16, 30 + i) for i, H in enumerate((4, 2, 2, 4)))
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=0.125)
    want = bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, scale=0.125)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        o, l = bsp.bsp_window_attention(W, Q, K, V, scale=0.125)
        got = bsp.bsp_window_attention_backward(W, Q, K, V, o, dO, l, scale=0.125)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert torch.equal(a, c)


def test_two_streams_at_once(bsp, path):
    """Two calls of one handle on two streams, each with its own workspace."""
    W = bsp.bsp_window_create(300, 4)
    ins = [[randn((1, 8, 2000, 128), torch.bfloat16, 10 * j + i) for i in range(3)] for j in range(2)]
    want = [bsp.bsp_window_attention(W, *x, scale=0.09)[0] for x in ins]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, x in zip(streams, ins):
            s.wait_stream(torch.cuda.current_stream())
            got.append(bsp.bsp_window_attention(W, *x, scale=0.09, stream=s)[0])
        torch.cuda.synchronize()
        for a, c in zip(want, got):
            assert torch.equal(a, c)


def test_no_tokens_no_keys(bsp, path):
    W = bsp.bsp_window_create(10, 1)
    e = lambda *s: torch.empty(*s, device="cuda", dtype=torch.bfloat16)
    O, lse = bsp.bsp_window_attention(W, e(2, 2, 5, 64).fill_(1), e(2, 1, 0, 64), e(2, 1, 0, 64))
    assert bool((O == 0).all()) and bool((lse == -math.inf).all())
    dQ, dK, dV = bsp.bsp_window_attention_backward(W, e(2, 2, 5, 64).fill_(1), e(2, 1, 0, 64), e(2, 1, 0, 64), O,
                                                   e(2, 2, 5, 64).fill_(1), lse)
    assert bool((dQ == 0).all()) and dK.numel() == 0
    O, lse = bsp.bsp_window_attention(W, e(2, 2, 0, 64), e(2, 1, 5, 64), e(2, 1, 5, 64))
    assert O.numel() == 0
    _, dK, dV = bsp.bsp_window_attention_backward(W, e(2, 2, 0, 64), e(2, 1, 5, 64), e(2, 1, 5, 64), O, O, lse)
    assert bool((dK == 0).all()) and bool((dV == 0).all())
    O, lse = bsp.bsp_window_attention(W, e(0, 2, 5, 64), e(0, 1, 5, 64), e(0, 1, 5, 64))
    assert O.numel() == 0
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    O, lse = bsp.bsp_paged_attention(W, e(0, 2, 64), e(3, 1, 16, 64), e(3, 1, 16, 64), i(0, 0), i(5), i(0)[None])
    assert O.numel() == 0
    assert bsp.bsp_window_status(W) == 0


# ------------------------------------------------------- refusals, bad pages --

def test_bad_pages_and_lengths_are_reported(bsp, path):
    b = Paged([1, 2, 1], [40, 50, 60], 2, 1, 64, 16, torch.bfloat16, 4)
    W = bsp.bsp_window_create()
    good = b.table.clone()
    for bad in (b.n_pages, -1, 2 ** 31 - 1):
        b.table.copy_(good)
        b.table[1, 3] = bad  # the page of the new tokens
        b.attend(bsp, W)
        assert bsp.bsp_window_status(W) == -7
        bsp.bsp_paged_append(W, b.Q[:, :1], b.Q[:, :1], b.Kc, b.Vc, b.q_start, b.kv_len, b.table)
        assert bsp.bsp_window_status(W) == -7
        assert bsp.bsp_window_status(W) == 0
    b.table.copy_(good)
    O, _ = b.attend(bsp, W)
    for arr, at, bad in (("kv_len", 1, -1), ("kv_len", 1, b.table.shape[1] * 16 + 1), ("q_start", 2, 99),
                         ("q_start", 2, 0)):
        t = getattr(b, arr)
        keep = t.clone()
        t[at] = bad
        out = torch.full_like(b.Q, 7.0)
        b.attend(bsp, W, O=out)
        assert bsp.bsp_window_status(W) == -7, (arr, bad)
        if arr == "kv_len":  # the other sequences are served, the bad one's rows left alone
            assert torch.equal(out[0], O[0]) and torch.equal(out[3], O[3]) and bool((out[1:3] == 7.0).all())
        t.copy_(keep)
    O2, _ = b.attend(bsp, W)
    assert bsp.bsp_window_status(W) == 0


@pytest.mark.parametrize("new", [[40, 0, 30, 25], [1] * 90, [1] * 700], ids=len)
def test_descending_offsets_attend_to_nothing(bsp, path, new):
    """Sequences that overlap could hold more tiles than the call's sizes allow
    for: reported, and no row is written."""
    b = Paged(new, [50] * len(new), 2, 1, 64, 16, torch.bfloat16, 6)
    W = bsp.bsp_window_create()
    t = b.q_start.clone()
    b.q_start[2:] = (t[2:] - t[2]).clamp(min=0)  # the third sequence begins at row 0 again
    O, lse = torch.full_like(b.Q, 7.0), torch.full(b.Q.shape[:2], 7.0, device="cuda")
    b.attend(bsp, W, O=O, lse=lse)
    assert bsp.bsp_window_status(W) == -7
    assert bool((O == 7).all()) and bool((lse == 7).all())
    b.q_start.copy_(t)
    O, lse = b.attend(bsp, W, scale=0.1)
    b.check(O, lse, 0.1, 0, 0)
    assert bsp.bsp_window_status(W) == 0


def test_refusals(bsp):
    W = bsp.bsp_window_create(10, 1)
    x = lambda *s, dt=torch.bfloat16: torch.zeros(*s, device="cuda", dtype=dt)
    ok = (x(1, 2, 8, 64), x(1, 1, 8, 64), x(1, 1, 8, 64))
    bsp.bsp_window_attention(W, *ok)
    with pytest.raises(bsp.BspError):
        bsp.bsp_window_attention(W, *ok, scale=0.0)
    with pytest.raises(bsp.BspError):
        bsp.bsp_window_attention(W, *ok, scale=float("nan"))
    with pytest.raises(ValueError):
        bsp.bsp_window_attention(W, x(1, 3, 8, 64), x(1, 2, 8, 64), x(1, 2, 8, 64))
    with pytest.raises(ValueError):
        bsp.bsp_window_attention(W, x(1, 2, 8, 64), x(1, 1, 8, 64), x(1, 1, 9, 64))
    with pytest.raises(TypeError):
        bsp.bsp_window_attention(W, x(1, 2, 8, 64), x(1, 1, 8, 64), x(1, 1, 8, 64, dt=torch.float16))
    with pytest.raises(TypeError):
        bsp.bsp_window_attention(W, *[x(1, 1, 8, 64, dt=torch.float64)] * 3)
    with pytest.raises(ValueError):
        bsp.bsp_window_attention(W, x(1, 2, 8, 64).cpu(), ok[1], ok[2])
    with pytest.raises(bsp.BspError):  # D
        bsp.bsp_window_attention(W, *[x(1, 1, 8, 24)] * 3)
    with pytest.raises(bsp.BspError):
        bsp.bsp_window_attention(W, *[x(1, 1, 8, 144)] * 3)
    with pytest.raises(bsp.BspError):  # 65 heads a group
        bsp.bsp_window_attention(W, x(1, 65, 8, 64), ok[1], ok[2])
    with pytest.raises(ValueError):  # last dimension not contiguous
        bsp.bsp_window_attention(W, x(1, 2, 64, 8).transpose(2, 3), ok[1], ok[2])
    with pytest.raises(bsp.BspError):  # a row stride of 65 elements
        bsp.bsp_window_attention(W, x(1, 2, 8, 65)[..., :64], ok[1], ok[2])
    with pytest.raises(bsp.BspError):  # expanded: stride 0
        bsp.bsp_window_attention(W, ok[0], x(1, 1, 1, 64).expand(1, 1, 8, 64), ok[2])
    with pytest.raises(bsp.BspError):  # an output that overlaps itself
        bsp.bsp_window_attention(W, *ok, O=x(1, 1, 20, 64).as_strided((1, 2, 8, 64), (64, 64, 64, 1)))
    with pytest.raises(ValueError):
        bsp.bsp_window_attention(W, *ok, lse=x(1, 2, 8))
    same = x(1, 2, 8, 64)
    with pytest.raises(bsp.BspError):  # in place of an input
        bsp.bsp_window_attention(W, same, ok[1], ok[2], O=same)
    O, l = bsp.bsp_window_attention(W, *ok)
    with pytest.raises(bsp.BspError):  # two gradients in one place
        bsp.bsp_window_attention_backward(W, *ok, O, x(1, 2, 8, 64), l, dK=ok[1].clone(), dV=ok[1])
    both = torch.empty_like(ok[1])
    with pytest.raises(bsp.BspError):
        bsp.bsp_window_attention_backward(W, *ok, O, x(1, 2, 8, 64), l, dK=both, dV=both)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    q, kc = x(2, 2, 64), x(3, 1, 16, 64)
    bsp.bsp_paged_attention(W, q, kc, kc, i(0, 2), i(5), i(0, 1)[None].contiguous())
    with pytest.raises(bsp.BspError):  # page of 24 slots
        bsp.bsp_paged_attention(W, q, x(3, 1, 24, 64), x(3, 1, 24, 64), i(0, 2), i(5), i(0)[None])
    with pytest.raises(ValueError):
        bsp.bsp_paged_attention(W, q, kc, kc, i(0, 2), i(5), i(0)[None].long())
    with pytest.raises(ValueError):
        bsp.bsp_paged_attention(W, q, kc, kc, i(0, 1, 2), i(5), i(0)[None])
    with pytest.raises(ValueError):
        bsp.bsp_paged_append(W, q, q, kc, kc, i(0, 2), i(5), i(0)[None])
    # the C entry itself: workspace and alignment
    L = bsp.lib()
    t = [bsp._heads(a) for a in (*ok, x(1, 2, 8, 64))]
    ws = torch.empty(int(L.bsp_window_attention_workspace(1, 2, 1, 8, 0)), dtype=torch.uint8, device="cuda")

    def call(ptr, n, lse=None, dtype=1):
        return L.bsp_window_attention(W.handle, dtype, *t, lse, 1, 2, 1, 8, 8, 64, 1.0, ctypes.c_void_p(ptr), n, None)

    assert call(ws.data_ptr(), ws.numel()) == 0
    assert call(0, ws.numel()) == -1
    assert call(ws.data_ptr(), ws.numel() - 1) == -1
    assert call(ws.data_ptr() + 16, ws.numel()) == -3
    assert call(ws.data_ptr(), ws.numel(), ctypes.c_void_p(ws.data_ptr() + 4)) == -3
    assert call(ws.data_ptr(), ws.numel(), None, 9) == -1
    torch.cuda.synchronize()
    assert bsp.bsp_window_status(W) == 0


# --------------------------------------------------- what no query may reach --

def _gradients(bsp, W, Q, K, V, dO, scale=0.125):
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=scale)
    return (O, lse, *bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, scale=scale))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(4, 2, 300, 170, 64, 40, 2), (1, 1, 700, 1, 128, 0, 0), (6, 2, 901, 400, 80, 60, 9)],
                         ids=str)
def test_gradient_of_queries_that_see_nothing(bsp, path, shape, dtype):
    """More queries than keys: the first ones see nothing, whatever they and
    their output gradient hold, their dQ is 0 and the rest is as without them."""
    Hq, Hkv, Sq, Sk, D, window, sinks = shape
    Q, dO = (randn((2, Hq, Sq, D), DT[dtype], 110 + i, "rows") for i in range(2))
    K, V = (randn((2, Hkv, Sk, D), DT[dtype], 112 + i) for i in range(2))
    W = bsp.bsp_window_create(window, sinks)
    n = Sq - Sk
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=0.125)
    want = bsp.bsp_window_attention_backward(W, Q[:, :, n:], K, V, O[:, :, n:], dO[:, :, n:],
                                             lse[:, :, n:].contiguous(), scale=0.125)
    r = ref.dense(Q, K, V, 0.125, window, sinks, dO)
    for value in (None, math.nan, math.inf):
        if value is not None:
            Q[:, :, :n] = value
            dO[:, :, :n] = value
        O, lse, dQ, dK, dV = _gradients(bsp, W, Q, K, V, dO)
        assert bool((O[:, :, :n] == 0).all()) and bool((lse[:, :, :n] == -math.inf).all())
        assert bool((dQ[:, :, :n] == 0).all())
        for name, got in (("dQ", dQ), ("dK", dK), ("dV", dV)):
            check(got, r[name], r["e" + name[-1]], name)
        assert torch.equal(dQ[:, :, n:], want[0]) and torch.equal(dK, want[1]) and torch.equal(dV, want[2])
    # a key of no number reaches those that see it, not the queries that see nothing
    K[:, :, 0] = math.nan
    dQ = _gradients(bsp, W, Q, K, V, dO)[2]
    assert bool((dQ[:, :, :n] == 0).all())
    assert bsp.bsp_window_status(W) == 0


# (Hq, Hkv, Sq, Sk, D, window, sinks): queries fewer than keys, so that the keys
# before every window are seen by nobody
UNSEEN = [(2, 1, 100, 1000, 64, 50, 0), (4, 2, 16, 256, 128, 32, 0), (6, 2, 130, 700, 80, 60, 5),
          (1, 1, 1, 130, 64, 1, 1), (2, 2, 400, 5000, 128, 300, 200)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", UNSEEN, ids=str)
def test_gradient_without_the_keys_that_nobody_sees(bsp, path, shape, dtype):
    """K and V rows before every window may hold anything: no gradient changes
    by a bit, and their own is 0."""
    Hq, Hkv, Sq, Sk, D, window, sinks = shape
    Q, dO = (randn((2, Hq, Sq, D), DT[dtype], 120 + i) for i in range(2))
    K, V = (randn((2, Hkv, Sk, D), DT[dtype], 122 + i, "rows") for i in range(2))
    W = bsp.bsp_window_create(window, sinks)
    want = _gradients(bsp, W, Q, K, V, dO)
    r = ref.dense(Q, K, V, 0.125, window, sinks, dO)
    for i, name in ((2, "dQ"), (3, "dK"), (4, "dV")):
        check(want[i], r[name], r["e" + name[-1]], name)
    unseen = torch.zeros(Sk, dtype=torch.bool, device="cuda")
    unseen[sinks:Sk - Sq - window + 1] = True
    assert bool(unseen.any())
    for value in (math.nan, math.inf, -60000.0):
        for both in ((K,), (V,), (K, V)):
            k, v = (t.clone() for t in (K, V))
            for t in (k if x is K else v for x in both):
                t[:, :, unseen] = value
            got = _gradients(bsp, W, Q, k, v, dO)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), value
            assert bool((got[3][:, :, unseen] == 0).all()) and bool((got[4][:, :, unseen] == 0).all())
    assert bsp.bsp_window_status(W) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-4, 1e-3, 1.0])
def test_gradient_of_a_small_output_gradient(bsp, path, dtype, size):
    """dS over 6000 keys is 1e-4 of dO and below 16 bits' range where dO is
    small; dQ, dK and dV are in it.  Their norms are off by at most 4 u: one
    rounding each of P or dS, of the O in delta, and of the result, which are
    independent and so add up as the terms themselves do, and the fp32 sums; and
    by the rounding of subnormal results."""
    dt = DT[dtype]
    Q = randn((1, 4, 200, 64), dt, 130) * 0.08
    K = randn((1, 2, 6000, 64), dt, 131) * 0.08
    V = randn((1, 2, 6000, 64), dt, 132)
    dO = (randn((1, 4, 200, 64), torch.float32, 133) * size).to(dt)
    W = bsp.bsp_window_create()
    got = _gradients(bsp, W, Q, K, V, dO, 16.0)[2:]
    r = ref.dense(Q, K, V, 16.0, 0, 0, dO)
    for name, g in zip(("dQ", "dK", "dV"), got):
        check(g, r[name], r["e" + name[-1]], name)
        off = (g.double() - r[name]).norm().item()
        assert off <= 4 * ref.U[dt] * r[name].norm().item() + ref.AB[dt] * math.sqrt(g.numel()), name


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gradient_of_a_large_output_gradient(bsp, path, dtype):
    """dS beyond 65504 with gradients that are far below it."""
    dt = DT[dtype]
    Q, K = (randn((1, H, 5, 64), dt, 140 + H) for H in (4, 2))
    V = randn((1, 2, 5, 64), dt, 142) * 16
    dO = randn((1, 4, 5, 64), dt, 143) * 4000
    W = bsp.bsp_window_create(0, 0)
    got = _gradients(bsp, W, Q, K, V, dO, 0.01)[2:]
    r = ref.dense(Q, K, V, 0.01, 0, 0, dO)
    for name, g in zip(("dQ", "dK", "dV"), got):
        assert r[name].abs().max().item() < 40000
        check(g, r[name], r["e" + name[-1]], name)
        off = (g.double() - r[name]).norm().item()
        assert off <= 4 * ref.U[dt] * r[name].norm().item(), name


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128])
def test_the_type_decides_the_kernels(bsp, path, D, dtype):
    """Both widths of every kernel of a family; nothing falls to the other."""
    W = bsp.bsp_window_create(60, 2)
    assert bsp.bsp_diag_window_family(W) == "none"
    want = "tensor cores" if path == "tc" and dtype != "f32" else "CUDA cores"
    Q, K, V, dO = (randn((2, H, 150, D), DT[dtype], 150 + i, "rows") for i, H in enumerate((6, 2, 2, 6)))
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=0.1)
    assert bsp.bsp_diag_window_family(W) == want
    bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, scale=0.1)
    assert bsp.bsp_diag_window_family(W) == want
    for new in ([1, 1], [30, 2], [1] * 3 + [0] * 600):  # plain and ragged splits
        P = bsp.bsp_window_create(60, 2)
        b = Paged(new, [50 + n for n in new], 6, 2, D, 32, DT[dtype], 155)
        b.check(*b.attend(bsp, P, scale=0.1), 0.1, 60, 2)
        assert bsp.bsp_diag_window_family(P) == want and bsp.bsp_window_status(P) == 0


@pytest.mark.parametrize("limit", [1, 2, 3, 5])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", ["dense", "gradient", "plain", "ragged"])
def test_a_wait_that_runs_out_is_reported(bsp, monkeypatch, what, D, limit):
    """Tiles of 48 steps take tens of microseconds, the limits are 1.4 to 7: every
    role stops, the call ends with its status, and the next one is right."""
    import time
    monkeypatch.delenv("BSP_FORCE_SIMT", raising=False)
    W = bsp.bsp_window_create(0, 0)
    if what in ("dense", "gradient"):
        Q, K, V, dO = (randn((1, H, 6144, D), torch.bfloat16, 160 + i) for i, H in enumerate((4, 2, 2, 4)))
        O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=0.1)
        if what == "dense":
            run = lambda: bsp.bsp_window_attention(W, Q, K, V, scale=0.1)
        else:
            run = lambda: bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, scale=0.1)
    else:
        new = [1] * 150 if what == "plain" else [30, 1] * 75
        b = Paged(new, [6144] * 150, 4, 2, D, 64, torch.bfloat16, 165)
        run = lambda: b.attend(bsp, W, scale=0.1)
    want = run()
    assert bsp.bsp_window_status(W) == 0
    bsp.bsp_diag_window_wait_limit(W, limit)
    t0 = time.perf_counter()
    run()
    assert bsp.bsp_window_status(W) == -6
    assert time.perf_counter() - t0 < 2.0
    assert bsp.bsp_window_status(W) == 0
    bsp.bsp_diag_window_wait_limit(W)
    for _ in range(2):
        assert all(torch.equal(a, c) for a, c in zip(run(), want))
    assert bsp.bsp_window_status(W) == 0


def test_status_of_two_streams(bsp):
    """A report stays until a reader takes it, on any stream of the device, and
    is taken once."""
    b = Paged([1, 1], [40, 50], 2, 1, 64, 16, torch.bfloat16, 170)
    b.table[1, 0] = b.n_pages
    W = bsp.bsp_window_create()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        one.wait_stream(torch.cuda.current_stream())
        b.attend(bsp, W, stream=one)
        assert bsp.bsp_window_status(W, one) == -7
        assert bsp.bsp_window_status(W, two) == 0 and bsp.bsp_window_status(W, one) == 0
        b.attend(bsp, W, stream=one)
        one.synchronize()
        assert bsp.bsp_window_status(W, two.cuda_stream) == -7 and bsp.bsp_window_status(W) == 0


def test_no_keys_for_queries_that_overlap(bsp, path):
    """Without keys, nothing beyond Q's own rows is addressed, however they lie:
    entries 8 elements apart here."""
    W = bsp.bsp_window_create(10, 1)
    room = torch.ones(8 * 299 + 64, dtype=torch.bfloat16, device="cuda")
    Q = room.as_strided((300, 1, 1, 64), (8, 64, 64, 1))
    none = torch.empty(300, 1, 0, 64, dtype=torch.bfloat16, device="cuda")
    O, lse = bsp.bsp_window_attention(W, Q, none, none)
    assert bool((O == 0).all()) and bool((lse == -math.inf).all())
    assert bsp.bsp_window_status(W) == 0


def test_gradients_over_inputs_are_refused_on_one_side_too(bsp):
    """Without queries, or without keys, a gradient in an input's place would be
    zeros over the input."""
    W = bsp.bsp_window_create(10, 1)
    x = lambda *s: torch.ones(*s, device="cuda", dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 0, device="cuda")
    none, K, V = x(1, 2, 0, 64), x(1, 1, 8, 64), x(1, 1, 8, 64)
    both = x(1, 1, 8, 64)
    for dK, dV in ((K, None), (None, V), (None, K), (both, both)):
        with pytest.raises(bsp.BspError):
            bsp.bsp_window_attention_backward(W, none, K, V, none, none, lse, dK=dK, dV=dV)
    Q, O, dO, nokey = x(1, 2, 8, 64), x(1, 2, 8, 64), x(1, 2, 8, 64), x(1, 1, 0, 64)
    lse = torch.zeros(1, 2, 8, device="cuda")
    for dQ in (Q, O, dO):
        with pytest.raises(bsp.BspError):
            bsp.bsp_window_attention_backward(W, Q, nokey, nokey, O, dO, lse, dQ=dQ)
    for t in (K, V, Q, O, dO):
        assert bool((t == 1).all())
    e = x(1, 2, 0, 64), x(1, 1, 0, 64)
    bsp.bsp_window_attention_backward(W, e[0], e[1], e[1], e[0], e[0], torch.zeros(1, 2, 0, device="cuda"))
    assert bsp.bsp_window_status(W) == 0


def test_long_windowed_sequences(bsp, path):
    """256 k tokens of 64 heads over 8: more (row tile, key tile) pairs than 2^31,
    of which a window of 64 leaves few steps.  Rows in the middle and at the end
    against the keys of their windows."""
    S, window, n = 262144, 64, 100
    W = bsp.bsp_window_create(window, 0)
    Q, dO = (randn((1, 64, S, 16), torch.bfloat16, 180 + i, "rows") for i in range(2))
    K, V = (randn((1, 8, S, 16), torch.bfloat16, 182 + i) for i in range(2))
    O, lse, dQ, dK, dV = _gradients(bsp, W, Q, K, V, dO, 0.25)
    assert bsp.bsp_window_status(W) == 0
    for end in (S // 2, S):
        rows, keys = slice(end - n, end), slice(end - n - window + 1, end)
        r = ref.dense(Q[:, :, rows], K[:, :, keys], V[:, :, keys], 0.25, window, 0, dO[:, :, rows])
        check(O[:, :, rows], r["O"], r["eO"], "O")
        check(lse[:, :, rows], r["lse"], r["else_"], "lse")
        check(dQ[:, :, rows], r["dQ"], r["eQ"], "dQ")
        # keys whose queries are all among the rows
        own = slice(end - n, end if end == S else end - window)
        for name, got in (("dK", dK), ("dV", dV)):
            at = slice(window - 1, window - 1 + own.stop - own.start)
            check(got[:, :, own], r[name][:, :, at], r["e" + name[-1]][:, :, at], name)


def test_long_windowed_pages(bsp, path):
    """A chunk of 16 k tokens under a table of 16 M keys, of which a window leaves
    few."""
    S, window, n, page = 16384, 100, 50, 128
    W = bsp.bsp_window_create(window, 0)
    Q = randn((1, 64, S, 16), torch.bfloat16, 190)[0].transpose(0, 1).contiguous()
    Kc, Vc = (randn((S // page, 8, page, 16), torch.bfloat16, 191 + i) for i in range(2))
    table = torch.full((1, 1 << 17), -1, dtype=torch.int32, device="cuda")
    table[0, :S // page] = torch.arange(S // page, dtype=torch.int32, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    O, lse = bsp.bsp_paged_attention(W, Q, Kc, Vc, i(0, S), i(S), table, scale=0.25)
    assert bsp.bsp_window_status(W) == 0
    K, V = (c.transpose(0, 1).reshape(1, 8, S, 16)[:, :, S - n - window + 1:] for c in (Kc, Vc))
    r = ref.dense(Q[S - n:].transpose(0, 1)[None], K, V, 0.25, window, 0)
    check(O[S - n:].transpose(0, 1)[None], r["O"], r["eO"], "O")
    check(lse[S - n:].T[None], r["lse"], r["else_"], "lse")


def test_more_steps_than_31_bits_are_refused(bsp, path):
    """Full attention of 2^21 tokens in 64 heads: refused before anything runs."""
    W = bsp.bsp_window_create(0, 0)
    S = 1 << 21
    x = torch.empty(S + 64, 16, dtype=torch.bfloat16, device="cuda")
    Q, K = (x.as_strided((1, H, S, 16), (S * 16, 8, 16, 1)) for H in (64, 8))  # heads that overlap
    O = torch.full((1, 64, S, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, 64, S), 7.0, device="cuda")
    with pytest.raises(bsp.BspError) as e:
        bsp.bsp_window_attention(W, Q, K, K, O=O, lse=lse)
    assert e.value.code == -2
    with pytest.raises(bsp.BspError) as e:
        bsp.bsp_window_attention_backward(W, Q, K, K, O, O.clone(), lse, dQ=O.clone())
    assert e.value.code == -2
    assert bool((O == 7).all()) and bool((lse == 7).all())
    assert bsp.bsp_window_status(W) == 0


def _tiles_that_meet(S, tokens, window, lo, hi):
    """[S] rows whose tile of `tokens` tokens has a row that sees a key of lo .. hi."""
    t = torch.arange(S, device="cuda") // tokens * tokens
    last = (t + tokens - 1).clamp(max=S - 1)
    return (last >= lo) & ((t - window + 1).clamp(min=0) <= hi)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_how_far_non_finite_rows_reach(bsp, path, dtype):
    """Three heads a group: 42 tokens are 126 rows.  Rows that the header does not
    name keep their bits, those that see the row have NaN."""
    S, window, j = 600, 100, 300
    W = bsp.bsp_window_create(window, 0)
    Q, K, V, dO = (randn((1, H, S, 64), DT[dtype], 200 + i) for i, H in enumerate((6, 2, 2, 6)))
    want = _gradients(bsp, W, Q, K, V, dO)
    pos = torch.arange(S, device="cuda")
    sees = (pos >= j) & (pos - j < window)
    # a V row: pieces of 16 keys
    V2 = V.clone()
    V2[0, 0, j] = math.nan
    O, lse, dQ, dK, dV = _gradients(bsp, W, Q, K, V2, dO)
    near = _tiles_that_meet(S, 42, window, j // 16 * 16, j // 16 * 16 + 15)
    assert torch.equal(O[:, 3:], want[0][:, 3:]) and torch.equal(lse, want[1])
    assert torch.equal(O[:, :3, ~near], want[0][:, :3, ~near]) and bool(O[:, :3, sees].isnan().all())
    near = _tiles_that_meet(S, 42, window, j // 128 * 128, j // 128 * 128 + 127)
    assert torch.equal(dQ[:, 3:], want[2][:, 3:]) and torch.equal(dQ[:, :3, ~near], want[2][:, :3, ~near])
    # a K row
    K2 = K.clone()
    K2[0, 1, j] = math.inf
    O, lse, dQ, dK, dV = _gradients(bsp, W, Q, K2, V, dO)
    for got, ref_ in ((O, want[0]), (lse, want[1])):
        assert torch.equal(got[:, :3], ref_[:, :3]) and torch.equal(got[:, 3:, ~sees], ref_[:, 3:, ~sees])
    assert torch.equal(dQ[:, :3], want[2][:, :3]) and torch.equal(dQ[:, 3:, ~near], want[2][:, 3:, ~near])
    # rows of Q and dO: the keys that their tile's rows see
    first = j // 42 * 42
    keys = (pos >= max(first - window + 1, 0) // 128 * 128) & (pos < (first + 41) // 128 * 128 + 128)
    for which in (0, 3):
        x = [Q, K, V, dO]
        x[which] = x[which].clone()
        x[which][0, 1, j] = math.nan
        O, lse, dQ, dK, dV = _gradients(bsp, W, *x)
        assert bool(dQ[0, 1, j].isnan().all())
        same = torch.ones(6, S, dtype=torch.bool, device="cuda")
        same[1, j] = False
        assert torch.equal(dQ[0][same], want[2][0][same])
        for got, ref_ in ((dK, want[3]), (dV, want[4])):
            assert torch.equal(got[:, 1], ref_[:, 1]) and torch.equal(got[:, 0, ~keys], ref_[:, 0, ~keys])
    assert bsp.bsp_window_status(W) == 0


def test_workspace_of_many_short_sequences(bsp):
    """One token each in 32768 (batch entry, KV head) pairs: 64 rows' statistics a
    pair, not the partial results of a long one."""
    size = bsp.lib().bsp_window_attention_workspace
    assert size(4096, 8, 8, 1, 1) - size(0, 8, 8, 1, 1) <= 32768 * 1024
    W = bsp.bsp_window_create()
    Q, K, V, dO = (randn((4096, 8, 1, 16), torch.float16, 210 + i) for i in range(4))
    O, lse, dQ, dK, dV = _gradients(bsp, W, Q, K, V, dO)
    assert torch.equal(O, V) and torch.equal(dV, dO)  # one key: P = 1
    # and dS = 0 but for dP and delta, one sum in two orders: gamma(16) = 5e-6 of
    # |dO||V| < 300, times scale |K| < 1
    assert dQ.abs().max().item() <= 1e-2 and dK.abs().max().item() <= 1e-2
    assert bsp.bsp_window_status(W) == 0


@pytest.mark.parametrize("size", [1.0, 2.0 ** -12])
@pytest.mark.parametrize("shape", JOINED, ids=str)
def test_tiles_of_many_pieces_in_fp16(bsp, path, shape, size):
    """Partial results leave fp16's factors behind, for output gradients of either
    size; the bound of the norms is that of test_gradient_of_a_small_output_gradient."""
    Z, Hq, Hkv, Sq, Sk, D, window, sinks = shape
    Q, dO = (randn((Z, Hq, Sq, D), torch.float16, sum(shape) + i) for i in range(2))
    K, V = (randn((Z, Hkv, Sk, D), torch.float16, sum(shape) + 2 + i) for i in range(2))
    dO = (dO * size).half()
    W = bsp.bsp_window_create(window, sinks)
    scale = 1.0 / math.sqrt(D)
    O, lse, dQ, dK, dV = _gradients(bsp, W, Q, K, V, dO, scale)
    r = ref.dense(Q, K, V, scale, window, sinks, dO)
    for name, got in (("O", O), ("dQ", dQ), ("dK", dK), ("dV", dV)):
        check(got, r[name], r["e" + name[-1]], name)
        off = (got.double() - r[name]).norm().item()
        assert off <= 4 * ref.U[torch.float16] * r[name].norm().item() + ref.AB[torch.float16] * math.sqrt(got.numel()), name
    assert all(torch.equal(a, b) for a, b in zip(_gradients(bsp, W, Q, K, V, dO, scale), (O, lse, dQ, dK, dV)))
    assert bsp.bsp_window_status(W) == 0
