"""Verification of drafted tokens where entries are no probabilities, against the
walk in fp64 over the rows with such entries set to 0."""

import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

import draft_ref as ref

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def counted(rows):
    """The rows in fp64 on the host, entries that count as 0 set to it."""
    return torch.where(rows > 0, rows, torch.zeros_like(rows)).double().cpu().numpy()


def agrees(bsp, W, parents, target, draft, tok, accept, sample):
    """Every sequence's path, count and token are those of the walk in fp64."""
    starts = [0]
    for t in parents:
        starts.append(starts[-1] + len(t))
    got = bsp.bsp_draft_verify(W, target, draft, tok, ints(starts), ints([x for t in parents for x in t]), accept, sample)
    path, count, token = (x.tolist() for x in got)
    p, q = counted(target), None if draft is None else counted(draft)
    tl, al, sl = tok.tolist(), accept.double().tolist(), sample.double().tolist()
    for i, t in enumerate(parents):
        a, b = starts[i], starts[i + 1]
        want, nxt = ref.verify(p[a:b], None if q is None else q[a:b], tl[a:b], t, al[a:b], sl[i])
        assert (count[i], path[a:b], token[i]) == (len(want), want + [-1] * (b - a - len(want)), nxt), i
    assert bsp.bsp_window_status(W) == 0
    return got


@pytest.mark.parametrize("chosen", [False, True], ids=["drawn", "chosen"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [5, 37, 3000])
def test_entries_that_count_as_nothing(bsp, V, dtype, chosen):
    """Negative entries, NaN and -inf in a third of the places of both rows, at the
    children's tokens and elsewhere."""
    W, n_seq = bsp.bsp_window_create(), 48
    r, g = random.Random(V), torch.Generator(device="cuda").manual_seed(V)
    parents = [[-1] + [r.randrange(max(0, i - 5), i) for i in range(1, 9)] for _ in range(n_seq)]
    T = 9 * n_seq
    rows = []
    for _ in range(2):
        x = torch.softmax(2 * torch.randn(T, V, generator=g, device="cuda"), -1)
        kind = torch.randint(0, 9, (T, V), generator=g, device="cuda")
        x = torch.where(kind == 0, -x, x)
        x = torch.where(kind == 1, torch.full_like(x, math.nan), x)
        rows.append(torch.where(kind == 2, torch.full_like(x, -math.inf), x).to(DT[dtype]))
    # tokens from the likely entries of the parents' rows, without their signs, and bad ones
    tok = torch.zeros(T, dtype=torch.int32, device="cuda")
    for s, t in enumerate(parents):
        for i in range(1, 9):
            row = rows[r.randrange(2)][9 * s + t[i]].float()
            bad = (~(row > 0)).nonzero()[:, 0].tolist()
            likely = row.abs().nan_to_num(0.0, posinf=0.0).argsort(descending=True)[:4].tolist()
            tok[9 * s + i] = r.choice(bad if bad and r.random() < 0.5 else likely)
    for low in (0.0, 0.8):  # then mostly rejected
        accept = low + (1 - low) * torch.rand(T, generator=g, device="cuda")
        sample = torch.rand(n_seq, generator=g, device="cuda")
        agrees(bsp, W, parents, rows[0], None if chosen else rows[1], tok, accept.clamp(max=1 - 2.0 ** -24), sample)


@pytest.mark.parametrize("bad", [-0.2, math.nan, -math.inf, -0.0])
def test_rejected_entries_that_count_as_nothing(bsp, bad):
    W = bsp.bsp_window_create()
    target = torch.tensor([[0.3, bad, 0.1, 0.3, 0.3]] * 3, device="cuda")
    for u in (0.0, 0.1, 0.45, 0.9):
        agrees(bsp, W, [[-1, 0, 0]], target, None, ints([0, 0, 1]), torch.full((3,), 0.9, device="cuda"), torch.full((1,), u, device="cuda"))
    # a draft's entry that counts as nothing leaves the target's as it is, and gives no
    # token that the target excludes
    target = torch.tensor([[0.5, 0.0, 0.25, 0.25]] * 3, device="cuda")
    draft = torch.tensor([[0.6, bad, bad, 0.4]] * 3, device="cuda")
    for tokens in ([0, 0, 1], [0, 1, 0], [0, 1, 2], [0, 0, 3]):
        for u in (0.0, 0.3, 0.6, 0.95):
            agrees(bsp, W, [[-1, 0, 0]], target, draft, ints(tokens), torch.full((3,), 0.9, device="cuda"),
                   torch.full((1,), u, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_all_of_a_run_rejected(bsp, dtype):
    """Chosen drafts that are all that a stretch of the vocabulary holds, of 0.06 to
    1e-13: what rounding leaves of the stretch's sum when they are taken away holds
    no token, and the next one, for the number 0, lies behind it."""
    W, n_seq, V = bsp.bsp_window_create(), 64, 32000
    g, r = torch.Generator().manual_seed(7), random.Random(7)
    target = torch.zeros(10 * n_seq, V)
    tok = torch.zeros(n_seq, 10, dtype=torch.int32)
    for s in range(n_seq):
        at = r.sample(range(256), 9)
        target[10 * s:10 * s + 10, at] = torch.tensor([10.0 ** -r.uniform(1.2, 13) for _ in at])
        target[10 * s:10 * s + 10, r.sample(range(1000, V), 20)] = 0.025
        tok[s, 1:] = torch.tensor(at)
    accept = torch.full((10 * n_seq,), 0.999, device="cuda")
    args = [[-1] + [0] * 9] * n_seq, target.to(DT[dtype]).cuda(), None, tok.view(-1).cuda(), accept
    for u in (0.0, 2.0 ** -149, 0.3, 1 - 2.0 ** -24):
        _, count, token = agrees(bsp, W, *args, torch.full((n_seq,), u, device="cuda"))
        assert bool((count == 1).all()) and bool((token >= 1000).all())
    # the same behind everything else, where a number that is too large falls to the last entry
    back = args[1].flip(1).contiguous(), None, (V - 1 - args[3]).contiguous()
    for u in (0.0, 1 - 2.0 ** -24, 1.0):
        _, count, token = agrees(bsp, W, args[0], *back, accept, torch.full((n_seq,), u, device="cuda"))
        assert bool((count == 1).all()) and bool((token < V - 1000).all())


def beside(border):
    """The float32 numbers next to a border, and its least distance from them."""
    x = np.float32(float(border))
    below, above = (x, np.nextafter(x, np.float32(2))) if Fraction(float(x)) < border else (np.nextafter(x, np.float32(0)), x)
    return float(below), float(above), min(border - Fraction(float(below)), Fraction(float(above)) - border) / border


@pytest.mark.parametrize("chosen", [False, True], ids=["drawn", "chosen"])
def test_sums_of_many_terms(bsp, chosen):
    """16 million entries to one block, 65536 to a thread, all but two the same, so that
    rounding errors add up: the sum decides on the second child, whose numbers are
    the two next to the border, 2^-26 of it away at least (V is chosen so)."""
    v, Z, q = 0.1 * 2.0 ** -20, 0.5, 0.25  # the rows' entries, the second child's
    v = float(np.float32(v))
    rest = Fraction(Z) - (0 if chosen else Fraction(q))
    for V in range(2 ** 24 + 1, 2 ** 24 + 400):
        total = (V - 2) * Fraction(v) + rest
        low, high, margin = beside(rest / total if chosen else rest / (Fraction(q) * total))
        if margin >= Fraction(1, 2 ** 26):
            break
    assert 0 < low < high < 1 and margin >= Fraction(1, 2 ** 26)
    x1, x2 = 5, V // 2
    target, draft = torch.full((3, V), v, device="cuda"), torch.zeros(3, V, device="cuda")
    target[:, x1], target[:, x2] = 0.0, Z
    draft[:, x1], draft[:, x2] = 0.5, q
    W, n_seq = bsp.bsp_window_create(), 400  # (the others without nodes)
    starts, parent, tok = ints([0] + [3] * n_seq), ints([-1, 0, 0]), ints([0, x1, x2])
    sample = torch.full((n_seq,), 0.5, device="cuda")
    for u, want in ((low, 2), (high, 1)):
        accept = torch.tensor([0.0, 0.5, u], device="cuda")
        _, count, _ = bsp.bsp_draft_verify(W, target, None if chosen else draft, tok, starts, parent, accept, sample)
        assert count[0].item() == want
    # and the next token, of a row of equal entries: the one that the number falls into
    target.fill_(v)
    for at in (3, 77777, 5555555, 12345678, 2 ** 24 - 9):
        u = float(np.float32((at + 0.5) / V))
        if not 0.25 <= u * V - int(u * V) <= 0.75:
            continue
        _, count, token = bsp.bsp_draft_verify(W, target, None, tok, starts, ints([-1, -1, -1]), accept, sample * 0 + u)
        assert count[0].item() == 1 and token[0].item() == int(Fraction(u) * V)
    assert bsp.bsp_window_status(W) == 0
