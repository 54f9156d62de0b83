"""Rotary positions and their gradient against the formula, entry by entry.

Bounds, per pair.  The fraction of a turn is off by 2^-32 (the fraction's lower
half is cut off), its remainder after the nearest quarter turn, at most 1/4 of a
half turn, by 2^-24 of itself when it becomes fp32: 2 pi 2^-32 + pi / 4 2^-24,
together below 0.82 * 2^-24 radians.  sincospif is off by one unit in the last
place at most, 2^-24 for values below 1; the amplitude's own rounding and its
product's round by 2^-24 each, each product and sum of the rotation by 2^-24 of
|x_a| + |x_b| times the amplitude.  Together below 6 * 2^-24 A (|x_a| + |x_b|), and
the output rounds by u |y| (fp16: or 2^-25, half its subnormals' spacing)."""

import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from gpu_util import U
from window_ref import AB

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


def randn(shape, dtype, seed, order="heads"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Z, H, S, D = shape
    if order == "rows":
        return torch.randn(Z, S, H, D, generator=g, device="cuda").to(dtype).transpose(1, 2)
    if order == "fused":
        return torch.randn(Z, S, H, 2 * D, generator=g, device="cuda").to(dtype)[..., :D].transpose(1, 2)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def turned(x, pos, freq, amplitude, pairs, inverse=False):
    """x [Z, H, S, D], pos [Z, S]: the values in fp64 and their bounds."""
    n = len(freq)
    phi = pos.double()[:, None, :, None] * torch.from_numpy(np.asarray(freq)).to(x.device)
    return turned_by(x, torch.cos(phi), torch.sin(phi) * (-1 if inverse else 1), amplitude, pairs, n)


def turned_by(x, c, s, amplitude, pairs, n):
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if pairs else (slice(0, n), slice(n, 2 * n))
    x64 = x.double()
    y, e = x64.clone(), torch.zeros_like(x64)
    xa, xb = x64[..., a], x64[..., b]
    y[..., a] = amplitude * (xa * c - xb * s)
    y[..., b] = amplitude * (xb * c + xa * s)
    e[..., a] = e[..., b] = 6 * 2.0 ** -24 * abs(amplitude) * (xa.abs() + xb.abs())
    e[..., :2 * n] += U[x.dtype] * y[..., :2 * n].abs() + AB[x.dtype]
    return y, e


def check(got, want, bound, what):
    same = (got.double() - want).abs() <= bound
    assert got.shape == want.shape and bool(same.all()), (what, (~same).nonzero()[:3].tolist())


# (Z, Hq, Hkv, S, D, rotated columns)
SHAPES = [(1, 1, 1, 1, 16, 16), (1, 1, 0, 3, 16, 2), (2, 3, 1, 65, 64, 64), (1, 5, 2, 130, 80, 20), (3, 2, 2, 33, 48, 22),
          (1, 4, 4, 257, 128, 128), (2, 8, 1, 100, 96, 24), (1, 2, 1, 70, 112, 110), (1, 1, 1, 5000, 32, 12), (1, 32, 8, 9, 128, 64),
          (2, 40, 1, 700, 16, 10)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_the_formula(bsp, shape, pairs, dtype):
    Z, Hq, Hkv, S, D, rot = shape
    dt, seed = DT[dtype], sum(shape)
    order = ("heads", "rows", "fused")[seed % 3]
    Q, K = randn((Z, Hq, S, D), dt, seed, order), randn((Z, Hkv, S, D), dt, seed + 1) if Hkv else None
    freq, amp = bsp.rotary_frequencies(rot, scaling=("none", "linear", "base", "parts")[seed % 4], factor=4.0)
    R = bsp.bsp_rotary_create(freq, amp, pairs)
    g = torch.Generator().manual_seed(seed)
    each = torch.randint(0, 200000, (Z, S), generator=g).to(torch.int32).cuda()
    shared = torch.randint(-5000, 5000, (S,), generator=g).to(torch.int32).cuda()
    rows = torch.arange(S, device="cuda").expand(Z, S)
    for given, pos in ((None, rows), (shared, shared.expand(Z, S)), (each, each)):
        for inverse in (False, True):
            q, k = bsp.bsp_rotary(R, Q, K, given, inverse=inverse)
            check(q, *turned(Q, pos, freq, amp, pairs, inverse), "Q")
            if Hkv:
                check(k, *turned(K, pos, freq, amp, pairs, inverse), "K")
            else:
                assert k is None
    # in their own places, into given tensors of other strides, and one alone: the same bits
    q, k = bsp.bsp_rotary(R, Q, K, each)
    Q2, K2 = Q.clone(), None if K is None else K.clone()
    bsp.bsp_rotary(R, Q2, K2, each, Q2, K2)
    assert torch.equal(Q2, q) and (K is None or torch.equal(K2, k))
    wide = torch.full((Z, S, Hq, 2 * D), 7.0, dtype=dt, device="cuda")
    bsp.bsp_rotary(R, Q, None, each, Q_out=wide[..., D:].transpose(1, 2))
    assert torch.equal(wide[..., D:].transpose(1, 2), q) and bool((wide[..., :D] == 7).all())
    if K is not None:
        Q3 = Q.clone()
        _, k3 = bsp.bsp_rotary(R, Q3, K, each, Q_out=Q3)
        assert torch.equal(Q3, q) and torch.equal(k3, k)


@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
def test_ragged_rows(bsp, pairs):
    """[T, H, D] tokens, as the paged calls take them."""
    freq, amp = bsp.rotary_frequencies(64)
    R = bsp.bsp_rotary_create(freq, amp, pairs)
    Q, K = randn((1, 6, 77, 64), torch.bfloat16, 1, "rows"), randn((1, 2, 77, 64), torch.bfloat16, 2, "rows")
    pos = torch.randint(0, 30000, (77,), dtype=torch.int32).cuda()
    want = bsp.bsp_rotary(R, Q, K, pos)
    got = bsp.bsp_rotary(R, Q[0].transpose(0, 1), K[0].transpose(0, 1), pos)
    for a, b in zip(got, want):
        assert torch.equal(a.transpose(0, 1), b[0])


def test_a_fused_projection_in_place(bsp):
    """Q and K as slices of one [T, heads, D] tensor, turned where they are; V beside
    them stays."""
    freq, amp = bsp.rotary_frequencies(64)
    for dtype, pairs in ((torch.float16, False), (torch.float32, True)):
        R = bsp.bsp_rotary_create(freq, amp, pairs)
        x = randn((1, 6 + 2 + 2, 91, 64), dtype, 4, "rows")[0].transpose(0, 1)
        assert x.is_contiguous()
        pos = torch.arange(91, dtype=torch.int32, device="cuda") * 7
        q, k = bsp.bsp_rotary(R, x[:, :6], x[:, 6:8], pos)
        v = x[:, 8:].clone()
        bsp.bsp_rotary(R, x[:, :6], x[:, 6:8], pos, x[:, :6], x[:, 6:8])
        assert torch.equal(x[:, :6], q) and torch.equal(x[:, 6:8], k) and torch.equal(x[:, 8:], v)


def test_far_positions(bsp):
    """Angles at any 32-bit position, against 50 decimal digits."""
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    pos = [0, 1, -1, 12345678, 2 ** 24 + 1, 999999937, 2 ** 30, 2 ** 31 - 1, -2 ** 31]
    freq, _ = bsp.rotary_frequencies(32)
    freq = np.concatenate([freq, [3.0, -1.25, 0.0, 6.5, 1e-9, 100.0, 2.0 ** -40, 0.7]])
    n = len(freq)
    turns = np.array([[float((Decimal(p) * Decimal(float(f)) / two_pi) % 1) for f in freq] for p in pos])
    x = randn((1, 2, len(pos), 48), torch.float32, 3)
    c, s = (torch.from_numpy(f(2 * np.pi * turns)).cuda()[None, None] for f in (np.cos, np.sin))
    for pairs in (False, True):
        R = bsp.bsp_rotary_create(freq, 1.0, pairs)
        q, _ = bsp.bsp_rotary(R, x, positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
        check(q, *turned_by(x, c, s, 1.0, pairs, n), "far positions")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
def test_gradient(bsp, pairs, dtype):
    """The transposed map; the second gradient is the map again."""
    dt = DT[dtype]
    freq, amp = bsp.rotary_frequencies(48, scaling="parts", factor=8.0)
    R = bsp.bsp_rotary_create(freq, amp, pairs)
    pos = torch.randint(0, 9000, (2, 50), dtype=torch.int32).cuda()
    Q, K = randn((2, 4, 50, 64), dt, 5, "rows").requires_grad_(), randn((2, 1, 50, 64), dt, 6).requires_grad_()
    dQ, dK = randn((2, 4, 50, 64), dt, 7), randn((2, 1, 50, 64), dt, 8, "rows")
    q, k = bsp.rotary(R, Q, K, pos)
    gq, gk = torch.autograd.grad((q, k), (Q, K), (dQ, dK), retain_graph=True)
    check(gq, *turned(dQ, pos, freq, amp, pairs, True), "dQ")
    check(gk, *turned(dK, pos, freq, amp, pairs, True), "dK")
    # one output alone, a broadcast gradient, a tensor that the kernels do not take
    g1, = torch.autograd.grad(k, K, dK, retain_graph=True)
    assert torch.equal(g1, gk)
    g2, = torch.autograd.grad(q.sum(), Q, retain_graph=True)
    check(g2, *turned(torch.ones_like(Q), pos, freq, amp, pairs, True), "dQ of a sum")
    odd = randn((2, 4, 50, 65), dt, 9)[..., 1:]
    assert torch.equal(bsp.rotary(R, odd, None, pos)[0], bsp.bsp_rotary(R, odd.contiguous(), None, pos)[0])
    v = dQ.clone().requires_grad_()
    g3, = torch.autograd.grad(bsp.rotary(R, Q, None, pos)[0], Q, v, create_graph=True)
    w = randn((2, 4, 50, 64), dt, 10)
    g4, = torch.autograd.grad(g3, v, w)
    check(g4, *turned(w, pos, freq, amp, pairs), "second gradient")
    assert torch.equal(bsp.rotary(R, Q.detach(), K.detach(), pos)[1], k)


def test_gradient_of_ragged_rows(bsp):
    """[T, heads, D] tokens, with shared, strided and missing gradients."""
    freq, amp = bsp.rotary_frequencies(64)
    R = bsp.bsp_rotary_create(freq, amp)
    pos = torch.randint(0, 500, (41,), dtype=torch.int32).cuda()
    Q, K = (randn((1, H, 41, 64), torch.float32, 30 + H, "rows")[0].transpose(0, 1).requires_grad_() for H in (4, 2))
    dQ, dK = randn((1, 4, 41, 64), torch.float32, 40)[0].transpose(0, 1), randn((1, 1, 41, 64), torch.float32, 41)[0].transpose(0, 1)
    dK = dK.expand(41, 2, 64)
    for positions, at in ((pos, pos), (None, torch.arange(41, device="cuda"))):
        q, k = bsp.rotary(R, Q, K, positions)
        gq, gk = torch.autograd.grad((q, k), (Q, K), (dQ, dK), retain_graph=True)
        for got, d in ((gq, dQ), (gk, dK)):
            want, bound = turned(d.transpose(0, 1)[None], at[None], freq, amp, False, True)
            check(got.transpose(0, 1)[None], want, bound, "gradient")
        only, = torch.autograd.grad(k, K, dK)
        assert torch.equal(only, gk)
    q, k = bsp.rotary(R, Q, K, pos)
    pos += 1
    with pytest.raises(RuntimeError):
        torch.autograd.grad(q, Q, dQ)


def test_gradient_by_differences(bsp):
    """The map is linear: f(x + h d) - f(x - h d) is 2 h times the derivative but
    for rounding, 6 * 2^-24 A (|x_a| + |x_b|) per entry, against dot products of
    some thousand entries of size 1: with h = 1 within 1e-3 of the norm."""
    freq, amp = bsp.rotary_frequencies(32)
    R = bsp.bsp_rotary_create(freq, amp)
    x, d, g = (randn((1, 2, 40, 32), torch.float32, 11 + i) for i in range(3))
    x.requires_grad_()
    grad, = torch.autograd.grad(bsp.rotary(R, x)[0], x, g)
    f = [(bsp.bsp_rotary(R, x.detach() + sgn * d)[0].double() * g.double()).sum().item() for sgn in (1, -1)]
    want = (grad.double() * d.double()).sum().item()
    assert abs((f[0] - f[1]) / 2 - want) <= 1e-3 * math.sqrt(g.numel())


def test_relative_positions(bsp):
    """Scores of rotated rows depend on the distance of their positions alone."""
    freq, amp = bsp.rotary_frequencies(64)
    R = bsp.bsp_rotary_create(freq, amp)
    Q, K = randn((1, 1, 1, 64), torch.float32, 1).expand(1, 1, 20, 64).contiguous(), \
        randn((1, 1, 1, 64), torch.float32, 2).expand(1, 1, 20, 64).contiguous()
    pos = (torch.arange(20, dtype=torch.int32) * 50001).cuda()
    q, _ = bsp.bsp_rotary(R, Q, None, pos)
    k, _ = bsp.bsp_rotary(R, K, None, pos - 17)
    s = (q.double() * k.double()).sum(-1)
    # each row entry is off by 6 * 2^-24 of its pair, both factors
    bound = 8 * 6 * 2.0 ** -24 * (Q.abs().sum() / 20 * K.abs().max() * 2).item()
    assert (s - s[..., :1]).abs().max().item() <= bound


def test_largest_and_empty(bsp):
    freq, amp = bsp.rotary_frequencies(16)
    R = bsp.bsp_rotary_create(freq, amp)
    for shape in ((0, 2, 5, 16), (1, 2, 0, 16)):
        q, k = bsp.bsp_rotary(R, torch.empty(*shape, device="cuda"), torch.empty(*shape, device="cuda"))
        assert q.shape == shape and k.shape == shape
    # element offsets beyond 2^31
    S = 1 << 19
    Q = torch.randn(1, S, 33, 128, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    q, _ = bsp.bsp_rotary(R, Q)
    at = torch.tensor([0, 5, S - 1], device="cuda")
    check(q[:, :, at], *turned(Q[:, :, at], at[None], freq, amp, False), "rows")


def test_streams_and_graphs(bsp):
    freq, amp = bsp.rotary_frequencies(64)
    R = bsp.bsp_rotary_create(freq, amp)
    Q, K = randn((1, 4, 64, 64), torch.float16, 1), randn((1, 2, 64, 64), torch.float16, 2)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    want = bsp.bsp_rotary(R, Q, K, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bsp.bsp_rotary(R, Q, K, pos, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, k = bsp.bsp_rotary(R, Q, K, pos)
    pos += 1000
    Q.copy_(Q.flip(2))
    g.replay()
    torch.cuda.synchronize()
    want = bsp.bsp_rotary(R, Q, K, pos)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_gradient_in_a_graph(bsp):
    freq, amp = bsp.rotary_frequencies(64)
    R = bsp.bsp_rotary_create(freq, amp, True)
    Q, K, dQ, dK = (randn((2, H, 33, 64), torch.bfloat16, 20 + i) for i, H in enumerate((4, 2, 4, 2)))
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    Q.requires_grad_()
    K.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(bsp.rotary(R, Q, K, pos), (Q, K), (dQ, dK))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq, gk = torch.autograd.grad(bsp.rotary(R, Q, K, pos), (Q, K), (dQ, dK))
    pos += 77
    dQ.normal_()
    graph.replay()
    torch.cuda.synchronize()
    at = pos.expand(2, 33)
    check(gq, *turned(dQ, at, freq, amp, True, True), "dQ")
    check(gk, *turned(dK, at, freq, amp, True, True), "dK")


def test_refusals(bsp):
    R = bsp.bsp_rotary_create([1.0, 0.5])
    Q, K = torch.zeros(1, 2, 8, 32, device="cuda"), torch.zeros(1, 1, 8, 32, device="cuda")
    bsp.bsp_rotary(R, Q, K)
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    for args in ((Q, K, pos.long()), (Q, K, pos[:7]), (Q, K, pos.cpu()), (Q, K, torch.zeros(2, 8, dtype=torch.int32, device="cuda")),
                 (Q, K[:, :, :7]), (Q, K[..., :16]), (Q, K[0]), (Q[0, 0], None), (Q, None, None, None, K), (Q.cpu(), None),
                 (Q, K[:, :0])):
        with pytest.raises(ValueError):
            bsp.bsp_rotary(R, *args)
    with pytest.raises(TypeError):
        bsp.bsp_rotary(R, Q, K.half())
    with pytest.raises(TypeError):
        bsp.bsp_rotary(R, Q.double())
    flat = torch.zeros(4096, device="cuda")
    bad = [((flat[1:513].view(1, 2, 8, 32), None), -3),                     # alignment
           ((torch.zeros(1, 2, 8, 34, device="cuda")[..., :32], None), -3),
           ((torch.zeros(1, 2, 8, 24, device="cuda"), None), -1),          # head size
           ((torch.zeros(1, 1, 8, 32, device="cuda").expand(1, 2, 8, 32), None), -1),
           ((Q, K, None, torch.empty_strided((1, 2, 8, 32), (512, 0, 32, 1), device="cuda")), -1),
           ((Q, Q, None, Q, Q), -1)]                                       # two outputs in one place
    for args, code in bad:
        with pytest.raises(bsp.BspError) as e:
            bsp.bsp_rotary(R, *args)
        assert e.value.code == code, args
    with pytest.raises(bsp.BspError) as e:  # its own memory in another order
        bsp.bsp_rotary(R, Q, None, None, Q.view(1, 8, 2, 32).transpose(1, 2))
    assert e.value.code == -1
    with pytest.raises(bsp.BspError) as e:  # 17 pairs of 32 columns
        bsp.bsp_rotary(bsp.bsp_rotary_create([1.0] * 17), Q)
    assert e.value.code == -1
    for freq, amp, code in (([], 1.0, -1), ([math.nan], 1.0, -1), ([math.inf], 1.0, -1), ([1.0], math.nan, -1), ([1.0], 1e39, -1),
                            ([1.0] * 65, 1.0, -2)):
        with pytest.raises(bsp.BspError) as e:
            bsp.bsp_rotary_create(freq, amp)
        assert e.value.code == code
