"""Drafted tokens, pages and rotary positions without a device: argument errors,
the frequencies, and the plain forms that the GPU tests compare with."""

import ctypes
import math
import random

import numpy as np
import pytest
import torch

import draft_ref as ref
from sparse_attention_layout_gb300 import bsp, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bsp.lib()


def test_refusals_without_a_handle(lib):
    r = bytes(32)  # a bsp_tensor_t of zeros
    assert lib.bsp_draft_tree(None, None, None, None, None, None, 1, 1, 1, None) == -1
    assert lib.bsp_paged_tree_attention(None, 1, r, r, r, r, None, None, None, None, None, None, 1, 1, 1, 1, 16, 1, 1, 64, 1, 1.0,
                                        None, 0, None) == -1
    for words, code in ((0, -1), (-1, -1), (33, -2)):
        assert lib.bsp_paged_tree_attention(None, 1, r, r, r, r, None, None, None, None, None, None, 1, 1, 1, 1, 16, 1, 1, 64, words,
                                            1.0, None, 0, None) == code
    assert lib.bsp_draft_verify(None, 0, None, 8, None, 8, None, None, None, None, None, None, None, None, 1, 1, 8, None) == -1
    assert lib.bsp_paged_keep(None, 1, r, r, None, None, None, None, None, 1, 1, 1, 1, 16, 1, 64, None) == -1
    assert lib.bsp_paged_copy(None, 1, r, r, None, None, 1, 1, 16, 1, 64, None) == -1
    assert lib.bsp_pages_free(None, None, None, None, 1, 1, 1, 16, None) == -1
    assert lib.bsp_pages_fork(None, None, None, None, None, 1, 1, 1, 16, None, 0, None) == -1
    assert lib.bsp_pages_reserve(None, None, None, None, None, None, None, 1, 1, 1, 16, None, 0, None) == -1
    assert lib.bsp_pages_compact(None, None, None, None, None, None, None, 1, 1, 1, None, 0, None) == -1
    assert lib.bsp_rotary(None, 1, r, r, None, None, None, 0, 0, 1, 1, 0, 1, 64, None) == -1
    assert lib.bsp_rotary_destroy(None) == 0


def test_refusals_of_a_rotary_handle(lib):
    f = (ctypes.c_double * 65)(*[1.0] * 65)
    h = ctypes.c_void_p()
    assert lib.bsp_rotary_create(f, 4, 1.0, 0, None) == -1
    assert lib.bsp_rotary_create(None, 4, 1.0, 0, ctypes.byref(h)) == -1
    assert lib.bsp_rotary_create(f, 0, 1.0, 0, ctypes.byref(h)) == -1
    assert lib.bsp_rotary_create(f, 65, 1.0, 0, ctypes.byref(h)) == -2
    assert lib.bsp_rotary_create(f, 4, math.inf, 0, ctypes.byref(h)) == -1
    assert lib.bsp_rotary_create(f, 4, 1.0, 2, ctypes.byref(h)) == -1
    f[3] = math.nan
    assert lib.bsp_rotary_create(f, 4, 1.0, 0, ctypes.byref(h)) == -1 and not h.value


def test_workspace_of_the_book(lib):
    for n_seq, max_pages, n_pages in ((1, 1, 1), (64, 1000, 70000), (16384, 60000, 5), (0, 5, 9)):
        n = lib.bsp_pages_workspace(n_seq, max_pages, n_pages)
        assert n >= 4 * n_seq * max_pages + 4 * n_seq and n >= 12 * n_pages and n % 256 == 0
    for sizes in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (16385, 1, 1), (16384, 65537, 5)):
        assert lib.bsp_pages_workspace(*sizes) == 0


def wrapper(name):
    """The Python entry point without its stream."""
    f = getattr(bsp, name).__wrapped__
    return lambda W, *a, **kw: f(W, *a, stream=0, **kw)


@pytest.fixture
def handle(monkeypatch):
    """A handle of the CPU, so that the checks before the library's can be met; the
    library itself must not be reached."""
    W = object.__new__(bsp.Window)
    W.handle, W.device = None, torch.device("cpu")

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_workspace"):
                    return 256
                raise AssertionError("the call was not refused")
            return call

    monkeypatch.setattr(bsp, "lib", Lib)
    yield W
    bsp._paged_workspace.cache_clear()
    bsp._pages_bytes.cache_clear()


def test_wrong_tensors_are_refused(handle):
    W = handle
    i32 = dict(dtype=torch.int32)
    K = torch.zeros(6, 2, 16, 32)
    starts, kv, table, rows = torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 4, **i32), torch.zeros(5, **i32)
    bits, Q = torch.zeros(5, 1, **i32), torch.zeros(5, 4, 32)
    p, u, s, refs = torch.zeros(5, 9), torch.zeros(5), torch.zeros(2), torch.zeros(6, **i32)
    calls = {
        "bsp_draft_tree": ([starts, kv, rows, 3], {0: kv, 1: rows, 2: u}),
        "bsp_draft_verify": ([p, p.clone(), rows, starts, rows, u, s], {0: p[:4], 1: p[:, :8], 2: kv, 3: kv, 4: kv, 5: s, 6: u}),
        "bsp_paged_tree_attention": ([Q, K, K.clone(), starts, kv, table, rows, bits],
                                     {0: Q[:4], 1: K[:5], 2: K[..., :16], 3: kv, 4: rows, 5: table[:1], 6: kv, 7: bits[:4]}),
        "bsp_paged_keep": ([K, K.clone(), starts, kv, table, rows, kv], {0: K[0], 1: K[:, :1], 2: kv, 3: s, 4: table[0], 5: bits, 6: rows}),
        "bsp_paged_copy": ([K, K.clone(), kv, kv], {0: K[0], 1: K[:5], 2: s, 3: rows}),
        "bsp_pages_free": ([refs, table, kv, 16], {0: table, 1: refs, 2: rows}),
        "bsp_pages_fork": ([refs, table, kv, kv, 16], {0: p, 1: K, 2: rows, 3: rows}),
        "bsp_pages_reserve": ([refs, table, kv, kv, 16], {0: p, 1: K, 2: rows, 3: s}),
        "bsp_pages_compact": ([refs, table], {0: table, 1: table.long()}),
    }
    for name, (args, wrong) in calls.items():
        with pytest.raises(AssertionError):
            wrapper(name)(W, *args)
        for i, bad in wrong.items():
            with pytest.raises((ValueError, TypeError)):
                wrapper(name)(W, *args[:i], bad, *args[i + 1:])
        for i, a in enumerate(args):  # every other column of a wider tensor
            if isinstance(a, torch.Tensor) and a.dim() < 4:
                with pytest.raises((ValueError, TypeError)):
                    wrapper(name)(W, *args[:i], torch.stack([a, a], -1)[..., 0], *args[i + 1:])


def test_wrong_rows_are_refused(handle):
    R, Q, K = handle, torch.zeros(2, 4, 6, 32), torch.zeros(2, 1, 6, 32)
    turn = wrapper("bsp_rotary")
    with pytest.raises(AssertionError):
        turn(R, Q, K, torch.zeros(2, 6, dtype=torch.int32))
    for args in ((Q, K, torch.zeros(2, 6)), (Q, K, torch.zeros(2, dtype=torch.int32)), (Q, K[:1]), (Q, K[:, :, :5]), (Q, K[0]),
                 (Q, None, None, None, K), (Q, K, None, K), (Q[0, 0],), (Q[..., ::2],), (Q, K.double()), (Q.long(),)):
        with pytest.raises((ValueError, TypeError)):
            turn(R, *args)


def test_frequencies():
    f, a = bsp.rotary_frequencies(64)
    assert a == 1.0 and f[0] == 1.0 and np.allclose(f, [10000.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-15)
    lin, a = bsp.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert a == 1.0 and np.array_equal(lin, f / 4)
    base, a = bsp.rotary_frequencies(64, scaling="base", factor=4.0)
    assert a == 1.0 and base[0] == 1.0 and math.isclose(base[-1], f[-1] / 4, rel_tol=1e-14)
    parts, a = bsp.rotary_frequencies(64, scaling="parts", factor=4.0, length=2048)
    assert math.isclose(a, 1 + 0.1 * math.log(4.0))
    turns = 2048 * f / (2 * math.pi)
    assert np.array_equal(parts[turns >= 32], f[turns >= 32]) and np.allclose(parts[turns <= 1], f[turns <= 1] / 4, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (parts[between] < f[between]).all() and (parts[between] > f[between] / 4).all()
    assert len(bsp.rotary_frequencies(2, scaling="base", factor=3.0)[0]) == 1
    for args in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=0.0), dict(rot_dim=8, scaling="other"),
                 dict(rot_dim=8, scaling="parts", fast=1.0, slow=1.0), dict(rot_dim=8, factor=-1.0)):
        with pytest.raises(ValueError):
            bsp.rotary_frequencies(**args)


def test_lists_of_a_book_agree():
    r = random.Random(1)
    b = ref.Book(50, 6, 10, 16)
    for _ in range(200):
        want = [min(160, n + r.randint(0, 30)) for n in b.kv]
        src, dst, enough = b.reserve(want)
        assert b.agrees() and all((a < 0) == (c < 0) for a, c in zip(src, dst))
        b.kv = [max(a, c) for a, c in zip(b.kv, want)] if enough else [0 if r.random() < 0.4 else n for n in b.kv]
        b.free()
        b.fork([r.choice((i, r.randrange(6), -1)) for i in range(6)])
        high, low = b.compact()
        assert b.agrees() and all(x >= 0 for x in b.refs)
        live = sum(n > 0 for n in b.refs)
        assert all(n > 0 for n in b.refs[:live])


def test_plain_verification_follows_the_target():
    """Of the reference itself: the first token is distributed as the target's row."""
    r = np.random.default_rng(3)
    p, q = np.array([0.5, 0.1, 0.4]), np.array([0.2, 0.7, 0.1])
    N, hits = 20000, np.zeros(3)
    for _ in range(N):
        tok = [0, *r.choice(3, 2, p=q)]
        path, nxt = ref.verify(np.stack([p] * 3), np.stack([q] * 3), tok, [-1, 0, 0], r.random(3), r.random())
        hits[tok[path[1]] if len(path) > 1 else nxt] += 1
    assert (np.abs(hits - N * p) <= 6 * np.sqrt(N * p * (1 - p))).all()


def test_trees_bit_by_bit():
    m = ref.tree_mask([-1, 0, 0, 1, 3], 10, 0, 0)
    assert [np.flatnonzero(x).tolist() for x in m] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4]]
    m = ref.tree_mask([-1, 0, 0, 1, 3], 10, 2, 11)  # the first node stands at a sink's position
    assert [np.flatnonzero(x).tolist() for x in m] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 3, 4]]
    assert ref.pack(m, 2).tolist() == [[1, 0], [3, 0], [5, 0], [11, 0], [25, 0]]
