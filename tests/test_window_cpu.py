"""The windowed operators' work geometry against a direct enumeration, and
their argument errors that need no device."""

import ctypes

import numpy as np
import pytest

from sparse_attention_layout_gb300 import bsp, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bsp.lib()


def visible(p, j, window, sinks):
    return j <= p and ((not window) or p - j < window or j < sinks)


def tiles(lib, window, sinks, a, b, shift):
    n = ctypes.c_int()
    buf = np.full(4096, -1, np.int32)
    rc = lib.bsp_diag_window_tiles(window, sinks, a, b, shift, ctypes.byref(n), ctypes.c_void_p(buf.ctypes.data), buf.size)
    assert rc == 0
    return buf[:n.value].tolist()


@pytest.mark.parametrize("window", [0, 1, 5, 16, 33, 200])
@pytest.mark.parametrize("sinks", [0, 1, 16, 17, 70])
def test_key_tiles_cover_the_visible_keys_once(lib, window, sinks):
    rng = np.random.default_rng(window * 100 + sinks)
    for shift in (4, 6, 7):
        for _ in range(40):
            a = int(rng.integers(-40, 700))
            b = a + int(rng.integers(0, 128))
            got = tiles(lib, window, sinks, a, b, shift)
            want = sorted({j >> shift for p in range(max(a, 0), b + 1) for j in range(p + 1) if visible(p, j, window, sinks)})
            if not want:
                assert got == [0]
                continue
            assert got == sorted(set(got)) and set(want) <= set(got), (a, b, shift)
            # no tile beyond the first sink tiles and the window's range
            lo = max(0, max(a, 0) - (window or 1 << 30) + 1)
            assert all(t in want or (t << shift) >= lo or (t << shift) < sinks for t in got)


@pytest.mark.parametrize("window", [0, 1, 7, 64, 150])
@pytest.mark.parametrize("sinks", [0, 3, 64, 90])
def test_query_tiles_cover_the_rows_that_see_a_key_tile(lib, window, sinks):
    rng = np.random.default_rng(window * 100 + sinks)
    for shift in (6, 7):
        for _ in range(25):
            Sq, Sk = int(rng.integers(1, 400)), int(rng.integers(1, 400))
            tok = int(rng.choice([1, 2, 9, 16, 42, 64, 128]))
            for t in range((Sk + (1 << shift) - 1) >> shift):
                f, n = ctypes.c_int(), ctypes.c_int()
                assert lib.bsp_diag_window_queries(window, sinks, Sq, Sk, tok, shift, t, ctypes.byref(f), ctypes.byref(n)) == 0
                keys = np.arange(t << shift, min(Sk, (t + 1) << shift))
                p = np.arange(Sq) + Sk - Sq
                see = np.array([any(visible(int(x), int(j), window, sinks) for j in (keys[0], keys[-1])) or
                                bool(((keys <= x) & ((window == 0) | (x - keys < window) | (keys < sinks))).any())
                                for x in p])
                want = sorted({int(i) // tok for i in np.flatnonzero(see)})
                got = list(range(f.value, f.value + n.value))
                if not want:
                    assert n.value >= 1
                else:
                    assert set(want) <= set(got), (Sq, Sk, tok, t)
                    assert got[0] == want[0] and (sinks > keys[0] or got[-1] == want[-1])
                assert got[-1] <= (Sq - 1) // tok


def test_largest_positions_do_not_overflow(lib):
    top = 1 << 30
    assert tiles(lib, 2 ** 31 - 1, 0, 100, 200, 7) == [0, 1]
    got = tiles(lib, 256, 5, top - 128, top - 1, 7)
    assert got[0] == 0 and got[-1] == (top - 1) >> 7 and len(got) == 4
    assert tiles(lib, 256, 2 ** 31 - 1, 0, 127, 7) == [0]


def test_refusals_without_a_handle(lib):
    r = bytes(32)  # a bsp_tensor_t of zeros
    assert lib.bsp_window_create(-1, 0, None, ctypes.byref(ctypes.c_void_p())) == -1
    assert lib.bsp_window_create(0, -1, None, ctypes.byref(ctypes.c_void_p())) == -1
    assert lib.bsp_window_create(0, 0, None, None) == -1
    assert lib.bsp_window_destroy(None) == 0
    assert lib.bsp_window_info(None, None, None) == -1
    assert lib.bsp_window_status(None, None) == -1
    assert lib.bsp_window_attention(None, 1, r, r, r, r, None, 1, 1, 1, 1, 1, 64, 1.0, None, 0, None) == -1
    assert lib.bsp_window_attention_backward(None, 1, r, r, r, r, r, None, r, r, r, 1, 1, 1, 1, 1, 64, 1.0, None, 0, None) == -1
    assert lib.bsp_paged_append(None, 1, r, r, r, r, None, None, None, 1, 1, 1, 1, 16, 1, 64, None) == -1
    assert lib.bsp_paged_attention(None, 1, r, r, r, r, None, None, None, None, 1, 1, 1, 1, 16, 1, 1, 64, 1.0, None, 0, None) == -1
    n = ctypes.c_int()
    assert lib.bsp_diag_window_tiles(0, 0, 5, 4, 7, ctypes.byref(n), None, 0) == -1
    assert lib.bsp_diag_window_tiles(0, 0, 0, 4, 9, ctypes.byref(n), None, 0) == -1
    assert lib.bsp_diag_window_queries(0, 0, 4, 4, 1, 7, 1, ctypes.byref(n), ctypes.byref(n)) == -1


def test_family_without_a_handle(lib):
    assert lib.bsp_diag_window_family(None) == -1


def test_wait_limits_grow_with_a_tile(lib):
    """A legal wait takes up to a tile's steps, of about a microsecond; an attempt
    takes tens of cycles (20 ns) at the least."""
    for steps in (1, 16384, 28000, 1 << 20, 1 << 23):
        n = lib.bsp_diag_window_attempts(steps)
        assert n * 20e-9 >= 2 * steps * 1e-6 and n < 2 ** 31
    assert lib.bsp_diag_window_attempts(1 << 40) == 2 ** 31 - 1
    assert lib.bsp_diag_window_wait_limit(None, 1) == -1


def test_status_is_read_behind_the_handles_device(monkeypatch):
    """With another device current, the word is read on the current stream of the
    handle's own device, with that device current."""
    import torch

    cuda1 = torch.device("cuda", 1)
    entered, read = [], []

    class Stream:
        def __init__(self, device):
            self.device = device

    class Using:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            entered.append(self.stream)

        def __exit__(self, *a):
            entered.append(None)

    class Lib:
        @staticmethod
        def bsp_window_status(handle, stream):
            read.append((handle, stream, entered[-1].device))
            return -7

    streams = {0: Stream(torch.device("cuda", 0)), 1: Stream(cuda1)}
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", Using)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: streams[0 if d is None else torch.device(d).index])
    monkeypatch.setattr(bsp, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(bsp, "_stream", lambda s: 1000)
    monkeypatch.setattr(bsp, "lib", lambda: Lib)
    W = object.__new__(bsp.Window)
    W.handle, W.device = 5, cuda1
    try:
        assert bsp.bsp_window_status(W) == -7
        assert read == [(5, 1001, cuda1)] and entered[-1] is None
        with pytest.raises(ValueError):  # another device's stream
            bsp.bsp_window_status(W, streams[0])
    finally:
        W.handle = None
