"""Calls as serving programs make them: from two host threads at once, in inference
mode, with pages far into a cache."""

import ctypes
import threading

import pytest
import torch

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


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# (head size, sequences) of two threads whose calls launch the same kernel with
# different amounts of shared memory
@pytest.mark.parametrize("pair", [((112, 1), (80, 1)), ((128, 1), (96, 3)), ((64, 1), (16, 2)), ((16, 16384), (48, 1))], ids=str)
def test_trees_of_two_threads(bsp, pair):
    """Each thread with its own handle, stream, workspace and sizes, over CUDA cores."""
    lib, calls = bsp.lib(), []
    for i, (D, n_seq) in enumerate(pair):
        W, stream = bsp.bsp_window_create(), torch.cuda.Stream()
        K, V, Q = randn(9, 2, 16, D, seed=i), randn(9, 2, 16, D, seed=i + 2), randn(5, 4, D, seed=i + 4)
        starts, kv = ints([0] + [5] * n_seq), ints([100] + [0] * (n_seq - 1))
        table = ints([[8, 3, 1, 0, 5, 2, 7]]).expand(n_seq, 7).contiguous()
        pos, bits = bsp.bsp_draft_tree(W, starts, kv, ints([-1, 0, 0, 1, 3]), 5)
        want, _ = bsp.bsp_paged_tree_attention(W, Q, K, V, starts, kv, table, pos, bits, scale=0.1)
        assert bsp.bsp_window_status(W) == 0
        n = lib.bsp_paged_attention_workspace()
        ws, O = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros_like(Q)
        args = (W.handle, 0, bsp._rows(Q), bsp._heads(K), bsp._heads(V), bsp._rows(O), None,
                *(t.data_ptr() for t in (starts, kv, table, pos, bits)), 5, n_seq, 7, 9, 16, 4, 2, D, 1, 0.1, ws.data_ptr(), n,
                stream.cuda_stream)
        calls.append((args, O, want, (W, K, V, Q, starts, kv, table, pos, bits, ws, stream)))
    torch.cuda.synchronize()
    together, codes = threading.Barrier(2), [[], []]

    def run(i):
        call, args = lib.bsp_paged_tree_attention, calls[i][0]
        together.wait()
        for _ in range(1500):
            codes[i].append(call(*args))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [[x for x in c if x] for c in codes] == [[], []]
    for _, O, want, _ in calls:
        assert torch.equal(O, want)


def test_rotary_positions_in_inference_mode(bsp):
    """Positions made in inference mode, there and, for a gradient, outside of it."""
    R = bsp.bsp_rotary_create(bsp.rotary_frequencies(64)[0])
    Q, K = randn(2, 4, 9, 64, seed=1), randn(2, 2, 9, 64, seed=2)
    rows = torch.randint(0, 5000, (2, 9), dtype=torch.int32).cuda()
    want = bsp.bsp_rotary(R, Q, K, rows)
    leaf = Q.clone().requires_grad_()
    with torch.inference_mode():
        pos = rows.clone()
        inside = Q.clone()
        for q in (Q, leaf, inside):  # (a weight's output, and tensors of the mode)
            got = bsp.rotary(R, q, K, pos)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not got[0].requires_grad
        assert torch.equal(bsp.rotary(R, inside)[0], bsp.bsp_rotary(R, Q)[0])
    with torch.no_grad():
        assert torch.equal(bsp.rotary(R, leaf, None, pos)[0], want[0])
    dQ = randn(2, 4, 9, 64, seed=3)
    back, _ = bsp.bsp_rotary(R, dQ, None, rows, inverse=True)
    q, _ = bsp.rotary(R, leaf, K, pos)
    assert torch.equal(q, want[0])
    with torch.inference_mode():
        pos.zero_()  # the gradient's own positions stay
    assert torch.equal(torch.autograd.grad(q, leaf, dQ)[0], back)
    # positions of no mode that change before the gradient: refused as before
    pos = rows.clone()
    q, _ = bsp.rotary(R, leaf, K, pos)
    pos.zero_()
    with pytest.raises(RuntimeError, match="changed in place"):
        torch.autograd.grad(q, leaf, dQ)


def test_tensor_maps_leave_the_current_context(bsp):
    """A thread that works in a driver context of its own still does after a tensor map
    was encoded there, and one without a context has one afterwards.  (The encoder that
    the tensor-core calls share; nothing is launched in that context.)"""
    cuda, lib = ctypes.CDLL("libcuda.so.1"), bsp.lib()
    encode = lib._ZN3bsp12make_tmap_2dEP14CUtensorMap_stPKvimmjji
    encode.argtypes = [ctypes.c_void_p] * 2 + [ctypes.c_int] + [ctypes.c_uint64] * 2 + [ctypes.c_uint32] * 2 + [ctypes.c_int]
    rows = torch.zeros(256, 64, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    results = {}

    def current():
        c = ctypes.c_void_p()
        assert cuda.cuCtxGetCurrent(ctypes.byref(c)) == 0
        return c.value

    def map_of(base):
        room = ctypes.create_string_buffer(256)
        at = -(-ctypes.addressof(room) // 64) * 64
        return encode(at, base, 1, 256, 64, 128, 64, 128)

    def own():
        dev, ctx, base = ctypes.c_int(), ctypes.c_void_p(), ctypes.c_uint64()
        assert cuda.cuInit(0) == 0 and cuda.cuDeviceGet(ctypes.byref(dev), torch.cuda.current_device()) == 0
        assert cuda.cuCtxCreate_v2(ctypes.byref(ctx), 0, dev) == 0
        try:
            assert cuda.cuMemAlloc_v2(ctypes.byref(base), ctypes.c_size_t(256 * 64 * 2)) == 0
            results["own"] = map_of(base.value), current() == ctx.value, map_of(base.value), current() == ctx.value
            assert cuda.cuCtxSetCurrent(ctx) == 0 and cuda.cuMemFree_v2(base) == 0
        finally:
            cuda.cuCtxDestroy_v2(ctx)

    def none():
        first = current()
        results["none"] = first, map_of(rows.data_ptr()), current()
        assert cuda.cuCtxSetCurrent(None) == 0
        results["again"] = map_of(rows.data_ptr()), current()

    for f in (own, none):
        t = threading.Thread(target=f)
        t.start()
        t.join()
    primary = current()
    assert results["own"] == (0, True, 0, True)
    assert results["none"] == (None, 0, primary) and results["again"] == (0, primary)


def test_kept_rows_behind_32_bit_offsets(bsp):
    """Accepted rows that move within and between pages behind 2^31 elements."""
    n_pages, Hkv, page, D = 16500, 8, 128, 128  # 2.16e9 elements a cache
    K, V = (torch.zeros(n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, n, kv = [3, n_pages - 2, n_pages - 1], 20, 270  # nodes at 250 .. 269, six of them in the second page
    for i, c in enumerate((K, V)):
        for x in table:
            c[x] = randn(Hkv, page, D, seed=10 * i + x % 10, dtype=torch.bfloat16)
    kept = [0, 2, 3, 5, 6, 7, 8, 11, 12, 15, 17, 19]
    want = []
    for c in (K, V):
        rows = torch.cat([c[x] for x in table], 1)  # [Hkv, positions, D]
        rows[:, 250:250 + len(kept)] = rows[:, [250 + x for x in kept]]
        want.append(rows)
    W = bsp.bsp_window_create()
    bsp.bsp_paged_keep(W, K, V, ints([0, n]), ints([kv]), ints([table]), ints(kept + [-1] * (n - len(kept))), ints([len(kept)]))
    assert bsp.bsp_window_status(W) == 0
    for c, rows in zip((K, V), want):
        assert torch.equal(torch.cat([c[x] for x in table], 1), rows)
        assert not bool(c[:3].any()) and not bool(c[4:n_pages - 2].any())
