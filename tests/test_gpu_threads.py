"""Calls from a thread that has made no CUDA call before, as autograd's own threads
may be: their tensor maps are encoded with the device's context current."""

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


def in_a_new_thread(call):
    out = []
    t = threading.Thread(target=lambda: out.append(call()))
    t.start()
    t.join()
    torch.cuda.synchronize()
    return out[0]


def randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("backward", [False, True])
def test_windowed_attention(bsp, backward):
    W, lib = bsp.bsp_window_create(50, 2), bsp.lib()
    Q, K, V, dO = (randn(1, H, 200, 64, seed=i) for i, H in enumerate((4, 2, 2, 4)))
    O, lse = bsp.bsp_window_attention(W, Q, K, V, scale=0.1)
    want = bsp.bsp_window_attention_backward(W, Q, K, V, O, dO, lse, scale=0.1) if backward else (O,)
    n = lib.bsp_window_attention_workspace(1, 4, 2, 200, int(backward))
    ws, got = torch.empty(n, dtype=torch.uint8, device="cuda"), [torch.zeros_like(t) for t in want]
    args = [bsp._heads(t) for t in (Q, K, V)]
    outs = [bsp._heads(t) for t in got]
    sizes = (1, 4, 2, 200, 200, 64, 0.1, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    if backward:
        args += [bsp._heads(O), bsp._heads(dO), lse.data_ptr(), *outs]
        rc = in_a_new_thread(lambda: lib.bsp_window_attention_backward(W.handle, 1, *args, *sizes))
    else:
        args += [*outs, None]
        rc = in_a_new_thread(lambda: lib.bsp_window_attention(W.handle, 1, *args, *sizes))
    assert rc == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_trees_over_pages(bsp):
    W, lib = bsp.bsp_window_create(50, 2), bsp.lib()
    K, V, Q = randn(9, 2, 16, 64, seed=1), randn(9, 2, 16, 64, seed=2), randn(5, 4, 64, seed=3)
    starts, kv, table = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 5], [100], [[8, 3, 1, 0, 5, 2, 7]]))
    pos, bits = bsp.bsp_draft_tree(W, starts, kv, torch.tensor([-1, 0, 0, 1, 3], dtype=torch.int32, device="cuda"), 5)
    want, _ = bsp.bsp_paged_tree_attention(W, Q, K, V, starts, kv, table, pos, bits, scale=0.1)
    n = lib.bsp_paged_attention_workspace()
    ws, O = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros_like(Q)
    args = (bsp._rows(Q), bsp._heads(K), bsp._heads(V), bsp._rows(O), None, *(t.data_ptr() for t in (starts, kv, table, pos, bits)),
            5, 1, 7, 9, 16, 4, 2, 64, 1, 0.1, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert in_a_new_thread(lambda: lib.bsp_paged_tree_attention(W.handle, 1, *args)) == 0
    assert torch.equal(O, want)


def test_block_sparse_attention(bsp):
    from sparse_attention_layout_gb300 import workloads
    L, lib = bsp.bsp_layout_compile(workloads.layout_band(8, 2, 2), 64), bsp.lib()
    for dtype, code in ((torch.bfloat16, 1), (torch.float32, 0)):
        Q, K, V = (randn(1, 2, 512, 64, seed=i).to(dtype) for i in range(3))
        want = bsp.bsp_attention(L, Q, K, V, scale=0.1)
        O = torch.zeros_like(Q)
        args = (*(t.data_ptr() for t in (Q, K, V, O)), 1, 64, 0.1, 0, None, torch.cuda.current_stream().cuda_stream)
        assert in_a_new_thread(lambda: lib.bsp_attention(L.handle, code, *args)) == 0
        assert torch.equal(O, want)


def test_others(bsp):
    """The calls without tensor maps."""
    W, lib, R = bsp.bsp_window_create(), bsp.lib(), bsp.bsp_rotary_create(bsp.rotary_frequencies(64)[0])
    Q = randn(1, 2, 70, 64, seed=4)
    want, _ = bsp.bsp_rotary(R, Q)
    got, stream = torch.zeros_like(Q), torch.cuda.current_stream().cuda_stream
    q, o = bsp._heads(Q), bsp._heads(got)
    assert in_a_new_thread(lambda: lib.bsp_rotary(R.handle, 1, q, o, None, None, None, 0, 0, 1, 2, 0, 70, 64, stream)) == 0
    assert torch.equal(got, want)
    starts, kv, parent, pos, bits = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [9], [-1, 0, 0], [0] * 3, [0] * 3))
    ptrs = [t.data_ptr() for t in (starts, kv, parent, pos, bits)]
    assert in_a_new_thread(lambda: lib.bsp_draft_tree(W.handle, *ptrs, 3, 1, 1, stream)) == 0
    assert pos.tolist() == [6, 7, 7] and bits.tolist() == [1, 3, 5]
    assert in_a_new_thread(lambda: lib.bsp_window_status(W.handle, stream)) == 0
