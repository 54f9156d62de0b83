"""Calls as serving programs make them: from two host threads at once, in inference
mode, with pages far into a cache."""

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
