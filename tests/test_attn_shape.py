"""Which launch paged attention takes, as its workspace shows (no device needed)."""

import os

import pytest


@pytest.fixture(scope="module")
def size():
    torch = pytest.importorskip("torch")
    from sparse_moe_02_amd import binding

    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    from sparse_moe_02_amd.attn import paged_attn_workspace

    def f(n_seqs, heads, max_kv, window=0, max_q=1):
        H, hk, D = heads
        return paged_attn_workspace(n_seqs * max_q, n_seqs, max_q, max_kv, H, hk, D, torch.bfloat16, window)

    return f


@pytest.mark.parametrize("heads", [(16, 2, 256), (32, 8, 128), (16, 16, 64)])
@pytest.mark.parametrize("window", [1, 128, 1000])
def test_a_window_bounds_the_keys_that_shape_the_launch(size, heads, window):
    """A decode of long sequences that see a short window is launched as one of short sequences."""
    for n in (64, 200):
        runs = size(n, heads, 16 * heads[2])
        assert size(n, heads, 16384) == size(n, heads, 131072) == runs  # without a window: equal runs
        assert size(n, heads, 16384, window) == size(n, heads, 131072, window) == size(n, heads, window + 1, window) != runs


@pytest.mark.parametrize("heads", [(16, 2, 256), (32, 8, 128), (16, 16, 64)])
def test_long_windows_take_equal_runs(size, heads):
    runs, D = size(64, heads, 131072), heads[2]
    assert size(64, heads, 131072, 32 * D) == size(64, heads, 32 * D, 131072) == runs
    assert size(64, heads, 131072, 31 * D) != runs
    assert size(64, heads, 32 * D - 1, 131072) != runs
