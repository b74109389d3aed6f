"""How the launches of attention of shared prefixes are shaped, as far as their workspaces tell: a row's partial results
are as many as a join holds, and hold no more than the blocks there are; sizes at their limits are taken."""

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def W():
    from sparse_moe_02_amd.attn import prefix_attn_workspace

    return prefix_attn_workspace


def _splits(W, T, seqs, groups, q, prefix, suffix, H, hk, D):
    """(fewest, most) splits that a workspace of this size can stand for"""
    n, rows = W(T, seqs, groups, q, prefix, suffix, H, hk, D), T * H
    s = n // (rows * (4 * D + 16))
    assert abs(n - s * rows * (4 * D + 16)) < 256, n
    return s


def test_splits(W):
    for T, seqs, groups, q in ((1, 1, 1, 1), (4, 4, 1, 1), (64, 64, 1, 1), (64, 64, 64, 1), (60, 23, 5, 4), (2048, 512, 3, 4)):
        for H, hk, D in ((16, 2, 256), (32, 8, 128), (16, 16, 64), (8, 1, 128)):
            for prefix in (0, 1, 31, 32, 33, 100, 1000, 5000, 16384, 131072, 1 << 20):
                for suffix in (0, 1, 60, 512, 4000, 1 << 20):
                    s = _splits(W, T, seqs, groups, q, prefix, suffix, H, hk, D)
                    blocks = max(1, -(-prefix // 32)) + max(1, -(-suffix // 32) + 1)
                    assert 2 <= s <= min(256, blocks), (T, seqs, groups, H, prefix, suffix, s)


def test_sizes_at_their_limits(W):
    from sparse_moe_02_amd import binding as B

    for seqs, groups in ((65535, 1), (65535, 65535)):
        assert W(8, seqs, groups, 1, 1 << 30, 1 << 30, 64, 64, 64) > 0
    assert W(1 << 17, 65535, 1, 1, 1 << 20, 1 << 20, 8, 1, 64) >= (1 << 20) * 2 * 256
    assert W(0, 1, 1, 1, 100, 100, 8, 1, 64) == 0
    for bad in ((1 << 18, 1, 1, 1, 1, 1, 8, 1, 64), (8, 65535, 1, 1, 1, 1, 128, 128, 64)):
        with pytest.raises(B.MoeError) as e:
            W(*bad)
        assert e.value.status == B.MOE_ERR_TOKENS
