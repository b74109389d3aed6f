"""Paged attention's launches, each reached on purpose: which one a call takes is read from the bytes of
workspace it asks for.  Tolerances as in ``test_gpu_attn``."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib
from test_gpu_attn import Case, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()


def _bytes(c, max_kv=None, window=0, max_q=None):
    from sparse_moe_02_amd.attn import paged_attn_workspace

    return paged_attn_workspace(c.T, len(c.new), max(c.new) if max_q is None else max_q,
                                max(c.total) if max_kv is None else max_kv, c.H, c.hk, c.D, c.q.dtype, window)


def _takes_runs(c, **kw):
    """Equal runs ask for the same bytes whatever the lengths are."""
    return _bytes(c, **kw) == _bytes(c, max_kv=10 ** 6, max_q=1)


# ------------------------------------------------------- equal runs under a window

@pytest.mark.parametrize("D,window", [(64, 32 * 64), (64, 2500), (128, 32 * 128), (256, 32 * 256)])
def test_runs_under_a_long_window(D, window):
    """Sequences longer than the window, of its length and around, short and empty ones; several tokens."""
    n = 24
    total = [window + 700, window, window + 1, window - 1, 3 * 32 + window] + [1 + 37 * i for i in range(n - 5)]
    new = [1, 1, 1, 2, 9] + [1, 0, 3] * (n // 3)
    c = Case(new[:n], total, 4, 2, D, page=32, seed=D)
    assert _takes_runs(c, window=window, max_kv=10 ** 6, max_q=1)
    out, lse = c.attn(max_q=1, max_kv=10 ** 6, window=window)
    c.check(out, lse, f"runs {D}, window {window}", window=window)


# ------------------------------------------------------------------- splits and their joins

def _splits(c, **kw):
    """Splits of the tile kernel: partial outputs and three numbers (of four) of each row and split."""
    return max(1, round(_bytes(c, **kw) / (c.T * c.H * (4 * c.D + 16))))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("splits", [2, 3, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_joins_of_few_splits(D, splits, dtype):
    """2, 3 and 4 splits of many one-token sequences, short (one split), long, and empty ones between."""
    n = {2: 300 if D == 64 else 200, 3: 200 if D == 64 else 150, 4: 150 if D == 64 else 100}[splits]
    top = 300 if splits == 4 else 900
    rng = np.random.default_rng(splits)
    total = [int(x) for x in rng.integers(1, top + 1, n)]
    total[0], total[1], total[2], total[-1] = top, 32, 33, top - 1
    new = [0 if i % 7 == 5 else 1 for i in range(n)]
    c = Case(new, total, 4, 1, D, dtype, page=16, pad=n - sum(new), seed=D + splits)
    assert _splits(c) == splits
    out, lse = c.attn()
    c.check(out, lse, f"{splits} splits of {D}")
    again = c.attn()
    at = int(c.q_start[-1])
    assert all((x[:at] == y[:at]).all() for x, y in zip((out, lse), again))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx,least", [(8300, 65), (16384, 129), (20011, 193)])
def test_joins_of_many_splits(D, ctx, least):
    """More splits with keys in them than one, two and three lane registers of the join hold."""
    c = Case([1], [ctx], 4, 1, D, "fp16" if D == 128 else "bf16", page=64, seed=ctx)
    assert _splits(c) >= least
    c.check(*c.attn(), f"{_splits(c)} splits of {D}")


def test_joins_of_many_splits_of_several_sequences():
    """The last splits of a short sequence are empty, of a long one full, and one sequence has one block."""
    c = Case([3, 1, 2], [17000, 9000, 20], 8, 2, 128, page=32, seed=51)
    assert _splits(c, max_q=1, max_kv=17000) > 64
    c.check(*c.attn(max_q=1), "uneven splits")


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_are_not_finite_in_partial_results(D, bad, few):
    """Values that some rows of a tile see and others do not, where the tile's keys are split over
    workgroups: the rows that see one get it, in its element alone, and all else stays as it is."""
    n = 100 if few else 3
    new = [40, 1, 1] + [1] * (n - 3)
    total = [900, 777, 20] + [50 + 5 * i for i in range(n - 3)]
    cases = [Case(new, total, 8, 2, D, page=16, seed=61) for _ in range(2)]
    c, ref = cases
    assert 2 <= _splits(c) <= 4 if few else _splits(c) > 4
    # (sequence, key, key/value head, element): seen by some of the first one's rows (its new tokens lie
    # at 860 and behind), by all of them but in a block that not all see whole, in the last block
    # of a split sequence, and of one that is not split
    spots = [(0, 880, 0, 5), (0, 859, 1, D - 1), (0, 899, 0, 0), (1, 770, 1, 17), (2, 19, 0, 33)]
    for s, key, h, e in spots:
        c.vc[c.table[s, key // 16], key % 16, h, e] = bad
        ref.vc[ref.table[s, key // 16], key % 16, h, e] = 1.0
    (out, lse), (ro, rl) = c.attn(), ref.attn()
    o, r = _np(out), _np(ro)
    hit = np.zeros(o.shape, bool)
    for s, key, h, e in spots:
        first = max(0, key - (total[s] - new[s]))  # of the new tokens that see it
        hit[c.q_start[s] + first:c.q_start[s + 1], 4 * h:4 * h + 4, e] = True
    assert hit.sum() == 4 * (20 + 40 + 1 + 1 + 1)
    want = np.broadcast_to(bad, o.shape)
    assert np.array_equal(o[hit], want[hit], equal_nan=True)
    # (beside them the reference's own value of 1 is in the elements that were hit alone)
    assert np.array_equal(o[~hit], r[~hit]) and np.isfinite(r).all()
    assert np.array_equal(_np(lse), _np(rl))
