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
