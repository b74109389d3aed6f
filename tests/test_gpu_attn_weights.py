"""Softmax weights of paged attention where their range matters: scores far from zero, and rows with
a dominant key and a long tail.

Tolerances as in ``test_gpu_attn``, with the mass (sum p |v|) of each element."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib, say
from test_gpu_attn import Case, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()


# ------------------------------------------------------------------------ scores far from zero

@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("times", [2 ** 5, 2 ** 9, 2 ** 12])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp16", 128), ("bf16", 256), ("fp16", 64)])
def test_sharp_scores(dtype, D, times, runs):
    """Scores of some 10 to 10^4 standard deviations, of both signs, in both kernels; chunks and decodes."""
    c = Case([1, 40, 1, 3, 1, 1], [700, 90, 33, 300, 1, 64], 8, 8, D, dtype, page=16, seed=D + times)
    c.q = c.q * times
    c.check(*c.attn(max_q=1 if runs else None, max_kv=10 ** 6 if runs else None), f"{dtype} {D} x {times} runs {runs}")


@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,size", [("bf16", 2.0 ** 30), ("bf16", 2.0 ** 50), ("fp16", 2.0 ** 15)])
def test_largest_scores(dtype, size, sign, runs):
    """Scores so large that neighbouring binary32 numbers lie several units apart: a row takes the value of
    its largest key (the scores of two keys differ by far more than a rounding of either, so other keys'
    weights are 0), and its log-sum-exp is that score."""
    D, n = 64, 500
    rng = np.random.default_rng(3)
    c = Case([1, 40, 1, 1, 1, 1], [n, n, 40, 33, 32, 1], 8, 8, D, dtype, page=16, seed=5)
    c.q[:] = 0
    c.q[:, :, 0] = c.dev(sign * size * rng.uniform(1.0, 1.9, (c.T, 8)))
    for b, length in enumerate(c.total):  # of each sequence distinct multiples of size / 512, in any order
        k = c.dev(size * (512 + rng.permutation(512)[:length]) / 512.0)
        if dtype == "bf16":  # 8 bits: several keys share a value, and one alone is the largest
            k = k.clamp(max=size * 1.75)
            k[k == size * 1.75] = size * 1.5
            k[int(rng.integers(length))] = size * 1.75 if sign > 0 else size * 0.5
        at = c.dev(np.arange(length))
        page = c.dev(c.table[b])[at // 16].long()
        c.kc[page, at % 16] = 0
        c.kc[page, at % 16, :, 0] = k.to(c.kc.dtype)[:, None]
    out, lse = (_np(x) for x in c.attn(max_q=1 if runs else None, max_kv=10 ** 6 if runs else None))
    q, kc, vc = _np(c.q), _np(c.kc), _np(c.vc)
    t = 0
    for b, (new, total) in enumerate(zip(c.new, c.total)):
        at = np.arange(total)
        k, v = kc[c.table[b][at // 16], at % 16, :, 0], vc[c.table[b][at // 16], at % 16]
        for i in range(new):
            see = total - new + i + 1
            for h in range(8):
                x = k[:see, h] * sign
                top = x == x.max()
                # (a value seen by several equal keys is their mean, whose sum rounds in binary32)
                want, score = v[:see, h][top].mean(0), q[t, h, 0] * k[:see, h][top][0] * D ** -0.5
                u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
                assert (np.abs(out[t, h] - want) <= u * np.abs(want) + 2.0 ** -16 * np.abs(v[:see, h][top]).mean(0)).all(), (b, i, h)
                assert abs(lse[t, h] - score) <= 2.0 ** -20 * abs(score) + 1e-6 * np.log(top.sum() + 1), (b, i, h)
            t += 1
    say(f"{dtype} {size} {sign} runs {runs}: every row its largest key")
