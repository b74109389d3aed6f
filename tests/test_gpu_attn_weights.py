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


# ------------------------------------------------------------------------ long tails in fp16

# The largest weight of a row is at least 2 to this power, so that fp16's smallest numbers (which round
# by at most 2^-25) lie that much further below it.
TILE, RUNS = 11, 15


def _given(c, k, v, q=8.0):
    """Every query is (q, 0, ...), and every sequence's keys are (k, 0, ...); v: [keys][D]."""
    c.q[:] = 0
    c.q[:, :, 0] = q
    for b, length in enumerate(c.total):
        at = c.dev(np.arange(length))
        page = c.dev(c.table[b])[at // c.page].long()
        c.kc[page, at % c.page] = 0
        c.kc[page, at % c.page, :, 0] = c.dev(k[:length]).to(c.kc.dtype)[:, None]
        c.vc[page, at % c.page] = c.dev(v[:length]).to(c.vc.dtype)[:, None]


def _check(c, launch, what, per_top):
    """per_top: keys for each key of the largest weight, at most."""
    from oracle import serve

    kw = {"unsplit": dict(max_kv=1), "split": {}, "runs": dict(max_q=1, max_kv=10 ** 6)}[launch]
    out, lse = (_np(x) for x in c.attn(scale=0.125, **kw))
    ro, rl, mass, _ = serve.paged_attn(_np(c.q), _np(c.kc), _np(c.vc), c.table, c.q_start, c.kv_len, 0.125)
    u = 2.0 ** -11
    # weights are rounded to 16 bits (u), or by 2^-25 below 2^-14; products here are exact, and a score of
    # up to 2^6 is off by 2^-18 as a base-2 exponent
    low = per_top * 2.0 ** -(25 + (RUNS if launch == "runs" else TILE)) * np.abs(_np(c.vc)).max()
    tol = u * np.abs(ro) + (u + 2.0 ** -16) * mass + low
    err = np.abs(out - ro) / tol
    say(f"{what}, {launch}: output error / tolerance {err.max():.3f}, tolerance / mass {(tol / mass).max():.2e}")
    assert (err <= 1.0).all(), what
    # the sum of the weights is taken block by block of 32 keys, one binary32 addition after the other
    # (each off by at most 2^-24 of the sum), which the logarithm takes as it is
    added = -(-max(c.total) // 32) * 2.0 ** -24
    assert (np.abs(lse - rl) <= 2.0 ** -20 * (1 + np.abs(rl)) + 2.0 ** -18 + added).all(), what


@pytest.mark.parametrize("launch", ["unsplit", "split", "runs"])
@pytest.mark.parametrize("every", [32, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tail_behind_a_sink(D, every, launch):
    """Keys of weight 1 whose values are zeros (one of `every`), the others at e^-15 to e^-18: the output
    is the tail's share."""
    n = 1000
    rng = np.random.default_rng(D)
    c = Case([1, 40, 1, 1, 1, 1], [n] * 6, 8, 8, D, "fp16", page=16, seed=D)
    k, v = rng.uniform(-2.0, 1.0, n), 500 * (1 + rng.random((n, D)))
    k[::every], v[::every] = 16.0, 0.0
    _given(c, k, v)
    _check(c, launch, f"tail of {D}, a sink of {every}", every)


@pytest.mark.parametrize("launch", ["unsplit", "split", "runs"])
@pytest.mark.parametrize("rise", [5.0, 20.0, -20.0])
@pytest.mark.parametrize("D", [64, 256])
def test_rising_scores(D, rise, launch):
    """Scores that rise (or fall) evenly along the keys, so that the reference follows in small steps."""
    n = 1000
    rng = np.random.default_rng(7)
    c = Case([1, 40, 1, 1, 1, 1], [n] * 6, 8, 8, D, "fp16", page=16, seed=D)
    _given(c, np.linspace(0, rise, n), 1 + rng.random((n, D)))
    _check(c, launch, f"scores rising by {rise}", n)


@pytest.mark.parametrize("launch", ["unsplit", "split"])
def test_tail_of_a_long_sequence(launch):
    """131072 keys behind one sink, their weights in the subnormal range."""
    n = 131072
    rng = np.random.default_rng(1)
    c = Case([1], [n], 1, 1, 64, "fp16", page=64, seed=1)
    k, v = rng.uniform(-2.5, -1.5, n), 500 * (1 + rng.random((n, 64)))
    k[0], v[0] = 16.0, 0.0
    _given(c, k, v)
    _check(c, launch, "long tail", n)


@pytest.mark.parametrize("launch", ["unsplit", "split", "runs"])
@pytest.mark.parametrize("diff", [17.6, 18.5, 19.2])
def test_sum_of_a_long_tail(diff, launch):
    """Values of 1 are their own mean, whatever their weights: a key at 0 and 131072 at e^-diff, each below
    the last bit of the sum that is divided by, and all of them above a rounding of fp16 (for the largest)."""
    n = 131072
    several = launch == "runs"  # (48 sequences choose equal runs, and the long one's spans several)
    c = Case([1] * (48 if several else 1), [n] + [1] * (47 if several else 0), 1, 1, 64, "fp16", page=64, seed=1)
    k = np.full(n, 16.0 - diff)
    k[0] = 16.0
    _given(c, k, np.ones((n, 64)))
    kw = {"unsplit": dict(max_kv=1), "split": {}, "runs": dict(max_q=1, max_kv=10 ** 6)}[launch]
    out = _np(c.attn(scale=0.125, **kw)[0])
    # weights' roundings are the same above and below; of the two sums, one binary32 addition a block of
    # 32 keys and one for 16, each off by at most 2^-24: 2^-12 and 2^-11
    say(f"e^-{diff} {launch}: {np.abs(out - 1).max() * 2.0 ** 11:.2f} roundings")
    assert (np.abs(out - 1) <= 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -11).all()
