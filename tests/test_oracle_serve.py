"""Pins for the serving operators' oracle (CPU only): each is checked against something that is not
its own loop -- complex multiplication, a dense softmax, the matrix form of a scan, invariants."""

import numpy as np
import pytest

from oracle import serve


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x, pos, f = rng.standard_normal((5, 3, 16)), np.array([0, 1, 7, 1000, 131071]), 10.0 ** -np.arange(4)
    turn = 1.5 * np.exp(1j * pos[:, None, None] * f)
    half = serve.rope(x, pos, f, 1.5)
    z = (x[..., :4] + 1j * x[..., 4:8]) * turn
    assert np.allclose(half[..., :4], z.real, atol=1e-12) and np.allclose(half[..., 4:8], z.imag, atol=1e-12)
    both = serve.rope(x, pos, f, 1.5, interleaved=True)
    z = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * turn
    assert np.allclose(both[..., 0:8:2], z.real, atol=1e-12) and np.allclose(both[..., 1:8:2], z.imag, atol=1e-12)
    assert np.array_equal(half[..., 8:], x[..., 8:]) and np.array_equal(both[..., 8:], x[..., 8:])


def test_rotated_products_depend_on_the_distance():
    rng = np.random.default_rng(1)
    q, k, f = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32)), 1e4 ** (-np.arange(16) / 16)
    at = lambda x, p: serve.rope(x, [p], f)[0, 0]
    near = at(q, 40) @ at(k, 33)
    assert abs(at(q, 90007) @ at(k, 90000) - near) < 1e-9 and abs(near - q[0, 0] @ k[0, 0]) > 1e-3


def _cache(rng, lens, page, hk, D, spare=3):
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need) + 1), -1)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return rng.standard_normal((len(order), page, hk, D)), rng.standard_normal((len(order), page, hk, D)), table


def _gather(cache, table, n):
    return np.concatenate([cache[p] for p in table[:-(-n // cache.shape[1])]])[:n]


@pytest.mark.parametrize("window,full", [(0, False), (3, False), (1, False), (0, True)])
def test_attention_is_a_masked_dense_softmax(window, full):
    rng = np.random.default_rng(2)
    lens, new, H, hk, D = [1, 9, 32, 20], [1, 9, 0, 7], 6, 2, 8
    kc, vc, table = _cache(rng, lens, 4, hk, D)
    qs = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((qs[-1] + 2, H, D))
    out, lse, mass, spread = serve.paged_attn(q, kc, vc, table, qs, lens, 0.7, window, full)
    assert np.isnan(out[qs[-1]:]).all()
    for b, (L, n) in enumerate(zip(lens, new)):
        K, V = _gather(kc, table[b], L).repeat(H // hk, 1), _gather(vc, table[b], L).repeat(H // hk, 1)
        s = 0.7 * np.einsum("qhd,khd->hqk", q[qs[b]:qs[b + 1]], K)
        p, j = np.arange(L - n, L)[:, None], np.arange(L)[None]
        see = np.ones((n, L), bool) if full else j <= p
        if window:
            see &= j > p - window
        e = np.where(see, np.exp(s), 0.0)
        assert np.allclose(out[qs[b]:qs[b + 1]], np.einsum("hqk,khd->qhd", e / e.sum(-1, keepdims=True), V), atol=1e-12)
        assert np.allclose(lse[qs[b]:qs[b + 1]], np.log(e.sum(-1)).T, atol=1e-12)
    assert (np.abs(out[:qs[-1]]) <= mass[:qs[-1]] + 1e-12).all()


def test_attention_of_what_sees_nothing_and_of_bad_places():
    rng = np.random.default_rng(3)
    kc, vc, table = _cache(rng, [8, 8], 4, 1, 4)
    q = rng.standard_normal((4, 2, 4))
    # more new tokens than positions: the first two lie before the sequence
    out, lse, _, _ = serve.paged_attn(q, kc, vc, table, [0, 4], [2, 8], 1.0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2], _gather(vc, table[0], 1)[:, 0])
    # a bad page's keys are absent, and a bad row is an empty sequence
    bad = table.copy()
    bad[1, 0] = 1000
    out, _, _, _ = serve.paged_attn(q, kc, vc, bad, [0, 2, 4], [8, 8], 1.0, full=True, row=[1, -1])
    K, V = _gather(kc, table[1], 8)[4:, 0], _gather(vc, table[1], 8)[4:, 0]
    w = np.exp(q[:2] @ K.T)
    assert np.allclose(out[:2], w @ V / w.sum(-1, keepdims=True), atol=1e-12) and (out[2:] == 0).all()


def test_append_fills_the_places_that_attention_reads():
    rng = np.random.default_rng(4)
    lens, new, hk, D, f = [5, 11, 3], [5, 4, 0], 2, 8, np.array([1.0, 0.1])
    kc, vc, table = _cache(rng, lens, 4, hk, D)
    qs = [0, 5, 9, 9]
    q, k, v = (rng.standard_normal((10, h, D)) for h in (4, hk, hk))
    qr, k2, v2 = serve.rope_append(q, k, v, kc, vc, table, qs, lens, f)
    for b, (L, n) in enumerate(zip(lens, new)):
        K, V = _gather(k2, table[b], L), _gather(v2, table[b], L)
        pos = np.arange(L - n, L)
        assert np.array_equal(K[:L - n], _gather(kc, table[b], L)[:L - n])
        assert np.allclose(K[L - n:], serve.rope(k[qs[b]:qs[b + 1]], pos, f), atol=0)
        assert np.array_equal(V[L - n:], v[qs[b]:qs[b + 1]])
    assert np.array_equal(qr[9], q[9])
    assert (k2 != kc).any((1, 2, 3)).sum() == 2 + 2  # pages of five and of the last four of eleven


def test_steps_are_the_scan():
    """Against the scan's oracle, whose pins are its own."""
    import oracle
    import synth

    g = synth.gdn_inputs(0, seed=5, nonzero_state=True)
    ro, rs = oracle.gdn_scan(g.q, g.k, g.v, g.alpha, g.beta, g.state)
    x = [synth.bf16_bits_to_f32(a).astype(np.float64) for a in (g.q, g.k, g.v)]
    T = len(g.alpha)
    out, S = serve.gdn_step(*x, g.alpha, g.beta, np.stack([np.ones_like(g.state), g.state]), [1] * T)
    assert np.allclose(out, ro, rtol=1e-10, atol=1e-10) and np.allclose(S[1], rs, rtol=1e-10, atol=1e-10)
    assert (S[0] == 1).all()
    out, S = serve.gdn_step(*x, g.alpha, g.beta, g.state[None], [-1, 1] * (T // 2) + [7] * (T % 2))
    assert (out == 0).all() and np.array_equal(S[0], g.state)


def _sound(pool):
    """Reference counts are what the tables say; content(s) of every sequence."""
    refs = np.zeros(len(pool.refs), int)
    for s in range(len(pool.lens)):
        held = pool._held(s)
        assert len(set(held)) == len(held)
        np.add.at(refs, held, 1)
    assert np.array_equal(refs, np.maximum(pool.refs, 0))
    return [pool.cache[:, pool._held(s)].copy() for s in range(len(pool.lens))]


def test_pool_keeps_counts_and_contents():
    rng = np.random.default_rng(6)
    pool = serve.Pool(np.zeros((8, 6)), np.zeros(8), np.zeros(30), 4, rng.integers(0, 1 << 30, (2, 30)))
    for _ in range(300):
        before, lens = _sound(pool), pool.lens.copy()
        op = rng.choice(["grow", "fork", "free", "compact"])
        seqs = list(rng.choice(8, rng.integers(1, 4), replace=False))
        if op == "grow":
            # (a shared page that is not full is never held: fork copies it)
            st = pool.grow(seqs, list(rng.integers(0, 6, len(seqs))))
        elif op == "fork":
            empty = [s for s in range(8) if lens[s] == 0][:2]
            st = pool.fork(list(rng.choice(8, len(empty))), empty)
            if not st:
                for d in empty:
                    assert pool.lens[d] % 4 == 0 or pool.refs[pool._held(d)[-1]] == 1
        elif op == "free":
            st = pool.free(seqs)
        else:
            st = pool.compact()
            used = pool.refs > 0
            assert not st and used[:used.sum()].all()
        after = _sound(pool)
        if st:
            assert np.array_equal(lens, pool.lens)
        for s in range(8):  # what a sequence held before stays
            if pool.lens[s] >= lens[s] > 0:
                assert np.array_equal(after[s][:, :before[s].shape[1]], before[s])


def test_pool_refusals():
    def pool():
        return serve.Pool(np.zeros((3, 2)), np.zeros(3), np.zeros(3), 4, np.zeros((1, 3)))

    assert pool().grow([0, 0], [1, 1]) == "shape" and pool().grow([3], [1]) == "shape" and pool().grow([0], [9]) == "shape"
    assert pool().grow([0, 1], [8, 8]) == "alloc" and pool().grow([0], [-1]) == "shape"
    p = pool()
    assert p.grow([0], [5]) == "" and p.fork([0], [0]) == "shape" and p.fork([0, 0], [1, 1]) == "shape"
    assert p.fork([0, 0], [1, 2]) == "alloc" and p.fork([0], [1]) == "" and list(p.refs) == [2, 1, 1]
    assert p.fork([0], [1]) == "shape" and p.free([0, 0]) == "shape" and p.free([0]) == "" and list(p.refs) == [1, 0, 1]
    assert p.compact() == "" and list(p.refs) == [1, 1, 0] and list(p.table[1]) == [0, 1]
