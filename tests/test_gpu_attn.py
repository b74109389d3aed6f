"""Rotary append and paged attention on the GPU against their plain binary64 forms.

Tolerances, from the arithmetic (u = eps / 2 of the 16-bit type, a rounding to it is off by at
most u relative to the value):
  - rotated elements: one rounding to 16 bits, u |y|; sine and cosine in binary32 from an angle
    whose rest of a turn is rounded to binary32 (at most 2 pi 2^-26) by a routine good to 2 ulp,
    and three binary32 roundings: below 1e-6 m (|a| + |b|).
  - attention: weights rounded to 16 bits (u each), scores off by at most
    d = scale * 2 D 2^-24 * sum |q k| + 2^-22 |score|, so with mass = sum p |v| the output is off
    by at most u |o| + (u + 2 d + 2^-18) mass, plus 2^-25 per key for fp16 weights below its
    normal range (the sum of weights is at least 1).
  - log-sum-exp: d + 2^-20 (1 + |lse|)."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()


def _dt(name):
    import torch

    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    """A ragged batch over a paged cache; layout: how the cache lies in memory."""

    def __init__(self, new, total, H, hk, D, dtype="bf16", page=32, layout="token", pad=0, seed=0, spare=2, fill=None):
        import torch

        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.hk, self.D, self.page = H, hk, D, page
        self.new, self.total = list(new), list(total)
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.q_start[-1]) + pad
        counts = [-(-max(t, 0) // page) for t in total]
        self.n_pages = sum(counts) + spare
        order = rng.permutation(self.n_pages)
        cols = max(counts) + 1
        self.table = np.full((len(new), cols), -1, np.int32)
        at = 0
        for i, c in enumerate(counts):
            self.table[i, :c] = order[at:at + c]
            at += c
        self.kv_len = np.array(total, np.int32)
        dt = _dt(dtype)

        def rnd(*s):
            return torch.randn(s, generator=g, device="cuda").to(dt)

        P = self.n_pages
        if layout == "token":
            kc, vc = rnd(P, page, hk, D), rnd(P, page, hk, D)
        elif layout == "head":
            kc, vc = rnd(P, hk, page, D).transpose(1, 2), rnd(P, hk, page, D).transpose(1, 2)
        else:  # one allocation, keys and values page by page, rows with room behind them
            both = rnd(P, 2, page, hk, D + 16)
            kc, vc = both[:, 0, :, :, :D], both[:, 1, :, :, :D]
        if fill is not None:  # what no sequence holds
            used = torch.zeros((P, page), dtype=torch.bool, device="cuda")
            for i, t in enumerate(total):
                for j in range(t):
                    used[self.table[i, j // page], j % page] = True
            kc[~used] = fill
            vc[~used] = fill
        self.kc, self.vc = kc, vc
        proj = rnd(self.T, H + 2 * hk, D)  # one projection's rows: q, k and v are slices
        self.q, self.k, self.v = proj[:, :H], proj[:, H:H + hk], proj[:, H + hk:]

    def dev(self, a):
        import torch

        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    def args(self):
        return self.dev(self.table), self.dev(self.q_start), self.dev(self.kv_len)

    def attn(self, max_q=None, max_kv=None, q=None, **kw):
        from sparse_moe_02_amd.attn import paged_attn

        return paged_attn(self.q if q is None else q, self.kc, self.vc, *self.args(),
                          max(self.new) if max_q is None else max_q, max(self.total) if max_kv is None else max_kv,
                          return_lse=True, **kw)

    def check(self, out, lse, what, scale=None, window=0, full=False, row=None, table=None, kv_len=None):
        import torch

        from oracle import serve

        scale = self.D ** -0.5 if scale is None else scale
        ro, rl, mass, spread = serve.paged_attn(_np(self.q), _np(self.kc), _np(self.vc),
                                                self.table if table is None else table, self.q_start,
                                                self.kv_len if kv_len is None else kv_len, scale, window, full, row)
        n = int(self.q_start[-1])
        go, gl = _np(out)[:n], _np(lse)[:n]
        ro, rl, mass, spread = ro[:n], rl[:n], mass[:n], spread[:n]
        u = torch.finfo(out.dtype).eps / 2
        d = abs(scale) * 2 * self.D * 2.0 ** -24 * spread + 2.0 ** -22 * np.abs(np.where(np.isfinite(rl), rl, 0))
        tol = u * np.abs(ro) + (u + 2 * d[..., None] + 2.0 ** -18) * mass
        if out.dtype == torch.float16:
            tol = tol + max(self.total) * 2.0 ** -25 * float(np.nanmax(np.abs(_np(self.vc)))) + 2.0 ** -25
        err = np.abs(go - ro) / np.maximum(tol, 1e-30)
        err = np.where((go == ro), 0.0, err)
        say(f"{what}: output error / tolerance {err.max() if err.size else 0:.3f}")
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl)), what
        fin = np.isfinite(rl)
        el = np.abs(gl - rl)[fin] / (d[fin] + 2.0 ** -20 * (1 + np.abs(rl[fin])))
        assert (err <= 1.0).all(), what
        assert (el <= 1.0).all(), (what, el.max())


SHAPES = [(16, 2, 256), (8, 8, 64), (12, 3, 128), (7, 1, 128), (40, 1, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,hk,D", SHAPES)
def test_decode(H, hk, D, dtype):
    c = Case([1] * 5, [1, 31, 32, 33, 500], H, hk, D, dtype, seed=H)
    out, lse = c.attn()
    c.check(out, lse, f"decode {H}/{hk}/{D} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,hk,D", SHAPES)
def test_ragged_chunks(H, hk, D, dtype):
    c = Case([3, 0, 17, 1, 70, 33], [3, 40, 17, 129, 200, 64], H, hk, D, dtype, page=16, pad=5, seed=D + H)
    q0 = _np(c.q)
    import torch

    out = torch.full((c.T, H, D), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((c.T, H), 7.0, device="cuda")
    c.attn(out=out, lse=lse)
    c.check(out, lse, f"ragged {H}/{hk}/{D} {dtype}")
    assert (out[-5:] == 7).all() and (lse[-5:] == 7).all()  # padding tokens are left as they were
    assert np.array_equal(q0, _np(c.q))


@pytest.mark.parametrize("window", [1, 16, 33, 100])
@pytest.mark.parametrize("D", [64, 256])
def test_window(window, D):
    c = Case([1, 40, 9], [300, 90, 9], 8, 2, D, page=16, seed=window)
    c.check(*c.attn(window=window), f"window {window}", window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_full(D):
    c = Case([5, 40, 1], [5, 100, 77], 8, 2, D, page=64, seed=D)
    c.check(*c.attn(full=True), "full", full=True)


@pytest.mark.parametrize("layout", ["head", "pairs"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_layouts(layout, page):
    c = Case([1, 37, 4], [290, 60, 5], 12, 4, 128, page=page, layout=layout, seed=page)
    c.check(*c.attn(), f"layout {layout} page {page}")


@pytest.mark.parametrize("scale", [0.0, 0.5, -0.2, 3.0, 1e-38, -1e-44])
def test_scale(scale):
    c = Case([1, 20], [100, 20], 4, 2, 64, seed=3)
    c.check(*c.attn(scale=scale), f"scale {scale}", scale=scale)


@pytest.mark.parametrize("H,hk,D", [(16, 2, 256), (4, 4, 64), (64, 2, 128)])
def test_long_chunk(H, hk, D):
    """Several hundred rows per sequence: every tile shape, against lengths that end anywhere."""
    c = Case([150, 333, 1, 64], [150, 700, 411, 1000], H, hk, D, page=32, seed=9)
    c.check(*c.attn(), f"long chunk {H}/{hk}/{D}")


@pytest.mark.parametrize("bounds", [(0, 0), (1, 1), (10 ** 6, 10 ** 6), (4, 100000)])
def test_bounds_shape_the_launch_only(bounds):
    c = Case([1, 4, 2], [900, 300, 2], 16, 2, 256, seed=4)
    c.check(*c.attn(max_q=bounds[0], max_kv=bounds[1]), f"bounds {bounds}")


def test_rows_that_see_nothing():
    """Empty sequences, and more new tokens than positions."""
    c = Case([2, 6, 1, 3], [0, 4, 0, 3], 8, 2, 128, page=16, seed=5)
    out, lse = c.attn()
    c.check(out, lse, "nothing visible")
    assert (out[:2] == 0).all() and (out[2:4] == 0).all() and (out[8] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_unseen_places_have_no_influence(bad, D):
    """NaN and infinities in free pages, behind the lengths, and at later positions."""
    c = Case([1, 20, 45], [77, 20, 131], 8, 2, D, page=32, seed=6, fill=bad)
    c.check(*c.attn(), f"fill {bad}")
    # positions 100.. of the last sequence (new tokens from 86 on) are bad: queries before see none
    for p in (100, 117):
        c.kc[c.table[2, p // 32], p % 32] = bad
        c.vc[c.table[2, p // 32], p % 32] = bad
    ref = Case([1, 20, 45], [77, 20, 131], 8, 2, D, page=32, seed=6, fill=0.0)
    out, lse = c.attn()
    ro, rl = ref.attn()
    t = 21 + (100 - 86)
    assert np.array_equal(_np(out)[:t], _np(ro)[:t]) and np.array_equal(_np(lse)[:t], _np(rl)[:t])
    assert not np.isfinite(_np(out)[t:]).all()
    # with a window that has passed them, later queries are free of them again
    out, lse = c.attn(window=8)
    ro, rl = ref.attn(window=8)
    ok = [i for i in range(45) if not any(86 + i - 8 < p <= 86 + i for p in (100, 117))]
    o, r = _np(out)[21:][ok], _np(ro)[21:][ok]
    assert np.array_equal(o, r)


def test_values_of_infinity_that_are_seen():
    c = Case([1, 3], [50, 40], 4, 2, 64, seed=8)
    c.vc[c.table[0, 0], 3, 0, 5] = float("inf")
    out, _ = c.attn()
    o = _np(out)
    assert np.isposinf(o[0, :2, 5]).all()
    o[0, :2, 5] = 0
    assert np.isfinite(o).all()


def test_bad_rows_pages_and_lengths():
    """Row and page numbers outside their arrays count as absent; lengths are cut at the table."""
    import torch

    from sparse_moe_02_amd.attn import paged_attn

    c = Case([1, 5, 2, 1], [100, 70, 64, 90], 8, 2, 128, page=16, seed=11)
    table, kv = c.table.copy(), c.kv_len.copy()
    table[0, 2], table[1, 0], table[1, 4] = c.n_pages, -7, 2 ** 31 - 1
    kv[3] = 10 ** 6
    row = np.array([2, 1, 0, 3], np.int32)
    for r in (row, np.array([2, 9, -1, 3], np.int32)):
        out, lse = paged_attn(c.q, c.kc, c.vc, c.dev(table), c.dev(c.q_start), c.dev(kv), 5, 128, row=c.dev(r),
                              return_lse=True)
        torch.cuda.synchronize()
        c.check(out, lse, f"bad rows {r}", row=r, table=table, kv_len=kv)


def test_one_split_and_many_agree():
    """The same batch in launches of different shape, each against the definition, and repeatable."""
    c = Case([1, 1], [2000, 37], 16, 2, 256, seed=12)
    for mk in (1, 128, 2000, 10 ** 6):
        a, b = c.attn(max_kv=mk), c.attn(max_kv=mk)
        assert all((x == y).all() for x, y in zip(a, b))
        c.check(*a, f"max_kv {mk}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx", [150, 190, 700, 2200, 5000])
def test_splits_of_every_number(D, ctx):
    """One token over one sequence: one launch, joins of few splits, of one round and of more."""
    c = Case([1], [ctx], 4, 1, D, seed=21)
    c.check(*c.attn(), f"{D} over {ctx}")


def test_places_beyond_32_bits():
    """Pages whose elements lie beyond 2^32 bytes and 2^32 elements of a plane's start."""
    import torch

    from sparse_moe_02_amd.attn import paged_attn, rope_append, rope_freqs

    c = Case([1, 20], [100, 20], 16, 2, 256, page=32, seed=13)
    n = (2 ** 32 // (32 * 2 * 256)) + c.n_pages + 4
    far = n - c.n_pages
    big_k = torch.empty((n, 32, 2, 256), dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty((n, 32, 2, 256), dtype=torch.bfloat16, device="cuda")
    big_k[far:], big_v[far:] = c.kc, c.vc
    table = np.where(c.table >= 0, c.table + far, -1).astype(np.int32)
    out, lse = paged_attn(c.q, big_k, big_v, c.dev(table), c.dev(c.q_start), c.dev(c.kv_len), 20, 100, return_lse=True)
    c.check(out, lse, "far pages")
    f, m = rope_freqs(64, device="cuda")
    q = rope_append(c.q, c.k, c.v, big_k, big_v, c.dev(table), c.dev(c.q_start), c.dev(c.kv_len), f, mscale=m)
    q2 = rope_append(c.q, c.k, c.v, c.kc, c.vc, *c.args(), f, mscale=m)
    assert (q == q2).all() and (big_k[far:] == c.kc).all() and (big_v[far:] == c.vc).all()


@pytest.mark.parametrize("n,window", [(2, 0), (17, 0), (64, 0), (64, 50), (65, 0), (130, 40)])
def test_tiles_of_many_uneven_sequences(n, window):
    """Sequences with and without new tokens, long and short, up to and above a wave's lanes."""
    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.integers(0, 40, n)]
    new[0], new[-1] = 90, 0
    lens = [a + int(x) for a, x in zip(new, rng.integers(0, 2, n) * rng.integers(0, 500, n))]
    c = Case(new, lens, 8, 2, 64, seed=n)
    c.check(*c.attn(window=window), f"{n} sequences, window {window}", window=window)


def test_calls_on_two_streams_at_once():
    """Two batches attended to at the same time, each many times, against each alone."""
    import torch

    cs = [Case([1] * 6, [900, 31, 32, 33, 500, 77], 16, 2, 256, seed=41), Case([64, 200], [64, 900], 8, 2, 128, seed=42)]
    alone = [c.attn() for c in cs]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in st:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cs, st)):
            with torch.cuda.stream(s):
                got[i].append(c.attn())
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all((o == alone[i][0]).all() and (m == alone[i][1]).all() for o, m in got[i])


def test_one_workspace_for_two_graphs():
    """Two captured calls of different shape share a workspace, replayed in turn on one stream."""
    import torch

    from sparse_moe_02_amd.attn import paged_attn_workspace

    cs = [Case([1, 1], [2000, 700], 16, 2, 256, seed=43), Case([40, 3], [900, 60], 16, 2, 256, seed=44)]
    n = max(paged_attn_workspace(c.T, 2, max(c.new), max(c.total), 16, 2, 256) for c in cs)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    eager = [c.attn() for c in cs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        args = c.args()
        from sparse_moe_02_amd.attn import paged_attn

        with torch.cuda.graph(g, stream=st):
            outs.append(paged_attn(c.q, c.kc, c.vc, *args, max(c.new), max(c.total), return_lse=True, workspace=ws))
        graphs.append((g, args))
    for _ in range(4):
        for i in (0, 1):
            graphs[i][0].replay()
            torch.cuda.synchronize()
            assert (outs[i][0] == eager[i][0]).all() and (outs[i][1] == eager[i][1]).all()
        ws.random_()


def test_graph_replays_follow_the_lengths():
    """A captured step is replayed with other lengths, tables and queries, on a stream of its own,
    with eager calls and synchronisations between the replays."""
    import torch

    from sparse_moe_02_amd.attn import paged_attn, rope_append, rope_freqs

    c = Case([1] * 4, [400, 300, 200, 100], 16, 2, 256, seed=14)
    table, qs, kv = c.args()
    q, k, v = c.q.clone(), c.k.clone(), c.v.clone()
    f, m = rope_freqs(64, 1e6, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def step():
        r = rope_append(q, k, v, c.kc, c.vc, table, qs, kv, f, mscale=m)
        return paged_attn(r, c.kc, c.vc, table, qs, kv, 1, 400, return_lse=True)

    with torch.cuda.stream(st):
        step()
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        go, gl = step()
    for i in range(4):
        kv.copy_(torch.tensor([400 - 90 * i, 5 + i, 200, 100 - 3 * i], dtype=torch.int32))
        q.copy_(torch.randn_like(q, dtype=torch.float32))
        torch.cuda.synchronize()
        eo, el = (x.clone() for x in step())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert (go == eo).all() and (gl == el).all(), i


# ------------------------------------------------- few rows over many long sequences (equal runs)
# (bounds of one token and 10^6 keys, with 48 or more sequences x key/value heads, choose that
# launch whatever the lengths are)

def _runs(c, **kw):
    assert len(c.new) * c.hk >= 48
    return c.attn(max_q=1, max_kv=10 ** 6, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,hk,D", [(16, 8, 256), (24, 12, 64), (48, 16, 128), (16, 16, 256)])
def test_runs_decode(H, hk, D, dtype):
    c = Case([1] * 6, [1, 31, 32, 33, 500, 1300], H, hk, D, dtype, page=16, seed=H)
    a, b = _runs(c), _runs(c)
    c.check(*a, f"runs {H}/{hk}/{D} {dtype}")
    assert all((x == y).all() for x, y in zip(a, b))


@pytest.mark.parametrize("window", [0, 1, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_runs_ragged(D, window):
    """Several tokens, several tiles of rows a sequence (more than the bound says), sequences
    without tokens or keys, padding."""
    c = Case([3, 0, 40, 1, 0, 0, 5, 2], [3, 40, 41, 129, 0, 7, 700, 1], 32, 8, D, page=32, pad=3, seed=D + window)
    c.check(*_runs(c, window=window), f"runs ragged {D} {window}", window=window)


def test_runs_full_and_negative_scale():
    c = Case([2, 3, 1, 9, 1, 1], [200, 3, 100, 65, 31, 33], 16, 8, 128, page=16, layout="head", seed=31)
    c.check(*_runs(c, full=True), "runs full", full=True)
    for scale in (0.0, -0.3):
        c.check(*_runs(c, scale=scale), f"runs scale {scale}", scale=scale)


@pytest.mark.parametrize("n", [63, 64, 65, 300])
def test_runs_over_many_sequences(n):
    """More sequences than a wave has lanes, most of them short, some empty."""
    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.integers(0, 3, n)]
    total = [a + int(x) for a, x in zip(new, rng.integers(0, 90, n))]
    total[n // 2] += 900
    c = Case(new, total, 4, 2, 64, page=16, layout="pairs", seed=n)
    row = rng.permutation(n).astype(np.int32)
    # rows in another order: lengths and new tokens no longer match, so some tokens see nothing
    out, lse = _runs(c, row=c.dev(row))
    c.check(out, lse, f"runs over {n}", row=row)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 256])
def test_runs_unseen_places(bad, D):
    new, total = [1, 20, 45, 1, 1, 1], [77, 20, 131, 64, 33, 1]
    c = Case(new, total, 16, 8, D, page=32, seed=6, fill=bad)
    c.check(*_runs(c), f"runs fill {bad}")
    ref = Case(new, total, 16, 8, D, page=32, seed=6, fill=0.0)
    for p in (100, 117):
        c.kc[c.table[2, p // 32], p % 32] = bad
        c.vc[c.table[2, p // 32], p % 32] = bad
    (out, lse), (ro, rl) = _runs(c), _runs(ref)
    t = 21 + (100 - 86)
    assert np.array_equal(_np(out)[:t], _np(ro)[:t]) and np.array_equal(_np(lse)[:t], _np(rl)[:t])
    assert not np.isfinite(_np(out)[t:66]).all()
    assert np.array_equal(_np(out)[66:], _np(ro)[66:])


def test_runs_bad_rows_and_pages():
    c = Case([1, 5, 2, 1, 1, 1], [100, 70, 64, 90, 600, 30], 16, 8, 128, page=16, seed=11)
    table, kv = c.table.copy(), c.kv_len.copy()
    table[0, 2], table[1, 0], table[1, 4], table[4, 7] = c.n_pages, -7, 2 ** 31 - 1, -1
    kv[3] = 10 ** 6
    row = np.array([2, 9, -1, 3, 4, 0], np.int32)
    from sparse_moe_02_amd.attn import paged_attn

    out, lse = paged_attn(c.q, c.kc, c.vc, c.dev(table), c.dev(c.q_start), c.dev(kv), 1, 10 ** 6, row=c.dev(row),
                          return_lse=True)
    c.check(out, lse, "runs bad rows", row=row, table=table, kv_len=kv)


def test_runs_values_of_infinity_that_are_seen():
    c = Case([1] * 6, [50, 400, 40, 33, 64, 1], 16, 8, 64, seed=8)
    c.vc[c.table[1, 4], 3, 0, 5] = float("inf")
    c.vc[c.table[1, 4], 4, 7, 6] = float("nan")
    o = _np(_runs(c)[0])
    assert np.isposinf(o[1, :2, 5]).all() and np.isnan(o[1, 14:, 6]).all()
    o[1, :2, 5] = o[1, 14:, 6] = 0
    assert np.isfinite(o).all()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 64)])
def test_bad_page_beside_values_that_are_not_finite(D, page):
    """A block of keys with one half in a bad page and a NaN that is seen in the other half."""
    for runs in (False, True):
        c = Case([1, 1, 1, 1, 1, 1], [200] * 6, 16, 8, D, page=16, seed=page)
        table = c.table.copy()
        table[0, 3] = -1                                 # keys 48 .. 63
        c.vc[table[0, 2], 5, 0, 7] = float("nan")        # key 37
        from sparse_moe_02_amd.attn import paged_attn

        out = _np(paged_attn(c.q, c.kc, c.vc, c.dev(table), c.dev(c.q_start), c.dev(c.kv_len), 1, 10 ** 6 if runs else 1))
        assert np.isnan(out[0, :2, 7]).all()
        out[0, :2, 7] = 0
        assert np.isfinite(out).all(), runs


# ------------------------------------------------------------------------ rotary append

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 64), (256, 256), (64, 54), (128, 118), (128, 2), (64, 0)])
def test_rope_append(D, rot, interleaved, dtype):
    import torch

    from oracle import serve
    from sparse_moe_02_amd.attn import rope_append, rope_freqs

    c = Case([3, 0, 20, 1, 2], [3, 9, 500, 129, 1], 5, 3, D, dtype, page=16, layout="head", pad=2, seed=rot + D)
    f, m = (None, 1.3) if rot == 0 else rope_freqs(rot, 1e4, "yarn", 4.0, 64, device="cuda")
    fr = np.zeros(0) if f is None else f.cpu().numpy()
    q, k, v = _np(c.q), _np(c.k), _np(c.v)
    rq, rk, rv = serve.rope_append(q, k, v, _np(c.kc), _np(c.vc), c.table, c.q_start, c.kv_len, fr, m, interleaved)
    out = torch.full((c.T, 5, D), 9.0, dtype=c.q.dtype, device="cuda")
    rope_append(c.q, c.k, c.v, c.kc, c.vc, *c.args(), f, mscale=m, interleaved=interleaved, q_out=out)
    u = torch.finfo(c.q.dtype).eps / 2
    n = int(c.q_start[-1])
    assert (out[n:] == 9).all()
    big = 1e-6 * m * 2 * max(np.abs(q).max(), np.abs(k).max())
    for got, ref, what in ((_np(out)[:n], rq[:n], "q"), (_np(c.kc), rk, "k"), (_np(c.vc), rv, "v")):
        err = np.abs(got - ref) - u * np.abs(ref)
        # fp16 below its normal range rounds by half of 2^-24
        assert (err <= (0 if what == "v" else big + 2.0 ** -25)).all(), (what, err.max())
    assert np.array_equal(_np(out)[:n, :, rot:], q[:n, :, rot:])  # the rest of the head passes unchanged
    assert np.array_equal(_np(c.vc), rv)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 200])
@pytest.mark.parametrize("most", [2, 40])
def test_rope_append_of_many_sequences(n, most):
    """Up to and above a wave's lanes, with empty sequences first, last and between, and padding."""
    import torch

    from oracle import serve
    from sparse_moe_02_amd.attn import rope_append, rope_freqs

    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.integers(0, most, n)]
    new[0], new[n // 2] = (0 if n > 1 else 3), 3
    c = Case(new, [x + int(y) for x, y in zip(new, rng.integers(0, 60, n))], 4, 2, 64, page=16, pad=3, seed=n + most)
    f, m = rope_freqs(64, device="cuda")
    row = rng.permutation(n).astype(np.int32)  # so lengths may be less than the new tokens: places before the sequence
    q, k, v = _np(c.q), _np(c.k), _np(c.v)
    rq, rk, rv = serve.rope_append(q, k, v, _np(c.kc), _np(c.vc), c.table, c.q_start, c.kv_len, f.cpu().numpy(), m, row=row)
    out = torch.full_like(c.q, 9.0)
    rope_append(c.q, c.k, c.v, c.kc, c.vc, *c.args(), f, mscale=m, row=c.dev(row), q_out=out)
    end = int(c.q_start[-1])
    u, big = 2.0 ** -8, 2e-6 * max(np.abs(q).max(), np.abs(k).max())
    assert (out[end:] == 9).all() and np.array_equal(_np(c.vc), rv)
    assert (np.abs(_np(out)[:end] - rq[:end]) <= u * np.abs(rq[:end]) + big).all()
    assert (np.abs(_np(c.kc) - rk) <= u * np.abs(rk) + big).all()


def test_rope_in_place_positions_and_rows():
    """q_out = q inside one projection's rows, given positions far out, rows in another order."""
    import torch

    from oracle import serve
    from sparse_moe_02_amd.attn import rope_append, rope_freqs

    c = Case([2, 4, 1], [50, 4, 33], 8, 2, 128, page=16, seed=21)
    f, m = rope_freqs(128, 1e6, "ntk", 8.0, device="cuda")
    pos = np.array([0, 1, 2 ** 31 - 1, 131071, -5, 10 ** 6, 7], np.int32)
    row = np.array([2, 0, 1], np.int32)
    q, k, v = _np(c.q), _np(c.k), _np(c.v)
    rq, rk, rv = serve.rope_append(q, k, v, _np(c.kc), _np(c.vc), c.table, c.q_start, c.kv_len, f.cpu().numpy(), m,
                                   pos=pos, row=row)
    back = rope_append(c.q, c.k, c.v, c.kc, c.vc, *c.args(), f, mscale=m, pos=c.dev(pos), row=c.dev(row), q_out=c.q)
    assert back.data_ptr() == c.q.data_ptr()
    u = torch.finfo(c.q.dtype).eps / 2
    # a position of 2^31 keeps its turn to 2^31 2^-53 2 turns in binary64: no part of the bound
    big = 2e-6 * max(np.abs(q).max(), np.abs(k).max())
    assert (np.abs(_np(c.q) - rq) <= u * np.abs(rq) + big).all()
    assert (np.abs(_np(c.kc) - rk) <= u * np.abs(rk) + big).all()
    assert np.array_equal(_np(c.vc), rv) and np.array_equal(_np(c.k), k)


def test_rope_append_skips_bad_places():
    from oracle import serve
    from sparse_moe_02_amd.attn import rope_append, rope_freqs

    c = Case([6, 3, 2], [4, 40, 17], 4, 2, 64, page=16, seed=22)  # the first sequence has negative positions
    table, kv = c.table.copy(), c.kv_len.copy()
    table[1, 2] = c.n_pages
    kv[2] = 1000
    f, m = rope_freqs(64, device="cuda")
    ref = serve.rope_append(_np(c.q), _np(c.k), _np(c.v), _np(c.kc), _np(c.vc), table, c.q_start, kv, f.cpu().numpy())
    rope_append(c.q, c.k, c.v, c.kc, c.vc, c.dev(table), c.dev(c.q_start), c.dev(kv), f, mscale=m)
    assert np.array_equal(_np(c.vc), ref[2])
    assert (np.abs(_np(c.kc) - ref[1]) <= 2.0 ** -8 * np.abs(ref[1]) + 1e-5).all()


def test_rope_values_that_are_not_finite_stay_in_their_pair():
    from sparse_moe_02_amd.attn import rope_append, rope_freqs

    c = Case([2], [2], 2, 1, 64, page=16, seed=23)
    c.q[0, 0, 3] = float("nan")
    c.q[1, 1, 60] = float("inf")
    f, m = rope_freqs(32, device="cuda")
    out = _np(rope_append(c.q, c.k, c.v, c.kc, c.vc, *c.args(), f, mscale=m))
    bad = np.argwhere(~np.isfinite(out)).tolist()
    assert bad == [[0, 0, 3], [0, 0, 19], [1, 1, 60]]
