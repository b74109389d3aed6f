"""Attention of sequences that share prefixes (moe_prefix_attn) against its binary64 form.

Tolerances as for paged attention (u = eps / 2 of the 16-bit type): weights rounded to 16 bits, scores off by
at most d = scale * 2 D 2^-24 * sum |q k| + 2^-22 |score|, so with mass = sum p |v| an output is off by
at most u |o| + (u + 2 d + 2^-18) mass, plus 2^-25 per key for fp16 weights below its normal range; the
log-sum-exp by d + 2^-20 (1 + |lse|)."""

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


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    """groups: a list of (prefix length, [(new tokens, length behind the prefix), ...])."""

    def __init__(self, groups, H, hk, D, dtype="bf16", page=32, pad=0, seed=0, layout="token"):
        import torch

        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.hk, self.D, self.page = H, hk, D, page
        self.prefix = [p for p, _ in groups]
        self.new = [n for _, s in groups for n, _ in s]
        self.total = [p + t for p, s in groups for _, t in s]
        self.suffix = [t for _, s in groups for _, t in s]
        self.group_start = np.concatenate([[0], np.cumsum([len(s) for _, s in groups])]).astype(np.int32)
        self.q_start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.q_start[-1]) + pad
        cols = max(-(-t // page) for t in self.total) + 1
        rows, at = [], 0
        for p, s in groups:
            shared = list(range(at, at + p // page))
            at += len(shared)
            for _, t in s:
                more = -(-(p + t) // page) - len(shared)
                rows.append(shared + list(range(at, at + more)))
                at += more
        self.n_pages = at + 2
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(rows), cols), -1, np.int32)
        for i, r in enumerate(rows):
            self.table[i, :len(r)] = order[r]
        self.kv_len = np.array(self.total, np.int32)
        dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
        if layout == "token":
            self.kc, self.vc = rnd(self.n_pages, page, hk, D), rnd(self.n_pages, page, hk, D)
        else:
            self.kc, self.vc = (rnd(self.n_pages, hk, page, D).transpose(1, 2) for _ in range(2))
        for i, p in enumerate(self.prefix):  # the prefix's rest, in pages of each sequence's own
            if p % page:
                b0, b1 = self.group_start[i], self.group_start[i + 1]
                mine = self.table[b0:b1, p // page]
                for c in (self.kc, self.vc):
                    for m in mine[1:]:
                        c[int(m), :p % page] = c[int(mine[0]), :p % page]
        self.q = rnd(self.T, H + 3, D)[:, 1:H + 1]

    def dev(self, a):
        import torch

        return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()

    def args(self):
        return [self.dev(x) for x in (self.table, self.q_start, self.kv_len, self.group_start, self.prefix)]

    def run(self, most=None, **kw):
        from sparse_moe_02_amd.attn import prefix_attn

        most = (max(self.new), max(self.prefix), max(self.suffix)) if most is None else most
        return prefix_attn(self.q, self.kc, self.vc, *self.args(), *most, return_lse=True, **kw)

    def check(self, what="", most=None, scale=None, full=False, row=None, **kw):
        import torch

        from oracle import step

        out, lse = self.run(most, scale=scale, full=full, row=None if row is None else self.dev(row), **kw)
        s = self.D ** -0.5 if scale is None else scale
        ro, rl, mass, spread = step.prefix_attn(_np(self.q), _np(self.kc), _np(self.vc), self.table, self.q_start, self.kv_len,
                                                self.group_start, self.prefix, s, full, row)
        n = int(self.q_start[-1])
        go, gl = _np(out)[:n], _np(lse)[:n]
        ro, rl, mass, spread = ro[:n], rl[:n], mass[:n], spread[:n]
        u = torch.finfo(out.dtype).eps / 2
        d = abs(s) * 2 * self.D * 2.0 ** -24 * spread + 2.0 ** -22 * np.abs(np.where(np.isfinite(rl), rl, 0))
        tol = u * np.abs(ro) + (u + 2 * d[..., None] + 2.0 ** -18) * mass
        if out.dtype == torch.float16:
            tol = tol + max(self.total) * 2.0 ** -25 * float(np.nanmax(np.abs(_np(self.vc)))) + 2.0 ** -25
        err = np.where(go == ro, 0.0, np.abs(go - ro) / np.maximum(tol, 1e-30))
        say(f"{what}: output error / tolerance {err.max() if err.size else 0:.3f}")
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl)) and (err <= 1).all(), what
        fin = np.isfinite(rl)
        assert (np.abs(gl[fin] - rl[fin]) <= d[fin] + 2.0 ** -20 * (1 + np.abs(rl[fin]))).all(), what
        return out, lse


SHAPES = [(16, 2, 256), (8, 8, 64), (12, 3, 128), (7, 1, 128), (40, 1, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,hk,D", SHAPES)
def test_one_group(H, hk, D, dtype):
    for prefix in (0, 1, 31, 32, 33, 64, 500):
        Case([(prefix, [(1, 1), (1, 30), (1, 32), (1, 33), (1, 90)])], H, hk, D, dtype, seed=prefix).check(f"{H}/{hk}/{D} behind {prefix}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,hk,D", SHAPES)
def test_groups_drafts_and_empty_sequences(H, hk, D, dtype):
    groups = [(100, [(3, 3), (0, 5), (1, 70)]), (0, [(2, 9)]), (257, [(0, 0), (0, 1)]), (64, [(4, 4)]), (15, [(1, 1)] * 9)]
    for layout, page in (("token", 16), ("head", 64)):
        c = Case(groups, H, hk, D, dtype, page=page, pad=3, seed=D, layout=layout)
        c.check(f"{H}/{hk}/{D} {layout}")
        c.check("full", full=True)


@pytest.mark.parametrize("n,q", [(1, 1), (33, 1), (64, 2), (65, 1), (150, 1), (70, 3), (200, 1)])
def test_many_sequences(n, q):
    """One tile and several of a prefix, up to and above a wave's lanes; one group and one a sequence."""
    rng = np.random.default_rng(n)
    seqs = [(int(rng.integers(0, q + 1)) if q > 1 else 1, int(rng.integers(q, 50))) for _ in range(n)]
    Case([(130, seqs)], 4, 2, 64, page=16, seed=n).check(f"{n} in one group")
    Case([(int(rng.integers(0, 70)), [s]) for s in seqs], 4, 2, 64, page=16, seed=n).check(f"{n} alone")
    Case([(77, [(1, 3)] * 24), (40, [(2, 40)] * 17)], 16, 2, 128, page=16, seed=n).check("two groups")


def test_bounds_shape_the_launch_only():
    c = Case([(700, [(1, 40), (2, 300)]), (90, [(1, 1), (3, 11)])], 16, 2, 128, seed=5)
    for most in ((0, 0, 0), (1, 1, 1), (3, 10 ** 6, 5), (3, 100, 10 ** 6), (10 ** 6, 700, 300), (3, 0, 300), (3, 700, 0), (2, 128, 64)):
        c.check(f"bounds {most}", most=most)


def test_long_prefix_many_splits():
    Case([(9000, [(1, 5), (1, 200)])], 8, 1, 64, seed=6).check("9000")
    Case([(40000, [(1, 9)] * 3)], 2, 1, 64, seed=7).check("40000")


def test_rows_scales_and_lengths_that_do_not_fit():
    c = Case([(50, [(1, 20), (2, 5), (1, 1)]), (20, [(1, 7), (1, 2)])], 8, 2, 128, page=16, seed=8)
    c.check("rows in another order", row=np.array([2, 0, 1, 4, 3]))
    c.check("rows outside", row=np.array([0, -1, 2, 7, 3]))       # a sequence; a group's first one
    c.check("negative scale", scale=-0.3)
    c.check("scale 0", scale=0.0)
    c.check("large scale", scale=1e4)
    c.kv_len = c.kv_len.copy()
    c.kv_len[0], c.kv_len[1], c.kv_len[3] = 10 ** 6, 30, -5           # behind the table; inside the prefix; negative
    c.check("lengths")
    c.prefix = [10 ** 6, -3]
    c.check("prefixes")


def test_bad_pages_and_values_that_are_not_seen():
    import torch

    c = Case([(70, [(1, 20), (1, 60)]), (33, [(2, 9)])], 8, 2, 128, page=16, seed=9)
    want, lw = c.run()
    for i, t in enumerate(c.total):  # what lies behind the sequences, and the second sequence's own copy of the prefix's rest
        c.kc[int(c.table[i, t // 16]), t % 16:] = float("nan") if t % 16 else c.kc[int(c.table[i, t // 16])]
        c.vc[int(c.table[i, t // 16]), t % 16:] = float("inf") if t % 16 else c.vc[int(c.table[i, t // 16])]
    c.kc[int(c.table[1, 4]), :6] = float("nan")
    c.vc[int(c.table[1, 4]), :6] = float("inf")
    got, lg = c.run()
    assert torch.equal(got, want) and torch.equal(lg, lw)
    table = c.table.copy()
    c = Case([(70, [(1, 20), (1, 60)]), (33, [(2, 9)])], 8, 2, 128, page=16, seed=9)
    c.table = table
    c.table[0, 1], c.table[1, 5], c.table[2, 0] = -1, 10 ** 9, c.n_pages
    c.check("bad pages")
    # what is seen and is no number stays in the rows that see it
    c.vc[int(c.table[1, 6]), 3, 0, 5] = float("nan")     # key 99 of the second sequence
    c.vc[int(c.table[2, 2]), 9, 1, 7] = float("inf")     # key 41 of the third, its last token's only
    out = _np(c.run()[0])
    bad = {tuple(x) for x in np.argwhere(~np.isfinite(out)).tolist()}
    assert bad == {(1, h, 5) for h in range(4)} | {(3, h, 7) for h in range(4, 8)}


def test_padding_and_given_arrays_stay():
    import torch

    c = Case([(40, [(2, 9), (1, 3)])], 8, 2, 64, pad=5, seed=10)
    out, lse = torch.full_like(c.q, 7.0), torch.full((c.T, 8), 7.0, device="cuda")
    got = c.run(out=out, lse=lse)
    assert got[0].data_ptr() == out.data_ptr() and (out[3:] == 7).all() and (lse[3:] == 7).all()
    assert torch.equal(out[:3], c.run()[0][:3])


def test_agrees_with_paged_attention():
    """The same batch without groups: each result within the other's rounding."""
    import torch

    from sparse_moe_02_amd.attn import paged_attn

    for H, hk, D in SHAPES:
        c = Case([(300, [(1, 33), (3, 70), (0, 4)]), (64, [(2, 2)])], H, hk, D, seed=11)
        out, lse = c.run()
        o2, l2 = paged_attn(c.q, c.kc, c.vc, *c.args()[:3], 3, max(c.total), return_lse=True)
        assert ((lse - l2).abs() <= 2.0 ** -16).all()
        assert ((out.float() - o2.float()).abs() <= 2.0 ** -6 * c.vc.float().abs().max()).all()


def test_streams_and_graphs():
    import torch

    c = Case([(600, [(1, 40)] * 6)], 16, 2, 256, seed=12)
    args = c.args()
    from sparse_moe_02_amd.attn import prefix_attn

    run = lambda: prefix_attn(c.q, c.kc, c.vc, *args, 1, 600, 40)
    want = run()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append(run())
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run()
    for i in range(3):
        c.q.copy_(torch.randn_like(c.q))
        args[4].fill_(600 - 37 * i)  # (the same keys, shared in part)
        graph.replay()
        assert torch.equal(o, run())


def test_refusals():
    import torch

    from sparse_moe_02_amd import binding as B
    from sparse_moe_02_amd.attn import prefix_attn

    c = Case([(40, [(1, 9), (1, 3)])], 8, 2, 64, seed=13)
    table, q_start, kv_len, gs, pl = c.args()
    call = lambda gs=gs, pl=pl, **kw: prefix_attn(c.q, c.kc, c.vc, table, q_start, kv_len, gs, pl, 1, 40, 9, **kw)
    for kw in (dict(gs=gs.long()), dict(pl=pl.float()), dict(gs=gs[:1]), dict(pl=pl.cpu()), dict(pl=torch.cat([pl, pl]))):
        with pytest.raises((ValueError, B.MoeError)):
            call(**kw)
    for kw, status in ((dict(gs=c.dev([0, 1, 2, 2]), pl=c.dev([1, 1, 1])), B.MOE_ERR_SHAPE),
                       (dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), B.MOE_ERR_WORKSPACE),
                       (dict(scale=float("inf")), B.MOE_ERR_SHAPE)):
        with pytest.raises(B.MoeError) as e:
            call(**kw)
        assert e.value.status == status
