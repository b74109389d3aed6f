"""The paged cache's bookkeeping on the GPU against its plain form: whole numbers and bits, so
everything is equal.  Then a server's steps together: grow, append, attend, fork, free,
compact."""

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


def _i32(x):
    import torch

    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Both:
    """A pool on the GPU and its plain form, with the same calls."""

    def __init__(self, n_pages, page, seqs, cols, planes=2, width=8, seed=0):
        import torch

        from oracle.serve import Pool
        from sparse_moe_02_amd.pages import PagePool

        g = torch.Generator().manual_seed(seed)
        self.cache = torch.randint(-2 ** 15, 2 ** 15, (planes, n_pages, width), generator=g, dtype=torch.int16).cuda()
        self.pool = PagePool(n_pages, page, seqs, cols)
        self.pool.table.fill_(-1)
        self.ref = Pool(-np.ones((seqs, cols)), np.zeros(seqs), np.zeros(n_pages), page, self.cache.cpu().numpy())

    def call(self, name, *args, apart=False):
        from sparse_moe_02_amd import binding as B

        say(f"{name} {[list(a)[:8] for a in args]} apart={apart}")
        pool = self.pool
        old = [t.clone() for t in (pool.table, pool.lens, pool.refs)]
        want = {"": 0, "shape": B.MOE_ERR_SHAPE, "alloc": B.MOE_ERR_ALLOC}[getattr(self.ref, name)(*map(list, args))]
        dev = [_i32(a) for a in args] + ([self.cache] if name in ("fork", "compact") else [])
        out = None
        if apart:
            out = pool.like()
            for t in (out.table, out.lens, out.refs):
                t.fill_(99)
        got = getattr(pool, name)(*dev, out=out)
        assert got is (out if apart else pool)
        if apart:
            assert all((a == b).all() for a, b in zip(old, (pool.table, pool.lens, pool.refs)))
            self.pool = out
        assert self.pool.check() == want, name
        self.pool.clear_error()
        self.same()
        return want

    def same(self):
        for name in ("table", "lens", "refs"):
            a, b = getattr(self.pool, name).cpu().numpy(), getattr(self.ref, name)
            assert np.array_equal(a, b), (name, np.argwhere(a != b)[:5].tolist())
        assert np.array_equal(self.cache.cpu().numpy(), self.ref.cache)


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("n_pages,page,seqs,cols,planes,width", [
    (40, 16, 6, 9, 2, 8), (300, 1, 20, 40, 1, 24), (9000, 32, 64, 200, 3, 8), (64, 64, 3, 21, 20, 3000)])
def test_random_calls(n_pages, page, seqs, cols, planes, width, apart):
    rng = np.random.default_rng(n_pages)
    b = Both(n_pages, page, seqs, cols, planes, width, seed=n_pages)
    seen = set()
    for step in range(40):
        op = rng.choice(["grow", "grow", "grow", "fork", "free", "compact"])
        ids = list(rng.permutation(seqs)[:rng.integers(1, seqs + 1)])
        if op == "grow":
            most = max(1, 2 * n_pages * page // seqs)
            r = b.call("grow", ids, rng.integers(0, min(most, cols * page // 2) + 1, len(ids)), apart=apart)
        elif op == "fork":
            empty = [s for s in range(seqs) if b.ref.lens[s] == 0]
            live = [s for s in range(seqs) if b.ref.lens[s] > 0] or ids
            dst = empty[:rng.integers(1, len(empty) + 1)] if empty else ids[:1]
            r = b.call("fork", rng.choice(live, len(dst)), dst, apart=apart)
        elif op == "free":
            r = b.call("free", ids[:max(1, len(ids) // 2)], apart=apart)
        else:
            r = b.call("compact", apart=apart)
        seen.add((str(op), r))
    assert len(seen) >= 4


def _start(seed=1):
    b = Both(50, 16, 8, 6, seed=seed)
    b.call("grow", [3, 0, 5], [40, 16, 1])
    return b


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("name,args", [
    ("grow", ([1, 2, 1], [1, 1, 1])), ("grow", ([8], [1])), ("grow", ([-1], [1])), ("grow", ([1], [-1])),
    ("grow", ([3], [57])), ("grow", ([1], [2 ** 31 - 1])), ("fork", ([3], [5])), ("fork", ([3, 3], [1, 1])),
    ("fork", ([3, 1], [1, 2])), ("fork", ([9], [1])), ("fork", ([3], [8])), ("free", ([3, 3],)), ("free", ([2 ** 31 - 1],)),
])
def test_bad_requests_change_nothing(name, args, apart):
    from sparse_moe_02_amd import binding as B

    assert _start().call(name, *args, apart=apart) == B.MOE_ERR_SHAPE


def test_too_few_pages():
    from sparse_moe_02_amd import binding as B

    b = Both(10, 16, 8, 12)
    assert b.call("grow", [0, 1], [100, 49]) == B.MOE_ERR_ALLOC
    assert b.call("grow", [0, 1], [100, 47]) == 0  # 7 + 3: the last page
    assert b.call("grow", [2], [1]) == B.MOE_ERR_ALLOC
    assert b.call("fork", [0], [2]) == B.MOE_ERR_ALLOC
    assert b.call("grow", [1], [1]) == 0  # room in its last page
    assert b.call("fork", [1], [2]) == 0  # a full last page is shared: no fresh one
    assert b.call("fork", [0], [3], apart=True) == B.MOE_ERR_ALLOC


@pytest.mark.parametrize("call", [("free", [3]), ("fork", [3], [1]), ("compact",)])
@pytest.mark.parametrize("bad", [50, -1, 2 ** 31 - 1])
def test_bad_table_entries(call, bad):
    from sparse_moe_02_amd import binding as B

    b = _start()
    b.pool.table[3, 1] = bad
    b.ref.table[3, 1] = bad
    assert b.call(*call) == B.MOE_ERR_SHAPE
    assert b.call("free", [0]) == 0  # other sequences go on


@pytest.mark.parametrize("length", [-5, 97, 2 ** 31 - 1])
def test_bad_lengths(length):
    from sparse_moe_02_amd import binding as B

    b = _start()
    b.pool.lens[3] = length
    b.ref.lens[3] = length
    for call in (("free", [3]), ("fork", [3], [1]), ("grow", [3], [1]), ("compact",)):
        assert b.call(*call) == B.MOE_ERR_SHAPE


def test_no_requests():
    b = _start()
    for apart in (False, True):
        for name, k in (("grow", 2), ("fork", 2), ("free", 1)):
            b.call(name, *([[]] * k), apart=apart)


def test_first_error_stays():
    from sparse_moe_02_amd import binding as B

    b = _start()
    b.pool.grow(_i32([1]), _i32([96]))
    b.pool.grow(_i32([1]), _i32([1]))             # behind the table
    b.pool.grow(_i32([0, 2, 4, 6, 7, 5]), _i32([80, 96, 96, 96, 96, 95]))  # too few pages
    b.pool.free(_i32([1]))
    assert b.pool.check() == B.MOE_ERR_SHAPE
    b.pool.clear_error()
    assert b.pool.check() == 0


def test_full_pool_and_empty_pool_compact():
    b = Both(12, 16, 4, 12)
    b.call("compact")
    b.call("grow", [1, 2], [96, 96])
    b.call("compact")
    b.call("free", [1])
    b.call("compact")
    b.call("free", [2])
    b.call("compact", apart=True)


def test_many_sequences():
    """More requests than the plan's workgroup has threads, forks of one source."""
    n = 3000
    b = Both(20000, 16, n + 2500, 8, planes=1, width=8)
    b.call("grow", range(n), [i % 60 for i in range(n)])
    b.call("fork", [7] * 1200 + [n - 1] * 1300, range(n, n + 2500))
    b.call("free", range(0, n, 2))
    b.call("compact")


def test_copy_pages():
    import torch

    from sparse_moe_02_amd.pages import copy_pages

    for shape in ((3, 20, 8), (1, 9, 16, 5, 24), (20, 6, 40000)):
        cache = torch.randn(shape, device="cuda").to(torch.bfloat16)
        ref = cache.clone()
        n = shape[1]
        src, dst = [1, 3, n, 0, -1], [0, 2, 1, n + 5, 4]
        copy_pages(cache, _i32(src), _i32(dst))
        for s, d in zip(src, dst):
            if 0 <= s < n and 0 <= d < n:
                ref[:, d] = ref[:, s]
        assert torch.equal(cache, ref)
    # pages interleaved with other memory, which keeps its bits
    wide = torch.randn((4, 10, 3, 64), device="cuda")
    ref = wide.clone()
    copy_pages(wide[1:3, :, 1], _i32([9]), _i32([0]))
    ref[1:3, 0, 1] = ref[1:3, 9, 1]
    assert torch.equal(wide, ref)


def test_pages_beyond_32_bits():
    import torch

    from sparse_moe_02_amd.pages import copy_pages

    cache = torch.empty((2, 2 ** 16 + 3, 32768), dtype=torch.int16, device="cuda")
    n = cache.shape[1]
    cache[:, n - 2] = torch.arange(32768, device="cuda").to(torch.int16)
    cache[:, n - 1] = 0
    copy_pages(cache, _i32([n - 2, n - 2]), _i32([n - 1, 0]))
    assert (cache[:, n - 1] == cache[:, n - 2]).all() and (cache[:, 0] == cache[:, n - 2]).all()


def test_graph_replays():
    """A captured decode step's bookkeeping replayed on the pool in place, with eager calls and
    synchronisations between the replays."""
    import torch

    b = Both(200, 16, 8, 20)
    b.call("grow", [0, 1, 2, 3], [30, 5, 16, 200])
    seqs, tokens = _i32([2, 0, 3]), _i32([1, 20, 3])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        b.pool.grow(seqs, tokens)
        b.pool.compact(b.cache)
    for i in range(4):
        b.call("free", [1])
        b.call("grow", [1], [40 + i])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.ref.grow([2, 0, 3], [1, 20, 3])
        b.ref.compact()
        assert b.pool.check() == 0
        b.same()


def test_serving_steps_together():
    """Prompts in chunks, parallel sampling, single tokens, an end and a compaction, through two
    attention layers' caches; every step's attention against binary64 over dense copies of the
    keys and values that were appended."""
    import torch

    from oracle import serve
    from sparse_moe_02_amd.attn import paged_attn, rope_append, rope_freqs
    from sparse_moe_02_amd.pages import PagePool

    H, hk, D, page, layers = 8, 2, 128, 16, 2
    rng = np.random.default_rng(3)
    g = torch.Generator(device="cuda").manual_seed(3)
    pool, spare = PagePool(64, page, 6, 16), None
    spare = pool.like()
    cache = torch.randn((2 * layers, 64, page, hk, D), generator=g, device="cuda").bfloat16()
    f, m = rope_freqs(64, 1e6, device="cuda")
    fr = f.cpu().numpy()
    dense = {}  # sequence -> per layer (keys, values) in binary64, as stored

    def step(seqs, new):
        nonlocal pool
        pool.grow(_i32(seqs), _i32(new))
        T = sum(new)
        qs = _i32(np.concatenate([[0], np.cumsum(new)]))
        for la in range(layers):
            proj = torch.randn((T, H + 2 * hk, D), generator=g, device="cuda").bfloat16()
            q, k, v = proj[:, :H], proj[:, H:H + hk], proj[:, H + hk:]
            kc, vc = cache[2 * la], cache[2 * la + 1]
            qr = rope_append(q, k, v, kc, vc, pool.table, qs, pool.lens, f, mscale=m, row=_i32(seqs))
            out, lse = paged_attn(qr, kc, vc, pool.table, qs, pool.lens, max(new), 256, row=_i32(seqs), return_lse=True)
            at = 0
            for s, n in zip(seqs, new):
                old = dense.setdefault(s, [None] * layers)[la]
                base = 0 if old is None else len(old[0])
                kk = serve.rope(k[at:at + n].double().cpu().numpy(), np.arange(base, base + n), fr, m)
                # stored keys are rounded to bf16
                kk = torch.from_numpy(kk).bfloat16().double().numpy()
                vv = v[at:at + n].double().cpu().numpy()
                K, V = (kk, vv) if old is None else (np.concatenate([old[0], kk]), np.concatenate([old[1], vv]))
                dense[s][la] = (K, V)
                Q = qr[at:at + n].double().cpu().numpy()
                for i in range(n):
                    for h in range(H):
                        x = D ** -0.5 * (K[:base + i + 1, h // 4] @ Q[i, h])
                        w = np.exp(x - x.max())
                        ref = w @ V[:base + i + 1, h // 4] / w.sum()
                        mass = w @ np.abs(V[:base + i + 1, h // 4]) / w.sum()
                        o = out[at + i, h].double().cpu().numpy()
                        # a key's fp32 angle may round it to the other neighbour in bf16: one step of
                        # 2^-7 in some of its elements moves a score by at most 2^-7 sum |q k|
                        d = 2.0 ** -7 * D ** -0.5 * 2 * np.abs(Q[i, h]).max() * np.abs(K[:, h // 4]).max()
                        assert (np.abs(o - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * d) * mass).all(), (s, i, h)
                at += n

    step([4, 1], [50, 17])
    step([4, 1, 0], [33, 1, 5])
    pool.fork(_i32([4, 4, 1]), _i32([2, 3, 5]), cache, out=spare)
    pool, spare = spare, pool
    for a, b in ((4, 2), (4, 3), (1, 5)):
        dense[b] = list(dense[a])
    step([0, 1, 2, 3, 4, 5], [1] * 6)
    pool.free(_i32([4, 0]))
    for s in (4, 0):
        del dense[s]
    pool.compact(cache, out=spare)
    pool, spare = spare, pool
    used = int((pool.refs > 0).sum())
    assert (pool.refs[:used] > 0).all() and (pool.refs[used:] == 0).all()
    step([5, 3, 2, 1], [1, 2, 1, 20])
    assert pool.check() == 0 and spare.check() == 0
