"""The C ABI of the operators around the mixers on the CPU: host checks return the documented
statuses before a device is touched (made-up pointers that are never read)."""

import os

import pytest

M = 1 << 30  # made-up arrays lie this far apart
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, TOKENS, DEVICE, ALIAS = 1, 2, 3, 4, 5, 6, 7, 9


@pytest.fixture(scope="module")
def B():
    from sparse_moe_02_amd import binding

    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return binding


@pytest.fixture(autouse=True)
def no_gpu():
    """A valid call stops at the missing GPU."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


def _status(B, fn, *args):
    try:
        fn(*args)
    except B.MoeError as e:
        return e.status
    return 0


# ------------------------------------------------------------------------------- norm

def _norm(B, T=5, n=3, W=256, dtype=0, x=None, r=None, s=None, w=8 * M, offset=0.0, eps=1e-6, to=0, out=None, group=0, scale=None):
    h = lambda i: B.moe_heads(i * M, n * W, W)
    return _status(B, B.moe_rms_norm, T, n, W, dtype, x or h(1), r, s, w, offset, eps, to, out or h(4), group, scale, 0)


def test_norm_valid_calls_reach_the_device_check(B):
    H = B.moe_heads
    assert _norm(B) == DEVICE and _norm(B, dtype=B.MOE_FP16, to=B.MOE_FP16) == DEVICE
    assert _norm(B, r=H(2 * M, 768, 256), s=H(3 * M, 768, 256), w=None) == DEVICE
    for to in (B.MOE_INT8, B.MOE_FP8):
        for group in (0, 32, 64, 128):
            assert _norm(B, to=to, scale=9 * M, group=group) == DEVICE
    # in place; slices of one projection; odd places without groups; strides of 0 where it is read
    x, r = H(M, 768, 256), H(2 * M, 768, 256)
    assert _norm(B, x=x, out=x) == DEVICE and _norm(B, x=x, r=r, s=x, out=r) == DEVICE and _norm(B, x=x, r=r, s=r, out=x) == DEVICE
    assert _norm(B, x=H(M, 2048, 256), out=H(M + 2 * 768, 2048, 256)) == DEVICE
    assert _norm(B, x=H(M + 2, 769, 257), out=H(4 * M + 6, 771, 257), W=255) == DEVICE
    assert _norm(B, x=H(M + 2, 768, 256), to=B.MOE_INT8, scale=9 * M, out=H(4 * M + 1, 768, 256)) == DEVICE
    assert _norm(B, x=H(M, 0, 256), r=H(2 * M, 0, 0)) == DEVICE
    assert _norm(B, T=0, x=H(0, 0, 0), out=H(0, 0, 0), w=None) == 0


def test_norm_refusals(B):
    H = B.moe_heads
    assert _norm(B, T=-1) == TOKENS and _norm(B, T=(1 << 20) + 1) == TOKENS and _norm(B, T=1 << 20, n=257) == TOKENS
    for kw in (dict(n=0), dict(n=4097), dict(W=0), dict(W=(1 << 20) + 1), dict(eps=-1e-6), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(offset=float("nan")), dict(group=64), dict(to=B.MOE_INT8, scale=9 * M, group=16),
               dict(to=B.MOE_INT8, scale=9 * M, group=64, W=96), dict(to=B.MOE_INT8, scale=9 * M, group=-64),
               dict(x=H(M, -8, 256)), dict(out=H(M, 768, 128)), dict(out=H(M, 0, 256)), dict(s=H(3 * M, 256, 256))):
        assert _norm(B, **kw) == SHAPE, kw
    for kw in (dict(dtype=B.MOE_FP32), dict(to=B.MOE_FP16), dict(to=B.MOE_FP32), dict(dtype=B.MOE_INT8, to=B.MOE_INT8)):
        assert _norm(B, **kw) == DTYPE, kw
    for kw in (dict(x=H(0, 768, 256)), dict(out=H(0, 768, 256)), dict(to=B.MOE_INT8), dict(scale=9 * M), dict(r=H(0, 8, 8))):
        assert _norm(B, **kw) == NULL, kw
    for kw in (dict(x=H(M + 1, 768, 256)), dict(w=8 * M + 1), dict(to=B.MOE_INT8, scale=9 * M + 2),
               dict(to=B.MOE_INT8, scale=9 * M, group=64, x=H(M + 2, 768, 256)),
               dict(to=B.MOE_INT8, scale=9 * M, group=64, out=H(4 * M + 4, 768, 256)),
               dict(to=B.MOE_INT8, scale=9 * M, group=64, w=8 * M + 2),
               dict(to=B.MOE_INT8, scale=9 * M, group=64, r=H(2 * M, 769, 256))):
        assert _norm(B, **kw) == ALIGN, kw
    x, r = H(M, 768, 256), H(2 * M, 768, 256)
    size = 5 * 3 * 256
    for kw in (dict(x=x, out=H(M + 16, 768, 256)), dict(x=x, r=r, out=H(2 * M + 2, 768, 256)), dict(x=x, s=H(M, 776, 256)),
               dict(s=H(4 * M, 768, 256)), dict(w=4 * M + 2 * size - 2), dict(s=H(8 * M, 768, 256)),
               dict(to=B.MOE_INT8, scale=9 * M, out=x), dict(to=B.MOE_INT8, scale=M + 2 * size - 4),
               dict(to=B.MOE_INT8, scale=4 * M + size - 4), dict(to=B.MOE_INT8, scale=8 * M),
               dict(to=B.MOE_INT8, scale=9 * M, s=H(4 * M, 768, 256))):
        assert _norm(B, **kw) == ALIAS, kw


# ----------------------------------------------------------------------------- linear

def _linear(B, w=None, T=5, x=4 * M, xld=192, xt=0, xs=None, group=0, out=5 * M, old=100, to=0, **kw):
    d = dict(codes=M, scale=2 * M, bias=3 * M, n=100, k=192, qparam_dtype=B.MOE_FP16)
    d.update(kw)
    return _status(B, B.moe_linear, w or B.moe_linear_weights(**d), T, x, xld, xt, xs, group, out, old, to, 0)


def test_linear_valid_calls_reach_the_device_check(B):
    for xt in (B.MOE_BF16, B.MOE_FP16):
        for to in (B.MOE_BF16, B.MOE_FP16, B.MOE_FP32):
            assert _linear(B, xt=xt, to=to, qparam_dtype=B.MOE_BF16) == DEVICE
    assert _linear(B, xt=B.MOE_INT8, xs=6 * M) == DEVICE and _linear(B, xt=B.MOE_INT8, xs=6 * M, group=64) == DEVICE
    assert _linear(B, xt=B.MOE_INT8, xs=6 * M, group=128, k=256, xld=256) == DEVICE
    assert _linear(B, T=1, xld=0, old=0) == DEVICE and _linear(B, xld=0) == DEVICE and _linear(B, T=70) == DEVICE
    assert _linear(B, out=5 * M + 2) == DEVICE
    assert _linear(B, T=0, x=None, out=None) == 0


def test_linear_refusals(B):
    for kw in (dict(n=0), dict(n=(1 << 24) + 1), dict(k=0), dict(k=32), dict(k=96), dict(k=(1 << 17) + 64), dict(group=64),
               dict(xt=B.MOE_INT8, xs=6 * M, group=32), dict(xt=B.MOE_INT8, xs=6 * M, group=128), dict(xld=-192), dict(old=99)):
        assert _linear(B, **kw) == SHAPE, kw
    for kw in (dict(qparam_dtype=B.MOE_FP32), dict(xt=B.MOE_FP32), dict(xt=B.MOE_FP8), dict(to=B.MOE_INT8)):
        assert _linear(B, **kw) == DTYPE, kw
    assert _linear(B, T=-1) == TOKENS and _linear(B, T=(1 << 20) + 1) == TOKENS and _linear(B, T=1 << 20, n=1 << 21) == TOKENS
    for kw in (dict(codes=None), dict(scale=None), dict(bias=None), dict(x=None), dict(out=None), dict(xt=B.MOE_INT8), dict(xs=6 * M)):
        assert _linear(B, **kw) == NULL, kw
    assert _status(B, B.moe_linear, None, 1, M, 64, 0, None, 0, 2 * M, 64, 0, 0) == NULL
    for kw in (dict(codes=M + 8), dict(scale=2 * M + 2), dict(bias=3 * M + 8), dict(x=4 * M + 8), dict(xld=196), dict(out=5 * M + 1),
               dict(out=5 * M + 2, to=B.MOE_FP32), dict(xt=B.MOE_INT8, xs=6 * M + 2), dict(xt=B.MOE_INT8, xs=6 * M, xld=200)):
        assert _linear(B, **kw) == ALIGN, kw
    # 112 padded rows of 256 padded k: 14336 bytes of codes, 896 of scales
    for kw in (dict(out=4 * M + 2), dict(out=M + 14334), dict(out=2 * M + 894), dict(out=3 * M), dict(out=M - 2 * (4 * 100 + 100) + 2),
               dict(xt=B.MOE_INT8, xs=5 * M + 4)):
        assert _linear(B, **kw) == ALIAS, kw
    assert _linear(B, out=M + 14336) == DEVICE


# ----------------------------------------------------------------------------- sample

def _sample(B, R=5, V=1000, l=M, ld=1000, t=2, u=2 * M, temperature=None, k=None, p=None, m=None, token=3 * M, prob=None, ws=4 * M,
            wsn=1 << 28):
    return _status(B, B.moe_sample, R, V, l, ld, t, u, temperature, k, p, m, token, prob, ws, wsn, 0)


def test_sample_valid_calls_reach_the_device_check(B):
    for t in (B.MOE_FP32, B.MOE_BF16, B.MOE_FP16):
        assert _sample(B, t=t) == DEVICE
    more = dict(temperature=5 * M, k=6 * M, p=7 * M, m=8 * M, prob=9 * M)
    assert _sample(B, **more) == DEVICE and _sample(B, V=1 << 20, ld=1 << 20) == DEVICE and _sample(B, ld=0) == DEVICE
    assert _sample(B, l=M + 2, t=B.MOE_BF16) == DEVICE and _sample(B, temperature=2 * M) == DEVICE
    assert _sample(B, R=0, l=None, u=None, token=None, ws=None, wsn=0) == 0
    need = B.moe_sample_workspace(5, 1000)
    assert need >= 5 * 128 * 12 and _sample(B, wsn=need) == DEVICE and _sample(B, wsn=need - 1) == WORKSPACE
    assert B.moe_sample_workspace(0, 10) == 0


def test_sample_refusals(B):
    assert _sample(B, R=-1) == TOKENS and _sample(B, R=65536) == TOKENS
    for kw in (dict(V=0), dict(V=(1 << 20) + 1), dict(ld=-1)):
        assert _sample(B, **kw) == SHAPE, kw
    assert _sample(B, t=B.MOE_INT8) == DTYPE and _sample(B, t=7) == DTYPE
    for kw in (dict(l=None), dict(u=None), dict(token=None)):
        assert _sample(B, **kw) == NULL, kw
    assert _sample(B, ws=None) == WORKSPACE
    for kw in (dict(l=M + 2), dict(u=2 * M + 1), dict(token=3 * M + 2), dict(prob=9 * M + 1), dict(k=6 * M + 2), dict(ws=4 * M + 128)):
        assert _sample(B, **kw) == ALIGN, kw
    size = 4 * 5 * 1000
    for kw in (dict(token=M + size - 4), dict(prob=M), dict(token=2 * M), dict(prob=3 * M + 16), dict(token=4 * M), dict(prob=4 * M),
               dict(temperature=3 * M), dict(k=9 * M, prob=9 * M + 16), dict(ws=M - 256), dict(ws=2 * M)):
        assert _sample(B, **kw) == ALIAS, kw
    for args, status in (((-1, 10), TOKENS), ((70000, 10), TOKENS), ((5, 0), SHAPE), ((5, (1 << 20) + 1), SHAPE)):
        assert _status(B, B.moe_sample_workspace, *args) == status


# ------------------------------------------------------------------------------ prefix

def _prefix(B, T=6, max_q=3, max_prefix=100, max_suffix=20, H=8, lse=None, scale=0.1, flags=0, ws=10 * M, wsn=1 << 29, groups=True,
            gs=11 * M, pl=11 * M + 4096, n_groups=2, n_seqs=4, q=4 * M, out=5 * M, **kw):
    d = dict(k=M, v=2 * M, page_stride=32 * 2 * 128, token_stride=2 * 128, head_stride=128, n_pages=10, page_size=32, n_kv_heads=2,
             head_dim=128, dtype=B.MOE_BF16)
    d.update(kw)
    b = B.moe_batch(3 * M, 3 * M + 4096, 3 * M + 8192, None, n_seqs, max(n_seqs, 1), 5)
    g = B.moe_prefix_groups(gs, pl, n_groups) if groups else None
    return _status(B, B.moe_prefix_attn, B.moe_paged_kv(**d), b, g, T, max_q, max_prefix, max_suffix, B.moe_heads(q, 8 * 128, 128), H,
                   B.moe_heads(out, 8 * 128, 128), lse, scale, flags, ws, wsn, 0)


def test_prefix_calls_and_refusals(B):
    assert _prefix(B) == DEVICE and _prefix(B, lse=12 * M, flags=B.MOE_ATTN_FULL, dtype=B.MOE_FP16) == DEVICE
    assert _prefix(B, max_q=0, max_prefix=0, max_suffix=0) == DEVICE and _prefix(B, n_groups=4) == DEVICE
    assert _prefix(B, T=0, ws=None, wsn=0) == 0
    for kw in (dict(n_groups=0), dict(n_groups=5), dict(max_prefix=-1), dict(max_suffix=-1), dict(max_q=-1), dict(n_seqs=0), dict(H=3),
               dict(head_dim=96), dict(flags=2), dict(scale=float("nan"))):
        assert _prefix(B, **kw) == SHAPE, kw
    for kw in (dict(groups=False), dict(gs=None), dict(pl=None), dict(q=None), dict(out=None)):
        assert _prefix(B, **kw) == NULL, kw
    for kw in (dict(gs=11 * M + 2), dict(pl=11 * M + 1), dict(ws=10 * M + 64), dict(lse=12 * M + 2)):
        assert _prefix(B, **kw) == ALIGN, kw
    assert _prefix(B, T=(1 << 17) + 1) == TOKENS and _prefix(B, dtype=B.MOE_FP32) == DTYPE
    kv = B.moe_paged_kv(None, None, 0, 0, 0, 1, 16, 2, 128, B.MOE_BF16)
    need = B.moe_prefix_attn_workspace(kv, 6, 4, 2, 3, 100, 20, 8)
    assert need >= 6 * 8 * 2 * 128 * 4 and _prefix(B, wsn=need) == DEVICE and _prefix(B, wsn=need - 1) == WORKSPACE
    for kw in (dict(out=11 * M - 4096), dict(lse=11 * M + 4100), dict(ws=11 * M), dict(lse=11 * M + 8), dict(lse=10 * M), dict(out=4 * M)):
        assert _prefix(B, **kw) == ALIAS, kw


def test_prefix_launches_stay_within_what_a_join_holds(B):
    kv = B.moe_paged_kv(None, None, 0, 0, 0, 1, 16, 2, 128, B.MOE_BF16)
    for T, seqs, groups, mq, mp, ms in ((1, 1, 1, 1, 1 << 30, 1 << 30), (6, 3, 3, 2, 0, 0), (1 << 17, 1 << 15, 7, 4, 16384, 500),
                                         (64, 64, 1, 1, 16384, 512), (2, 2, 2, 1, 1 << 40, 3)):
        n = B.moe_prefix_attn_workspace(kv, T, seqs, groups, mq, mp, ms, 8)
        slots = n / (T * 8 * (128 * 4 + 16))
        assert 2 <= slots <= 256.01, (T, slots)
