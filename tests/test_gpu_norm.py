"""The norm (moe_rms_norm) against its binary64 form.

Tolerances, u = 2^-24: the sum of squares adds, on a lane's path, at most 128 terms one by one (rows of
32768 elements over 256 lanes; 64 in rows of up to 16384) and joins lanes in 8 more steps; all terms are
positive, so it is off by less than 137 u relative, its root by half of that, and the root, quotient and
two products by 5 u more: y is off by less than 74 u < 2^-17 relative before it is rounded once, by 2^-8
(bf16) or 2^-11 (fp16) relative, 2^-25 absolute among fp16's small numbers.  h = x + r is rounded in
binary32 (u) and once more.  In 8 bits a scale is off by 2^-17 relative too and y / s by twice that; a code is then at
most half a step from it: 0.5 (int8), or 2^-4 relative and 2^-10 absolute (e4m3)."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib, say

pytestmark = pytest.mark.gpu

SLOP = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()


def _np(t):
    return t.double().cpu().numpy()


def _make(shape, dtype, seed, of=None):
    """x, residual, weight; x a slice of rows of `of` elements."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = (rnd(*shape[:-1], of or shape[-1]) * torch.exp(rnd(shape[0], *[1] * (len(shape) - 1)))).to(dt)[..., :shape[-1]]
    return x, (3 * rnd(*shape)).to(dt), (1 + 0.3 * rnd(shape[-1])).to(dt)


def _check(x, r, w, kind, group=0, offset=0.0, eps=1e-6, what="", **kw):
    import torch

    from oracle import step
    from sparse_moe_02_amd.norm import rms_norm

    ry, rh = step.rms_norm(_np(x), None if w is None else _np(w), eps, offset, None if r is None else _np(r))
    u = torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    got = rms_norm(x, w, eps, offset=offset, residual=r, out_dtype=kind, group=group, **kw)
    got = got if isinstance(got, tuple) else (got,)
    if kind is None:
        err = np.abs(_np(got[0]) - ry) / ((u + SLOP) * np.abs(ry) + tiny + 1e-300)
        say(f"{what}: error / tolerance {err.max():.3f}")
        assert got[0].dtype == x.dtype and (err <= 1).all(), what
        hs = got[1:]
    else:
        most = 127.0 if kind == torch.int8 else 448.0
        rs = step.group_scales(ry, most, group)
        codes, scale = got[0], _np(got[1])
        assert codes.dtype == kind and scale.shape == rs.shape
        assert (np.abs(scale - rs) <= SLOP * rs).all(), what
        v = ry.reshape(*rs.shape, -1) / np.where(rs == 0, 1, rs)[..., None]
        c = codes.float().double().cpu().numpy().reshape(v.shape)
        tol = 0.5 if kind == torch.int8 else 2.0 ** -4 * np.abs(v) + 2.0 ** -10
        assert (np.abs(c - v) <= tol + 2 * SLOP * np.abs(v)).all(), what
        assert np.abs(c).max() <= most
        hs = got[2:]
    assert len(hs) == (1 if r is not None or kw.get("sum") is not None else 0)
    for h in hs:
        assert h.dtype == x.dtype
        assert (np.abs(_np(h) - rh) <= (u + 2.0 ** -23) * np.abs(rh) + tiny).all(), what
    return got


WIDTHS = [1, 7, 8, 63, 64, 65, 120, 128, 136, 248, 256, 264, 511, 512, 520, 1000, 1024, 1032, 2047, 2048, 2056, 4096, 8191, 8192,
          8200, 8201, 16384, 16392, 32768]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    for T in (1, 5, 67):
        x, r, w = _make((T, width), dtype, width + T)
        _check(x, r, w, None, what=f"{T} x {width} {dtype}")
    _check(x, None, None, None, offset=1.25, eps=0.1, what="no residual, no weight")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("width", [8, 32, 64, 96, 128, 192, 256, 384, 640, 1024, 1920, 2048, 8192, 8320, 20480, 33, 1023, 9001])
def test_eight_bits(width, kind, dtype):
    import torch

    kind = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    for i, group in enumerate((0, 32, 64, 128)):
        if group and width % group:
            continue
        x, r, w = _make((13, width), dtype, width + i)
        _check(x, r if i % 2 else None, w, kind, group, what=f"{width} by {group}")


def test_heads_of_a_fused_projection():
    import torch

    for n, D in ((16, 256), (5, 64), (3, 128), (2, 7), (4, 72)):
        proj, _, w = _make((31, n + 3, D), "bf16", n)
        x = proj[:, 1:n + 1]
        _check(x, None, w, None, offset=1.0, what=f"{n} heads of {D}")
        if D == 128:
            _check(x, None, w, torch.int8, 128, what="heads in 8 bits")
        # in place, between rows that stay as they were
        want = _check(x, None, w, None)[0].clone()
        before = proj.clone()
        from sparse_moe_02_amd.norm import rms_norm

        assert rms_norm(x, w, out=x).data_ptr() == x.data_ptr()
        assert torch.equal(x, want) and torch.equal(proj[:, 0], before[:, 0]) and torch.equal(proj[:, n + 1:], before[:, n + 1:])


@pytest.mark.parametrize("width", [7, 64, 2048, 2047, 8200, 9001])
def test_in_place(width):
    import torch

    from sparse_moe_02_amd.norm import rms_norm

    x, r, w = _make((9, width), "bf16", width)
    y, h = rms_norm(x, w, residual=r)
    for place in ("sum over residual, y over x", "sum over x, y over residual"):
        a, b = x.clone(), r.clone()
        s, o = (b, a) if place.startswith("sum over residual") else (a, b)
        gy, gh = rms_norm(a, w, residual=b, sum=s, out=o)
        assert gh.data_ptr() == s.data_ptr() and gy.data_ptr() == o.data_ptr()
        assert torch.equal(gy, y) and torch.equal(gh, h), place


def test_rows_of_nothing_and_of_no_numbers():
    import torch

    from sparse_moe_02_amd.norm import rms_norm

    inf, nan = float("inf"), float("nan")
    x, r, w = _make((6, 256), "bf16", 3)
    x[0], r[0] = 0, 0
    x[1, 5] = nan
    x[2, 5] = inf
    x[3], r[3] = 1e-30, 0  # (squares vanish: eps alone)
    y = rms_norm(x, w, residual=r)[0]
    assert (y[0] == 0).all() and y[1].isnan().all() and y[2, 5].isnan() and (y[2, 6:] == 0).all()
    assert torch.equal(y[3], (x[3].float() * 1e3 * w.float()).bfloat16())
    for kind in (torch.int8, torch.float8_e4m3fn):
        for group in (0, 64):
            c, s, _ = rms_norm(x, w, residual=r, out_dtype=kind, group=group)
            c = c.float()
            assert (c[0] == 0).all() and (s[0] == 0).all()
            assert s[1].isnan().all() and (c[1] == 0).all()
            assert (s[2, 0].isnan() or s[2, 0].isinf()) and (c[2] == 0).all()
            assert s[4:].isfinite().all() and (c[4:].abs().amax(-1) == (127 if kind == torch.int8 else 448)).all()
            if group:
                assert (s[2, 1:] == 0).all()  # the row's other elements are 0
    for T in (0, 3):
        e = torch.empty((T, 0 if T else 5), dtype=torch.bfloat16, device="cuda")
        assert rms_norm(e, e.new_empty(e.shape[1])).shape == e.shape


def test_far_strides_and_many_rows():
    """Places behind 2^31 elements; rows behind the first 2^16 workgroups."""
    import torch

    big = torch.zeros((3, 1 << 30), dtype=torch.bfloat16, device="cuda")
    x, _, w = _make((3, 2048), "bf16", 1)
    big[:, -2048:] = x
    _check(big[:, -2048:], None, w, None, what="far rows")
    del big
    x, r, w = _make((70001, 8), "fp16", 2)
    _check(x, r, w, None, what="70001 rows")
    x, r, w = _make((66000, 2056), "bf16", 2)
    _check(x[::1000], None, w, None, what="every 1000th row")


def test_streams_and_graphs():
    import torch

    from sparse_moe_02_amd.norm import rms_norm

    x, r, w = _make((64, 2048), "bf16", 5)
    want = rms_norm(x, w, residual=r, out_dtype=torch.int8, group=128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = rms_norm(x, w, residual=r, out_dtype=torch.int8, group=128)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rms_norm(x, w, residual=r, out_dtype=torch.int8, group=128)
    for seed in range(3):
        x2, r2, _ = _make((64, 2048), "bf16", seed)
        x.copy_(x2)
        r.copy_(r2)
        graph.replay()
        want = rms_norm(x2, w, residual=r2, out_dtype=torch.int8, group=128)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    import torch

    from sparse_moe_02_amd import binding as B
    from sparse_moe_02_amd.norm import rms_norm

    x, r, w = _make((4, 256), "bf16", 1)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x[:, ::2]), dict(x=x[0]), dict(weight=w.half()), dict(weight=w[1:]),
                dict(residual=r[:3]), dict(residual=r.half()), dict(out_dtype=torch.float32), dict(out=x.float()), dict(out=x[:, :8]),
                dict(sum=x[:3]), dict(scale=x.float())):
        with pytest.raises(ValueError):
            rms_norm(**{**dict(x=x, weight=w, residual=r), **bad})
    for bad, status in ((dict(group=64), B.MOE_ERR_SHAPE), (dict(out_dtype=torch.int8, group=100), B.MOE_ERR_SHAPE),
                        (dict(eps=-1.0), B.MOE_ERR_SHAPE), (dict(eps=float("nan")), B.MOE_ERR_SHAPE),
                        (dict(offset=float("inf")), B.MOE_ERR_SHAPE), (dict(sum=x, out=x), B.MOE_ERR_ALIAS)):
        with pytest.raises(B.MoeError) as e:
            rms_norm(**{**dict(x=x, weight=w, residual=r), **bad})
        assert e.value.status == status, bad
    odd = torch.empty(4 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 256)
    with pytest.raises(B.MoeError) as e:
        rms_norm(odd, w, out_dtype=torch.int8, group=64)
    assert e.value.status == B.MOE_ERR_ALIGN


@pytest.mark.parametrize("width", [1, 6, 8, 17, 120, 256, 771, 2048, 3326, 8195, 20003])
@pytest.mark.parametrize("start", [1, 2, 5])
def test_rows_that_start_anywhere(width, start):
    """Every array aligned to its elements only, rows an odd distance apart, between elements that stay as they were."""
    import torch

    def place(t):
        buf = torch.full((t.shape[0], t.shape[1] + 3), 7, dtype=torch.float32, device="cuda").to(t.dtype).flatten()
        buf = torch.cat([buf, buf[:start]])
        v = buf[start:].view(t.shape[0], -1)[:, :width]
        v.copy_(t)
        return buf, v

    for kind in (None, torch.int8):
        x, r, w = _make((11, width), "bf16", width + start)
        (_, x), (_, r), (_, w) = place(x), place(r), place(w[None])
        w = w[0]
        ob, o = place(torch.zeros((11, width), dtype=torch.bfloat16 if kind is None else kind, device="cuda"))
        sb, s = place(torch.zeros((11, width), dtype=torch.bfloat16, device="cuda"))
        _check(x, r, w, kind, out=o, sum=s, what=f"{width} from {start}")
        for b in (ob, sb):
            inside = torch.zeros(b.shape, dtype=torch.bool, device="cuda")
            inside[start:].view(11, -1)[:, :width] = True
            assert (b[~inside].float() == 7).all()
