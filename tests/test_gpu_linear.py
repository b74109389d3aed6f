"""Products with 4-bit weights (moe_linear) against their binary64 form.

Tolerances, u = 2^-24.  With A = sum_k |x| (31 |s| + |b|): a group's 64 products (exact, of codes up to 31
with the offset) are summed in the matrix units, off by at most 64 * 2 u of their magnitudes where these
truncate; X, scale and bias add less than 24 u; groups are added one by one (k / 64 at most) and waves (16).  So a
result is off by less than (168 + k / 64) u A before it is rounded once: 2^-8 (bf16) or 2^-11 (fp16) relative,
2^-25 absolute among fp16's small numbers, or not at all."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()


def _np(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, n, k, seed=0, qdtype="fp16"):
        import torch

        from sparse_moe_02_amd.linear import QLinear

        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.k = n, k
        self.codes = torch.randint(-2 ** 31, 2 ** 31, (n, k // 8), generator=self.g, device="cuda", dtype=torch.int64).int()
        qd = {"fp16": torch.float16, "bf16": torch.bfloat16}[qdtype]
        self.scale = (0.02 * torch.rand((n, k // 64), generator=self.g, device="cuda")).to(qd)
        self.bias = (0.1 * torch.randn((n, k // 64), generator=self.g, device="cuda")).to(qd)
        self.lin = QLinear(self.codes, self.scale, self.bias)

    def rows(self, T, kind, cols=1):
        """(x, x_scale)"""
        import torch

        x = torch.randn((T, self.k), generator=self.g, device="cuda")
        if kind == "int8":
            return (torch.randint(-127, 128, (T, self.k), generator=self.g, device="cuda", dtype=torch.int32).to(torch.int8),
                    0.01 + torch.rand((T, cols), generator=self.g, device="cuda"))
        return x.to({"bf16": torch.bfloat16, "fp16": torch.float16}[kind]), None

    def check(self, out, x, xs, what=""):
        import torch

        from oracle import step

        ref, _ = step.linear(_np(x), self.codes.cpu().numpy(), _np(self.scale), _np(self.bias), None if xs is None else _np(xs))
        ax = np.abs(_np(x))
        if xs is not None:
            ax = ax * np.repeat(_np(xs), self.k // xs.shape[1], 1)
        A = ax @ np.repeat(31 * np.abs(_np(self.scale)) + np.abs(_np(self.bias)), 64, 1).T
        u = torch.finfo(out.dtype).eps / 2 if out.dtype != torch.float32 else U
        tol = u * np.abs(ref) + (168 + self.k / 64) * U * A * (1 + u) + (2.0 ** -25 if out.dtype == torch.float16 else 0)
        err = np.abs(_np(out) - ref) / tol
        say(f"{what} {self.n} x {self.k}, {x.shape[0]} rows {x.dtype}: error / tolerance {err.max():.3f}")
        assert out.shape == ref.shape and (err <= 1).all(), what

    def run(self, T, kind, cols=1, **kw):
        x, xs = self.rows(T, kind, cols)
        out = self.lin(x, xs, **kw)
        self.check(out, x, xs)
        return out


@pytest.mark.parametrize("kind", ["bf16", "fp16", "int8"])
@pytest.mark.parametrize("n,k", [(1, 64), (16, 128), (17, 192), (31, 64), (48, 320), (100, 1024), (257, 2048), (33, 2112), (15, 4096),
                                 (40, 4160), (16, 8192), (3, 16448)])
def test_shapes(n, k, kind):
    c = Case(n, k, n + k, "bf16" if n % 2 else "fp16")
    for T in (1, 2, 15, 16, 17, 33, 64, 70):
        c.run(T, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "int8"])
def test_output_types_and_many_rows_of_weights(kind):
    import torch

    c = Case(9001, 256, 3)  # more tiles than workgroups
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        for T in (1, 20, 130):
            assert c.run(T, kind, out_dtype=dt).dtype == dt
    c = Case(70000, 64, 4)
    c.run(5, kind, out_dtype=torch.float32)


def test_int8_scales_by_group():
    c = Case(100, 1280, 5)
    for cols in (1, 10, 20):
        for T in (1, 18, 40):
            c.run(T, "int8", cols)


def test_int8_sums_are_exact():
    """Scales and biases that are powers of two times small numbers: every step is exact, the largest codes and
    values included."""
    import torch

    from sparse_moe_02_amd.linear import QLinear

    n, k = 32, 512
    g = torch.Generator(device="cuda").manual_seed(6)
    codes = torch.full((n, k // 8), -1, dtype=torch.int32, device="cuda")
    codes[1:] = torch.randint(-2 ** 31, 2 ** 31, (n - 1, k // 8), generator=g, device="cuda", dtype=torch.int64).int()
    s = torch.full((n, k // 64), 0.5, device="cuda").half()
    b = torch.full((n, k // 64), -4.0, device="cuda").half()
    x = torch.randint(-128, 128, (5, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    x[0], x[1] = 127, -128
    from oracle import step

    ref, _ = step.linear(_np(x), codes.cpu().numpy(), _np(s), _np(b), np.full((5, 1), 0.25))
    got = QLinear(codes, s, b)(x, torch.full((5, 1), 0.25, device="cuda"), out_dtype=torch.float32)
    assert np.array_equal(_np(got), ref)


def test_strided_rows_and_what_stays():
    import torch

    c = Case(1000, 512, 7)
    x, _ = c.rows(9, "bf16")
    wide = torch.full((9, 1024), float("nan"), device="cuda").bfloat16()
    wide[:, 256:768] = x
    out = torch.full((9, 1003), 7.0, device="cuda")
    got = c.lin(wide[:, 256:768], out=out[:, 1:1001])
    c.check(got, x, None, "strided")
    assert (out[:, 0] == 7).all() and (out[:, 1001:] == 7).all()
    assert torch.equal(got, c.lin(x, out_dtype=torch.float32))
    # one row of x for all
    c.check(c.lin(x[:1].expand(9, 512)), x[:1].expand(9, 512), None, "expanded")
    # padding of the weights holds nothing that a result sees
    c.lin.codes.view(-1)[-8:] = -1
    assert c.lin(x[:0]).shape == (0, 1000)


def test_values_that_are_not_finite_stay_in_their_rows():
    import torch

    c = Case(50, 256, 8)
    x, _ = c.rows(20, "bf16")
    want = c.lin(x)
    x[3, 5], x[17, 200] = float("nan"), float("inf")
    got = c.lin(x)
    rest = [i for i in range(20) if i not in (3, 17)]
    assert got[3].isnan().all() and not got[17].isfinite().any() and torch.equal(got[rest], want[rest])


def test_rows_do_not_depend_on_their_number():
    """A row's result is bitwise the same alone and among up to 16 others."""
    import torch

    for kind in ("bf16", "int8"):
        c = Case(300, 2048, 9)
        x, xs = c.rows(16, kind)
        whole = c.lin(x, xs, out_dtype=torch.float32)
        for i in (0, 7, 15):
            assert torch.equal(c.lin(x[i:i + 1], None if xs is None else xs[i:i + 1], out_dtype=torch.float32)[0], whole[i])


def test_streams_and_graphs():
    import torch

    c = Case(2000, 1024, 10)
    x, _ = c.rows(4, "bf16")
    want = c.lin(x)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(c.lin(x))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = c.lin(x)
    for _ in range(3):
        x.copy_(c.rows(4, "bf16")[0])
        graph.replay()
        assert torch.equal(o, c.lin(x))


def test_refusals():
    import torch

    from sparse_moe_02_amd import binding as B
    from sparse_moe_02_amd.linear import QLinear

    c = Case(32, 128, 11)
    for args in ((c.codes[:, :4], c.scale, c.bias), (c.codes.long(), c.scale, c.bias), (c.codes, c.scale.float(), c.bias.float()),
                 (c.codes, c.scale[:3], c.bias), (c.codes, c.scale, c.bias.bfloat16()), (c.codes[0], c.scale, c.bias)):
        with pytest.raises(ValueError):
            QLinear(*args)
    with pytest.raises(ValueError):
        QLinear(c.codes, c.scale, c.bias, device="cpu")
    x, _ = c.rows(3, "bf16")
    i8, xs = c.rows(3, "int8", 2)
    for args, kw in (((x.float(),), {}), ((x.cpu(),), {}), ((x[:, :64],), {}), ((x[0],), {}), ((x, xs), {}), ((i8,), {}), ((i8, xs[:2]), {}),
                     ((i8, xs.half()), {}), ((i8, torch.ones((3, 3), device="cuda")), {}), ((x,), dict(out_dtype=torch.int8)),
                     ((x,), dict(out=torch.empty((3, 31), device="cuda"))), ((x,), dict(out=torch.empty((3, 32), dtype=torch.int8, device="cuda"))),
                     ((x.t().contiguous().t(),), {})):
        with pytest.raises(ValueError):
            c.lin(*args, **kw)
    odd = torch.empty(3 * 130, dtype=torch.bfloat16, device="cuda").view(3, 130)[:, :128]
    for bad, kw, status in ((odd, {}, B.MOE_ERR_ALIGN), (x, dict(out=x[:, :32]), B.MOE_ERR_ALIAS),
                            (x, dict(out=torch.empty((1, 32), device="cuda").expand(3, 32)), B.MOE_ERR_SHAPE)):
        with pytest.raises(B.MoeError) as e:
            c.lin(bad, **kw)
        assert e.value.status == status
