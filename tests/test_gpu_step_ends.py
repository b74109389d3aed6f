"""The norm, the 4-bit products, the choice of tokens and attention of shared prefixes at the ends of the sizes that they
accept.  Tolerances as in each operator's own tests, but for the norm's: a lane of 256 adds up to 4096 squares of a row of
2^20 one by one, so their sum is off by less than (4096 + 9) 2^-24 relative, its root by half of that, and the root,
quotient and two products by 5 2^-24 more: y by less than 2^-12.9, 2^-12 below."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib
from test_gpu_prefix import Case
from test_gpu_sample_tail import _check

pytestmark = pytest.mark.gpu

SLOP = 2.0 ** -12


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()
    yield
    torch.cuda.empty_cache()


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------- norm

WHOLE = [(1 << 20, 0), ((1 << 20) - 1, 0), ((1 << 20) - 8, 0), (32768 + 8, 0), (100003, 0)]
GROUPS = [(1 << 20, 32), (1 << 20, 128), (131072, 64)]


@pytest.mark.parametrize("width, group, kind", [(*c, k) for c in WHOLE for k in ("bf16", "fp16")] +
                         [(*c, k) for c in WHOLE + GROUPS for k in ("int8", "fp8")])
def test_norm_of_the_longest_rows(width, group, kind):
    import torch

    from oracle import step
    from sparse_moe_02_amd.norm import rms_norm

    dt = torch.float16 if kind == "fp16" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(width + group)
    x, r = (torch.randn((3, width), generator=g, device="cuda").to(dt) for _ in range(2))
    w = (1 + 0.3 * torch.randn(width, generator=g, device="cuda")).to(dt)
    ry, rh = step.rms_norm(_np(x), _np(w), residual=_np(r))
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if kind == "fp16" else 0.0
    if kind in ("bf16", "fp16"):
        y, h = rms_norm(x, w, residual=r)
        assert (np.abs(_np(y) - ry) <= (u + SLOP) * np.abs(ry) + tiny).all()
    else:
        most, out = (127.0, torch.int8) if kind == "int8" else (448.0, torch.float8_e4m3fn)
        codes, scale, h = rms_norm(x, w, residual=r, out_dtype=out, group=group)
        rs = step.group_scales(ry, most, group)
        assert scale.shape == rs.shape and (np.abs(_np(scale) - rs) <= SLOP * rs).all()
        v = ry.reshape(*rs.shape, -1) / rs[..., None]
        c = codes.float().double().cpu().numpy().reshape(v.shape)
        tol = 0.5 if kind == "int8" else 2.0 ** -4 * np.abs(v) + 2.0 ** -10
        assert (np.abs(c - v) <= tol + 2 * SLOP * np.abs(v)).all()
    assert (np.abs(_np(h) - rh) <= (u + 2.0 ** -23) * np.abs(rh) + tiny).all()
    # in place: the row is read in several passes
    if kind in ("bf16", "fp16"):
        a, b = x.clone(), r.clone()
        rms_norm(a, w, residual=b, sum=b, out=a)
        assert torch.equal(a, y) and torch.equal(b, h)


def test_norm_of_many_heads():
    import torch

    from oracle import step
    from sparse_moe_02_amd.norm import rms_norm

    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((33, 4096, 72), generator=g, device="cuda").bfloat16()[..., :64]
    y = rms_norm(x, None, offset=1.0)
    ry, _ = step.rms_norm(_np(x), None, offset=1.0)
    assert (np.abs(_np(y) - ry) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(ry)).all()


def test_norm_without_eps():
    """The formula as it stands: a row of zeros has no number, others need no eps."""
    import torch

    from oracle import step
    from sparse_moe_02_amd.norm import rms_norm

    x = torch.randn((3, 256), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    x[1] = 0
    y = rms_norm(x, None, 0.0, offset=1.0)
    ry, _ = step.rms_norm(_np(x[::2]), None, 0.0, 1.0)
    assert y[1].isnan().all() and (np.abs(_np(y[::2]) - ry) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(ry)).all()
    codes, scale = rms_norm(x, None, 0.0, offset=1.0, out_dtype=torch.int8)
    assert scale[1].isnan().all() and (codes[1] == 0).all() and scale[::2].isfinite().all()


# --------------------------------------------------------------------------- products

@pytest.mark.parametrize("kind, qdtype", [("bf16", "fp16"), ("fp16", "bf16"), ("int8", "fp16"), ("int8", "bf16")])
@pytest.mark.parametrize("n, k", [(20, 1 << 17), (9000, (1 << 17) - 64), (1 << 24, 64), ((1 << 24) - 15, 64)])
def test_products_of_the_largest_weights(n, k, kind, qdtype):
    import torch

    from oracle import step
    from sparse_moe_02_amd.linear import QLinear

    g = torch.Generator(device="cuda").manual_seed(n + k)
    qd = {"fp16": torch.float16, "bf16": torch.bfloat16}[qdtype]
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), generator=g, device="cuda", dtype=torch.int32)
    scale = (0.02 * torch.rand((n, k // 64), generator=g, device="cuda")).to(qd)
    bias = (0.1 * torch.randn((n, k // 64), generator=g, device="cuda")).to(qd)
    lin = QLinear(codes, scale, bias)
    rows = sorted({0, 15, n // 2 - 1, n // 2, n - 17, n - 16, n - 2, n - 1} | {(i * n) // 61 for i in range(61)})
    rows = [r for r in rows if 0 <= r < n]
    c, s, b = codes[rows].cpu().numpy(), _np(scale[rows]), _np(bias[rows])
    for T in (1, 17):
        if kind == "int8":
            x = torch.randint(-127, 128, (T, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
            xs = 0.01 + torch.rand((T, k // 64), generator=g, device="cuda")
        else:
            x, xs = torch.randn((T, k), generator=g, device="cuda").to({"bf16": torch.bfloat16, "fp16": torch.float16}[kind]), None
        out = _np(lin(x, xs, out_dtype=torch.float32)[:, rows])
        ref, _ = step.linear(_np(x), c, s, b, None if xs is None else _np(xs))
        ax = np.abs(_np(x)) if xs is None else np.abs(_np(x)) * np.repeat(_np(xs), 64, 1)
        A = ax @ np.repeat(31 * np.abs(s) + np.abs(b), 64, 1).T
        assert (np.abs(out - ref) <= 2.0 ** -24 * np.abs(ref) + (168 + k / 64) * 2.0 ** -24 * A * (1 + 2.0 ** -24)).all(), T


def test_products_of_the_largest_numbers():
    """bfloat16 rows up to 2^117 with the largest codes: no sum of a group overflows (31 * 64 * 2^117 < 2^128)."""
    import torch

    from oracle import step
    from sparse_moe_02_amd.linear import QLinear

    n, k = 20, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), generator=g, device="cuda", dtype=torch.int32)
    codes[:2] = -1
    scale, bias = (2.0 ** -10 * torch.rand((n, k // 64), generator=g, device="cuda")).half(), torch.zeros((n, k // 64), device="cuda").half()
    x = torch.full((18, k), 2.0 ** 117, device="cuda").bfloat16()
    x[1:] *= torch.rand((17, k), generator=g, device="cuda").bfloat16()
    out = QLinear(codes, scale, bias)(x, out_dtype=torch.float32)
    ref, _ = step.linear(_np(x), codes.cpu().numpy(), _np(scale), _np(bias))
    A = np.abs(_np(x)) @ np.repeat(31 * np.abs(_np(scale)), 64, 1).T
    assert (np.abs(_np(out) - ref) <= 2.0 ** -24 * np.abs(ref) + (168 + k / 64) * 2.0 ** -24 * A * (1 + 2.0 ** -24)).all()


# ----------------------------------------------------------------------------- tokens

@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V, skip", [(1 << 20, 0), (1 << 20, 3), ((1 << 20) - 3, 1)])
def test_tokens_of_the_largest_vocabularies(V, skip, dtype):
    """257 chunks where a row starts inside a 16-byte block."""
    import torch

    from sparse_moe_02_amd.sample import sample

    dt = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(V + skip)
    sharp = torch.tensor([0.01, 1.0, 2.5, 4.0, 4.0, 6.0, 3.0], device="cuda")
    R = len(sharp)
    buf = torch.full((R * (V + 5) + 8,), 6e4, device="cuda").to(dt)
    l = buf[skip:skip + R * (V + 5)].view(R, V + 5)[:, :V]
    l.copy_(torch.randn((R, V), generator=g, device="cuda") * sharp[:, None])
    l[6, :] = -12.0 + 0.5 * l[6]
    l[6, V - 1] = 9.0  # (one likely token, the last one)
    rng = np.random.default_rng(V + skip)
    params = (np.array([1.0, 0.8, 1.0, 1.0, 0.7, 1.0, 1.0]), np.array([0, 0, 400000, 0, 50, 0, 900000]),
              np.array([0.4, 0.9, 0.9, 1.0, 0.95, 0.99, 1.0]), np.array([0, 0, 0, 1e-3, 0.01, 1e-9, 1e-11]))
    u = rng.random((3, R))
    for i in range(3):
        u[i, 6] *= 1e-4  # (in front of the likely token)
        _check(l, u[i], *params, f"{V} behind {skip} {dtype}")
    # the same rows among enough others for the launches of many rows
    f = lambda x, d=torch.float32: torch.tensor(np.asarray(x), dtype=d, device="cuda")
    args = f(u[0]), f(params[0]), f(params[1], torch.int32), f(params[2]), f(params[3])
    few = sample(l, *args, return_prob=True)
    for r in (0, 2, 6):
        n = 1300
        many = sample(l[r:r + 1].expand(n, V), *(a[r:r + 1].expand(n).contiguous() for a in args), return_prob=True)
        assert all((m == x[r]).all() for m, x in zip(many, few)), r
    # the largest logits at both ends, equal; one at the end
    l[0, 0] = l[0, V - 1] = 60.0
    l[1, V - 1] = 60.0
    assert sample(l, f(u[0]), torch.zeros(R, device="cuda"))[:2].tolist() == [0, V - 1]
    one = torch.ones(R, dtype=torch.int32, device="cuda")
    assert sample(l, f(u[0]), None, one)[:2].tolist() == [0, V - 1]


def test_tokens_of_the_most_rows():
    import torch

    from sparse_moe_02_amd.sample import sample

    R, V = 65535, 333
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn((R, V), generator=g, device="cuda") * torch.linspace(0.1, 5, R, device="cuda")[:, None]
    u, t = torch.rand(R, generator=g, device="cuda"), 0.5 + torch.rand(R, generator=g, device="cuda")
    k = torch.randint(0, 50, (R,), generator=g, device="cuda", dtype=torch.int32)
    p = 0.5 + 0.5 * torch.rand(R, generator=g, device="cuda")
    token, prob = sample(l, u, t, k, p, 0.01 * t, return_prob=True)
    for a in (0, 32000, 65472):
        s = slice(a, a + 63)
        q, w = sample(l[s], u[s], t[s], k[s], p[s], 0.01 * t[s], return_prob=True)
        assert torch.equal(q, token[s]) and torch.equal(w, prob[s])
    f = lambda x: x[::4096].cpu().numpy()
    _check(l[::4096], f(u), f(t), f(k), f(p), f(0.01 * t), "65535 rows")


# -------------------------------------------------------------------------- attention

def test_prefixes_of_many_heads_and_of_the_largest_pages():
    Case([(70, [(1, 20), (2, 33)]), (5, [(1, 1)])], 512, 256, 64, page=16, seed=1).check("256 key/value heads")
    Case([(40, [(1, 20), (1, 33)])], 1024, 2, 64, page=16, seed=2).check("512 heads of one")
    Case([(70000, [(1, 20), (2, 33)]), (5, [(1, 1)])], 4, 2, 64, page=65536, seed=3).check("pages of 65536")
