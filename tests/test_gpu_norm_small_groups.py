"""8-bit outputs of the norm (moe_rms_norm) of groups whose largest element is near 2^-120, the least that has a scale.

With eps 1, no weight and offset 1 the norm of such rows is the identity (their squares are 0 beside eps), so y is x as it
stands.  With t = max|y| the scale t / 127 (448) is below binary32's normal range: rounded to a multiple of 2^-149, it is off
by 2^-150 at most, and one quotient before that, 2^-24 relative.  A code is y times a quotient of 2^-24, at most 2^-23 off
y / (t / 127), and half a step from it: 0.5 (int8), or 2^-4 relative and 2^-10 absolute (e4m3).  Zeros are codes of 0, and
the largest element the largest code."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu

# in units of 2^-120: below the least, the least, around 1.75 (above which 448 / t is finite), and normal ones
TOPS = [2.0 ** -8, 0.5, 255 / 256, 1.0, 129 / 128, 1.25, 1.5, 223 / 128, 1.75, 225 / 128, 255 / 128, 2.0, 3.0, 448.0, 2.0 ** 20, 2.0 ** 100]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("width, group", [(8, 0), (33, 0), (64, 32), (96, 32), (256, 64), (256, 128), (256, 0), (1000, 0), (2048, 128), (2056, 0),
                                          (8192, 32), (20480, 0), (20480, 128), (20481, 0)])
def test_scales_and_codes(kind, width, group):
    import torch

    from sparse_moe_02_amd.norm import rms_norm

    dt, most = (torch.int8, 127.0) if kind == "int8" else (torch.float8_e4m3fn, 448.0)
    g = group or width
    rng = np.random.default_rng(width + group)
    # each group its own largest element, with zeros of both signs among the others
    tops = np.array([[TOPS[(i + 5 * j) % len(TOPS)] for j in range(width // g)] for i in range(len(TOPS))])
    part = rng.uniform(-1, 1, (len(TOPS), width // g, g)) * 2.0 ** -rng.integers(0, 12, (len(TOPS), width // g, g))
    part[..., ::3] = 0.0
    part[..., 3::6] = -0.0
    part[..., 1], part[..., 4] = 1.0, -1.0
    x = torch.from_numpy((part * tops[..., None] * 2.0 ** -120).reshape(len(TOPS), width)).to(torch.bfloat16)
    y = x.double().numpy().reshape(part.shape)
    assert (np.abs(y).max(-1) == tops * 2.0 ** -120).all()
    codes, scale = rms_norm(x.cuda(), None, 1.0, offset=1.0, out_dtype=dt, group=group)
    codes, scale = codes.float().double().cpu().numpy().reshape(part.shape), scale.double().cpu().numpy()
    some = tops >= 1
    want = np.where(some, tops, 0.0) * 2.0 ** -120 / most
    assert (np.abs(scale - want) <= 2.0 ** -150 + 2.0 ** -24 * want).all()
    assert (codes[~some] == 0).all() and (codes[y == 0] == 0).all()
    assert (codes[some][..., 1] == most).all() and (codes[some][..., 4] == -most).all()
    v = y[some] / want[some][..., None]
    tol = 0.5 if kind == "int8" else 2.0 ** -4 * np.abs(v) + 2.0 ** -10
    assert (np.abs(codes[some] - v) <= tol + 2.0 ** -23 * np.abs(v)).all()


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_groups_of_large_elements(kind):
    """Up to the largest bfloat16: no step overflows."""
    import torch

    from sparse_moe_02_amd.norm import rms_norm

    dt, most = (torch.int8, 127.0) if kind == "int8" else (torch.float8_e4m3fn, 448.0)
    # (mean(h^2) = 1 for rows of +-1, so y is the weight but for the root's rounding)
    x = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.full((64,), float(torch.finfo(torch.bfloat16).max), dtype=torch.bfloat16, device="cuda")
    w[1::2], w[2::4] = -w[0], 0.0
    for group in (0, 32):
        codes, scale = rms_norm(x, w, 0.0, out_dtype=dt, group=group)
        assert torch.equal(codes.float(), torch.sign(w.float()).expand(2, 64) * most)
        assert ((scale.double() * most / float(w[0]) - 1).abs() <= 2.0 ** -22).all()
