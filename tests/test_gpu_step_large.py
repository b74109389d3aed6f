"""The norm, the 4-bit products, the choice of tokens and attention of shared prefixes where offsets pass 2^32 elements
or workgroups of one launch pass 2^24.  Tolerances as in each operator's own tests."""

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
    yield
    torch.cuda.empty_cache()


def test_norm_of_many_rows():
    """2^24 + 64 rows of a workgroup each, 17 GB of codes out of 64 rows for all tokens: every token's codes are the
    first one's, and those are a small call's."""
    import torch

    from sparse_moe_02_amd.norm import rms_norm

    T, n, W = (1 << 18) + 1, 64, 1032
    x = torch.randn((1, n, W), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").bfloat16()
    want, scale = rms_norm(x, None, out_dtype=torch.int8)
    got, scales = rms_norm(x.expand(T, n, W), None, out_dtype=torch.int8)
    assert torch.equal(scales, scale.expand(T, n, 1))
    for t in range(0, T, 1 << 14):
        assert (got[t:t + (1 << 14)] == want).all(), t


def test_product_of_many_rows():
    """Pairs of a weight tile and 16 rows of x beyond 2^22, and an output of more than 2^32 elements."""
    import torch

    from oracle import step
    from sparse_moe_02_amd.linear import QLinear

    T, n, k = 270000, 16384, 4160
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-2 ** 31, 2 ** 31, (n, k // 8), generator=g, device="cuda", dtype=torch.int64).int()
    s = 0.01 + 0.01 * torch.rand((n, k // 64), generator=g, device="cuda")
    scale, bias = s.half(), (-7.5 * s).half()
    x = torch.randn((T, k), generator=g, device="cuda", dtype=torch.bfloat16)
    out = QLinear(codes, scale, bias)(x)
    rows = [0, 17, 65535, 65536, 131072, 262143, 262144, T - 17, T - 1]
    f = lambda t: t.double().cpu().numpy()
    xr, cols = f(x[rows]), slice(n - 300, n)
    c, sc, b = codes[cols].cpu().numpy(), f(scale[cols]), f(bias[cols])
    ref, _ = step.linear(xr, c, sc, b)
    mass = np.abs(xr) @ np.repeat(31 * np.abs(sc) + np.abs(b), 64, 1).T
    assert (np.abs(f(out[rows][:, cols]) - ref) <= 2.0 ** -8 * np.abs(ref) + (168 + k / 64) * 2.0 ** -24 * mass).all()
    # a sample of the rest against the same rows alone: two results, each off by 2^-8 of itself and 233 u A < 0.03
    # (A < 2000), where the largest ones are above 16
    lin = QLinear(codes, scale, bias)
    for t in range(5, T, T // 20):
        a, b = out[t:t + 32].float(), lin(x[t:t + 32]).float()
        assert (a - b).abs().max() <= 2.0 ** -6 * b.abs().max(), t


@pytest.mark.parametrize("filters", [False, True])
def test_tokens_of_rows_far_apart(filters):
    import torch

    from sparse_moe_02_amd.sample import sample

    V, far = 5003, (1 << 32) + 8
    buf = torch.empty(far + V, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn((2, V), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    logits = buf.as_strided((2, V), (far, 1))
    logits.copy_(rows)
    u = torch.tensor([0.3, 0.7], device="cuda")
    p = (None, torch.tensor([50, 0], dtype=torch.int32, device="cuda"), torch.tensor([0.9, 0.5], device="cuda")) if filters else ()
    for a, b in zip(sample(logits, u, *p, return_prob=True), sample(rows, u, *p, return_prob=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("new", [1, 40])
def test_prefix_in_far_pages(new):
    """Pages whose places lie behind 2^32 elements of the cache, against the same pages of a small one."""
    import torch

    from sparse_moe_02_amd.attn import prefix_attn

    page, hk, D, H = 64, 2, 128, 8
    size = page * hk * D
    pages = (1 << 32) // size + 64
    g = torch.Generator(device="cuda").manual_seed(3)
    small = torch.randn((2, 40, page, hk, D), generator=g, device="cuda").bfloat16()
    big = torch.empty((2, pages, page, hk, D), dtype=torch.bfloat16, device="cuda")
    at = pages - 40
    big[:, at:] = small
    q = torch.randn((3 * new, H, D), generator=g, device="cuda").bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    shared = list(range(16))
    table = [shared + [16 + 3 * i + j for j in range(3)] for i in range(3)]
    lens = [1024 + 150, 1024 + 64, 1024 + 129]
    args = i32([0, new, 2 * new, 3 * new]), i32(lens), i32([0, 3]), i32([1024]), new, 1024, 192
    a, la = prefix_attn(q, small[0], small[1], i32(table), *args, return_lse=True)
    b, lb = prefix_attn(q, big[0], big[1], i32(table) + at, *args, return_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    say(f"pages from {at} of {pages}")


def test_prefixes_of_many_sequences_without_tokens():
    """65535 sequences, each a group, 3 of them with a token: groups times splits of their bounds pass 2^24
    workgroups."""
    import torch

    from sparse_moe_02_amd.attn import prefix_attn

    n, page, hk, D, H = 65535, 16, 4, 64, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    kc, vc = (torch.randn((8, page, hk, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((3, H, D), generator=g, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    has = [0, 33333, n - 1]
    start = torch.zeros(n + 1, **i32)
    for b in has:
        start[b + 1:] += 1
    table = torch.zeros((n, 2), **i32)
    lens, prefix = torch.zeros(n, **i32), torch.zeros(n, **i32)
    small = torch.tensor([[0, 1], [2, 3], [4, 5]], **i32)
    table[has], lens[has], prefix[has] = small, torch.tensor([20, 32, 5], **i32), torch.tensor([16, 9, 0], **i32)
    most = 1, 1 << 20, 1 << 20
    a, la = prefix_attn(q, kc, vc, table, start, lens, torch.arange(n + 1, **i32), prefix, *most, return_lse=True)
    b, lb = prefix_attn(q, kc, vc, small, start[[0, *(x + 1 for x in has)]], lens[has], torch.arange(4, **i32), prefix[has], 1, 16, 32,
                        return_lse=True)
    assert (a.double() - b.double()).abs().max() <= 2.0 ** -7 * vc.abs().max() and (la - lb).abs().max() <= 2.0 ** -18 * (1 + lb.abs().max())
