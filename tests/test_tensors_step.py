"""The tensor reader's rows and groups: what they return, and what they refuse (with an exception, whatever the
argument is)."""

import struct

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def N():
    from sparse_moe_02_amd._device import N

    return N


def test_host_tensors_and_other_things_are_refused(N):
    t = torch.zeros((2, 64), dtype=torch.bfloat16)
    for bad in (t, t[None], t[0], None, 3, "t", [t], torch.zeros(3, dtype=torch.int32)):
        for index in (-1, 0):
            with pytest.raises(ValueError):
                N.rows("t", bad, -1, -1, -1, N.BF16, index)
            with pytest.raises(ValueError):
                N.groups(bad, bad, index)
    for f in (N.rows, N.groups):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        N.rows(b"t", t, -1, -1, -1, N.BF16, 0)
    with pytest.raises(TypeError):
        N.rows("t", t, "2", -1, -1, N.BF16, 0)


def test_the_wrappers_refuse_host_tensors(N):
    from sparse_moe_02_amd.attn import prefix_attn
    from sparse_moe_02_amd.linear import QLinear
    from sparse_moe_02_amd.norm import rms_norm
    from sparse_moe_02_amd.sample import sample

    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        rms_norm(x, None)
    with pytest.raises(ValueError):
        sample(x, torch.zeros(2))
    with pytest.raises(ValueError):
        prefix_attn(x[:, None], x[None, None], x[None, None], i[None], i, i[:1], i, i[:1], 1, 1, 1)
    with pytest.raises(ValueError):
        QLinear(torch.zeros((16, 8), dtype=torch.int32), torch.zeros((16, 1)).half(), torch.zeros((16, 1)).half(), device="cpu")


@pytest.mark.gpu
def test_what_they_return(N):
    z = lambda *n, **k: torch.zeros(*n, device="cuda", **k)
    t = z(5, 8, 192, dtype=torch.float16)[:, 1:7:2, 64:128]
    got = N.rows("t", t, -1, 3, 64, N.FP16, 0)
    assert got[1:] == (5, 3, 64) and struct.unpack("Pqq", got[0]) == (t.data_ptr(), 8 * 192, 2 * 192)
    t = z(5, 192, dtype=torch.int8)[:, 64:128]
    got = N.rows("t", t, 5, 1, -1, N.INT8, 0)
    assert got[1:] == (5, 1, 64) and struct.unpack("Pqq", got[0]) == (t.data_ptr(), 192, 0)
    starts, lens = z(4, dtype=torch.int32), z(3, dtype=torch.int32)
    got, n = N.groups(starts, lens, 0)
    assert n == 3 and struct.unpack("PPi4x", got) == (starts.data_ptr(), lens.data_ptr(), 3)
    for bad in (dict(T=4), dict(heads=2), dict(D=32), dict(type=N.FP8), dict(index=1)):
        a = dict(T=-1, heads=1, D=-1, type=N.INT8, index=0)
        a.update(bad)
        with pytest.raises(ValueError):
            N.rows("t", t, *a.values())
    with pytest.raises(ValueError):
        N.rows("t", z(5, 64, dtype=torch.int8).t(), -1, 1, -1, N.INT8, 0)
    with pytest.raises(ValueError):
        N.groups(starts, lens[:2], 0)
    with pytest.raises(ValueError):
        N.groups(starts.long(), lens, 0)
