"""The wrappers' tensor reader: what it returns, and what it refuses (with an exception, whatever the
argument is)."""

import struct

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def N():
    from sparse_moe_02_amd._device import N

    return N


def test_host_tensors_and_other_things_are_refused(N):
    z = torch.zeros
    t = z((2, 3, 64), dtype=torch.bfloat16)
    for bad in (t, None, 3, "t", [t]):
        for index in (-1, 0):
            with pytest.raises(ValueError):
                N.address("t", bad, N.BF16, index, 2, 3, 64)
            with pytest.raises(ValueError):
                N.heads("t", bad, -1, -1, 64, N.BF16, index)
            with pytest.raises(ValueError):
                N.cache(bad, bad, index)
            with pytest.raises(ValueError):
                N.memory(bad, 3, index)
            with pytest.raises(ValueError):
                N.batch(bad, bad, bad, None, index)
    for f in (N.address, N.heads, N.cache, N.batch, N.memory):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        N.address("t", t, N.BF16, 0, *[1] * 9)
    with pytest.raises(TypeError):
        N.address("t", t, "bf16", 0)
    with pytest.raises(TypeError):
        N.address(b"t", t, N.BF16, 0)
    with pytest.raises(OverflowError):
        N.address("t", t, N.BF16, 0, 1 << 64)


@pytest.mark.gpu
def test_what_it_returns(N):
    z = lambda *n, **k: torch.zeros(*n, device="cuda", **k)
    t = z(5, 8, 192, dtype=torch.float16)[:, 1:7:2, 64:128]
    got, T, H = N.heads("t", t, -1, 3, 64, N.FP16, 0)
    assert (T, H) == (5, 3) and struct.unpack("Pqq", got) == (t.data_ptr(), 8 * 192, 2 * 192)
    assert struct.unpack("Pqq", N.heads("t", t[:1, :1], 1, 1, 64, N.FP16, 0)[0]) == (t.data_ptr(), 0, 0)
    k = z(2, 6, 16, 4, 128, dtype=torch.bfloat16)
    got = N.cache(k[0], k[1], 0)
    assert got[1:3] == (4, 128) and got[3] == N.BF16
    from sparse_moe_02_amd import binding as B

    assert struct.unpack("PPqqqiiiii4x", got[0]) == (k[0].data_ptr(), k[1].data_ptr(), 16 * 4 * 128, 4 * 128, 128, 6, 16, 4,
                                                     128, B.MOE_BF16)
    i32 = dict(dtype=torch.int32)
    table, q_start, kv_len, row = z(7, 9, **i32), z(4, **i32), z(7, **i32), z(3, **i32)
    got, n = N.batch(table, q_start, kv_len, row, 0)
    want = (q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), row.data_ptr(), 3, 7, 9)
    assert n == 3 and struct.unpack("PPPPiii4x", got) == want
    assert struct.unpack("PPPPiii4x", N.batch(table, q_start, kv_len, None, 0)[0])[3] == 0
    assert struct.unpack("Pqqqi4x", N.memory(k, 6, 0)) == (k.data_ptr(), 6 * 16 * 4 * 128 * 2, 16 * 4 * 128 * 2,
                                                           16 * 4 * 128 * 2, 2)
    assert N.address("k", k, N.BF16, 0) == N.address("k", k, N.BF16, 0, 2, -1, 16, 4, 128) == k.data_ptr()


@pytest.mark.gpu
def test_refusals_on_the_device(N):
    z = lambda *n, **k: torch.zeros(*n, device="cuda", **k)
    t = z(2, 3, 64, dtype=torch.bfloat16)
    for args in ((N.FP16, 0, 2, 3, 64), (N.BF16, 1, 2, 3, 64), (N.BF16, -1, 2, 3, 64), (N.BF16, 0, 2, 3), (N.BF16, 0, 2, 4, 64)):
        with pytest.raises(ValueError):
            N.address("t", t, *args)
    with pytest.raises(ValueError):
        N.address("t", t[:, :, ::2], N.BF16, 0)
    for bad in (t[:, :, ::2], t.float(), t[0], t[:, :, :32]):
        with pytest.raises(ValueError):
            N.heads("t", bad, -1, -1, 64, N.BF16, 0)
    with pytest.raises(ValueError):
        N.heads("t", t, 3, 3, 64, N.BF16, 0)
    with pytest.raises((ValueError, RuntimeError)):  # no strides
        N.address("t", t.float().to_sparse(), N.FP32, 0)
    k = z(6, 16, 4, 128, dtype=torch.bfloat16)
    for k0, v0 in ((k, k.half()), (k.float(), k.float()), (k, k[:5]), (k, k.transpose(1, 2).contiguous().transpose(1, 2)),
                   (k[0], k[0]), (k[..., ::2], k[..., ::2]), (k, k.cpu())):
        with pytest.raises(ValueError):
            N.cache(k0, v0, 0)
    i32 = dict(dtype=torch.int32)
    table, q_start, kv_len, row = z(7, 9, **i32), z(4, **i32), z(7, **i32), z(3, **i32)
    for bad in ((table.long(), q_start, kv_len, row), (table[:, :3], q_start, kv_len, row), (table, table, kv_len, row),
                (table, q_start, kv_len[1:], row), (table, q_start, kv_len, row[1:]), (table, q_start.cpu(), kv_len, row)):
        with pytest.raises(ValueError):
            N.batch(*bad, 0)
    for bad in (k, z(2, 6), z(2, 6, 4, 4).transpose(2, 3), z(0, 6, 8)):
        with pytest.raises(ValueError):
            N.memory(bad, 6 if bad is not k else 5, 0)
