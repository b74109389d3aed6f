"""Products of few rows with 4-bit weights on device tensors (argument marshalling for
``include/linear.h``; every step runs in the HIP kernels).

Calls are enqueued on torch's current stream of the weights' device and never wait for it.
"""

from __future__ import annotations

import torch

from . import binding as B
from ._device import N, on, stream

_TYPES = {torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16, torch.float32: B.MOE_FP32, torch.int8: B.MOE_INT8}


class QLinear:
    """Weights [n][k] of 4 bits: code * scale + bias, one scale and one bias for each group of 64
    along k, in the library's tiles, which are whole when this returns.

    codes: int32 [n][k / 8], element k in bits 4 (k % 8) of word k / 8; scale, bias: float16 or
    bfloat16 [n][k / 64]; all row-major, on any device.  They are laid out once, here; the tensors
    given are not kept."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, bias: torch.Tensor, device="cuda:0"):
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("weights live on a GPU")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        if codes.dim() != 2 or codes.dtype != torch.int32 or codes.shape[0] < 1 or codes.shape[1] < 8 or codes.shape[1] % 8:
            raise ValueError("codes: int32 [n][k / 8], k a multiple of 64, required")
        self.n, self.k = codes.shape[0], 8 * codes.shape[1]
        if scale.dtype not in (torch.float16, torch.bfloat16) or scale.shape != (self.n, self.k // 64):
            raise ValueError(f"scale: float16 or bfloat16 [{self.n}][{self.k // 64}] required")
        if bias.dtype != scale.dtype or bias.shape != scale.shape:
            raise ValueError("bias must have scale's type and shape")
        # whole tiles: rows and groups of zeros behind the last ones
        rows, k = -(-self.n // 16) * 16, -(-self.k // 128) * 128
        s = stream(self.device.index)

        def tiled(t, width, pack):
            t = t.to(self.device)
            if t.shape != (rows, width):
                t = torch.nn.functional.pad(t, (0, width - t.shape[1], 0, rows - t.shape[0]))
            t = t.contiguous()
            o = torch.empty_like(t)
            pack(t.data_ptr(), o.data_ptr(), rows, k, s)
            return o

        with on(self.device.index):
            self.codes = tiled(codes, k // 8, B.moe_pack_codes)
            self.scale, self.bias = (tiled(t, k // 64, B.moe_pack_qparams) for t in (scale, bias))
            torch.cuda.current_stream().synchronize()  # (calls may come on any stream)
        self._index = self.device.index
        self._w = B.moe_linear_weights(self.codes.data_ptr(), self.scale.data_ptr(), self.bias.data_ptr(), self.n, self.k,
                                       _TYPES[scale.dtype])
        self._c = bytes(self._w)

    def __call__(self, x: torch.Tensor, x_scale: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None) -> torch.Tensor:
        """x W^T (see ``moe_linear``).  x: [T][k], 16-byte aligned rows any distance apart, bfloat16 or float16, or int8 with
        x_scale float32 [T][1, k / 64 or k / 128], as ``rms_norm`` gives them.  out: [T][n] of bfloat16, float16 or
        float32, by default a new tensor of out_dtype (x's type, or bfloat16)."""
        t = _TYPES.get(x.dtype)
        if t is None or t == B.MOE_FP32:
            raise ValueError("x: bfloat16, float16 or int8 required")
        hx, T, _, _ = N.rows("x", x, -1, 1, self.k, (N.BF16, N.FP16, 0, N.INT8)[t], self._index)
        if out is None:
            if out_dtype is None:
                out_dtype = torch.bfloat16 if t == B.MOE_INT8 else x.dtype
            if out_dtype not in (torch.bfloat16, torch.float16, torch.float32):
                raise ValueError("out_dtype: bfloat16, float16 or float32 required")
            out = x.new_empty((T, self.n), dtype=out_dtype)
        o = _TYPES.get(out.dtype, B.MOE_INT8)
        if o == B.MOE_INT8:
            raise ValueError("out: bfloat16, float16 or float32 required")
        N.rows("out", out, T, 1, self.n, (N.BF16, N.FP16, N.FP32)[o], self._index)
        sp, group = None, 0
        if (x_scale is not None) != (t == B.MOE_INT8):
            raise ValueError("x_scale: with int8 x, and only with it")
        if x_scale is not None:
            sp = N.address("x_scale", x_scale, N.FP32, self._index, T, -1)
            cols = x_scale.shape[1]
            if cols not in (1, self.k // 64) and 128 * cols != self.k:
                raise ValueError("x_scale: [T][1, k / 64 or k / 128] required")
            group = 0 if cols == 1 else self.k // cols
        if T:
            with on(self._index):
                st = (B._lib or B.lib()).moe_linear(self._c, T, x.data_ptr(), x.stride(0) if T > 1 else 0, t, sp, group,
                                                    out.data_ptr(), out.stride(0) if T > 1 else 0, o, stream(self._index))
            if st:
                raise B.MoeError("moe_linear", st)
        return out
