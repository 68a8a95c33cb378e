"""RMS norm with the residual's addition and 8-bit outputs, and its backward
pass: the ctypes layer over include/ge_rms_norm.h (argument marshalling only;
every step runs in the library's HIP kernels)."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .binding import (DTYPE_CODE, ELEM_SIZE, GE_ERR_DTYPE, GE_ERR_SHAPE, TORCH_DTYPE, GemmEpilogError, _check,
                      _stream, ge_norm_desc, lib, mx_scale_ld)

GE_NORM_PLAIN, GE_NORM_E4M3_ROW, GE_NORM_MX = 0, 1, 2
NORM_OUT_CODE = {"plain": GE_NORM_PLAIN, "e4m3_row": GE_NORM_E4M3_ROW, "mx": GE_NORM_MX}


class RmsNorm:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * gamma, on rows of
    `cols` values.

    dtype  "f32", "f16" or "bf16": x, residual, h, gamma, and the gradients
    out    "plain" (y in dtype), "e4m3_row" (E4M3 codes, one fp32 scale per
           row) or "mx" (E4M3 codes, one E8M0 scale byte per 32 columns, rows
           of mx_scale_ld(cols) bytes)
    rows   the most rows of a call; forward and backward take fewer with rows=
    ld     row stride in elements of x, residual, h and the gradients; ldy of y
           (both default to cols rounded up to 16 bytes)
    """

    def __init__(self, rows, cols, dtype, out="plain", eps=1e-6, ld=None, ldy=None):
        self.h = None
        t = DTYPE_CODE[dtype] if not isinstance(dtype, int) else dtype
        o = NORM_OUT_CODE[out] if isinstance(out, str) else out
        e = 16 // ELEM_SIZE[t]
        ey = e if o == GE_NORM_PLAIN else 16
        self.desc = ge_norm_desc(rows, cols, t, o, -(-cols // e) * e if ld is None else ld,
                                 -(-cols // ey) * ey if ldy is None else ldy, eps)
        h = ctypes.c_void_p()
        self._lib = lib()
        _check(self._lib.ge_rms_norm_create(ctypes.byref(h), ctypes.byref(self.desc)), "ge_rms_norm_create")
        self.h = h.value
        self.rows, self.cols, self.ld, self.ldy = rows, cols, self.desc.ld, self.desc.ldy
        self.dtype = TORCH_DTYPE[t]
        self.out_dtype = self.dtype if o == GE_NORM_PLAIN else torch.float8_e4m3fn
        self.scale_dtype, self.scale_ld = ((torch.uint8, mx_scale_ld(cols)) if o == GE_NORM_MX else (torch.float32, 1))
        s = ctypes.c_size_t()
        _check(self._lib.ge_rms_norm_workspace_size(self.h, ctypes.byref(s)), "ge_rms_norm_workspace_size")
        self.workspace_bytes = s.value

    def alloc_outputs(self, device="cuda"):
        """(y, scales) for a full call; scales is None for the plain output."""
        y = torch.empty(self.rows, self.ldy, dtype=self.out_dtype, device=device)[:, :self.cols]
        if self.desc.out == GE_NORM_E4M3_ROW:
            return y, torch.empty(self.rows, dtype=torch.float32, device=device)
        if self.desc.out == GE_NORM_MX:
            return y, torch.full((self.rows, mx_scale_ld(self.cols)), 127, dtype=torch.uint8, device=device)
        return y, None

    def _matrix(self, t, ld, dtype, rows, what) -> Optional[int]:
        """The address of a matrix of at least `rows` rows of cols values, row stride ld."""
        if t is None:
            return None
        if t.dtype is not dtype:
            raise GemmEpilogError(GE_ERR_DTYPE, what)
        if t.numel() < rows * self.cols or (rows > 1 and t.stride(0) != ld):
            raise GemmEpilogError(GE_ERR_SHAPE, what)
        return t.data_ptr()

    def _vector(self, t, dtype, count, what) -> Optional[int]:
        """The address of `count` packed values."""
        if t is None:
            return None
        if t.dtype is not dtype:
            raise GemmEpilogError(GE_ERR_DTYPE, what)
        if t.numel() < count or not t.is_contiguous():
            raise GemmEpilogError(GE_ERR_SHAPE, what)
        return t.data_ptr()

    def forward(self, x, gamma, y, residual=None, h=None, scales=None, rstd=None, rows=None, stream=None):
        """Writes y (and scales, h, rstd where given) for `rows` rows."""
        n = self.rows if rows is None else rows
        _check(self._lib.ge_rms_norm_forward(
            self.h, n, self._matrix(x, self.ld, self.dtype, n, "RmsNorm.forward: x"),
            self._matrix(residual, self.ld, self.dtype, n, "RmsNorm.forward: residual"),
            self._vector(gamma, self.dtype, self.cols, "RmsNorm.forward: gamma"),
            self._matrix(h, self.ld, self.dtype, n, "RmsNorm.forward: h"),
            self._matrix(y, self.ldy, self.out_dtype, n, "RmsNorm.forward: y"),
            self._vector(scales, self.scale_dtype, n * self.scale_ld, "RmsNorm.forward: scales"),
            self._vector(rstd, torch.float32, n, "RmsNorm.forward: rstd"), _stream(stream)), "ge_rms_norm_forward")

    def backward(self, dy, h, gamma, rstd, dx, dgamma=None, dh=None, workspace=None, rows=None, stream=None):
        """Writes dx (the gradient of x and of the residual) and, if given,
        dgamma, which needs a workspace of workspace_bytes."""
        n = self.rows if rows is None else rows
        _check(self._lib.ge_rms_norm_backward(
            self.h, n, self._matrix(dy, self.ld, self.dtype, n, "RmsNorm.backward: dy"),
            self._matrix(h, self.ld, self.dtype, n, "RmsNorm.backward: h"),
            self._vector(gamma, self.dtype, self.cols, "RmsNorm.backward: gamma"),
            self._vector(rstd, torch.float32, n, "RmsNorm.backward: rstd"),
            self._matrix(dh, self.ld, self.dtype, n, "RmsNorm.backward: dh"),
            self._matrix(dx, self.ld, self.dtype, n, "RmsNorm.backward: dx"),
            self._vector(dgamma, self.dtype, self.cols, "RmsNorm.backward: dgamma"),
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream)),
            "ge_rms_norm_backward")

    def describe(self) -> str:
        buf = ctypes.create_string_buffer(256)
        _check(self._lib.ge_rms_norm_describe(self.h, buf, 256), "ge_rms_norm_describe")
        return buf.value.decode()

    def free(self):
        if self.h:
            self._lib.ge_rms_norm_free(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
