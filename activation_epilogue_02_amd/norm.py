"""RMS norm with the residual's addition and 8-bit outputs, and its backward
pass: the ctypes layer over include/ge_rms_norm.h (argument marshalling only;
every step runs in the library's HIP kernels)."""
from __future__ import annotations

import ctypes

import torch

from .binding import (DTYPE_CODE, ELEM_SIZE, TORCH_DTYPE, _check, _device, _stream, ge_norm_desc, lib, mx_scale_ld,
                      tensor_args)

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
        self._lib, self._args = lib(), tensor_args()
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

    def forward(self, x, gamma, y, residual=None, h=None, scales=None, rstd=None, rows=None, stream=None):
        """Writes y (and scales, h, rstd where given) for `rows` rows.

        Every tensor has to hold those rows in the handle's types and strides: GemmEpilogError with GE_ERR_DTYPE or
        GE_ERR_SHAPE otherwise (GE_ERR_HIP: not on the current GPU, whose stream takes the launch)."""
        n, cols, ld, t = self.rows if rows is None else rows, self.cols, self.ld, self.dtype
        matrix, vector = self._args.matrix, self._args.vector
        first = y if y is not None else gamma   # (the library refuses what is missing)
        dev = -1 if first is None else _device(first, "RmsNorm.forward: y")
        xp = None if x is None else matrix(x, n, cols, ld, t, dev, "RmsNorm.forward: x")
        rp = None if residual is None else matrix(residual, n, cols, ld, t, dev, "RmsNorm.forward: residual")
        gp = None if gamma is None else vector(gamma, cols, t, dev, "RmsNorm.forward: gamma")
        hp = None if h is None else matrix(h, n, cols, ld, t, dev, "RmsNorm.forward: h")
        yp = None if y is None else matrix(y, n, cols, self.ldy, self.out_dtype, dev, "RmsNorm.forward: y")
        sp = None
        if scales is not None:
            sp = (self._args.scale_rows(scales, n, self.scale_ld, dev, "RmsNorm.forward: scales")
                  if self.scale_dtype is torch.uint8 else
                  vector(scales, n, torch.float32, dev, "RmsNorm.forward: scales"))
        vp = None if rstd is None else vector(rstd, n, torch.float32, dev, "RmsNorm.forward: rstd")
        _check(self._lib.ge_rms_norm_forward(self.h, n, xp, rp, gp, hp, yp, sp, vp, _stream(stream)),
               "ge_rms_norm_forward")

    def backward(self, dy, h, gamma, rstd, dx, dgamma=None, dh=None, workspace=None, rows=None, stream=None):
        """Writes dx (the gradient of x and of the residual) and, if given,
        dgamma, which needs a workspace of workspace_bytes.  Checks as forward's."""
        n, cols, ld, t = self.rows if rows is None else rows, self.cols, self.ld, self.dtype
        matrix, vector = self._args.matrix, self._args.vector
        first = dx if dx is not None else gamma
        dev = -1 if first is None else _device(first, "RmsNorm.backward: dx")
        yp = None if dy is None else matrix(dy, n, cols, ld, t, dev, "RmsNorm.backward: dy")
        hp = None if h is None else matrix(h, n, cols, ld, t, dev, "RmsNorm.backward: h")
        gp = None if gamma is None else vector(gamma, cols, t, dev, "RmsNorm.backward: gamma")
        vp = None if rstd is None else vector(rstd, n, torch.float32, dev, "RmsNorm.backward: rstd")
        ep = None if dh is None else matrix(dh, n, cols, ld, t, dev, "RmsNorm.backward: dh")
        xp = None if dx is None else matrix(dx, n, cols, ld, t, dev, "RmsNorm.backward: dx")
        dp = None if dgamma is None else vector(dgamma, cols, t, dev, "RmsNorm.backward: dgamma")
        ws, size = None, 0
        if workspace is not None:
            ws, size = self._args.workspace(workspace, dev, "RmsNorm.backward: workspace")
        _check(self._lib.ge_rms_norm_backward(self.h, n, yp, hp, gp, vp, ep, xp, dp, ws, size, _stream(stream)),
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
