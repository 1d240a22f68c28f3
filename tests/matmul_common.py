"""What the tests of the products with 4-bit weights share: weights with known bytes, and the products in 64 bits (numpy,
on the host) with bounds on how far a result of the kernels' arithmetic may lie from them."""
import math

import numpy as np
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from kv_common import blocks_times, values
from oracle import ref

FMT = {"nvfp4": (B.FP4Q_NVFP4, ref.NVFP4, 16), "mxfp4": (B.FP4Q_MXFP4, ref.MXFP4, 32)}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


class Made:
    """A weight [n, k] with the oracle's bytes; `values`: what its bytes stand for, in the domain they are stored in."""

    def __init__(self, rng, fmt, n, k, rotate=False, S=0.013):
        f, rf, self.block = FMT[fmt]
        self.fmt, self.n, self.k, self.rotate, self.S = fmt, n, k, rotate, np.float32(S)
        self.format = f
        if n and k:
            q = ref.quantize(values(rng, (n, k)), fmt=rf, global_scale=float(self.S))
            self.codes, self.scales = q["codes"].reshape(-1), q["scales"].reshape(-1)
            y = ref.dequantize(q["codes"], q["scales"], float(self.S), n, k, fmt=rf)
        else:
            self.codes, self.scales = np.zeros(0, np.uint8), np.zeros(0, np.uint8)
            y = np.zeros((n, k))
        self.values = np.asarray(y, np.float64).reshape(n, k)

    def handle(self, device="cuda"):
        S = torch.tensor([self.S], device=device) if self.fmt == "nvfp4" else None
        return B.QuantizedWeight(torch.from_numpy(self.codes.copy()).to(device), torch.from_numpy(self.scales.copy()).to(device),
                                 S, self.n, self.k, format=self.format, rotate=self.block if self.rotate else 0,
                                 require_cuda=device != "cpu")


def rows_of_x(rng, m, k, dtype):
    return torch.from_numpy(values(rng, (m, k))).to(dtype) if m and k else torch.zeros(m, k, dtype=dtype)


def product64(w, x):
    """(x W^T, bound of |error| before the result's rounding), in 64 bits.

    A product passes through at most `depth` additions: those of the 32 products of a matrix instruction, one for each
    instruction and part of x along the row, and the joining of the waves and splits; an addition inside the matrix
    core may cut instead of rounding, so each is charged 2^-23 of the sum of magnitudes.  Rotated x: log2(block) + 1
    binary32 roundings of sums within a block.  Parts of x: NVFP4 in f16, rotated bf16 in one (half a step, 2^-11), binary32
    in two (2^-22), and what falls below f16's range under 2^-38 of the row's largest value; MXFP4 in bf16,
    rotated bf16 in two (half a step of what cutting to the first leaves, 2^-7 2^-8), binary32 in three (none).  The
    step fl32(s S) of a dequantized value is rounded once, where the kernels apply S once at the end: 2^-23."""
    v = x.double().numpy()
    n = w.block
    A = np.abs(v)
    nv = w.fmt == "nvfp4"
    parts, cut = ((3, 2.0 ** -22 if nv else 0.0) if x.dtype == torch.float32 else (1, 0.0))
    extra = np.zeros_like(v)
    if w.rotate and w.k:
        if x.dtype == torch.bfloat16:
            parts, cut = 2, 2.0 ** -11 if nv else 2.0 ** -15
        v = blocks_times(v, n)
        whole = np.repeat(A.reshape(-1, n).sum(-1), n).reshape(A.shape) / math.sqrt(n)
        extra = whole * (math.log2(n) + 1) * 2.0 ** -24
        A = np.abs(v)
    mag = np.abs(w.values)
    depth = 32 + parts * (w.k / 32 + 1) + 40
    tol = (A @ mag.T) * (depth * 2.0 ** -23 + 2.0 ** -22 + cut) + extra @ mag.T
    if nv and w.k and len(A):
        tol = tol + 2.0 ** -38 * A.max(-1, keepdims=True) * mag.sum(-1)
    return v @ w.values.T, tol


def rounded(y, tol, dtype):
    """The bound with the result's own rounding added."""
    return tol + HALF[dtype] * (np.abs(y) + tol) + 1e-37


def close(got, want, tol):
    off = np.abs(got.double().cpu().numpy() - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(off / tol):.3g} of the bound at {np.argwhere(bad)[:4].tolist()}"
