"""Products whose weights or activations lie at the ends of their types: the smallest and largest block scales, values of x below the
normal range of binary32 and parts of x below it, against 64 bits."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B

pytestmark = pytest.mark.gpu
FP4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def weight(rng, fmt, scale_bytes, cols):
    """A weight of a row for each scale byte, all blocks of it with that byte; its values in 64 bits, without the global scale."""
    n, block = len(scale_bytes), 32 if fmt == "mxfp4" else 16
    codes = rng.integers(0, 16, (n, cols))
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)
    scales = np.repeat(np.array(scale_bytes, np.uint8), cols // block)
    if fmt == "mxfp4":
        s = 2.0 ** (np.array(scale_bytes, np.float64) - 127)
    else:
        e, m = np.array(scale_bytes) >> 3, np.array(scale_bytes) & 7
        s = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    S = None if fmt == "mxfp4" else torch.ones(1, device="cuda")
    w = B.QuantizedWeight(torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), S, n, cols,
                          format=B.FP4Q_MXFP4 if fmt == "mxfp4" else B.FP4Q_NVFP4)
    return w, FP4[codes] * s[:, None]


@pytest.mark.parametrize("m", [3, 12, 48, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("power", [-126, -120, 0, 100, 120])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_ends(fmt, power, dtype, m):
    """x about 2^power.  Of MXFP4 those rows of the weight are looked at whose products lie well within binary32."""
    rng = np.random.default_rng(power + 1000)
    cols = 192
    tags = [0, 1, 2, 5, 30, 127, 200, 249, 252] if fmt == "mxfp4" else [0, 1, 2, 7, 8, 56, 0x7D, 0x7E]
    w, v = weight(rng, fmt, tags, cols)
    x = torch.from_numpy(rng.standard_normal((m, cols)) * 2.0 ** power).to(dtype)
    x = x.clamp(-2.0 ** 125, 2.0 ** 125)
    got = B.matmul(w, x.cuda()).double().cpu().numpy()
    xd = x.double().numpy()
    want, mag = xd @ v.T, np.abs(xd) @ np.abs(v).T
    # as the products' other tests have it: an addition charged 2^-23 of the magnitudes, of a depth of at most 32 + 3 (cols / 32 + 1)
    # + 40; binary32 x in two f16 parts 2^-22, and 2^-38 of the row's largest value; the result's rounding
    tol = mag * ((72 + 3 * (cols / 32 + 1)) * 2.0 ** -23 + 2.0 ** -22)
    if fmt == "nvfp4":
        tol = tol + 2.0 ** -38 * np.abs(xd).max(-1, keepdims=True) * np.abs(v).sum(-1)
    # bf16's steps are of 2^-133 at least: the last of a binary32 value's parts is rounded by up to half of one (and is exact where
    # the value is at least 2^-110, its last bit being 2^-133 then)
    if dtype == torch.float32:
        tol = tol + 2.0 ** -134 * np.abs(v).sum(-1)
    tol = tol + HALF[dtype] * (np.abs(want) + tol)
    # a product of a value and a weight, and the result, within the normal range, far enough for the bound's 2^-24
    keep = np.array([(abs(power + t - 127) < 95) if fmt == "mxfp4" else (-90 < power < 108) for t in tags])
    off = np.abs(got - want)[:, keep]
    assert (off <= tol[:, keep]).all(), f"worst {(off / tol[:, keep]).max():.3g} of the bound, rows {np.array(tags)[keep][np.unique(np.argwhere(~(off <= tol[:, keep]))[:, 1])]}"
