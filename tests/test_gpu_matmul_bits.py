"""All 24 bits of an activation reach the products: rows whose results are exact in binary32, so that any bit of x that is lost on
the way shows, whatever the number of rows."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROWS = [1, 2, 3, 5, 16, 17, 33, 100, 300, 1200]
# significands that end in the last bit of binary32, of each kind of parts: full ones, gaps, carries, all ones
FULL = [1 + 2.0 ** -23, 1 + 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -23, 2 - 2.0 ** -23, 1 + 2.0 ** -11 - 2.0 ** -23, 1.5 - 2.0 ** -23, 0xAAAAAB * 2.0 ** -23]


def signs(rng, fmt, n, k, rotate=0):
    """A weight of values 1 and -1 (a block's scale of 1), and those values."""
    bits = rng.integers(0, 2, (n, k))
    codes = (2 | bits << 3).astype(np.uint8)
    return handle(codes, fmt, n, k, rotate), 1.0 - 2.0 * bits


def handle(codes, fmt, n, k, rotate=0):
    block = 32 if fmt == "mxfp4" else 16
    packed = torch.from_numpy(codes[:, 0::2] | codes[:, 1::2] << 4).cuda()
    scales = torch.full((n * k // block,), 127 if fmt == "mxfp4" else 0x38, dtype=torch.uint8, device="cuda")
    S = None if fmt == "mxfp4" else torch.ones(1, device="cuda")
    return B.QuantizedWeight(packed, scales, S, n, k, format=B.FP4Q_MXFP4 if fmt == "mxfp4" else B.FP4Q_NVFP4, rotate=rotate)


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n,k", [(20, 576), (300, 1056)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_one_value_of_a_row(fmt, n, k, m):
    """A row with one value that needs all its bits, at every place in turn: the product is that value or its negative."""
    rng = np.random.default_rng(m + k)
    h, w = signs(rng, fmt, n, k)
    for first in range(0, min(k, 48 * m), m):
        at = (first + np.arange(m)) % k
        v = rng.choice(FULL, m).astype(np.float32) * (2.0 ** rng.integers(-40, 41, m)).astype(np.float32)
        x = np.zeros((m, k), np.float32)
        x[np.arange(m), at] = v
        got = B.matmul(h, torch.from_numpy(x).cuda()).cpu().numpy()
        want = v[:, None] * w[:, at].T
        assert (got == want).all(), f"values at {at[np.nonzero((got != want).any(1))[0][:4]]}"


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_large_values_beside_weights_of_zero(fmt, m):
    """A row whose largest values meet weights of zero: the small ones are all that its result has."""
    n, k = 40, 640
    rng = np.random.default_rng(m)
    codes = (2 | rng.integers(0, 2, (n, k)) << 3).astype(np.uint8)
    w = np.where(codes & 8, -1.0, 1.0)
    none = np.arange(k) % 5 == 0
    codes[:, none], w[:, none] = 0, 0.0
    h = handle(codes, fmt, n, k)
    for large in (2.0 ** 20, 2.0 ** 45, float(np.finfo(np.float32).min)):
        x = np.zeros((m, k), np.float32)
        x[:, none] = large
        at = 1 + 5 * rng.integers(0, k // 5, m)
        x[np.arange(m), at] = rng.choice(FULL, m)
        got = B.matmul(h, torch.from_numpy(x).cuda()).cpu().numpy()
        want = x[np.arange(m), at][:, None] * w[:, at].T
        assert (got == want).all()


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rotated_values_that_nearly_cancel(fmt, dtype, m):
    """A block (1, d, 0, ...) is c (1 + d) and c (1 - d) in turn once rotated, c = 1 / sqrt(block); a row of the weight that has 1
    and -1 at two neighbours gives 2 c d.  Each of the two values is rounded twice in binary32 at most, by 2^-24 c (1 + d)
    (with c = 1 / 4 not at all), and c itself by 2^-25 relative: 2^-21 c in all."""
    block = 32 if fmt == "mxfp4" else 16
    n, k = 24, 18 * block
    rng = np.random.default_rng(m)
    pair = rng.integers(0, k // 2, n)
    codes = np.zeros((n, k), np.uint8)
    codes[np.arange(n), 2 * pair], codes[np.arange(n), 2 * pair + 1] = 2, 2 | 8
    h = handle(codes, fmt, n, k, rotate=block)
    for d in (2.0 ** -10, 2.0 ** -14, 2.0 ** -18):
        x = np.zeros((m, k), np.float32)
        up = 2.0 ** rng.integers(-20, 21, (m, k // block))
        x[:, 0::block], x[:, 1::block] = up, up * d
        got = B.matmul(h, torch.from_numpy(x).to(dtype).cuda()).double().cpu().numpy()
        size = up[:, 2 * pair // block] / np.sqrt(block)
        half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24  # of the result's rounding
        tol = size * (0.0 if fmt == "nvfp4" else 2.0 ** -21 * (1 + half)) + size * 2 * d * (0.0 if fmt == "nvfp4" else half)
        assert (np.abs(got - 2 * d * size) <= tol).all()
