"""Products whose operands pass 32 bits of bytes: rows of x, of y and of the weight beyond 4 GiB."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from matmul_common import Made, close, product64, rounded

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("rotate", [False, True])
def test_many_rows_of_x(rotate):
    """600,000 rows of 4096 values (4.9 GB; rotated, their parts too)."""
    rng = np.random.default_rng(1)
    w = Made(rng, "nvfp4", 40, 4096, rotate)
    m = 600_000
    x = torch.randn(m, 4096, device="cuda", dtype=BF16, generator=torch.Generator(device="cuda").manual_seed(1))
    got = B.matmul(w.handle(), x)
    at = torch.tensor([0, 1, 127, 128, 262143, 262144, 524287, 524288, 599_998, 599_999])
    y, tol = product64(w, x[at.cuda()].cpu())
    close(got[at.cuda()], y, rounded(y, tol, BF16))


def test_many_values_of_y():
    """70,000 rows of 33,000 results (4.6 GB)."""
    rng = np.random.default_rng(2)
    w = Made(rng, "mxfp4", 33_000, 32)
    x = torch.randn(70_000, 32, device="cuda", dtype=BF16, generator=torch.Generator(device="cuda").manual_seed(2))
    got = B.matmul(w.handle(), x)
    at = torch.tensor([0, 1, 65_075, 65_076, 65_100, 69_999])
    y, tol = product64(w, x[at.cuda()].cpu())
    close(got[at.cuda()], y, rounded(y, tol, BF16))


@pytest.mark.parametrize("tokens", [2, 20, 70])
def test_many_rows_of_the_weight(tokens):
    """2,200,000 weight rows of 4096 values (4.5 GB of codes): those around 2^32 bytes and the last ones."""
    n, k = 2_200_000, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (n * k // 2,), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(40, 90, (n * k // 16,), dtype=torch.uint8, device="cuda", generator=g)
    x = torch.randn(tokens, k, device="cuda", dtype=BF16, generator=g)
    S = 0.01
    got = B.matmul(B.QuantizedWeight(codes, scales, torch.tensor([S], device="cuda"), n, k), x)
    at = [0, 1, 2_097_151, 2_097_152, 2_097_153, 2_199_999]
    w = Made(np.random.default_rng(0), "nvfp4", 1, 16, S=S)
    from oracle import ref
    rows = [np.asarray(ref.dequantize(codes[r * k // 2:(r + 1) * k // 2].cpu().numpy(), scales[r * k // 16:(r + 1) * k // 16].cpu().numpy(),
                                      S, 1, k), np.float64).reshape(k) for r in at]
    w.values, w.k = np.stack(rows), k
    y, tol = product64(w, x.cpu())
    close(got[:, at], y, rounded(y, tol, BF16))


@pytest.mark.parametrize("tokens,dtype,rotate", [(1, BF16, False), (16, BF16, True), (20, torch.float32, False), (130, BF16, False),
                                                 (130, BF16, True)])
def test_the_longest_rows(tokens, dtype, rotate):
    """2^22 columns, the most that there can be, of a weight whose scales differ along the row."""
    n, k = 20, 1 << 22
    rng = np.random.default_rng(4)
    w = Made(rng, "nvfp4", n, 16, rotate, S=0.01)
    w.codes, w.scales = rng.integers(0, 256, n * k // 2, dtype=np.uint8), rng.integers(40, 90, n * k // 16, dtype=np.uint8)
    from oracle import ref
    w.values, w.k = np.asarray(ref.dequantize(w.codes, w.scales, 0.01, n, k), np.float64).reshape(n, k), k
    x = torch.randn(tokens, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)
    got = B.matmul(w.handle(), x)
    at = sorted({0, tokens // 2, tokens - 1})
    y, tol = product64(w, x[at].cpu())
    close(got[at], y, rounded(y, tol, dtype))
