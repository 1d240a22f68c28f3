"""Every kernel that a product can be dispatched to (matmul_forms) against 64 bits, all results of each call."""
import math

import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from matmul_forms import ONE_PART, THREE_PARTS

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
FP4 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
KINDS = [("bf16", BF16, False, s) for s in ONE_PART] + [("f32", F32, False, s) for s in THREE_PARTS] + \
        [("rotated", BF16, True, s) for s in THREE_PARTS]


def weight(g, fmt, n, k, rotate):
    """Random codes under scales that make a sum over a row about 1, and what they stand for in 64 bits."""
    block = 32 if fmt == "mxfp4" else 16
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    v = torch.tensor(FP4, dtype=F64, device="cuda")[torch.stack((codes & 15, codes >> 4), -1).long()].reshape(n, k)
    small = -int(round(math.log2(3 * math.sqrt(max(k, 1)))))
    if fmt == "mxfp4":
        scales = torch.randint(126, 129, (n, k // block), dtype=torch.int32, device="cuda", generator=g) + small
        s, scales, S = torch.exp2(scales.to(F64) - 127), scales.to(torch.uint8), None
    else:
        scales = torch.randint(48, 64, (n, k // block), dtype=torch.uint8, device="cuda", generator=g)
        S = torch.tensor([2.0 ** small * 1.37], device="cuda")
        s = scales.view(torch.float8_e4m3fn).to(F64) * S.to(F64)
    w = B.QuantizedWeight(codes, scales, S, n, k, format=B.FP4Q_MXFP4 if fmt == "mxfp4" else B.FP4Q_NVFP4, rotate=block if rotate else 0)
    return w, (v.reshape(n, -1, block) * s[..., None]).reshape(n, k)


def turned(x, block):
    """Each block of x (64 bits) times the orthonormal Hadamard matrix."""
    h = torch.ones(1, 1, dtype=F64, device="cuda")
    while h.shape[0] < block:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return torch.mm(x.reshape(-1, block), h / math.sqrt(block)).reshape(x.shape)


def sums(x, v, block, rotate, parts):
    """(x W^T, a bound of its error) in 64 bits.  At most `depth` additions: 32 in a matrix instruction, one for each
    instruction and part along the row, and 40 to join waves and splits; each may be off by 2^-23 of the magnitudes that it
    adds, an addition in the matrix core being cut instead of rounded.  Rotated: log2(block) + 1 roundings of binary32 sums of a
    block.  The global scale is one rounding more."""
    k = x.shape[1]
    a, extra = x, None
    if rotate:
        a = turned(x, block)
        whole = x.abs().reshape(-1, k // block, block).sum(-1, keepdim=True) / math.sqrt(block)
        extra = whole.expand(-1, -1, block).reshape(x.shape) * ((math.log2(block) + 1) * 2.0 ** -24)
    depth = 32 + parts * (k / 32 + 1) + 40
    tol = torch.mm(a.abs(), v.abs().t()) * (depth * 2.0 ** -23 + 2.0 ** -24)
    if rotate:
        tol += torch.mm(extra, v.abs().t())
    return torch.mm(a, v.t()), tol


def block_of(fmt):
    return 32 if fmt == "mxfp4" else 16


def silu(g):
    return g / (1 + torch.exp(-g))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("weights", [1, 2])
@pytest.mark.parametrize("kind,dtype,rotate,size", KINDS, ids=[f"{c[0]}-{'x'.join(map(str, c[3]))}" for c in KINDS])
def test_against_64_bits(kind, dtype, rotate, size, weights, fmt):
    n, k, m = size
    gen = torch.Generator(device="cuda").manual_seed(n + 31 * k + 977 * m + weights)
    made = [weight(gen, fmt, n, k, rotate) for _ in range(weights)]
    x = torch.randn(m, k, device="cuda", generator=gen).to(dtype)
    parts = 1 if kind == "bf16" else 3
    got = B.matmul(made[0][0], x) if weights == 1 else B.gated(made[0][0], made[1][0], x)
    assert got.dtype == dtype and tuple(got.shape) == (m, n)
    both = [sums(x.to(F64), v, block_of(fmt), rotate, parts) for _, v in made]
    y, tol = both[0]
    if weights == 2:
        # silu's slope is at most 1.1, and its own arithmetic a few roundings and those of its exponent
        (u, tu), a = both[1], silu(y)
        ta = 1.1 * tol + a.abs() * ((8 + 8 * y.abs()) * 2.0 ** -24)
        y, tol = a * u, ta * u.abs() + a.abs() * tu + ta * tu + (a * u).abs() * 2.0 ** -24
    off = (got.to(F64) - y).abs()
    bad = ~(off <= tol + HALF[dtype] * (y.abs() + tol) + 1e-37)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[:4].tolist()}"
    if weights == 1 and kind == "f32":
        # values of both signs: a partial sum is of the size of the result's spread, not of the sum of magnitudes.  Each of the
        # additions is off by 2^-23 of it at most, so that the spread of the error is at most `depth` of them; twice
        # that for what a sample strays, and the result's own rounding
        spread = torch.mm(x.to(F64).square(), made[0][1].square().t()).sqrt()
        depth = 32 + parts * (k / 32 + 1) + 40
        ratio = float((off / spread).square().mean().sqrt())
        assert ratio <= 2 * depth * 2.0 ** -23 + 2.0 ** -24, f"spread of the error {ratio:.3g} of the results'"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("weights", [1, 2])
@pytest.mark.parametrize("size", THREE_PARTS, ids=lambda s: "x".join(map(str, s)))
def test_all_bits_of_a_single_value(size, weights, fmt):
    """Rows of one value of 24 bits each: its parts' products (14 bits each) add up exactly but for the last addition, which rounds
    or cuts to 24 bits, and the global scale; a part that were lost would be 2^-17 of the result or more."""
    n, k, m = size
    gen = torch.Generator(device="cuda").manual_seed(n + 31 * k + 977 * m + weights)
    made = [weight(gen, fmt, n, k, False) for _ in range(weights)]
    at = torch.randint(0, k, (m,), device="cuda", generator=gen)
    v = torch.randint(1 << 23, 1 << 24, (m,), device="cuda", generator=gen) | 0x0101  # each part has bits
    v = v.to(F64) * torch.exp2(torch.randint(-26, -20, (m,), device="cuda", generator=gen).to(F64))
    x = torch.zeros(m, k, device="cuda")
    x[torch.arange(m, device="cuda"), at] = v.to(F32)
    got = (B.matmul(made[0][0], x) if weights == 1 else B.gated(made[0][0], made[1][0], x)).to(F64)
    y = [v[:, None] * w[:, at].t() for _, w in made]
    if weights == 1:
        want, tol = y[0], 2.0 ** -23 + 2 * 2.0 ** -24
    else:  # the errors of both sums, silu's relative slope being 1 + |g| at most, and of the activation
        want, tol = silu(y[0]) * y[1], (2 + y[0].abs()) * (2.0 ** -23 + 2.0 ** -24) + (8 + 8 * y[0].abs()) * 2.0 ** -24 + 2 * 2.0 ** -24
    bad = ~((got - want).abs() <= tol * want.abs())
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[:4].tolist()}"
