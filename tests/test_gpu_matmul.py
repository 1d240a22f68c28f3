"""Products with 4-bit weights on the GPU against 64 bits, with bounds derived from the roundings (matmul_common)."""
import math

import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from matmul_common import Made, close, product64, rounded, rows_of_x

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FORMS = [(f, r, d) for f in ("nvfp4", "mxfp4") for r in (False, True) for d in (BF16, F32)]
IDS = [f"{f}{'-rotated' if r else ''}-{str(d)[6:]}" for f, r, d in FORMS]
# tokens, rows, cols (in units of 32): every form of the kernels, sizes at their tiles' ends, one less and one more
SIZES = [(1, 1, 1), (1, 16, 1), (1, 4096, 4), (2, 17, 3), (3, 33, 129), (4, 100, 32), (5, 31, 40), (8, 256, 17), (16, 32, 64),
         (17, 65, 9), (31, 64, 33), (32, 129, 8), (33, 63, 24), (48, 260, 68), (64, 128, 16), (65, 64, 5), (100, 127, 36),
         (16, 20, 500), (4, 33, 640), (128, 256, 8), (130, 300, 44), (255, 257, 12), (300, 515, 20), (513, 129, 67)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_matmul(form, size):
    fmt, rotate, dtype = form
    m, n, k = size
    rng = np.random.default_rng(m * 7919 + n * 31 + k + 1000003 * FORMS.index(form))
    # NVFP4: rows that end inside a step, and after the first block of two
    k = 32 * k - (16 if fmt == "nvfp4" and k % 4 == 1 else 0)
    w, x = Made(rng, fmt, n, k, rotate), rows_of_x(rng, m, k, dtype)
    got = B.matmul(w.handle(), x.cuda())
    y, tol = product64(w, x)
    assert got.dtype == dtype and tuple(got.shape) == (m, n)
    close(got, y, rounded(y, tol, dtype))


def act64(act, g):
    """The activation in 64 bits, and the largest slope of any of the three (1.13, at 1.5 or so) as a bound."""
    if act == B.FP4Q_ACT_SILU:
        return g / (1 + np.exp(-np.maximum(g, -700)))
    if act == B.FP4Q_ACT_GELU:
        return 0.5 * g * np.array([math.erfc(-v / math.sqrt(2)) for v in g.reshape(-1)]).reshape(g.shape)
    return 0.5 * g * (1 + np.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def gated64(w0, w1, x, act):
    """act(x W0^T) * (x W1^T) and the bound: the products' errors through the factors (slope at most 1.13), and the
    activation's own arithmetic.  exp, erf and their arguments (an exponent of up to 104 in a few roundings; the cube of
    the tanh form three more) are relative errors of 1 + exp or 1 + erf: for silu and the tanh form below
    (8 + 8 |z|) 2^-24 of the result with z the exponent, at most 104 where the result is not below 2^-149; for erf
    |g| 2^-22 absolute, as 1 + erf cancels."""
    (g, tg), (u, tu) = product64(w0, x), product64(w1, x)
    a = act64(act, g)
    z = np.abs(g) if act == B.FP4Q_ACT_SILU else 2 * math.sqrt(2 / math.pi) * np.abs(g + 0.044715 * g ** 3)
    ta = 1.13 * tg + (np.abs(g) * 2.0 ** -22 if act == B.FP4Q_ACT_GELU else np.abs(a) * (8 + 8 * np.minimum(z, 104)) * 2.0 ** -24)
    return a * u, ta * np.abs(u) + np.abs(a) * tu + ta * tu + np.abs(a * u) * 2.0 ** -23


@pytest.mark.parametrize("act", [B.FP4Q_ACT_SILU, B.FP4Q_ACT_GELU, B.FP4Q_ACT_GELU_TANH])
@pytest.mark.parametrize("size", [(1, 16, 4), (3, 31, 9), (4, 20, 300), (16, 100, 36), (13, 40, 512), (20, 100, 36), (32, 257, 17), (33, 65, 12),
                                  (70, 130, 8), (300, 257, 17)], ids=str)
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_gated(form, size, act):
    fmt, rotate, dtype = form
    m, n, k = size
    rng = np.random.default_rng(m * 7919 + n * 31 + k + 1000003 * FORMS.index(form) + act)
    k *= 32
    ws = [Made(rng, fmt, n, k, rotate, S) for S in (0.02, 0.011)]
    x = (rows_of_x(rng, m, k, F32) * (0.7 if fmt == "nvfp4" else 0.01)).to(dtype)
    got = B.gated(ws[0].handle(), ws[1].handle(), x.cuda(), activation=act)
    y, tol = gated64(*ws, x, act)
    close(got, y, rounded(y, tol, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m", [1, 20, 150])
def test_strides_and_untouched_memory(dtype, m):
    """Rows of x and of the output with gaps, unaligned outputs, outputs of an odd stride; what lies between stays."""
    rng = np.random.default_rng(m)
    w, x = Made(rng, "nvfp4", 37, 208), rows_of_x(rng, m, 208, dtype)
    wide = torch.full((m, 240), float("nan"), dtype=dtype)
    wide[:, 16:224] = x
    y, tol = product64(w, x)
    for first, stride in ((0, 37), (1, 39), (4, 44), (3, 128)):
        hold = torch.full((m * stride + 200,), 7.0, dtype=dtype, device="cuda")
        out = hold[first:].as_strided((m, 37), (stride, 1))
        got = B.matmul(w.handle(), wide.cuda()[:, 16:224], out=out)
        assert got is out
        close(out, y, rounded(y, tol, dtype))
        rest = torch.ones_like(hold, dtype=torch.bool)
        rest[first:].as_strided((m, 37), (stride, 1))[:] = False
        assert (hold[rest] == 7.0).all()


def test_shapes_of_x():
    """One row without a batch dimension, several leading ones, none at all, and empty ones."""
    rng = np.random.default_rng(5)
    w = Made(rng, "mxfp4", 24, 64)
    h, x = w.handle(), rows_of_x(rng, 12, 64, BF16).cuda()
    y = B.matmul(h, x)
    assert torch.equal(B.matmul(h, x[3]), B.matmul(h, x[3:4])[0])
    assert torch.equal(B.matmul(h, x.view(2, 3, 2, 64)), y.view(2, 3, 2, 24))
    out = torch.empty(3, 4, 24, dtype=BF16, device="cuda")
    assert B.matmul(h, x.view(3, 4, 64), out=out).data_ptr() == out.data_ptr() and torch.equal(out.view(12, 24), y)
    assert B.matmul(h, x[:0]).shape == (0, 24) and B.matmul(h, x.view(12, 1, 64)[:, :0]).shape == (12, 0, 24)
    none = Made(rng, "nvfp4", 0, 64).handle()
    assert B.matmul(none, x).shape == (12, 0)
    short = Made(rng, "nvfp4", 9, 0)  # a sum over nothing
    assert torch.equal(B.matmul(short.handle(), x[:, :0]), torch.zeros(12, 9, dtype=BF16, device="cuda"))
    assert torch.equal(B.gated(short.handle(), short.handle(), x[:1, :0]), torch.zeros(1, 9, dtype=BF16, device="cuda"))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m", [3, 24, 40, 300])
def test_values_that_are_not_finite_stay_in_their_row(m, fmt, rotate, dtype):
    rng = np.random.default_rng(m)
    w, x = Made(rng, fmt, 50, 160, rotate), rows_of_x(rng, m, 160, dtype)
    h = w.handle()
    clean = B.matmul(h, x.cuda())
    x[1, 37], x[2, 100] = float("nan"), float("inf")
    got = B.matmul(h, x.cuda())
    assert torch.isnan(got[1]).all()
    assert not torch.isfinite(got[2]).all()
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    assert torch.equal(got[keep], clean[keep])
    if not rotate:  # infinity times a weight: its sign, or NaN where the weight is zero
        v = torch.from_numpy(w.values[:, 100])
        want = torch.where(v == 0, float("nan"), torch.sign(v) * float("inf"))
        assert torch.equal(torch.nan_to_num(got[2].double().cpu(), 5.0), torch.nan_to_num(want.double(), 5.0))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m", [1, 50, 200])
def test_scales_that_are_none_stay_in_their_row(m, fmt):
    """A NaN scale byte of one weight row makes that column of y NaN, and no other."""
    rng = np.random.default_rng(m)
    w, x = Made(rng, fmt, 70, 480), rows_of_x(rng, m, 480, BF16).cuda()
    clean = B.matmul(w.handle(), x)
    w.scales[(41 * 480 + 479) // w.block] = 0xFF if fmt == "mxfp4" else 0x7F
    got = B.matmul(w.handle(), x)
    assert torch.isnan(got[:, 41]).all()
    keep = [n for n in range(70) if n != 41]
    assert torch.equal(got[:, keep], clean[:, keep])


@pytest.mark.parametrize("S", [2.0 ** -117, 2.0 ** -60, 2.0 ** 100])
def test_global_scales_at_the_ends(S):
    rng = np.random.default_rng(1)
    one = Made(rng, "nvfp4", 40, 256, S=1.0)
    x = rows_of_x(rng, 6, 256, F32)
    w = one.handle()
    base = B.matmul(w, x.cuda()).double()
    scaled = B.QuantizedWeight(w.tensors[0], w.tensors[1], torch.tensor([S], device="cuda"), 40, 256)
    assert torch.equal(B.matmul(scaled, x.cuda()).double(), base * S)  # a power of two: exact


@pytest.mark.parametrize("m", [2, 24, 60, 200])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_same_result_every_time_and_by_rows(m, fmt):
    """No order of sums changes between calls, and a row of x gives the same bits wherever it stands among the others."""
    rng = np.random.default_rng(m)
    w, x = Made(rng, fmt, 200, 1120, True), rows_of_x(rng, m, 1120, BF16).cuda()
    h = w.handle()
    y = B.matmul(h, x)
    for _ in range(3):
        assert torch.equal(B.matmul(h, x), y)
    turned = torch.roll(x, 1, 0)
    assert torch.equal(B.matmul(h, turned), torch.roll(y, 1, 0))
