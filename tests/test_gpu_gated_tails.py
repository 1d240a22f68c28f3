"""The gated block's activations far from zero, where they are small and the other factor is large: their relative error."""
import math

import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B

pytestmark = pytest.mark.gpu


def weight(fmt, n, k, at, code):
    """Every row has one value, of `code` at column `at`, under a scale of 1."""
    block = 32 if fmt == "mxfp4" else 16
    codes = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    codes[:, at // 2] = code << 4 * (at % 2)
    scales = torch.full((n * k // block,), 127 if fmt == "mxfp4" else 0x38, dtype=torch.uint8, device="cuda")
    return B.QuantizedWeight(codes.reshape(-1), scales, None if fmt == "mxfp4" else torch.ones(1, device="cuda"), n, k,
                             format=B.FP4Q_MXFP4 if fmt == "mxfp4" else B.FP4Q_NVFP4)


def wanted(act, g):
    if act == B.FP4Q_ACT_SILU:
        return g / (1 + math.exp(-g))
    if act == B.FP4Q_ACT_GELU:
        return 0.5 * g * math.erfc(-g / math.sqrt(2))
    return g / (1 + math.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def bound(act, g):
    """Relative error of the activation in binary32.  GELU: the argument g / sqrt 2 is off by its rounding and the constant's, 2^-23
    relative together at most, times the slope of log erfc, at most 2 z^2 + 1 = g^2 + 1; erfc itself by at most 16 units in
    the last place, OpenCL's limit, 2^-19; two products.  The others: an exponent z of a few roundings, 8 |z| 2^-24, exp, a sum and a
    quotient, 8 2^-24."""
    if act == B.FP4Q_ACT_GELU:
        return (g * g + 1) * 2.0 ** -23 + 2.0 ** -19 + 2 * 2.0 ** -24
    z = np.abs(g) if act == B.FP4Q_ACT_SILU else 2 * math.sqrt(2 / math.pi) * np.abs(g + 0.044715 * g ** 3)
    return (8 + 8 * z) * 2.0 ** -24


@pytest.mark.parametrize("act", [B.FP4Q_ACT_SILU, B.FP4Q_ACT_GELU, B.FP4Q_ACT_GELU_TANH])
@pytest.mark.parametrize("m", [1, 7, 40, 300])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_tails(fmt, m, act):
    """Gates and up-projections that are each one value of x: exact, so that the activation's error alone is left."""
    n, k = 5, 320
    low = {B.FP4Q_ACT_SILU: -80.0, B.FP4Q_ACT_GELU: -12.5, B.FP4Q_ACT_GELU_TANH: -9.0}[act]
    g = np.concatenate((np.linspace(low, 12.0, 295), [-5.0, -5.2, -5.5, -6.0, -8.9])).astype(np.float32)
    u = np.float32(2.0) ** np.random.default_rng(m).integers(0, 40, len(g))
    w0, w1 = weight(fmt, n, k, 7, 2), weight(fmt, n, k, 200, 2)
    x = np.zeros((len(g), k), np.float32)
    x[:, 7], x[:, 200] = g, u
    x = torch.from_numpy(x).cuda()
    got = torch.cat([B.gated(w0, w1, x[i:i + m], activation=act) for i in range(0, len(g), m)]).double().cpu().numpy()
    want = np.array([wanted(act, float(v)) for v in g]) * u
    tol = np.abs(want) * (bound(act, g.astype(np.float64)) + 2 * 2.0 ** -24)  # the product, and the result's rounding
    assert (np.abs(got - want[:, None]) <= tol[:, None]).all(), \
        f"worst {np.nanmax(np.abs(got - want[:, None]) / np.maximum(tol[:, None], 1e-300)):.3g} of the bound"
