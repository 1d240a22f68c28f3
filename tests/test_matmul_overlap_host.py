"""A product whose result would lie in its own x is refused on the host (no GPU needed: no call here is accepted)."""
import ctypes as C
import os

import pytest

from block_scaled_fp4_fp4q_amd import binding as B

X = 1 << 24
SHAPE, NULL = -3, -1


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libfp4q.so not built")
    return B.lib()


def call(L, y, tokens=8, n=256, k=256, xs=None, ys=None, dtype=B.FP4Q_F32):
    """The statuses of the product and of the gated block, without the workspace that they need."""
    s = B.make_spec(B.FP4Q_NVFP4)
    w = B.fp4q_weight(1 << 20, 1 << 21, 1 << 22, n, k)
    xs, ys = k if xs is None else xs, n if ys is None else ys
    return (L.fp4q_matmul(C.byref(s), C.byref(w), X, dtype, tokens, xs, y, ys, None, 0, None),
            L.fp4q_gated(C.byref(s), C.byref(w), C.byref(w), 0, X, dtype, tokens, xs, y, ys, None, 0, None))


# of 40 binary32 rows, which need a workspace: what is not refused for its places is refused for that
OVER = [dict(y=X), dict(y=X + 4), dict(y=X - 4), dict(y=X + 40 * 1024 - 4), dict(y=X - 40 * 1024 + 4),
        dict(y=X + 1024 - 4, xs=512, ys=512), dict(y=X + 2048, xs=512, ys=512), dict(y=X + 1024 + 4, xs=512, ys=512),
        dict(y=X, xs=0), dict(y=X + 512, xs=0), dict(y=X - 39 * 4096 + 1000, xs=256, ys=1024),
        dict(y=X + 1024, xs=512, ys=1024 + 256), dict(y=X, n=8), dict(y=X + 800, n=8, ys=64, xs=512)]
APART = [dict(y=X + 40 * 1024), dict(y=X - 40 * 1024), dict(y=X + 1024, xs=512, ys=512), dict(y=X - 1024, xs=512, ys=512),
         dict(y=X + 5120, xs=512, ys=512), dict(y=X + 1024, xs=0), dict(y=X + 1024, xs=512, ys=1024),
         dict(y=X + 1024, n=8, xs=512, ys=512)]


@pytest.mark.parametrize("case", OVER, ids=str)
def test_shared(L, case):
    assert call(L, tokens=40, **case) == (SHAPE, SHAPE)


@pytest.mark.parametrize("case", APART, ids=str)
def test_apart(L, case):
    assert call(L, tokens=40, **case) == (NULL, NULL)


def test_against_every_byte(L):
    """Small rows at all places near each other, by a look at every element."""
    for xs in (0, 16, 20, 32, 48):
        for ys in (7, 16, 20, 33):
            for at in range(-140, 161, 3):
                x = {i * xs + j for i in range(40) for j in range(16)}
                y = {at + i * ys + j for i in range(40) for j in range(7)}
                want = SHAPE if x & y else NULL
                assert call(L, X + 4 * at, tokens=40, n=7, k=16, xs=xs, ys=ys) == (want, want), (xs, ys, at)
