"""How the products' calls are cut into workgroups, asked of the plan itself on the host (no GPU needed)."""
import ctypes as C
import os
import shutil

import pytest

from matmul_forms import ONE_PART, THREE_PARTS, form
from matmul_plans import compiled, plans

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("plan"))


# weights, mx, rotate, bf16, rows, cols, tokens, and the kernel that was measured to take less time
MEASURED = [(2, 0, 0, 1, 4096, 4096, 20, "few"), (2, 0, 0, 1, 4096, 4096, 24, "many"), (2, 0, 0, 1, 4096, 4096, 32, "many"),
            (2, 1, 0, 1, 4096, 4096, 20, "few"), (2, 1, 0, 1, 4096, 4096, 24, "many"), (2, 1, 0, 1, 4096, 4096, 32, "many"),
            (2, 0, 0, 1, 14336, 4096, 20, "few"), (2, 0, 0, 1, 14336, 4096, 32, "many"), (2, 1, 0, 1, 14336, 4096, 32, "few"),
            (2, 0, 0, 1, 16384, 2048, 32, "few"), (1, 0, 0, 1, 14336, 4096, 32, "few"), (1, 0, 0, 1, 4096, 4096, 32, "few"),
            (1, 0, 0, 1, 4096, 14336, 17, "many"), (1, 0, 0, 0, 4096, 14336, 8, "many"), (1, 0, 0, 0, 4096, 14336, 4, "few"),
            (1, 0, 1, 1, 28672, 8192, 6, "few"), (1, 0, 1, 1, 28672, 8192, 12, "many"), (1, 0, 1, 1, 8192, 8192, 6, "few"),
            (2, 0, 1, 1, 1024, 4096, 12, "many"), (2, 1, 0, 0, 14336, 6144, 16, "few"), (1, 0, 1, 1, 1024, 4096, 6, "few"),
            (1, 0, 0, 0, 4096, 4096, 8, "few"), (1, 0, 0, 0, 4096, 4096, 16, "many"), (2, 0, 1, 1, 14336, 4096, 16, "few")]


@pytest.mark.parametrize("case", MEASURED, ids=str)
def test_the_faster_kernel_is_taken(exe, case):
    assert plans(exe, [case[:7]])[0].kernel == case[7]


def test_no_call_within_the_stated_limit_is_refused(exe):
    """ceil(rows / 64) * ceil(tokens / 32) below 2^23, at its ends; beyond it some are, and ask for no workspace."""
    forms = [(w, mx, rotate, bf16) for w in (1, 2) for mx in (0, 1) for rotate in (0, 1) for bf16 in (0, 1)]
    most = (1 << 23) - 1
    sizes = [(64 * most, 32, t) for t in (1, 2, 3, 16, 17, 32)] + [(64 * (most // 2), 4096, t) for t in (33, 64)]
    sizes += [(64, 32, 32 * most), (1, 1 << 22, 32 * most), (64 * 2896, 64, 32 * 2896), (64 * 65, 32, 32 * (most // 65))]
    assert not any(p.refused for p in plans(exe, [(*f, *s) for f in forms for s in sizes]))
    beyond = plans(exe, [(*f, 1 << 36, 32, t) for f in forms for t in (1, 20, 500)])
    assert all(p.refused for p in beyond)


def test_refused_calls_say_so():
    """Through the C ABI: the call's status, and no workspace asked for."""
    from block_scaled_fp4_fp4q_amd import binding as B
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libfp4q.so not built")
    L, s = B.lib(), B.make_spec(B.FP4Q_NVFP4)
    w = B.fp4q_weight(1 << 20, 1 << 21, 1 << 22, 1 << 36, 32)
    for tokens in (1, 20, 500):
        assert L.fp4q_matmul_workspace_bytes(C.byref(s), C.byref(w), tokens, B.FP4Q_F32) == 0
        assert L.fp4q_gated_workspace_bytes(C.byref(s), C.byref(w), tokens, B.FP4Q_F32) == 0
        assert L.fp4q_matmul(C.byref(s), C.byref(w), 1 << 23, B.FP4Q_F32, tokens, 32, 1 << 24, 1 << 36, None, 0, None) == -3
        assert L.fp4q_gated(C.byref(s), C.byref(w), C.byref(w), 0, 1 << 23, B.FP4Q_F32, tokens, 32, 1 << 24, 1 << 36, None, 0,
                            None) == -3


def test_every_kernel_has_a_size_among_the_compared_ones(exe):
    """The kernels that any of some 30,000 calls takes, and those of the sizes that are compared with 64 bits (matmul_forms)."""
    rows = (1, 20, 100, 515, 1003, 2051, 4100, 6160, 8200, 12304, 16400, 33000, 70000, 200000)
    cols = (32, 96, 256, 288, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 14336, 14368, 1 << 20)
    tokens = (1, 2, 3, 4, 5, 8, 12, 16, 17, 20, 24, 32, 33, 48, 64, 65, 100, 128, 129, 200, 300, 512, 1000, 2000, 4096, 8192, 30000)

    def taken(sizes):
        return {form(c, p): c for c, p in zip(sizes, plans(exe, sizes)) if not p.refused}
    some = taken([(w, mx, rotate, bf16, n, k, m) for w in (1, 2) for mx in (0, 1) for rotate, bf16 in ((0, 0), (0, 1), (1, 1))
                  for n in rows for k in cols for m in tokens])
    mine = taken([(w, mx, 0, bf16, *size) for w in (1, 2) for mx in (0, 1) for bf16, sizes in ((1, ONE_PART), (0, THREE_PARTS))
                  for size in sizes])
    assert not set(some) - set(mine), {f: some[f] for f in set(some) - set(mine)}
    assert len(some) >= 160
