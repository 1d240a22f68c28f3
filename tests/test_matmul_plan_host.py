"""How the products' calls are cut into workgroups, asked of the plan itself on the host (no GPU needed)."""
import shutil

import pytest

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
            (1, 0, 0, 0, 4096, 4096, 8, "few"), (1, 0, 0, 0, 4096, 4096, 16, "many"), (2, 0, 1, 1, 14336, 4096, 16, "few")]


@pytest.mark.parametrize("case", MEASURED, ids=str)
def test_the_faster_kernel_is_taken(exe, case):
    assert plans(exe, [case[:7]])[0].kernel == case[7]
