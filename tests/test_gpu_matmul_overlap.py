"""Results beside their x in one array, and in its place."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B
from matmul_common import Made, close, product64, rounded, rows_of_x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [1, 9, 70, 400])
def test_columns_of_one_array(m, dtype):
    rng = np.random.default_rng(m)
    w, x = Made(rng, "nvfp4", 96, 160), rows_of_x(rng, m, 160, dtype)
    y, tol = product64(w, x)
    for first in (160, 168):
        both = torch.full((m, 288), 3.0, dtype=dtype, device="cuda")
        both[:, :160] = x.cuda()
        close(B.matmul(w.handle(), both[:, :160], out=both[:, first:first + 96]), y, rounded(y, tol, dtype))
        assert torch.equal(both[:, :160].cpu(), x) and (both[:, 160:first] == 3.0).all() and (both[:, first + 96:] == 3.0).all()


@pytest.mark.parametrize("m", [1, 9, 70])
def test_in_place_is_refused(m):
    rng = np.random.default_rng(m)
    h, x = Made(rng, "mxfp4", 64, 64).handle(), rows_of_x(rng, m, 64, torch.float32).cuda()
    wide = torch.cat((x, x), 1)
    for a, out in ((x, x), (wide[:, :64], wide[:, 32:96]), (wide[:, 32:96], wide[:, :64])):
        keep = wide.clone(), x.clone()
        with pytest.raises(B.Fp4qError):
            B.matmul(h, a, out=out)
        with pytest.raises(B.Fp4qError):
            B.gated(h, h, a, out=out)
        assert torch.equal(wide, keep[0]) and torch.equal(x, keep[1])
